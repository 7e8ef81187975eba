// Norms of queries and keys with the position rotation (ss2d_qk_norm.hip): launch
// arguments, already validated by ss2d_delta_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ss2d {

struct QkSide {
  const void* x;
  const float* weight;  // or null
  const void* dy;       // gradients
  void* y;              // gradients: dx, dense
  float* dweight;       // gradients, or null
  int64_t x_stride[3], y_stride[3];  // sequence, token, head; y_stride: of y, gradients: of dy
};
struct QkArgs {
  QkSide side[2];  // queries, keys
  const float* table;        // (table_rows, rotated): cosines, then sines; or null
  const int32_t* positions;  // (sequences, length), or null: the token's number in its sequence
  float* partial;
  int64_t sequences, length, heads[2], dim, rotated, table_rows;
  bool interleaved;
  float eps;
  int dtype;
  hipStream_t stream;
};
hipError_t launch_qk_norm(const QkArgs& a);
hipError_t launch_qk_norm_backward(const QkArgs& a);
size_t qk_norm_backward_workspace_bytes(int64_t tokens, const int64_t (&heads)[2], int64_t dim, int64_t rotated);

}  // namespace ss2d
