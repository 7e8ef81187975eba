"""The build refuses kernels of the delta rule that spill vector registers (CPU; the kernels are only compiled)."""
import os
import subprocess

import pytest

import selective_scan_crossscan_amd as ss2d
from selective_scan_crossscan_amd import _build

SOURCE = """
#include <hip/hip_runtime.h>
__global__ __launch_bounds__(1024) void NAME(const float* x, float* y, int n) {
  float v[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = x[i * 1024 + threadIdx.x];
  for (int r = 0; r < n; ++r)
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = fmaf(v[i], v[(i * 7 + 3) % COUNT], y[r]);
#pragma unroll
  for (int i = 0; i < COUNT; ++i) y[i * 1024 + threadIdx.x] = v[i];
}
"""


def _compiled(folder, name, count):
    try:
        hipcc = _build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    src, obj = folder / f"{name}.hip", str(folder / f"{name}.o")
    src.write_text(SOURCE.replace("NAME", name).replace("COUNT", str(count)))
    subprocess.check_call([hipcc, *_build.HIPCC_FLAGS, "-c", "-o", obj, str(src)], stderr=subprocess.DEVNULL)
    return obj


def test_spilled_registers_are_found_and_refused(tmp_path):
    """1024 threads leave 128 registers each: 300 values do not fit, 8 do."""
    many, few, other = _compiled(tmp_path, "delta_many", 300), _compiled(tmp_path, "delta_few", 8), _compiled(tmp_path, "other", 300)
    (n,), (m,) = _build.vector_spills(many).values(), _build.vector_spills(few).values()
    assert n > 100 and m == 0
    _build.check_registers(few)
    _build.check_registers(other)
    with pytest.raises(RuntimeError, match="delta_many"):
        _build.check_registers(many)
    nothing = tmp_path / "nothing"
    nothing.write_bytes(b"no kernels")
    with pytest.raises(RuntimeError, match="metadata"):
        _build.check_registers(str(nothing))


def test_the_library_keeps_them():
    if not os.path.exists(ss2d.library_path()):
        pytest.skip("library not built")
    spills = _build.vector_spills(ss2d.library_path())
    assert sum("delta_" in k for k in spills) > 100  # every variant of storage type, keys and pass
    _build.check_registers(ss2d.library_path())
