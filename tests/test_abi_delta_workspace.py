"""Workspaces of the delta rule for packed sequences, on the CPU: what is kept for the segments of long sequences does not
grow with the number of sequences, however short they are."""
import ctypes

import pytest

import selective_scan_crossscan_amd as ss2d

CHUNK = {0: 32, 1: 64}


def need(name, S, T, H, K, V, packed, dtype):
    z = (ctypes.c_int64 * 24)(S, T, H, H, K, V, *([0] * 18))
    n = getattr(ss2d.lib(), name)(z, packed, dtype)
    assert n > 0
    return n


@pytest.mark.parametrize("name,states", [("ss2d_delta_rule_workspace", 1), ("ss2d_delta_rule_backward_workspace", 2)])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("H,K,V", [(16, 128, 128), (4, 64, 32), (1, 256, 320)])
def test_short_sequences_keep_no_segments(name, states, dtype, H, K, V):
    T, C = 65536, CHUNK[dtype]
    each = need(name, T // C, T, H, K, V, 0, dtype) / (T // C)  # sequences of one chunk: what a chunk takes, nothing cut
    # sequences are cut to give 1024 workgroups; a workgroup is a segment, a head and 64 values
    segments = 2 * 1024 // (H * -(-V // 64)) + 2
    kp = next(n for n in (32, 64, 128, 256) if n >= K)
    cut = segments * H * (states * K * V + kp * kp) * 4
    for S in (64, 1024, 4096, 60000):
        chunks = T // C + S  # each sequence's last chunk counts whole
        # 1 MiB: a workspace's parts are rounded up
        assert need(name, S, T, H, K, V, 1, dtype) <= chunks * each + cut + (1 << 20), S
