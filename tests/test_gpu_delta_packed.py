"""Many packed sequences, most too short to be cut and some cut into segments, whose states are then kept for the cut ones
alone (ss2d_delta_rule, _backward)."""
import numpy as np
import pytest

from delta_reference import check_forward, check_gradients, make, values
from test_gpu_delta import _host, packed
from test_gpu_delta_backward import run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LENS = [
    # a segment is 256 tokens in bf16, 128 in fp32: lengths around one, two and three of them between single tokens,
    # empty sequences, cut ones next to each other, first and last
    [600] + [1] * 12 + [300, 257, 0, 0, 2] + [70] * 6 + [513, 512, 256] + [0, 1] * 9 + [128, 129],
    [3, 0, 1] * 9 + [1100, 1] + [1, 0, 2] * 4 + [255, 385] + [1] * 5,
    [5] * 200 + [1030] + [4] * 100,
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=["many", "few", "one"])
def test_prompts_match_oracle(lens, dtype):
    args = make(lens, 1, 2, 40, 24, dtype, seed=len(lens))
    o, last = packed(args, lens, dtype, 0.2)
    check_forward("packed", _host(o), _host(last), args, lens, 0.2, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=["many", "few", "one"])
def test_gradients_match_oracle(lens, dtype):
    args = make(lens, 1, 2, 24, 40, dtype, seed=len(lens) + 1)
    r = np.random.default_rng(1)
    do = values(r.standard_normal(args[2].shape), dtype)
    dl = r.standard_normal(args[5].shape).astype(np.float32)
    check_gradients("packed", run(args, do, lens, dl, 0.2, dtype), args, do, lens, dl, 0.2, dtype)
