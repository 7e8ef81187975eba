"""The delta rule and the norms of its queries and keys around what they are given: results do not depend on what the
workspace holds, nothing is written behind it, and offsets that are wrong stay in range."""
import ctypes

import numpy as np
import pytest

from delta_reference import make, values
from oracle import delta
from test_gpu_delta import DT, _cu, _dev, _host, _lib
from test_gpu_qk_norm import EPS, _half

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

GUARD = 4096

CASES = [
    # lens, G, H, K, V: whole and cut sequences (a segment is 256 tokens or more in bf16, 128 in fp32), two sequences of
    # equal lengths, short ones beside cut ones, shared heads, values whose last tiles are padding, all padded key sizes
    ([100, 31], 1, 2, 20, 24),
    ([1100], 1, 1, 24, 24),
    ([800, 800], 2, 2, 64, 130),
    ([70, 0, 5], 1, 2, 128, 130),
    ([900, 1, 0, 300], 1, 3, 100, 130),
    ([100, 31], 1, 2, 256, 70),
    ([900], 1, 2, 256, 130),
    ([600] + [1] * 40 + [300, 0], 1, 2, 40, 72),
    ([800], 1, 2, 100, 3),
    ([130], 1, 1, 5, 200),
]


def _call(name, tensors, lens, G, H, K, V, code, fill, packed):
    """The C entry's outputs and status with a workspace of `fill` and a guard behind it; tensors: addresses of the inputs
    and of the outputs as the C entry takes them."""
    L = _lib().lib()
    T, S = sum(lens), len(lens)
    n = lens[0]
    three = (lambda h, d: (0 if packed else n * h * d, h * d, d))
    sizes = (ctypes.c_int64 * 24)(S, T, G, H, K, V, *three(G, K), *three(G, K), *three(H, V), *three(H, 1), *three(H, V),
                                  *three(H, 1))
    need = getattr(L, name + "_workspace")(sizes, int(packed), code)
    assert need > 0
    ws = torch.full((need + GUARD,), fill, dtype=torch.uint8, device="cuda")
    rc = getattr(L, name)(*(None if t is None else t.data_ptr() for t in tensors), sizes, 0.3, code, ws.data_ptr(), need,
                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert bool((ws[need:] == fill).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:40])
def test_workspace_may_hold_anything(case, dtype):
    lens, G, H, K, V = case
    code = 1 if dtype == "bf16" else 0
    args = make(lens, G, H, K, V, dtype, seed=K + V)
    x = [_dev(a, dtype if i < 3 else "f32") for i, a in enumerate(args)]
    do = _dev(values(np.random.default_rng(3).standard_normal(args[2].shape), dtype), dtype)
    dl = torch.randn(x[5].shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    for packed in (True, False) if len(set(lens)) == 1 else (True,):
        cu = _cu(lens) if packed else None
        forward, backward = [], []
        for fill in (0, 255):  # 255: NaN in either type
            outs = [torch.full_like(x[2], float("nan")), torch.full_like(x[5], float("nan"))]
            _call("ss2d_delta_rule", (*x, cu, *outs), lens, G, H, K, V, code, fill, packed)
            forward.append(outs)
            outs = [torch.full_like(x[i], float("nan")) for i in range(6)]
            _call("ss2d_delta_rule_backward", (*x, cu, do, dl, *outs), lens, G, H, K, V, code, fill, packed)
            backward.append(outs)
        for a, b in (forward, backward):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
            assert all(bool(torch.isfinite(s).all()) for s in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [2, 1])
def test_wrong_cu_seqlens_stay_in_range(dtype, H):
    """Offsets beyond the tokens, negative or decreasing: garbage at worst and a clean exit, forward (many sequences, where
    the segments of cut ones alone are kept) and gradients."""
    ss2d, T = _lib(), 1500
    args = make([T], 1, H, 16, 16, dtype, seed=11)
    d = [_dev(x, dtype if i < 3 else "f32") for i, x in enumerate(args[:5])]
    do = torch.randn(T, H, 16, device="cuda").to(DT[dtype])
    r = np.random.default_rng(0)
    for cu in ([0, 2 ** 31 - 1], [-5, 100, 50, 300], [1500, 0, 1500, 0], [-2 ** 31, -1], [700, 1500, 0, 1500],
               list(r.integers(-100, 1700, 60)), [0, 1500] * 30):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        _, last = ss2d.delta_rule(*d, cu_seqlens=c, final_state=True)
        out = ss2d.delta_rule_backward(*d, do, state=torch.zeros_like(last), dfinal_state=last, cu_seqlens=c)
        torch.cuda.synchronize()
        assert last.shape[0] == len(cu) - 1 and out["dstate"].shape == last.shape


def _in_order(T, heads, other, D):
    """The most additions that one of a weight's gradients goes through, one after the other.  Rows are taken in runs of
    two heads by groups of threads, one for eight channels (no rotation); 1024 workgroups at most for queries and keys
    together, shared by their runs; then sums over a workgroup's groups of threads, in pairs inside a wave and over the
    four waves, and over the workgroups' parts in 32 ranges, in order."""
    threads = 4
    while threads * 8 < D:
        threads *= 2
    runs, all_runs = T * -(-heads // 2), T * (-(-heads // 2) + -(-other // 2))
    groups = 256 // threads
    blocks = min(-(-runs // groups), max(1, 1024 * runs // all_runs))
    return 2 * -(-runs // (blocks * groups)) + 4 + 3 + -(-blocks // 32) + 32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk,D,T", [(16, 1, 32, 30000), (1, 16, 64, 20000), (16, 1, 128, 4097), (32, 2, 40, 5000)])
def test_weight_gradients_of_uneven_heads(Hq, Hk, D, T, dtype):
    """A side of few heads is summed by few workgroups.  Each term has two roundings more than the norm's own (the product,
    the sum's of the gradient), half steps of 2^-24 of its absolute value; so has each addition on its way."""
    r = np.random.default_rng(T)
    x = {n: values(r.standard_normal((T, h, D)), dtype) for n, h in (("q", Hq), ("k", Hk))}
    dy = {n: values(r.standard_normal(x[n].shape), dtype) for n in "qk"}
    w = {n: r.uniform(0.5, 1.5, D).astype(np.float32) for n in "qk"}
    out = _lib().qk_norm_backward(_dev(x["q"], dtype), _dev(x["k"], dtype), _dev(dy["q"], dtype), _dev(dy["k"], dtype),
                                  _dev(w["q"]), _dev(w["k"]), eps=EPS)
    torch.cuda.synchronize()
    for n, h, other in (("q", Hq, Hk), ("k", Hk, Hq)):
        ref = delta.head_norm_backward(x[n], dy[n], w[n], None, None, False, EPS)[1]
        xhat = np.abs(x[n]) / np.sqrt((np.asarray(x[n], np.float64) ** 2).mean(-1, keepdims=True) + EPS)
        size = (np.abs(dy[n]) * xhat).sum((0, 1))
        tol = (_half(D) + (_in_order(T, h, other, D) + 2) * 2.0 ** -24) * size
        worst = float(np.max(np.abs(_host(out[f"d{n}_weight"]) - ref) / tol))
        print(f"[qk] d{n}_weight {T} x {h} x {D}: {worst:.3f} of {_in_order(T, h, other, D)} additions", flush=True)
        assert worst <= 1
