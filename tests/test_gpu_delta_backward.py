"""GPU parity of the delta rule's gradients (ss2d_delta_rule_backward) against the float64 oracle in oracle/delta.py
(tolerances in delta_reference.py), against differences of the forward, and under capture."""
import numpy as np
import pytest

from delta_reference import check_gradients, make, values
from test_gpu_delta import DT, _cu, _dev, _host, _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAMES = ("dq", "dk", "dv", "dlog_decay", "dbeta", "dstate")


def run(args, do, lens, dl, scale, dtype):
    q, k, v, g, b, st = args
    out = _lib().delta_rule_backward(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), _dev(b), _dev(do, dtype),
                                     state=None if st is None else _dev(st),
                                     dfinal_state=None if dl is None else _dev(dl), cu_seqlens=_cu(lens), scale=scale)
    torch.cuda.synchronize()
    return [None if n not in out else _host(out[n]) for n in NAMES]


CASES = [
    # lens, G, H, K, V: one token, chunk borders, empty sequences, odd sizes, every padded key size, several value tiles,
    # shared keys, segments
    ([1], 1, 1, 1, 1),
    ([64], 1, 2, 32, 64),
    ([65], 2, 2, 33, 65),
    ([5, 0, 64, 1, 129, 0], 2, 4, 16, 32),
    ([150], 1, 3, 100, 40),
    ([40, 90], 2, 2, 128, 128),
    ([100, 31], 1, 2, 256, 70),
    ([33], 1, 1, 7, 300),
    ([70], 1, 1, 200, 200),
    ([1100], 1, 1, 24, 24),
    ([700, 0, 300, 1, 513], 1, 2, 40, 130),
    ([900], 1, 1, 130, 20),
    ([800], 1, 2, 100, 3),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gradients_match_oracle(case, dtype):
    lens, G, H, K, V = case
    print(f"[case] delta gradients {case} {dtype}", flush=True)
    args = make(lens, G, H, K, V, dtype, seed=len(lens) * K + V)
    r = np.random.default_rng(K)
    do = values(r.standard_normal(args[2].shape), dtype)
    dl = r.standard_normal(args[5].shape).astype(np.float32)
    check_gradients("gradients", run(args, do, lens, dl, K ** -0.5, dtype), args, do, lens, dl, K ** -0.5, dtype)


@pytest.mark.parametrize("decay,keys", [("none", "random"), ("strong", "random"), ("far", "random"), ("none", "same"),
                                        ("mixed", "zero")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_and_hard_systems(decay, keys, dtype):
    lens = [300, 70]
    args = make(lens, 1, 2, 48, 40, dtype, seed=3, decay=decay, keys=keys, state=False)
    do = values(np.random.default_rng(4).standard_normal(args[2].shape), dtype)
    check_gradients(f"{decay} {keys}", run(args, do, lens, None, 1.0, dtype), args, do, lens, None, 1.0, dtype)


def test_gradients_are_those_of_the_forward():
    """Central differences of the forward along random directions, fp32."""
    ss2d = _lib()
    lens = [150, 40]
    args = make(lens, 2, 4, 16, 24, "f32", seed=5)
    r = np.random.default_rng(6)
    d = [_dev(x) for x in args]
    do, dl = (_dev(r.standard_normal(x.shape)) for x in (args[2], args[5]))
    cu = _cu(lens)

    def loss(a):
        o, last = ss2d.delta_rule(*a[:5], state=a[5], cu_seqlens=cu, scale=0.4, final_state=True)
        return float((o.double() * do.double()).sum() + (last.double() * dl.double()).sum())

    got = ss2d.delta_rule_backward(*d[:5], do, state=d[5], dfinal_state=dl, cu_seqlens=cu, scale=0.4)
    for i, name in enumerate(NAMES):
        u = _dev(r.standard_normal(args[i].shape))
        e = 2e-3
        vals = [loss([x + s * u if j == i else x for j, x in enumerate(d)]) for s in (e, -e)]
        num, mine = (vals[0] - vals[1]) / (2 * e), float((got[name].double() * u.double()).sum())
        size = float(got[name].double().norm() * u.double().norm())
        print(f"[delta] {name}: {mine:.5f} {num:.5f}", flush=True)
        # the step's square times the third derivative, and fp32 rounding of the loss over the step
        assert abs(num - mine) <= 2e-3 * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_outside_the_sequences_are_left_alone(dtype):
    """Packed tokens outside the sequences hold NaN and are not read; their gradients' places are not written."""
    import ctypes

    lens, lead, tail, G, H, K, V = [70, 0, 9], 3, 40, 1, 2, 24, 24
    args = make(lens, G, H, K, V, dtype, seed=7)
    do = values(np.random.default_rng(8).standard_normal(args[2].shape), dtype)
    pad = [np.concatenate([np.full((lead,) + x.shape[1:], np.nan, np.float32), x,
                           np.full((tail,) + x.shape[1:], np.nan, np.float32)]) for x in (*args[:5], do)]
    T = len(do) + lead + tail
    sizes = (ctypes.c_int64 * 24)(len(lens), T, G, H, K, V, 0, K, K, 0, K, K, 0, H * V, V, 0, H, 1, 0, H * V, V, 0, H, 1)
    ss2d = _lib()
    L, code = ss2d.lib(), 1 if dtype == "bf16" else 0
    n = L.ss2d_delta_rule_backward_workspace(sizes, 1, code)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN
    ins = [_dev(x, dtype if i in (0, 1, 2, 5) else "f32") for i, x in enumerate(pad)]
    outs = [torch.full_like(ins[i], 7.0) for i in range(5)]
    st, ds, cu = _dev(args[5]), torch.empty(3, H, K, V, device="cuda"), _cu(lens, lead)
    rc = L.ss2d_delta_rule_backward(*(x.data_ptr() for x in ins[:5]), st.data_ptr(), cu.data_ptr(), ins[5].data_ptr(),
                                    None, *(x.data_ptr() for x in outs), ds.data_ptr(), sizes, 0.5, code, ws.data_ptr(),
                                    n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    for x in outs:
        assert bool((x[:lead] == 7).all()) and bool((x[-tail:] == 7).all())
    got = [_host(x)[lead:-tail] for x in outs] + [_host(ds)]
    check_gradients("inside", got, args, do, lens, None, 0.5, dtype)


def test_captured_while_an_eager_call_lives():
    """Gradients captured into a graph, replayed with eager calls between."""
    ss2d = _lib()
    args = make([600], 1, 2, 64, 64, "bf16", seed=9, state=False)
    d = [_dev(x, "bf16" if i < 3 else "f32")[None] for i, x in enumerate(args[:5])]
    do = torch.randn_like(d[2])
    want = ss2d.delta_rule_backward(*d, do)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ss2d.delta_rule_backward(*d, do)
    for _ in range(3):
        for x in out.values():
            x.fill_(float("nan"))
        g.replay()
        eager = ss2d.delta_rule_backward(*d, do)
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) and torch.equal(eager[n], want[n]) for n in want)
