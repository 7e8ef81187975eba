"""GPU parity of linear attention's gradients (ss2d_linear_attention_backward) against
the float64 oracle in oracle/tokens.py (itself pinned by central differences), and
against central differences of the GPU's own forward.

Tolerances.  With |.| the gradients on absolute values (every term added without
cancelling), fp32 results are off by at most c |.|, c = (T/8 + 256 + K + V) 2^-24: states
and their gradients take one product and at most eight accumulations per 64 tokens, a
term is a product of sums over K and V.  A decay's gradient subtracts two sums of one
chunk's terms, at most 64 of each token's |q||k||do||v| products: the oracle's |.| for it
is the sum over all tokens of its chunk, taken here as 64 times the largest within 64
tokens.  For bf16, dq, dk, dv add their own rounding 2^-8 and that of the masked products,
2^-8 |.|; where heads share keys the parts are fp32 and only the sum is rounded.
"""
import numpy as np
import pytest

from oracle import tokens
from test_gpu_attention import DT, _dev, _host, check, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _grads(seed, shape_o, shape_s, dtype):
    r = np.random.default_rng(seed)
    do = r.standard_normal(shape_o).astype(np.float32)
    if dtype == "bf16":
        import ss2d_inputs
        do = ss2d_inputs.round_to_bf16(do)
    return do, r.standard_normal(shape_s).astype(np.float32)


def _bounds(q, k, v, g, do, lens, st, dl, scale, dtype, ref):
    mag = tokens.linear_attention_backward(np.abs(q), np.abs(k), np.abs(v), g, np.abs(do), lens,
                                           None if st is None else np.abs(st), None if dl is None else np.abs(dl),
                                           abs(scale))
    c = (max(lens) / 8 + 256 + q.shape[2] + v.shape[2]) * 2.0 ** -24
    tol = []
    for i, (m, r) in enumerate(zip(mag, ref)):
        if i == 3:
            # own terms of the tokens of a chunk: |q_i . k_i| |do_i . v_i| enters the row and the column sums
            own = np.zeros_like(m)
            for h in range(m.shape[1]):
                gr = h * q.shape[1] // m.shape[1]
                own[:, h] = abs(scale) * np.abs(q[:, gr] * k[:, gr]).sum(-1) * np.abs(do[:, h] * v[:, h]).sum(-1)
            near = np.array([(m + own)[max(0, t - 63):t + 64].max(0) for t in range(len(m))])
            tol.append(c * 2 * near + 1e-37)
        elif dtype == "bf16" and i < 3:
            tol.append(c * m + 2.0 ** -8 * np.abs(r) + (2.0 ** -8 + 2.0 ** -15) * (1 + 2.0 ** -8) * m + 1e-37)
        else:
            tol.append(c * m + 1e-37)
    return tol


NAMES = ("dq", "dk", "dv", "dlog_decay", "dstate")

CASES = [
    ([1], 1, 1, 1, 1),
    ([64], 1, 1, 32, 64),
    ([65], 2, 2, 33, 65),
    ([5, 0, 64, 1, 129, 0], 2, 4, 16, 32),
    ([200], 1, 3, 100, 40),
    ([40, 40, 40], 2, 2, 128, 128),
    ([150, 31], 1, 2, 256, 70),
    ([90], 1, 1, 256, 256),
    ([33], 1, 1, 7, 300),
    ([1100], 1, 1, 24, 24),
    ([700, 0, 300, 1, 513], 1, 2, 40, 130),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gradients_match_oracle(case, dtype):
    lens, G, H, K, V = case
    print(f"[case] attention backward {case} {dtype}", flush=True)
    q, k, v, g, st = make(lens, G, H, K, V, dtype, seed=len(lens) * K + V + 1)
    do, dl = _grads(K, v.shape, st.shape, dtype)
    scale = K ** -0.5
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = _lib().linear_attention_backward(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), _dev(do, dtype),
                                           state=_dev(st), dfinal_state=_dev(dl), cu_seqlens=cu, scale=scale)
    torch.cuda.synchronize()
    ref = tokens.linear_attention_backward(q, k, v, g, do, lens, st, dl, scale)
    for name, r, t in zip(NAMES, ref, _bounds(q, k, v, g, do, lens, st, dl, scale, dtype, ref)):
        check(name, _host(out[name]), r, t)


@pytest.mark.parametrize("decay", ["none", "strong", "far"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays(decay, dtype):
    lens = [300, 70]
    q, k, v, g, st = make(lens, 2, 4, 48, 40, dtype, seed=21, decay=decay)
    do, _ = _grads(22, v.shape, st.shape, dtype)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = _lib().linear_attention_backward(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), _dev(do, dtype),
                                           state=_dev(st), cu_seqlens=cu)
    torch.cuda.synchronize()
    ref = tokens.linear_attention_backward(q, k, v, g, do, lens, st)
    for name, r, t in zip(NAMES, ref, _bounds(q, k, v, g, do, lens, st, None, 1.0, dtype, ref)):
        check(name, _host(out[name]), r, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_lengths_strided_without_states(dtype):
    """Equal lengths, q, k, v and do as slices with other tokens and heads between, a decay per head (stride 0)."""
    S, L, G, H, K, V = 3, 100, 1, 2, 24, 40
    q, k, v, _, _ = make([L] * S, G, H, K, V, dtype, seed=23)
    do, _ = _grads(24, v.shape, (1,), dtype)
    pad = _dev(np.concatenate([np.ones((S * L, 3)), q.reshape(S * L, -1), k.reshape(S * L, -1)], 1).reshape(S, L, -1), dtype)
    qd, kd = pad[..., 3:3 + K].unflatten(-1, (G, K)), pad[..., 3 + K:].unflatten(-1, (G, K))
    vd = _dev(v.reshape(S, L, H, V).transpose(2, 0, 1, 3), dtype).permute(1, 2, 0, 3)
    dd = _dev(do.reshape(S, L, H, V).transpose(0, 2, 1, 3), dtype).transpose(1, 2)
    gh = np.array([-0.02, -0.7], np.float32)
    out = _lib().linear_attention_backward(qd, kd, vd, _dev(gh).expand(S, L, H), dd, scale=0.2)
    torch.cuda.synchronize()
    assert set(out) == set(NAMES) - {"dstate"}
    g = np.broadcast_to(gh, (S * L, H))
    ref = tokens.linear_attention_backward(q, k, v, g, do, [L] * S, None, None, 0.2)
    for name, r, t in zip(NAMES[:4], ref, _bounds(q, k, v, g, do, [L] * S, None, None, 0.2, dtype, ref)):
        check(name, _host(out[name]).reshape(r.shape), r, t)


def test_gradients_by_differences_of_the_forward():
    """d/de of sum(o do) + sum(last dl) along a random direction, by central differences of the GPU forward in fp32."""
    ss2d = _lib()
    q, k, v, g, st = make([150], 2, 4, 20, 24, "f32", seed=25)
    do, dl = _grads(26, v.shape, st.shape, "f32")
    d = [_dev(x)[None] for x in (q, k, v, g)] + [_dev(st)]
    out = ss2d.linear_attention_backward(*d[:4], _dev(do)[None], state=d[4], dfinal_state=_dev(dl), scale=0.5)
    r = np.random.default_rng(27)
    for i, name in enumerate(NAMES):
        u = _dev(r.standard_normal(d[i].shape))
        vals = []
        for e in (2e-3, -2e-3):
            x = list(d)
            x[i] = x[i] + e * u
            o, last = ss2d.linear_attention(*x[:4], state=x[4], scale=0.5, final_state=True)
            vals.append(float((o.double() * _dev(do)[None].double()).sum() + (last.double() * _dev(dl).double()).sum()))
        num = (vals[0] - vals[1]) / 4e-3
        got = float((out[name].double() * u.double()).sum())
        size = float(out[name].double().norm() * u.double().norm())
        print(f"[attention] {name}: {got:.6f} {num:.6f}", flush=True)
        # q, k, v and the state enter linearly or (k with v, the decay) smoothly: step^2 of the third derivative, and
        # the forward's fp32 rounding of some 1e-6 of the loss's terms over the step
        assert abs(got - num) <= 2e-3 * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_outside_the_sequences_are_not_read(dtype):
    lens, lead, tail = [70, 0, 9], 3, 40
    q, k, v, g, st = make(lens, 1, 2, 20, 24, dtype, seed=28)
    do, dl = _grads(29, v.shape, st.shape, dtype)
    pad = [np.concatenate([np.full((lead,) + x.shape[1:], np.nan, np.float32), x,
                           np.full((tail,) + x.shape[1:], np.nan, np.float32)]) for x in (q, k, v, g, do)]
    cu = torch.tensor(lead + np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = _lib().linear_attention_backward(*(_dev(x, dtype) for x in pad[:3]), _dev(pad[3]), _dev(pad[4], dtype),
                                           state=_dev(st), dfinal_state=_dev(dl), cu_seqlens=cu)
    torch.cuda.synchronize()
    ref = tokens.linear_attention_backward(q, k, v, g, do, lens, st, dl)
    for name, r, t in zip(NAMES, ref, _bounds(q, k, v, g, do, lens, st, dl, 1.0, dtype, ref)):
        got = _host(out[name])
        check(name, got if name == "dstate" else got[lead:-tail], r, t)


def test_wrong_cu_seqlens_stay_in_range():
    q, k, v, g, st = make([300], 1, 2, 16, 16, "f32", seed=30)
    for cu in ([0, 2 ** 31 - 1], [-5, 100, 50, 300], [300, 0, 300, 0], [-2 ** 31, -1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        _lib().linear_attention_backward(_dev(q), _dev(k), _dev(v), _dev(g), _dev(v), cu_seqlens=c)
        torch.cuda.synchronize()


def test_results_repeat_and_graph_replays_match():
    ss2d = _lib()
    q, k, v, g, st = make([1500], 1, 2, 64, 64, "bf16", seed=31)
    do, dl = _grads(32, v.shape, st.shape, "bf16")
    d = [_dev(x, "bf16")[None] for x in (q, k, v)] + [_dev(g)[None], _dev(do, "bf16")[None]]
    kw = dict(state=_dev(st), dfinal_state=_dev(dl))
    eager = ss2d.linear_attention_backward(*d, **kw)
    again = ss2d.linear_attention_backward(*d, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(eager[n], again[n]) for n in NAMES)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ss2d.linear_attention_backward(*d, **kw)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        ss2d.linear_attention_backward(*(x[:, :300] for x in d))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], out[n]) for n in NAMES)
