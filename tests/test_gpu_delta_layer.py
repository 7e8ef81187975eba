"""The delta rule and the norms of its queries and keys as a layer uses them: packed prompts from slices of one
projection, then tokens on the states they leave; the gradients through both; a caller's stream; launches past 2^32
threads.

Every stage is held to the float64 oracle from the values it was given (the tolerances are those of delta_reference.py
and test_gpu_qk_norm.py); the gradients of both together to central differences of the float64 oracles.
"""
import numpy as np
import pytest

from delta_reference import check_forward, make
from oracle import delta
from test_gpu_delta import DT, _cu, _dev, _host, _lib
from test_gpu_qk_norm import EPS, check_out
from test_gpu_token_streams import _busy, _outputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

G, H, K, V, ROT = 2, 4, 40, 24, 16
WIDTH = [G * K, G * K, H * V, 3]  # a row of the projection: queries, keys, values, and what belongs to others


def _slices(row):
    q, k, v, _ = row.split(WIDTH, -1)
    return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))


def _rates(T, r):
    return -np.exp(r.uniform(-5, 0, (T, H))).astype(np.float32), r.uniform(0, 1, (T, H)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_then_tokens(dtype):
    ss2d, r = _lib(), np.random.default_rng(21)
    lens = [130, 1, 0, 77]
    scale, unit = K ** -0.5, torch.full((K,), K ** -0.5, device="cuda")
    table = ss2d.rotation_table(256, ROT, 100.0)
    weight = _dev(r.uniform(0.5, 1.5, V))

    def norms(name, row, pos):
        q, k, v = _slices(row)
        at = torch.from_numpy(pos.astype(np.int32)).cuda()
        qn, kn = ss2d.qk_norm(q, k, k_weight=unit, rotation=table, positions=at, eps=EPS)
        for what, got, x, w in (("q", qn, q, None), ("k", kn, k, unit)):
            check_out(f"{name} {what}", _host(got), _host(x), None if w is None else _host(w), _host(table), pos, False, dtype)
        return qn, kn, v

    def normed(name, o):
        y = _host(ss2d.rms_norm(o, weight, eps=EPS))
        x = _host(o)
        ref = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * _host(weight)
        # a sum of V squares, its root's reciprocal and two products, and the output's own rounding
        tol = ((V + 8) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)) * np.abs(ref) + 1e-37
        assert np.all(np.abs(y - ref) <= tol), name

    T = sum(lens)
    row = _dev(r.standard_normal((T, sum(WIDTH))), dtype)
    q, k, v = norms("prompts", row, np.concatenate([np.arange(n) for n in lens]))
    g, b = _rates(T, r)
    o, states = ss2d.delta_rule(q, k, v, _dev(g), _dev(b), cu_seqlens=_cu(lens), scale=scale, final_state=True)
    args = tuple(_host(x) for x in (q, k, v)) + (g, b, None)
    check_forward("prompts", _host(o), _host(states), args, lens, scale, dtype)
    normed("prompts", o)

    slots = np.array([3, 0, 2, 1])  # each token's row has a sequence's state; one row is padding
    for i in range(3):
        before = _host(states)
        row = _dev(r.standard_normal((5, sum(WIDTH))), dtype)
        index = np.append(slots, -1).astype(np.int32)
        q, k, v = norms(f"token {i}", row, np.append(np.array(lens)[slots] + i, 0))
        g, b = _rates(5, r)
        o = ss2d.delta_rule_step(q, k, v, _dev(g), _dev(b), states, torch.from_numpy(index).cuda(), scale=scale)
        args = tuple(_host(x)[:4] for x in (q, k, v)) + (g[:4], b[:4], before[slots])
        check_forward(f"token {i}", _host(o)[:4], _host(states)[slots], args, [1] * 4, scale, dtype)
        assert not _host(o)[4].any()
        normed(f"token {i}", o)


def test_gradients_through_both():
    """fp32: both gradients are off by some 2 sqrt(n) 2^-24 = 2e-6 of their terms' norms (n = K + V + 64), the terms
    being ten times a result at most; differences of step e = 1e-4 by e^2 of the third derivative: 1e-4 of the
    gradient's norm times the direction's leaves a factor of more than two for both."""
    ss2d, r = _lib(), np.random.default_rng(22)
    lens, scale = [70, 33], 0.4
    T = sum(lens)
    x = r.standard_normal((T, sum(WIDTH))).astype(np.float32)
    g, b = _rates(T, r)
    wq, wk = (r.uniform(0.5, 1.5, K).astype(np.float32) * s for s in (1, np.float32(K ** -0.5)))
    do = r.standard_normal((T, H, V)).astype(np.float32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    angle = np.arange(80)[:, None] * 0.5 ** np.arange(ROT // 2)
    angles = np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)

    def loss(x, wq, wk, g, b):
        q, k, v, _ = np.split(x, np.cumsum(WIDTH)[:3], -1)
        q = delta.head_norm(q.reshape(T, G, K), wq, angles, pos, True, EPS)
        k = delta.head_norm(k.reshape(T, G, K), wk, angles, pos, True, EPS)
        return float((delta.delta_rule(q, k, v.reshape(T, H, V), g, b, lens, None, scale)[0] * do).sum())

    q, k, v = _slices(_dev(x))
    kw = dict(q_weight=_dev(wq), k_weight=_dev(wk), rotation=_dev(angles), positions=torch.from_numpy(pos).cuda(),
              interleaved=True, eps=EPS)
    qn, kn = ss2d.qk_norm(q, k, **kw)
    d = ss2d.delta_rule_backward(qn, kn, v, _dev(g), _dev(b), _dev(do), cu_seqlens=_cu(lens), scale=scale)
    e = ss2d.qk_norm_backward(q, k, d["dq"], d["dk"], **kw)
    dx = np.concatenate([_host(e["dq"]).reshape(T, -1), _host(e["dk"]).reshape(T, -1), _host(d["dv"]).reshape(T, -1),
                         np.zeros((T, WIDTH[3]))], -1)
    mine = [dx, _host(e["dq_weight"]), _host(e["dk_weight"]), _host(d["dlog_decay"]), _host(d["dbeta"])]
    leaves = [np.asarray(t, np.float64) for t in (x, wq, wk, g, b)]
    for i, name in enumerate(("projection", "query weight", "key weight", "log decay", "beta")):
        u = r.standard_normal(leaves[i].shape)
        step = 1e-4
        hi, lo = (loss(*(t + s * u if j == i else t for j, t in enumerate(leaves))) for s in (step, -step))
        want, got = (hi - lo) / (2 * step), float((mine[i] * u).sum())
        size = np.linalg.norm(mine[i]) * np.linalg.norm(u)
        print(f"[layer] {name}: {got:.6f}, differences {want:.6f}, size {size:.3f}", flush=True)
        assert abs(got - want) <= 1e-4 * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("keys", [40, 256])
def test_gradients_of_repeated_values_are_those_of_copies(dtype, keys):
    """Gradients, rates and values whose strides repeat one (expand), and calls with other values in the workspace."""
    ss2d, T = _lib(), 150
    q, k, v, g, b, _ = make([T], 1, 2, keys, 70, dtype, seed=23, state=False)
    d = [_dev(x, dtype if i < 3 else "f32")[None] for i, x in enumerate((q, k, v, g, b))]
    d[2] = d[2][:, :1].expand(1, T, 2, 70)
    d[3], d[4] = (x[:, :, :1].expand(1, T, 2) for x in d[3:])
    do = torch.randn(70, device="cuda").to(DT[dtype]).expand(1, T, 2, 70)
    want = ss2d.delta_rule_backward(*(x.contiguous() for x in d), do.contiguous(), scale=0.3)
    for fill in (0, 255):
        torch.full((1 << 26,), fill, dtype=torch.uint8, device="cuda")
        got = ss2d.delta_rule_backward(*d, do, scale=0.3)
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_is_written_around_outputs(dtype):
    ss2d = _lib()
    for T, keys, vals in ((1, 5, 3), (70, 130, 65), (300, 33, 7)):
        q, k, v, g, b, _ = make([T], 1, 1, keys, vals, dtype, seed=T, state=False)
        d = [_dev(x, dtype if i < 3 else "f32")[None] for i, x in enumerate((q, k, v, g, b))]
        n = T * vals
        room = torch.full((n + 512,), 7.0, dtype=DT[dtype], device="cuda")
        ss2d.delta_rule(*d, out=room[256:256 + n].view(1, T, 1, vals))
        step = torch.full((n + 512,), 7.0, dtype=DT[dtype], device="cuda")
        states = torch.full((T * keys * vals + 512,), 7.0, device="cuda")
        ss2d.delta_rule_step(*(x[0] for x in d), states[256:-256].view(T, 1, keys, vals),
                             out=step[256:256 + n].view(T, 1, vals))
        torch.cuda.synchronize()
        for x in (room, step, states):
            assert bool((x[:256] == 7).all()) and bool((x[-256:] == 7).all())
            assert not bool((x[256:-256] == 7).any())


def _inputs(op, seed):
    """Tensors of a call of some 30 MB, each in a block of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def key(*shape):
        return torch.nn.functional.normalize(normal(*shape), dim=-1).to(torch.bfloat16)

    if op == "delta_rule_step":
        return [key(64, 8, 128), key(64, 8, 128), key(64, 8, 128), -normal(64, 8).abs(), normal(64, 8).sigmoid(),
                normal(64, 8, 128, 128)]
    if op.startswith("delta_rule"):
        x = [key(2, 2048, 8, 128) for _ in range(3)] + [-normal(2, 2048, 8).abs(), normal(2, 2048, 8).sigmoid()]
        return x + [key(2, 2048, 8, 128)] if op.endswith("backward") else x
    x = [key(4096, 8, 128) for _ in range(4 if op.endswith("backward") else 2)]
    return x + [normal(128), normal(128)]


@pytest.mark.parametrize("op", ["delta_rule", "delta_rule_backward", "delta_rule_step", "qk_norm", "qk_norm_backward"])
def test_inputs_and_outputs_outlive_their_names(op):
    """On a stream given by the caller, as test_gpu_token_streams.py asks of the others."""
    fn = getattr(_lib(), op)
    want = [t.clone() for t in _outputs(fn(*_inputs(op, 1)))]
    side = torch.cuda.Stream()
    _busy()
    with torch.cuda.stream(side):
        _busy()
    torch.cuda.synchronize()
    for _ in range(3):
        other, x = _inputs(op, 2), _inputs(op, 1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _busy()
        out = fn(*x, stream=side)
        sizes = [t.numel() * t.element_size() for t in x]
        del x
        spoilt = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]  # before `side` gets to the call
        torch.cuda.current_stream().wait_stream(side)
        _busy()
        got = [t.clone() for t in _outputs(out)]
        del out
        second = fn(*other, stream=side)  # writes at once, while this stream is busy
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del spoilt, second


@pytest.mark.parametrize("S,heads", [((1 << 20) + 3, 8), (65535, 130)], ids=["prompts", "steps"])
def test_sequences_or_rows_past_a_launch_axis(S, heads):
    """Single tokens, a workgroup of 256 threads per head, over 2^31 threads: as prompts, and as steps (rows 65535)."""
    ss2d = _lib()
    gen = torch.Generator(device="cuda").manual_seed(31)
    q, k, v = (torch.randn(S, 1, n, 4, generator=gen, device="cuda") for n in (1, 1, heads))
    b = torch.rand(S, 1, heads, generator=gen, device="cuda")
    g = torch.zeros(S, 1, heads, device="cuda")
    if S > 65535:
        o = ss2d.delta_rule(q, k, v, g, b)
    else:
        cache = torch.zeros(S, heads, 4, 4, device="cuda")
        o = ss2d.delta_rule_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], b[:, 0], cache)[:, None]
    torch.cuda.synchronize()
    q, k, v, b = (x.double() for x in (q, k, v, b[..., None]))
    want = b * (q * k).sum(-1, keepdim=True) * v
    # four products and their sum, beta, the value: ten roundings of the absolute values
    tol = 10 * 2.0 ** -24 * b * (q * k).abs().sum(-1, keepdim=True) * v.abs() + 1e-37
    assert bool(((o - want).abs() <= tol).all())


def test_norms_past_a_launch_axis():
    """Rows of 32 threads each, 2^26 and a few of them."""
    ss2d, T = _lib(), (1 << 25) + 5
    q, k = (torch.randn(1, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    want = ss2d.qk_norm(q[None], k[None])
    got = ss2d.qk_norm(q.expand(T, 1, 256), k.expand(T, 1, 256))
    torch.cuda.synchronize()
    for x, w in zip(got, want):
        assert all(bool((x[i:i + (1 << 22)] == w).all()) for i in range(0, T, 1 << 22))
