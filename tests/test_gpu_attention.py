"""GPU parity of linear attention with a decay per head (ss2d_linear_attention, _step)
against the float64 oracle in oracle/tokens.py, element by element.

Tolerances.  With |.| the operator on absolute values (all terms of an output added
without cancelling), a result in fp32 of a sequence of T tokens is off by at most
c |.|, c = (T/8 + 128 + K) 2^-24: per 64 tokens the state takes one product and at most
eight accumulations, each half a step of 2^-23; a term itself is a sum over K, a decay
(exp2 of a difference, a few steps) and two products.  For bf16 an output adds its own
rounding, 2^-8 |o|, and the rounding of the masked scores, 2^-8 |.|, and of the state
read in two parts, 2^-16 |.|.
"""
import numpy as np
import pytest

from oracle import tokens
import ss2d_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _values(a, dtype):
    a = np.asarray(a, dtype=np.float32)
    return ss2d_inputs.round_to_bf16(a) if dtype == "bf16" else a


def _dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DT[dtype]).cuda()


def _host(t):
    return t.double().cpu().numpy()


def make(lens, G, H, K, V, dtype, seed, decay="mixed", state=True):
    r = np.random.default_rng(seed)
    T = sum(lens)
    q, k, v = (_values(r.standard_normal((T, n, d)), dtype) for n, d in ((G, K), (G, K), (H, V)))
    g = {"mixed": -np.exp(r.uniform(np.log(1e-3), np.log(2.0), (T, H))), "none": np.zeros((T, H)),
         "strong": -r.uniform(5, 60, (T, H)), "far": -np.exp(r.uniform(-3, 0, (T, H)))}[decay].astype(np.float32)
    if decay == "far":  # tokens that forget everything, by the type's lowest value and by -Inf
        g[r.random((T, H)) < 0.05] = np.finfo(np.float32).min
        g[r.random((T, H)) < 0.05] = -np.inf
    st = r.standard_normal((len(lens), H, K, V)).astype(np.float32) if state else None
    return q, k, v, g, st


def bounds(q, k, v, g, st, lens, scale, dtype, ref_o):
    o_abs, s_abs = tokens.linear_attention(np.abs(q), np.abs(k), np.abs(v), g, lens,
                                           None if st is None else np.abs(st), abs(scale))
    c = (max(lens) / 8 + 128 + q.shape[2]) * 2.0 ** -24
    to = c * o_abs
    if dtype == "bf16":
        to = to + 2.0 ** -8 * np.abs(ref_o) + (2.0 ** -8 + 2.0 ** -16) * (1 + 2.0 ** -8) * o_abs
    return to + 1e-37, c * s_abs + 1e-37


def check(name, got, ref, tol):
    err = np.abs(got - ref)
    worst = float(np.max(err / tol)) if err.size else 0.0
    print(f"[attention] {name}: worst error / tolerance {worst:.3f}", flush=True)
    assert np.all(err <= tol), (name, worst, np.argwhere(~(err <= tol))[:5].tolist())


CASES = [
    # lens, G, H, K, V: one token, chunk borders, empty and one-token sequences among others, odd sizes, every
    # padded key size, several value tiles, shared keys, segments (one long sequence, few heads)
    ([1], 1, 1, 1, 1),
    ([63], 1, 2, 32, 64),
    ([64], 2, 2, 33, 65),
    ([65], 1, 1, 64, 16),
    ([5, 0, 64, 1, 129, 0], 2, 4, 16, 32),
    ([200], 1, 3, 100, 40),
    ([40, 40, 40], 2, 2, 128, 128),
    ([150, 31], 1, 2, 256, 70),
    ([33], 1, 1, 7, 300),
    ([1100], 1, 1, 24, 24),
    ([700, 0, 300, 1, 513], 1, 2, 40, 130),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_prompts_match_oracle(case, dtype):
    lens, G, H, K, V = case
    print(f"[case] attention {case} {dtype}", flush=True)
    q, k, v, g, st = make(lens, G, H, K, V, dtype, seed=len(lens) * K + V)
    scale = K ** -0.5
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    o, last = _lib().linear_attention(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), state=_dev(st),
                                      cu_seqlens=cu, scale=scale, final_state=True)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention(q, k, v, g, lens, st, scale)
    to, ts = bounds(q, k, v, g, st, lens, scale, dtype, ref_o)
    check("o", _host(o), ref_o, to)
    check("state", _host(last), ref_s, ts)


# heads enough for tiles of 128 value columns: in several segments, of packed sequences too, and in one each
WIDE = [
    ([2560], 1, 64, 16, 128),
    ([2000, 0, 700], 2, 64, 16, 100),
    ([512, 512], 1, 160, 8, 128),
    ([150, 600], 1, 80, 200, 90),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_wide_tiles_match_oracle(case, dtype):
    test_prompts_match_oracle(case, dtype)


@pytest.mark.parametrize("decay", ["none", "strong", "far"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays(decay, dtype):
    """No decay at all, decays that leave a few tokens, and tokens that forget everything (lowest value, -Inf)."""
    lens = [300, 70]
    q, k, v, g, st = make(lens, 2, 4, 48, 40, dtype, seed=7, decay=decay)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    o, last = _lib().linear_attention(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), state=_dev(st),
                                      cu_seqlens=cu, final_state=True)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention(q, k, v, g, lens, st)
    to, ts = bounds(q, k, v, g, st, lens, 1.0, dtype, ref_o)
    check("o", _host(o), ref_o, to)
    check("state", _host(last), ref_s, ts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views_and_expanded_decay(dtype):
    """q, k, v as slices of one projection at an odd offset, heads before tokens, one decay per head (stride 0)."""
    S, L, G, H, K, V = 2, 150, 2, 4, 24, 40
    q, k, v, _, _ = make([L] * S, G, H, K, V, dtype, seed=8)
    row = np.concatenate([np.zeros((S * L, 1)), q.reshape(S * L, -1), k.reshape(S * L, -1)], 1)
    qk = _dev(row.reshape(S, L, -1), dtype)
    qd = qk[..., 1:1 + G * K].unflatten(-1, (G, K))
    kd = qk[..., 1 + G * K:].unflatten(-1, (G, K))
    vd = _dev(v.reshape(S, L, H, V).transpose(0, 2, 1, 3), dtype).transpose(1, 2)  # stored (S, H, L, V)
    gh = -np.linspace(0.01, 1, H).astype(np.float32)
    gd = _dev(gh).expand(S, L, H)
    o = _lib().linear_attention(qd, kd, vd, gd, scale=0.3)
    torch.cuda.synchronize()
    g = np.broadcast_to(gh, (S * L, H))
    ref, _ = tokens.linear_attention(q, k, v, g, [L] * S, None, 0.3)
    to, _ = bounds(q, k, v, g, None, [L] * S, 0.3, dtype, ref)
    check("o", _host(o).reshape(ref.shape), ref, to)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_outside_the_sequences_are_left_alone(dtype):
    """Packed tokens before the first and behind the last sequence hold NaN: neither read nor written."""
    lens, lead, tail = [70, 0, 9], 3, 40
    q, k, v, g, st = make(lens, 1, 2, 20, 24, dtype, seed=9)
    pad = [np.concatenate([np.full((lead,) + x.shape[1:], np.nan, np.float32), x,
                           np.full((tail,) + x.shape[1:], np.nan, np.float32)]) for x in (q, k, v, g)]
    cu = torch.tensor(lead + np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = torch.full(pad[2].shape, 7.0, dtype=DT[dtype], device="cuda")
    _lib().linear_attention(_dev(pad[0], dtype), _dev(pad[1], dtype), _dev(pad[2], dtype), _dev(pad[3]),
                            state=_dev(st), cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    got = _host(out)
    assert np.all(got[:lead] == 7) and np.all(got[-tail:] == 7)
    ref, _ = tokens.linear_attention(q, k, v, g, lens, st)
    to, _ = bounds(q, k, v, g, st, lens, 1.0, dtype, ref)
    check("o", got[lead:-tail], ref, to)


def test_tokens_far_apart():
    """Values 2^24 - 1 elements apart, the largest stride taken: offsets beyond 2^31 elements and 2^32 bytes."""
    T, H, K, V, far = 150, 2, 16, 40, 2 ** 24 - 1
    q, k, v, g, _ = make([T], 1, H, K, V, "bf16", seed=20)
    room = torch.empty((T - 1) * far + H * V, dtype=torch.bfloat16, device="cuda")
    vd = room.as_strided((1, T, H, V), (0, far, V, 1))
    vd.copy_(_dev(v, "bf16")[None])
    o = _lib().linear_attention(_dev(q, "bf16")[None], _dev(k, "bf16")[None], vd, _dev(g)[None])
    torch.cuda.synchronize()
    ref, _ = tokens.linear_attention(q, k, v, g, [T])
    to, _ = bounds(q, k, v, g, None, [T], 1.0, "bf16", ref)
    check("o", _host(o)[0], ref, to)


def test_wrong_cu_seqlens_stay_in_range():
    """Offsets beyond the tokens, negative or decreasing: clamped, so finite garbage at worst and a clean exit."""
    q, k, v, g, st = make([300], 1, 2, 16, 16, "f32", seed=10)
    for cu in ([0, 2 ** 31 - 1], [-5, 100, 50, 300], [300, 0, 300, 0], [-2 ** 31, -1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        o, last = _lib().linear_attention(_dev(q), _dev(k), _dev(v), _dev(g), cu_seqlens=c, final_state=True)
        torch.cuda.synchronize()
        assert last.shape[0] == len(cu) - 1


def test_prompt_in_pieces_equals_whole_and_steps():
    """A prompt cut anywhere, continued from the kept state, and its tokens one by one, agree with the whole."""
    T, G, H, K, V = 200, 2, 4, 64, 48
    q, k, v, g, _ = make([T], G, H, K, V, "f32", seed=11)
    d = [_dev(x)[None] for x in (q, k, v, g)]
    ss2d = _lib()
    whole, last = ss2d.linear_attention(*d, final_state=True)
    st, parts = None, []
    for a, b in ((0, 1), (1, 90), (90, 154), (154, T)):
        o, st = ss2d.linear_attention(*(x[:, a:b] for x in d), state=st, final_state=True)
        parts.append(o)
    cache = torch.zeros(3, H, K, V, device="cuda")
    idx = torch.full((T,), 1, dtype=torch.int32, device="cuda")
    steps = ss2d.linear_attention_step(*(x[0].contiguous() for x in d), cache, idx)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention(q, k, v, g, [T])
    to, ts = bounds(q, k, v, g, None, [T], 1.0, "f32", ref_o)
    check("whole", _host(whole)[0], ref_o, to)
    check("pieces", _host(torch.cat(parts, 1))[0], ref_o, to)
    check("steps", _host(steps), ref_o, to)
    check("state whole", _host(last), ref_s, ts)
    check("state pieces", _host(st), ref_s, ts)
    check("state steps", _host(cache)[1:2], ref_s, ts)
    assert not _host(cache)[[0, 2]].any()


def test_state_may_be_updated_in_place():
    q, k, v, g, st = make([600, 3], 1, 2, 32, 32, "f32", seed=12)
    ss2d = _lib()
    cu = torch.tensor([0, 600, 603], dtype=torch.int32).cuda()
    dev = [_dev(x) for x in (q, k, v, g)]
    o1, last = ss2d.linear_attention(*dev, state=_dev(st), cu_seqlens=cu, final_state=True)
    # the C entry takes state_out == state_in
    s = _dev(st)
    from selective_scan_crossscan_amd import tokens as T
    sizes, _, S, G, H, K, V, code = T._attention_sizes(*dev, cu)
    n = ss2d.lib().ss2d_linear_attention_workspace(sizes, 1, code)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o2 = torch.empty_like(o1)
    rc = ss2d.lib().ss2d_linear_attention(*(x.data_ptr() for x in dev), s.data_ptr(), cu.data_ptr(), o2.data_ptr(),
                                          s.data_ptr(), sizes, 1.0, code, ws.data_ptr(), n,
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(s, last)


# ------------------------------------------------------------------ single tokens
STEPS = [(1, 1, 1, 1, 1, 1), (3, 5, 2, 4, 16, 32), (2, 2, 1, 3, 100, 65), (40, 64, 2, 2, 128, 128), (5, 6, 1, 2, 256, 300),
         (300, 300, 1, 2, 24, 40), (700, 900, 1, 2, 8, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_steps_match_oracle(case, dtype):
    """Every row its own slot, in any order, with padding rows among them; untouched slots keep their bits."""
    rows, slots, G, H, K, V = case
    print(f"[case] step {case} {dtype}", flush=True)
    r = np.random.default_rng(rows + K)
    q, k, v, g, _ = make([rows], G, H, K, V, dtype, seed=rows + V)
    st = r.standard_normal((slots, H, K, V)).astype(np.float32)
    idx = r.permutation(slots)[:rows].astype(np.int32)
    if rows > 2:
        idx[1], idx[-1] = -1, slots  # padding
    sd = _dev(st)
    o = _lib().linear_attention_step(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), sd,
                                     torch.from_numpy(idx).cuda(), scale=0.5)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention_step(q, k, v, g, st, idx, 0.5)
    abs_o, abs_s = tokens.linear_attention_step(abs(q), abs(k), abs(v), g, abs(st), idx, 0.5)
    c = (K + 16) * 2.0 ** -24
    check("o", _host(o), ref_o, c * abs_o + (2.0 ** -8 * np.abs(ref_o) if dtype == "bf16" else 0) + 1e-37)
    check("state", _host(sd), ref_s, 8 * 2.0 ** -24 * abs_s + 1e-37)
    idle = np.setdiff1d(np.arange(slots), idx)
    assert np.array_equal(_host(sd)[idle], st[idle].astype(np.float64))


def test_step_rows_of_one_slot_run_in_order():
    r = np.random.default_rng(13)
    rows, slots, G, H, K, V = 300, 4, 1, 2, 32, 70
    q, k, v, g, _ = make([rows], G, H, K, V, "f32", seed=14)
    st = r.standard_normal((slots, H, K, V)).astype(np.float32)
    idx = r.integers(-1, slots + 1, rows).astype(np.int32)
    sd = _dev(st)
    o = _lib().linear_attention_step(_dev(q), _dev(k), _dev(v), _dev(g), sd, torch.from_numpy(idx).cuda())
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention_step(q, k, v, g, st, idx)
    abs_o, abs_s = tokens.linear_attention_step(abs(q), abs(k), abs(v), g, abs(st), idx)
    c = (rows + K + 16) * 2.0 ** -24
    check("o", _host(o), ref_o, c * abs_o + 1e-37)
    check("state", _host(sd), ref_s, c * abs_s + 1e-37)


def test_step_without_index_and_with_strided_rows():
    q, k, v, g, _ = make([5], 2, 4, 24, 32, "bf16", seed=15)
    st = np.random.default_rng(16).standard_normal((7, 4, 24, 32)).astype(np.float32)
    row = np.concatenate([q.reshape(5, -1), k.reshape(5, -1), v.reshape(5, -1)], 1)
    x = _dev(row, "bf16")
    qd, kd, vd = x[:, :48].view(5, 2, 24), x[:, 48:96].view(5, 2, 24), x[:, 96:].view(5, 4, 32)
    sd = _dev(st)
    o = _lib().linear_attention_step(qd, kd, vd, _dev(g), sd)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention_step(q, k, v, g, st, np.arange(5))
    abs_o, abs_s = tokens.linear_attention_step(abs(q), abs(k), abs(v), g, abs(st), np.arange(5))
    check("o", _host(o), ref_o, 40 * 2.0 ** -24 * abs_o + 2.0 ** -8 * np.abs(ref_o) + 1e-37)
    check("state", _host(sd), ref_s, 8 * 2.0 ** -24 * abs_s)
    assert np.array_equal(_host(sd)[5:], st[5:].astype(np.float64))


# ------------------------------------------------------------------ streams and graphs
def test_graph_replays_match_eager():
    """A captured prompt (in segments, with a workspace) and step, replayed with eager work between."""
    ss2d = _lib()
    q, k, v, g, st = make([1500], 1, 2, 64, 64, "bf16", seed=17)
    d = [_dev(x, "bf16")[None] for x in (q, k, v)] + [_dev(g)[None], _dev(st)]
    row = [x[0, :2].contiguous() for x in d[:4]]
    idx = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    cache0 = torch.randn(2, 2, 64, 64, device="cuda")
    eager, last = ss2d.linear_attention(*d[:4], state=d[4], final_state=True)
    c_eager = cache0.clone()
    s_eager = ss2d.linear_attention_step(*row, c_eager, idx)
    torch.cuda.synchronize()
    cache = cache0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, end = ss2d.linear_attention(*d[:4], state=d[4], final_state=True)
        s = ss2d.linear_attention_step(*row, cache, idx)
    for i in range(4):
        cache.copy_(cache0)
        o.zero_()
        other = ss2d.linear_attention(*(x[:, :700] for x in d[:4]), state=d[4])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager) and torch.equal(end, last), i
        assert torch.equal(s, s_eager) and torch.equal(cache, c_eager), i
        assert torch.isfinite(other.float()).all()


def test_two_streams_at_once():
    ss2d = _lib()
    sets = []
    for i in range(2):
        q, k, v, g, st = make([2000], 1, 2, 64, 64, "bf16", seed=18 + i)
        d = [_dev(x, "bf16")[None] for x in (q, k, v)] + [_dev(g)[None]]
        sets.append((d, ss2d.linear_attention(*d)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = []
    for _ in range(3):
        outs.append([ss2d.linear_attention(*d, stream=st) for (d, _), st in zip(sets, streams)])
    torch.cuda.synchronize()
    for pair in outs:
        for got, (_, want) in zip(pair, sets):
            assert torch.equal(got, want)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 4096, 4097, 9000])
def test_many_short_sequences(count):
    """Sequences of 0 to 3 tokens, and one of 600 among them: every one is found, its states its own."""
    r = np.random.default_rng(count)
    lens = r.integers(0, 4, count).tolist()
    lens[count * 2 // 3] = 600
    q, k, v, g, st = make(lens, 1, 2, 8, 12, "f32", seed=count + 1)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    o, last = _lib().linear_attention(_dev(q), _dev(k), _dev(v), _dev(g), state=_dev(st), cu_seqlens=cu, final_state=True)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention(q, k, v, g, lens, st)
    to, ts = bounds(q, k, v, g, st, lens, 1.0, "f32", ref_o)
    check("o", _host(o), ref_o, to)
    check("state", _host(last), ref_s, ts)


def test_step_rows_far_apart():
    """Rows of v 2^31 + 3 elements apart: offsets beyond 32 bits."""
    B, H, K, V, far = 3, 2, 16, 40, 2 ** 31 + 3
    q, k, v, g, _ = make([B], 1, H, K, V, "bf16", seed=31)
    st = np.random.default_rng(32).standard_normal((B, H, K, V)).astype(np.float32)
    room = torch.empty((B - 1) * far + H * V, dtype=torch.bfloat16, device="cuda")
    vd = room.as_strided((B, H, V), (far, V, 1))
    vd.copy_(_dev(v, "bf16"))
    sd = _dev(st)
    o = _lib().linear_attention_step(_dev(q, "bf16"), _dev(k, "bf16"), vd, _dev(g), sd)
    torch.cuda.synchronize()
    ref_o, ref_s = tokens.linear_attention_step(q, k, v, g, st, np.arange(B))
    abs_o, abs_s = tokens.linear_attention_step(abs(q), abs(k), abs(v), g, abs(st), np.arange(B))
    check("o", _host(o), ref_o, (K + 16) * 2.0 ** -24 * abs_o + 2.0 ** -8 * np.abs(ref_o) + 1e-37)
    check("state", _host(sd), ref_s, 8 * 2.0 ** -24 * abs_s)
