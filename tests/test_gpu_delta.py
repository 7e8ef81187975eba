"""GPU parity of the gated delta rule (ss2d_delta_rule, _step) against the float64 oracle in oracle/delta.py; the
tolerances are derived in delta_reference.py."""
import numpy as np
import pytest

from delta_reference import check, check_forward, make, unit, values
from oracle import delta

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DT[dtype]).cuda()


def _host(t):
    return t.double().cpu().numpy()


def _cu(lens, lead=0):
    return torch.tensor(lead + np.cumsum([0] + lens), dtype=torch.int32).cuda()


def packed(args, lens, dtype, scale=1.0, **kw):
    q, k, v, g, b, st = args
    out = _lib().delta_rule(_dev(q, dtype), _dev(k, dtype), _dev(v, dtype), _dev(g), _dev(b),
                            state=None if st is None else _dev(st), cu_seqlens=_cu(lens), scale=scale,
                            final_state=True, **kw)
    torch.cuda.synchronize()
    return out


CASES = [
    # lens, G, H, K, V: one token, chunk borders, empty and one-token sequences among others, odd sizes, every padded
    # key size, several value tiles, shared keys, segments (long sequences, few heads)
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
    ([900], 1, 1, 130, 20),
    ([800], 1, 2, 100, 3),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_prompts_match_oracle(case, dtype):
    lens, G, H, K, V = case
    print(f"[case] delta {case} {dtype}", flush=True)
    args = make(lens, G, H, K, V, dtype, seed=len(lens) * K + V)
    o, last = packed(args, lens, dtype, K ** -0.5)
    check_forward("prompts", _host(o), _host(last), args, lens, K ** -0.5, dtype)


@pytest.mark.parametrize("decay", ["none", "strong", "far"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays(decay, dtype):
    """No decay at all, decays that leave a few tokens, and tokens that forget everything (lowest value, -Inf)."""
    lens = [300, 70]
    args = make(lens, 2, 4, 48, 40, dtype, seed=7, decay=decay)
    o, last = packed(args, lens, dtype)
    check_forward(decay, _host(o), _host(last), args, lens, 1.0, dtype)


@pytest.mark.parametrize("keys", ["same", "zero"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_hard_systems(keys, dtype):
    """The same key again and again with beta 1, and beta and keys of 0."""
    lens = [600, 3, 64]
    args = make(lens, 1, 2, 32, 24, dtype, seed=8, decay="none" if keys == "same" else "mixed", keys=keys)
    o, last = packed(args, lens, dtype)
    check_forward(keys, _host(o), _host(last), args, lens, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_lengths_strided_views_and_expanded_rates(dtype):
    """q, k, v as slices of one projection at an odd offset, heads before tokens, one decay and one beta per head."""
    S, L, G, H, K, V = 2, 150, 2, 4, 24, 40
    q, k, v, _, _, _ = make([L] * S, G, H, K, V, dtype, seed=9)
    row = np.concatenate([np.zeros((S * L, 1)), q.reshape(S * L, -1), k.reshape(S * L, -1)], 1)
    qk = _dev(row.reshape(S, L, -1), dtype)
    qd = qk[..., 1:1 + G * K].unflatten(-1, (G, K))
    kd = qk[..., 1 + G * K:].unflatten(-1, (G, K))
    vd = _dev(v.reshape(S, L, H, V).transpose(0, 2, 1, 3), dtype).transpose(1, 2)  # stored (S, H, L, V)
    gh, bh = -np.linspace(0.01, 1, H).astype(np.float32), np.linspace(0.2, 1, H).astype(np.float32)
    o = _lib().delta_rule(qd, kd, vd, _dev(gh).expand(S, L, H), _dev(bh).expand(S, L, H), scale=0.3)
    torch.cuda.synchronize()
    args = (q, k, v, np.broadcast_to(gh, (S * L, H)), np.broadcast_to(bh, (S * L, H)), None)
    check_forward("strided", _host(o).reshape(v.shape), None, args, [L] * S, 0.3, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_outside_the_sequences_are_left_alone(dtype):
    """Packed tokens before the first and behind the last sequence hold NaN: neither read nor written."""
    lens, lead, tail = [70, 0, 9], 3, 40
    args = make(lens, 1, 2, 20, 24, dtype, seed=10)
    pad = [np.concatenate([np.full((lead,) + x.shape[1:], np.nan, np.float32), x,
                           np.full((tail,) + x.shape[1:], np.nan, np.float32)]) for x in args[:5]]
    out = torch.full(pad[2].shape, 7.0, dtype=DT[dtype], device="cuda")
    _lib().delta_rule(*(_dev(x, dtype) for x in pad[:3]), _dev(pad[3]), _dev(pad[4]), state=_dev(args[5]),
                      cu_seqlens=_cu(lens, lead), out=out)
    torch.cuda.synchronize()
    got = _host(out)
    assert np.all(got[:lead] == 7) and np.all(got[-tail:] == 7)
    check_forward("inside", got[lead:-tail], None, args, lens, 1.0, dtype)


def test_wrong_cu_seqlens_stay_in_range():
    """Offsets beyond the tokens, negative or decreasing: clamped, so garbage at worst and a clean exit."""
    args = make([1000], 1, 2, 16, 16, "f32", seed=11)
    ss2d = _lib()
    d = [_dev(x) for x in args[:5]]
    for cu in ([0, 2 ** 31 - 1], [-5, 100, 50, 300], [1000, 0, 1000, 0], [-2 ** 31, -1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        o, last = ss2d.delta_rule(*d, cu_seqlens=c, final_state=True)
        torch.cuda.synchronize()
        assert last.shape[0] == len(cu) - 1


def test_prompt_in_pieces_equals_whole_and_steps():
    """A prompt cut anywhere, continued from the kept state, and its tokens one by one, agree with the whole."""
    T, G, H, K, V = 200, 2, 4, 64, 48
    args = make([T], G, H, K, V, "f32", seed=12, state=False)
    d = [_dev(x)[None] for x in args[:5]]
    ss2d = _lib()
    whole, last = ss2d.delta_rule(*d, final_state=True)
    st, parts = None, []
    for a, b in ((0, 1), (1, 90), (90, 154), (154, T)):
        o, st = ss2d.delta_rule(*(x[:, a:b] for x in d), state=st, final_state=True)
        parts.append(o)
    cache = torch.zeros(3, H, K, V, device="cuda")
    idx = torch.full((T,), 1, dtype=torch.int32, device="cuda")
    steps = ss2d.delta_rule_step(*(x[0].contiguous() for x in d), cache, idx)
    torch.cuda.synchronize()
    check_forward("whole", _host(whole)[0], _host(last), args, [T], 1.0, "f32")
    check_forward("pieces", _host(torch.cat(parts, 1))[0], _host(st), args, [T], 1.0, "f32")
    check_forward("steps", _host(steps), _host(cache)[1:2], args, [T], 1.0, "f32")
    assert not _host(cache)[[0, 2]].any()


@pytest.mark.parametrize("lens", [[1000, 3], [40, 3]])
def test_state_may_be_updated_in_place(lens):
    """state_out over state_in through the C ABI, in one segment and in several."""
    import ctypes

    args = make(lens, 1, 2, 32, 32, "f32", seed=13)
    ss2d = _lib()
    d = [_dev(x) for x in args]
    o, last = packed(args, lens, "f32")
    T, H, V, K = sum(lens), 2, 32, 32
    sizes = (ctypes.c_int64 * 24)(len(lens), T, 1, H, K, V, 0, K, K, 0, K, K, 0, H * V, V, 0, H, 1, 0, 0, 0, 0, H, 1)
    L = ss2d.lib()
    n = L.ss2d_delta_rule_workspace(sizes, 1, 0)
    ws, out, cu = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(d[2]), _cu(lens)
    rc = L.ss2d_delta_rule(*(x.data_ptr() for x in d), cu.data_ptr(), out.data_ptr(), d[5].data_ptr(), sizes, 1.0, 0,
                           ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(d[5], last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (3, 2, 4, 33, 5), (5, 1, 2, 128, 128), (7, 3, 3, 256, 66),
                                  (130, 2, 4, 64, 70), (40, 8, 16, 100, 128)], ids=str)
def test_steps_match_oracle(case, dtype):
    """Single tokens: slots in any order, padding rows, rows of one slot in order, strided rows."""
    B, G, H, K, V = case
    r = np.random.default_rng(B + K)
    slots = B + 3
    q, k, v, g, b, st = make([1] * slots, G, H, K, V, dtype, seed=B)
    q, k, v, g, b = (np.resize(x, (B,) + x.shape[1:]) for x in (q, k, v, g, b))
    idx = r.permutation(slots)[:B].astype(np.int32)
    if B > 2:
        idx[2] = idx[0]
        idx[-1] = [slots, -1][B % 2]
    row = _dev(np.concatenate([q.reshape(B, -1), k.reshape(B, -1), v.reshape(B, -1)], 1), dtype)
    parts = row.split([G * K, G * K, H * V], 1)
    cache = _dev(st)
    o = _lib().delta_rule_step(parts[0].unflatten(-1, (G, K)), parts[1].unflatten(-1, (G, K)),
                               parts[2].unflatten(-1, (H, V)), _dev(g), _dev(b), cache, torch.from_numpy(idx).cuda(),
                               scale=0.5)
    torch.cuda.synchronize()
    ref_o, ref_s = delta.delta_rule_step(q, k, v, g, b, st, idx, 0.5)
    n = 2 * (K + 16)  # two sums over K, one after the other, for rows of the same slot twice
    size = np.linalg.norm(st, axis=2).max() + np.abs(v).max() * 2
    check("step state", _host(cache), ref_s, size, n)
    ab = np.repeat(np.linalg.norm(q, axis=-1), H // G, 1)[..., None] * 0.5 * size
    err = np.abs(_host(o) - ref_o)
    tol = 2 * n * 2.0 ** -24 * ab + (2.0 ** -8 * np.abs(ref_o) if dtype == "bf16" else 0)
    assert np.all(err <= tol)
    if B > 2:
        assert not _host(o)[-1].any()


def test_results_do_not_depend_on_the_workspace_or_on_other_sequences():
    lens = [333, 64, 700]
    args = make(lens, 2, 4, 64, 64, "bf16", seed=14)
    first = packed(args, lens, "bf16")
    torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")  # NaN into what the allocator hands out next
    again = packed(args, lens, "bf16")
    assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_captured_calls_replay():
    """Two captures with their own workspaces, prompts and steps, replayed with eager work between."""
    ss2d = _lib()
    sets = []
    for seed in (15, 16):
        args = make([600], 1, 2, 64, 64, "bf16", seed=seed, state=False)
        d = [_dev(x, "bf16" if i < 3 else "f32")[None] for i, x in enumerate(args[:5])]
        want = ss2d.delta_rule(*d, final_state=True)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ss2d.delta_rule(*d, final_state=True)
        sets.append((g, out, want, d))
    for _ in range(3):
        for g, out, want, d in sets:
            for x in out:
                x.fill_(float("nan"))
            g.replay()
        ss2d.delta_rule(*sets[0][3])
        torch.cuda.synchronize()
        for g, out, want, d in sets:
            assert all(torch.equal(x, y) for x, y in zip(out, want))
