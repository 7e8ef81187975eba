"""Token-sequence operators at sizes whose workgroups' threads pass 2^32, the most that one axis
of a launch takes.  A row (a sequence, a head) does not depend on the others, so each call is held
to smaller calls of the same operator, whose values the other tests check: bit for bit where the
same kernel does the same arithmetic, else to the definition with the bounds of those tests."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _tiled(x, rows):
    """rows rows that repeat those of x."""
    out = torch.empty((rows,) + x.shape[1:], dtype=x.dtype, device=x.device)
    for i in range(0, rows, len(x)):
        out[i:i + len(x)] = x[:rows - i]
    return out


def _repeats(big, small):
    """big's rows repeat small's, bit for bit."""
    big, small = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (big, small))
    n, whole = len(small), len(big) // len(small)
    return (bool((big[:whole * n].view(whole, *small.shape) == small).all())
            and torch.equal(big[whole * n:], small[:len(big) - whole * n]))


# rows of 8 threads each, of a workgroup of 256 each, of 1024
@pytest.mark.parametrize("rows,dim", [((1 << 29) + 5, 1), ((1 << 24) + 3, 520), ((1 << 22) + 1, 8200)],
                         ids=lambda n: str(n))
def test_norm_rows(rows, dim):
    ss2d = _lib()
    x, r = (_randn((1 << 29) // dim // 512, dim, seed=i, dtype=torch.bfloat16) for i in (1, 2))
    want = ss2d.rms_norm(x, residual=r)
    xs, rs = _tiled(x, rows), _tiled(r, rows)
    ss2d.rms_norm(xs, residual=rs, out=xs, residual_out=rs)
    torch.cuda.synchronize()
    assert _repeats(xs, want[0]) and _repeats(rs, want[1])


def test_norm_fp8_rows():
    ss2d = _lib()
    x = _randn(1 << 20, 1, seed=3, dtype=torch.bfloat16)
    want = ss2d.rms_norm_fp8(x)
    got = ss2d.rms_norm_fp8(_tiled(x, (1 << 28) + 7))
    torch.cuda.synchronize()
    assert _repeats(got[0], want[0]) and _repeats(got[1], want[1])


def test_steps():
    """65535 rows of 272 heads: 2^24 workgroups of 256 threads."""
    ss2d = _lib()
    B, H = 65535, 272
    q, k = (_randn(B, 1, 1, seed=i) for i in (4, 5))
    v, g, state = _randn(B, H, 1, seed=6), -_randn(B, H, seed=7).abs(), _randn(B, H, 1, 1, seed=8)
    parts = state.clone()
    half = B // 2
    want = [ss2d.linear_attention_step(q[a:b], k[a:b], v[a:b], g[a:b], parts[a:b]) for a, b in ((0, half), (half, B))]
    got = ss2d.linear_attention_step(q, k, v, g, state)
    torch.cuda.synchronize()
    assert torch.equal(got, torch.cat(want)) and torch.equal(state, parts)


def test_prompts():
    """2^20 sequences of one token and 17 heads."""
    ss2d = _lib()
    S, H, K, V = (1 << 20) + 3, 17, 8, 8
    q, k, v = (_randn(S, 1, n, 8, seed=9 + n, dtype=torch.bfloat16) for n in (1, 1, H))
    g, state = -_randn(S, 1, H, seed=30).abs(), _randn(S, H, K, V, seed=31)
    o, last = ss2d.linear_attention(q, k, v, g, state=state, final_state=True)
    for a in range(0, S, 1 << 18):
        part = slice(a, min(S, a + (1 << 18)))
        wo, wl = ss2d.linear_attention(q[part], k[part], v[part], g[part], state=state[part], final_state=True)
        torch.cuda.synchronize()
        assert torch.equal(o[part], wo) and torch.equal(last[part], wl)


def _short_and_long(S, long, H, K, V, seed):
    """S - 1 packed sequences of one token and a long one behind them, fp32."""
    T = S - 1 + long
    q, k, v = (_randn(T, n, d, seed=seed + i) for i, (n, d) in enumerate(((1, K), (1, K), (H, V))))
    g, state = -0.1 * _randn(T, H, seed=seed + 3).abs(), _randn(S, H, K, V, seed=seed + 4)
    cu = torch.cat([torch.arange(S), torch.tensor([T])]).to(torch.int32).cuda()
    return q, k, v, g, state, cu


def test_packed_prompts_of_several_segments():
    """State passes and carries of 2^20 sequences, the last of which is cut; it is held to itself alone."""
    ss2d = _lib()
    S, long, H, K, V = 1 << 20, 100000, 17, 8, 8
    q, k, v, g, state, cu = _short_and_long(S, long, H, K, V, seed=40)
    o, last = ss2d.linear_attention(q, k, v, g, state=state, cu_seqlens=cu, final_state=True)
    n = S - 1
    h = state[:n].double() * g[:n].double().exp()[..., None, None] + k[:n, :, :, None].double() * v[:n, :, None, :].double()
    mag = (state[:n].abs() * g[:n].exp()[..., None, None] + k[:n, :, :, None].abs() * v[:n, :, None, :].abs()).double()
    c = (1 / 8 + 128 + K) * 2.0 ** -24
    assert bool(((last[:n] - h).abs() <= c * mag + 1e-37).all())
    q1 = q[:n, 0].double()
    assert bool(((o[:n] - torch.einsum("tk,thkv->thv", q1, h)).abs()
                 <= c * torch.einsum("tk,thkv->thv", q1.abs(), mag) + 1e-37).all())
    del h, mag
    tail = [x[n:][None] for x in (q, k, v, g)]
    alone = ss2d.linear_attention(*tail, state=state[n:], final_state=True)
    size = ss2d.linear_attention(*(x.abs() for x in tail[:3]), tail[3], state=state[n:].abs(), final_state=True)
    c = 2 * (long / 8 + 128 + K) * 2.0 ** -24  # two results, each within c of the definition
    for got, want, m in zip((o[n:][None], last[n:]), alone, size):
        assert bool(((got - want).abs() <= c * 1.1 * m + 1e-37).all())


def test_packed_gradients_of_several_segments():
    """The carries both ways of 32769 sequences: 2^24 workgroups. Single tokens to the formula, the long sequence to
    itself alone."""
    ss2d = _lib()
    S, long, H, K, V = (1 << 15) + 1, 20000, 16, 64, 64
    q, k, v, g, state, cu = _short_and_long(S, long, H, K, V, seed=50)
    do, dl = _randn(*v.shape, seed=60), _randn(*state.shape, seed=61)
    got = ss2d.linear_attention_backward(q, k, v, g, do, state=state, dfinal_state=dl, cu_seqlens=cu)
    torch.cuda.synchronize()
    n = S - 1
    c = (1 / 8 + 256 + K + V) * 2.0 ** -24

    def single(q, k, v, g, do, state, dl):
        """Gradients of sequences of one token, in 64 bits."""
        q, k, v, g, do, state, dl = (x.double() for x in (q[:, 0], k[:, 0], v, g, do, state, dl))
        a = g.exp()[..., None, None]
        h = a * state + k[:, None, :, None] * v[:, :, None, :]
        d = dl + q[:, None, :, None] * do[:, :, None, :]
        return {"dq": torch.matmul(h, do[..., None])[..., 0].sum(1, keepdim=True),
                "dk": torch.matmul(d, v[..., None])[..., 0].sum(1, keepdim=True),
                "dv": torch.matmul(k[:, None, None, :], d)[:, :, 0], "dlog_decay": (a * state * d).sum((-1, -2)),
                "dstate": a * d}

    for a in range(0, n, 4096):
        part = slice(a, min(n, a + 4096))
        x = [t[part] for t in (q, k, v, g, do, state, dl)]
        want = single(*x)
        mag = single(*(t if i == 3 else t.abs() for i, t in enumerate(x)))
        for name in want:
            near = mag[name]
            if name == "dlog_decay":  # the token's own term enters the row and the column sums
                near = near + (x[0] * x[1]).abs().sum(-1).double() * (x[4] * x[2]).abs().sum(-1).double()
                near = 2 * near
            assert bool(((got[name][part] - want[name]).abs() <= c * near + 1e-37).all()), name
    # the long one, in other segments: either result is within c of the definition's terms
    c = 2 * (long / 8 + 256 + K + V) * 2.0 ** -24
    tail = [x[n:][None] for x in (q, k, v, g, do)]
    kw = dict(state=state[n:], dfinal_state=dl[n:])
    alone = ss2d.linear_attention_backward(*tail, **kw)
    size = ss2d.linear_attention_backward(*(x if i == 3 else x.abs() for i, x in enumerate(tail)),
                                          **{name: t.abs() for name, t in kw.items()})
    torch.cuda.synchronize()
    for name in ("dq", "dk", "dv", "dstate"):
        err = (got[name][n:].reshape(alone[name].shape) - alone[name]).abs()
        assert bool((err <= c * 1.1 * size[name] + 1e-37).all()), name
