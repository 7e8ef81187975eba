"""GPU parity of the root-mean-square norm (ss2d_rms_norm, its 8-bit form and its
gradients) against the float64 oracle in oracle/tokens.py.

Tolerances.  The sum of squares has only positive terms, added in fp32 by at most
8 x 2 terms per thread, 6 steps in a wave and 16 across waves, so the norm is off by
less than 64 half steps of 2^-24 with the root, the division and the two products.
Dots (gradients) are bounded the same way against the sum of their terms' absolute
values.  An output rounded to bf16 is off by 2^-8 of itself more, one rounded to
e4m3 by 2^-4 of itself or half the smallest step, 2^-10 (times the block's scale).
"""
import numpy as np
import pytest

from oracle import tokens
import ss2d_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
C = 64 * 2.0 ** -24
EPS = 1e-5


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _case(rows, dim, dtype, seed):
    r = np.random.default_rng(seed)
    spread = np.exp(r.normal(0, 1, dim))
    a = [(r.standard_normal((rows, dim)) * spread).astype(np.float32) for _ in range(4)]
    if dtype == "bf16":
        a = [ss2d_inputs.round_to_bf16(x) for x in a]
    return (*a, r.uniform(0.5, 1.5, dim).astype(np.float32))


def _dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype]).cuda()


def _host(t):
    return t.double().cpu().numpy()


def _half(x, dtype):
    return np.abs(x) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)


# every workgroup shape (one wave, 4, 8, 16 waves, two passes of 16), ragged ends of a thread's
# eight channels, of a block of 128 and of a wave, one channel, odd counts of rows
SHAPES = [(1, 1), (3, 7), (5, 128), (9, 130), (2, 511), (4, 512), (3, 520), (7, 1000), (2, 2048), (3, 2049), (2, 4096),
          (1, 5000), (2, 8192), (1, 8200), (2, 16384), (1, 16383), (600, 96)]
# several rows of a wave, and a last group with fewer
SHAPES += [(20001, 8), (9000, 59), (17000, 64), (9001, 65), (5003, 128), (5000, 129), (4999, 250), (3001, 256), (3000, 257)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_matches_oracle(shape, dtype):
    print(f"[case] norm {shape} {dtype}", flush=True)
    x, res, _, _, w = _case(*shape, dtype, seed=sum(shape))
    ss2d = _lib()
    y, r = ss2d.rms_norm(_dev(x, dtype), _dev(w), residual=_dev(res, dtype), eps=EPS)
    y0 = ss2d.rms_norm(_dev(x, dtype), eps=EPS)
    torch.cuda.synchronize()
    ry, rr = tokens.rms_norm(x, w, res, EPS)
    # the sum's own rounding, 2^-24 of it, is inside C
    assert np.all(np.abs(_host(r) - rr) <= _half(rr, dtype) + 2.0 ** -24 * np.abs(rr))
    assert np.all(np.abs(_host(y) - ry) <= C * np.abs(ry) + _half(ry, dtype) * (1 + C))
    ry0, _ = tokens.rms_norm(x, None, None, EPS)
    assert np.all(np.abs(_host(y0) - ry0) <= C * np.abs(ry0) + _half(ry0, dtype) * (1 + C))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_fp8_matches_oracle(shape, dtype):
    print(f"[case] norm fp8 {shape} {dtype}", flush=True)
    x, res, _, _, w = _case(*shape, dtype, seed=sum(shape) + 1)
    q, s, r = _lib().rms_norm_fp8(_dev(x, dtype), _dev(w), residual=_dev(res, dtype), eps=EPS)
    torch.cuda.synchronize()
    ry, rr = tokens.rms_norm(x, w, res, EPS)
    rs = tokens.block_scales(ry)
    s, q = _host(s), _host(q)
    assert np.all(np.abs(s - rs) <= C * rs)
    assert np.all(np.abs(_host(r) - rr) <= _half(rr, dtype) + 2.0 ** -24 * np.abs(rr))
    per = np.repeat(s, 128, 1)[:, :shape[1]]
    step = np.maximum(np.abs(ry) * 2.0 ** -4, per * 2.0 ** -10)
    assert np.all(np.abs(q * per - ry) <= step * (1 + 1e-4) + C * np.abs(ry))
    # away from a rounding border (2 C of the value) the stored value is the nearest one exactly
    lo, hi = tokens.round_e4m3(ry / per * (1 - 2 * C)), tokens.round_e4m3(ry / per * (1 + 2 * C))
    same = lo == hi
    assert same.mean() > 0.99 or same.size < 200
    assert np.array_equal(q[same], lo[same])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + [(5000, 64), (1500, 2048)], ids=lambda s: "x".join(map(str, s)))
def test_norm_gradients_match_oracle(shape, dtype):
    print(f"[case] norm backward {shape} {dtype}", flush=True)
    x, dy, dr, _, w = _case(*shape, dtype, seed=sum(shape) + 2)
    ss2d = _lib()
    g = ss2d.rms_norm_backward(_dev(x, dtype), _dev(w), _dev(dy, dtype), dresidual=_dev(dr, dtype), eps=EPS)
    g0 = ss2d.rms_norm_backward(_dev(x, dtype), None, _dev(dy, dtype), eps=EPS)
    torch.cuda.synchronize()
    assert set(g0) == {"dx"}
    for got, wt, d in ((g["dx"], w, dr), (g0["dx"], None, None)):
        ref, _ = tokens.rms_norm_backward(x, wt, dy, d, EPS)
        rstd = 1 / np.sqrt((x.astype(np.float64) ** 2).mean(1, keepdims=True) + EPS)
        gy = np.abs(dy * (1 if wt is None else wt))
        terms = rstd * (gy + np.abs(x * rstd) * (gy * np.abs(x * rstd)).mean(1, keepdims=True))
        terms = terms + (0 if d is None else np.abs(d))
        assert np.all(np.abs(_host(got) - ref) <= C * terms + _half(ref, dtype) * (1 + C))
    _, dw = tokens.rms_norm_backward(x, w, dy, None, EPS)
    xh = np.abs(x / np.sqrt((x.astype(np.float64) ** 2).mean(1, keepdims=True) + EPS))
    # a column's sum runs over the rows of a workgroup, then over 16 ranges of workgroups
    bound = (shape[0] + 64) * 2.0 ** -24 * (np.abs(dy) * xh).sum(0)
    assert np.all(np.abs(_host(g["dweight"]) - dw) <= bound)


def test_norm_in_place():
    """residual_out may be the residual (the usual stream update), out may be x; same bits as out of place."""
    x, res, _, _, w = _case(33, 700, "bf16", seed=4)
    ss2d = _lib()
    y, r = ss2d.rms_norm(_dev(x, "bf16"), _dev(w), residual=_dev(res, "bf16"))
    xd, rd = _dev(x, "bf16"), _dev(res, "bf16")
    y2, r2 = ss2d.rms_norm(xd, _dev(w), residual=rd, out=xd, residual_out=rd)
    torch.cuda.synchronize()
    assert y2 is xd and r2 is rd and torch.equal(y, xd) and torch.equal(r, rd)


def test_norm_special_rows():
    """Zeros give zeros (8-bit: the least scale); a NaN or an infinity stays inside its row."""
    ss2d = _lib()
    x = np.random.default_rng(5).standard_normal((4, 300)).astype(np.float32)
    x[0] = 0
    x[2, 17] = np.nan
    x[3, 5] = np.inf
    y = _host(ss2d.rms_norm(_dev(x)))
    q, s = ss2d.rms_norm_fp8(_dev(x))
    torch.cuda.synchronize()
    assert not y[0].any() and not _host(q)[0].any() and np.all(_host(s)[0] == 2.0 ** -126)
    ref, _ = tokens.rms_norm(x[1], None, None, 1e-6)
    assert np.all(np.abs(y[1] - ref) <= (C + 2.0 ** -24) * np.abs(ref))
    assert np.isnan(y[2]).all() and np.isnan(_host(q)[2]).all()
    assert np.isnan(y[3, 5]) and not y[3, :5].any()


def test_norm_graph_replays_match_eager():
    ss2d = _lib()
    x, dy, dr, _, w = _case(200, 1024, "bf16", seed=6)
    d = [_dev(a, "bf16") for a in (x, dy, dr)]
    wd = _dev(w)
    y, s, r = ss2d.rms_norm_fp8(d[0], wd, residual=d[1])
    g = ss2d.rms_norm_backward(d[0], wd, d[1], dresidual=d[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2, r2 = ss2d.rms_norm_fp8(d[0], wd, residual=d[1])
        g2 = ss2d.rms_norm_backward(d[0], wd, d[1], dresidual=d[2])
    for _ in range(3):
        g2["dweight"].zero_()
        ss2d.rms_norm_backward(d[0], wd, d[2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2.view(torch.uint8), y.view(torch.uint8)) and torch.equal(s2, s) and torch.equal(r2, r)
        assert torch.equal(g2["dx"], g["dx"]) and torch.equal(g2["dweight"], g["dweight"])


@pytest.mark.parametrize("dim", [5, 59, 414, 1001, 8191, 9001])
def test_ragged_rows_in_place(dim):
    """Rows whose ends are loaded together with what lies before them, written over their own inputs."""
    ss2d = _lib()
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, r, dy, dr = (torch.randn(301, dim, generator=g, device="cuda").bfloat16() for _ in range(4))
    w = torch.rand(dim, generator=g, device="cuda")
    y, s = ss2d.rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    ss2d.rms_norm(x1, w, residual=r1, out=x1, residual_out=r1)
    x2, r2 = x.clone(), r.clone()
    ss2d.rms_norm(x2, w, residual=r2, out=r2, residual_out=x2)
    want = ss2d.rms_norm_backward(s, w, dy, dresidual=dr)
    L = ss2d.lib()
    n = L.ss2d_rms_norm_backward_workspace(301, dim, ss2d.SS2D_BF16)
    ws, dw = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(dim, device="cuda")
    for over in (0, 1):
        a, b = dy.clone(), dr.clone()
        rc = L.ss2d_rms_norm_backward(s.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(), 1e-6,
                                      (a, b)[over].data_ptr(), dw.data_ptr(), 301, dim, ss2d.SS2D_BF16, ws.data_ptr(), n,
                                      torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal((a, b)[over], want["dx"]) and torch.equal(dw, want["dweight"])
    torch.cuda.synchronize()
    assert torch.equal(x1, y) and torch.equal(r1, s) and torch.equal(r2, y) and torch.equal(x2, s)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_fp8_small_blocks(dtype, weighted):
    """Blocks of 128 whose largest value is 2^-145 .. 2^-95, zeros among them, beside one that sets the row's rstd (about
    140): the definition's values and scales, no NaN from a quotient past fp32's range.  Inputs under 2^-126 are exact;
    what the tolerances allow is that of test_norm_fp8_matches_oracle."""
    ss2d = _lib()
    r = np.random.default_rng(8)
    rows, dim = 51, 300
    x = np.zeros((rows, dim), np.float32)
    x[:, :128] = 0.01 * r.choice([-1, 1], (rows, 128))
    for i in range(rows):
        small = np.ldexp(r.uniform(-1, 1, dim - 128), -145 + i).astype(np.float32)
        small[r.random(dim - 128) < 0.2] = 0
        x[i, 128:] = small
    if dtype == "bf16":
        x = ss2d_inputs.round_to_bf16(x)
    w = r.uniform(0.5, 1.5, dim).astype(np.float32) if weighted else None
    q, s = ss2d.rms_norm_fp8(_dev(x, dtype), None if w is None else _dev(w), eps=1e-12)
    torch.cuda.synchronize()
    ry, _ = tokens.rms_norm(x, w, None, 1e-12)
    rs = tokens.block_scales(ry)
    s, q = _host(s), _host(q)
    assert np.isfinite(q).all() and not q[ry == 0].any()
    assert np.all(np.abs(s - rs) <= C * rs)
    per = np.repeat(s, 128, 1)[:, :dim]
    lo, hi = tokens.round_e4m3(ry / per * (1 - 2 * C)), tokens.round_e4m3(ry / per * (1 + 2 * C))
    same = lo == hi
    assert same.mean() > 0.99
    assert np.array_equal(q[same], lo[same])
