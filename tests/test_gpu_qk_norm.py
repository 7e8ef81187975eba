"""GPU parity of the norms of queries and keys with the position rotation (ss2d_qk_norm, _backward) against the float64
oracle in oracle/delta.py, element by element.

Tolerances.  The sum of D squares is off by at most (D/8 + 8) half steps of 2^-24, its root's reciprocal by half of that
and three more, an output by four more (norm, weight, two products and a sum of the rotation), of the pair's absolute
values; a bf16 output adds 2^-8 of itself.  A gradient has two such sums, and its weight's is a sum over the rows of one
workgroup's part (at most 1 + rows / 1024 in order for 2048 workgroups) and of the parts.
"""
import numpy as np
import pytest

from oracle import delta
from test_gpu_delta import _dev, _host, _lib
from delta_reference import values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-5


def _table(rows, rot, seed=0):
    angle = np.arange(rows)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


def _half(D):
    return (D / 8 + 24) * 2.0 ** -24


def pair_size(y, rot, interleaved):
    """|a| + |b| of each channel's pair (|y| of those that do not turn)."""
    a, b = delta._pairs(rot, interleaved)
    out = np.abs(y)
    out[..., a] = out[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out


def check_out(name, got, x, w, table, pos, inter, dtype):
    ref = delta.head_norm(x, w, table, pos, inter, EPS)
    flat = delta.head_norm(x, w, None, None, False, EPS)
    size = pair_size(flat, table.shape[1], inter) if table is not None else np.abs(flat)
    tol = 2 * _half(x.shape[-1]) * size + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + 1e-37
    worst = float(np.max(np.abs(got - ref) / tol))
    print(f"[qk] {name}: worst error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1, (name, worst)


def check_grad(name, dx, dw, x, dy, w, table, pos, inter, dtype):
    ref, refw = delta.head_norm_backward(x, dy, w, table, pos, inter, EPS)
    D = x.shape[-1]
    back = delta.rotate(dy, table, pos, inter, back=True) if table is not None else np.asarray(dy, np.float64)
    size = pair_size(np.asarray(dy, np.float64), table.shape[1], inter) if table is not None else np.abs(back)
    rstd = 1 / np.sqrt((np.asarray(x, np.float64) ** 2).mean(-1, keepdims=True) + EPS)
    xhat = np.abs(x) * rstd
    gy = size if w is None else size * np.abs(w)
    terms = rstd * (gy + xhat * (gy * xhat).mean(-1, keepdims=True))
    tol = 4 * _half(D) * terms + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + 1e-37
    worst = float(np.max(np.abs(dx - ref) / tol))
    print(f"[qk] {name}: worst error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1, (name, worst)
    if dw is not None:
        rows = x.shape[0] * x.shape[1]
        c = 2 * _half(D) + (rows / 1024 + 8 + 64 + 32) * 2.0 ** -24
        worst = float(np.max(np.abs(dw - refw) / (c * (size * xhat).sum((0, 1)) + 1e-37)))
        print(f"[qk] {name} weight: worst error / tolerance {worst:.3f}", flush=True)
        assert worst <= 1, (name, worst)


CASES = [
    # T, Hq, Hk, D, rotated, interleaved
    (1, 1, 1, 1, 0, False),
    (1, 1, 1, 2, 2, True),
    (3, 2, 1, 24, 10, True),
    (5, 3, 2, 24, 10, False),
    (7, 4, 4, 64, 64, False),
    (9, 16, 4, 128, 128, False),
    (33, 5, 1, 100, 100, False),
    (8, 2, 2, 255, 30, True),
    (6, 2, 1, 256, 256, False),
    (4, 1, 3, 250, 250, False),
    (11, 2, 2, 13, 6, False),
    (700, 6, 2, 96, 48, False),
    (3000, 2, 1, 32, 0, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norms_and_gradients_match_oracle(case, dtype):
    T, Hq, Hk, D, rot, inter = case
    print(f"[case] qk {case} {dtype}", flush=True)
    r = np.random.default_rng(T + D)
    # queries, keys and values as one projection leaves them, at an odd offset
    row = values(np.exp(r.standard_normal((T, 1))) * r.standard_normal((T, 1 + (Hq + 2 * Hk) * D)), dtype)
    x = {"q": row[:, 1:1 + Hq * D].reshape(T, Hq, D), "k": row[:, 1 + Hq * D:1 + (Hq + Hk) * D].reshape(T, Hk, D)}
    wq, wk = (r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    if T == 5:
        wk = None
    table = _table(50, rot) if rot else None
    pos = r.integers(0, 50, T).astype(np.int32)
    if T > 3:
        pos[:4] = [-3, 50, 2 ** 31 - 1, -2 ** 31]  # clamped
    rd = _dev(row, dtype)
    qd = rd[:, 1:1 + Hq * D].unflatten(-1, (Hq, D))
    kd = rd[:, 1 + Hq * D:1 + (Hq + Hk) * D].unflatten(-1, (Hk, D))
    extra = dict(rotation=None if table is None else _dev(table), interleaved=inter, eps=EPS,
                 positions=None if table is None else torch.from_numpy(pos).cuda())
    wd = [None if w is None else _dev(w) for w in (wq, wk)]
    q, k = _lib().qk_norm(qd, kd, *wd, **extra)
    dy = {n: values(r.standard_normal(x[n].shape), dtype) for n in "qk"}
    out = _lib().qk_norm_backward(qd, kd, _dev(dy["q"], dtype), _dev(dy["k"], dtype), *wd, **extra)
    torch.cuda.synchronize()
    assert ("dk_weight" in out) == (wk is not None)
    for n, y, w in (("q", q, wq), ("k", k, wk)):
        check_out(n, _host(y), x[n], w, table, pos, inter, dtype)
        dw = out.get(f"d{n}_weight")
        check_grad(n, _host(out["d" + n]), None if dw is None else _host(dw), x[n], dy[n], w, table, pos, inter, dtype)
    # over the inputs, as slices of one row: the values' part stays as it was
    before = rd.clone()
    _lib().qk_norm(qd, kd, *wd, out=(qd, kd), **extra)
    torch.cuda.synchronize()
    assert torch.equal(qd, q) and torch.equal(kd, k)
    assert torch.equal(rd[:, 1 + (Hq + Hk) * D:], before[:, 1 + (Hq + Hk) * D:]) and torch.equal(rd[:, :1], before[:, :1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_heads_first_and_default_positions(dtype):
    """(S, L) leading axes with heads before tokens in memory, positions counted in each sequence, repeated gradients."""
    S, L, Hq, Hk, D, rot = 3, 20, 4, 2, 40, 40
    r = np.random.default_rng(1)
    x = {n: values(r.standard_normal((S, h, L, D)), dtype) for n, h in (("q", Hq), ("k", Hk))}
    table = _table(L, rot)
    d = {n: _dev(x[n], dtype).transpose(1, 2) for n in "qk"}
    q, k = _lib().qk_norm(d["q"], d["k"], rotation=_dev(table), eps=EPS)
    dy = values(r.standard_normal((Hq, D)), dtype)
    grads = _lib().qk_norm_backward(d["q"], d["k"], _dev(dy, dtype).expand(S, L, Hq, D),
                                    _dev(dy[:Hk], dtype).expand(S, L, Hk, D), rotation=_dev(table), eps=EPS)
    torch.cuda.synchronize()
    pos = np.tile(np.arange(L), S)
    for n, y, h in (("q", q, Hq), ("k", k, Hk)):
        flat = x[n].transpose(0, 2, 1, 3).reshape(S * L, h, D)
        check_out(n, _host(y).reshape(flat.shape), flat, None, table, pos, False, dtype)
        check_grad(n, _host(grads["d" + n]).reshape(flat.shape), None, flat, np.broadcast_to(dy[:h], flat.shape), None,
                   table, pos, False, dtype)


def test_zeros_and_unit_keys():
    """A head of zeros gives zeros (eps keeps the root off 0), and a weight of D^-0.5 unit length."""
    D = 64
    x = torch.randn(5, 2, D, device="cuda")
    x[0] = 0
    q, k = _lib().qk_norm(x, x.clone(), k_weight=torch.full((D,), D ** -0.5, device="cuda"), eps=0.0 + 1e-12)
    torch.cuda.synchronize()
    assert not q[0].any() and torch.allclose(k[1:].norm(dim=-1), torch.ones(4, 2, device="cuda"), atol=1e-6)


def test_captured_calls_replay():
    ss2d = _lib()
    q, k = torch.randn(300, 4, 64, device="cuda"), torch.randn(300, 2, 64, device="cuda")
    w, t = torch.rand(64, device="cuda"), ss2d.rotation_table(300, 64)
    f = lambda: [*ss2d.qk_norm(q, k, w, w, rotation=t), *ss2d.qk_norm_backward(q, k, q, k, w, w, rotation=t).values()]  # noqa: E731
    want = f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    for _ in range(3):
        for x in out:
            x.fill_(float("nan"))
        g.replay()
        f()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
