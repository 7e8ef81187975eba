"""Pins of the token-sequence oracle (oracle/tokens.py): closed forms, the quadratic
form of linear attention, splits of a sequence, and central differences."""
import numpy as np
import pytest

from oracle import tokens


def _inputs(seed, lens, G, H, K, V):
    r = np.random.default_rng(seed)
    T = sum(lens)
    return (r.standard_normal((T, G, K)), r.standard_normal((T, G, K)), r.standard_normal((T, H, V)),
            -r.exponential(0.5, (T, H)), r.standard_normal((len(lens), H, K, V)))


def test_attention_equals_the_quadratic_form():
    q, k, v, g, _ = _inputs(0, [9], 1, 2, 3, 4)
    o, _ = tokens.linear_attention(q, k, v, g, [9], scale=0.5)
    for h in range(2):
        for i in range(9):
            want = sum(0.5 * np.exp(g[j + 1:i + 1, h].sum()) * (q[i, 0] @ k[j, 0]) * v[j, h] for j in range(i + 1))
            np.testing.assert_allclose(o[i, h], want, rtol=1e-12, atol=1e-13)


def test_attention_without_decay_sums_and_with_full_decay_forgets():
    q, k, v, g, _ = _inputs(1, [6], 1, 1, 2, 2)
    o, last = tokens.linear_attention(q, k, v, 0 * g, [6])
    np.testing.assert_allclose(last[0, 0], np.einsum("tk,tv->kv", k[:, 0], v[:, 0]), rtol=1e-12)
    o, _ = tokens.linear_attention(q, k, v, np.full_like(g, -np.inf), [6])
    np.testing.assert_allclose(o[:, 0], (q[:, 0] * k[:, 0]).sum(-1)[:, None] * v[:, 0], rtol=1e-12)


def test_attention_continues_from_a_state_and_steps_equal_prompts():
    q, k, v, g, st = _inputs(2, [5, 0, 3], 2, 4, 3, 2)
    o, last = tokens.linear_attention(q, k, v, g, [5, 0, 3], st, 0.7)
    np.testing.assert_array_equal(last[1], st[1])
    _, mid = tokens.linear_attention(q[:2], k[:2], v[:2], g[:2], [2], st[:1], 0.7)
    o2, end = tokens.linear_attention(q[2:5], k[2:5], v[2:5], g[2:5], [3], mid, 0.7)
    np.testing.assert_allclose(o2, o[2:5], rtol=1e-12)
    np.testing.assert_allclose(end[0], last[0], rtol=1e-12)
    so, cache = tokens.linear_attention_step(q, k, v, g, st, [0] * 5 + [2] * 3, 0.7)
    np.testing.assert_allclose(so, o, rtol=1e-12)
    np.testing.assert_allclose(cache, last, rtol=1e-12)
    so, cache = tokens.linear_attention_step(q[:2], k[:2], v[:2], g[:2], st, [-1, 3], 0.7)
    assert not so.any()
    np.testing.assert_array_equal(cache, st)


@pytest.mark.parametrize("lens", [[1], [4, 0, 3]])
def test_attention_gradients_by_central_differences(lens):
    ins = list(_inputs(3, lens, 2, 4, 3, 2))
    r = np.random.default_rng(4)
    do, dl = r.standard_normal(ins[2].shape), r.standard_normal(ins[4].shape)

    def loss(q, k, v, g, st):
        o, last = tokens.linear_attention(q, k, v, g, lens, st, 0.6)
        return (o * do).sum() + (last * dl).sum()

    q, k, v, g, st = ins
    grads = tokens.linear_attention_backward(q, k, v, g, do, lens, st, dl, 0.6)
    for i, gr in enumerate(grads):
        num = np.zeros_like(gr)
        for at in np.ndindex(*gr.shape):
            d = []
            for e in (1e-5, -1e-5):
                x = [a.copy() for a in ins]
                x[i][at] += e
                d.append(loss(*x))
            num[at] = (d[0] - d[1]) / 2e-5
        # differences of 64-bit sums: step^2 of the third derivative and 1e-16 / 1e-5 of rounding
        np.testing.assert_allclose(gr, num, rtol=1e-7, atol=1e-7)


def test_norm_closed_form_and_gradients():
    y, r = tokens.rms_norm([[3.0, 4.0]], [2.0, 1.0], [[0.0, 0.0]], eps=0.0)
    np.testing.assert_allclose(y, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])
    np.testing.assert_array_equal(r, [[3.0, 4.0]])
    rg = np.random.default_rng(5)
    x, w, dy, dr = (rg.standard_normal(s) for s in ((3, 5), (5,), (3, 5), (3, 5)))
    dx, dw = tokens.rms_norm_backward(x, w, dy, dr, 1e-3)

    def loss(x, w):
        return (tokens.rms_norm(x, w, None, 1e-3)[0] * dy).sum() + (x * dr).sum()

    for got, arr, which in ((dx, x, 0), (dw, w, 1)):
        for at in np.ndindex(*arr.shape):
            d = []
            for e in (1e-5, -1e-5):
                a = [x.copy(), w.copy()]
                a[which][at] += e
                d.append(loss(*a))
            assert abs(got[at] - (d[0] - d[1]) / 2e-5) <= 1e-7 * (1 + abs(got[at]))


def test_e4m3_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.linspace(-448, 448, 4001), np.geomspace(1e-4, 448, 4001), np.arange(0, 64) * 2.0 ** -11,
                        [17.0, 19.0, 0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(tokens.round_e4m3(x), want)


def test_block_scales_and_product():
    y = np.zeros((2, 130))
    y[0, 5], y[0, 129] = -896.0, 44.8
    np.testing.assert_allclose(tokens.block_scales(y), [[2.0, 0.1], [2.0 ** -126] * 2])
    rg = np.random.default_rng(6)
    a, b = rg.standard_normal((3, 200)), rg.standard_normal((150, 200))
    sa, sb = rg.uniform(1, 2, (3, 2)), rg.uniform(1, 2, (2, 2))
    out = tokens.matmul_fp8(a, sa, b, sb)
    want = sum(a[2, k] * sa[2, k // 128] * b[140, k] * sb[1, k // 128] for k in range(200))
    np.testing.assert_allclose(out[2, 140], want, rtol=1e-12)


def test_torch_reference_is_the_oracle():
    """tests/token_reference.py, which the tests of long sequences use, against the oracle: both in 64 bits."""
    torch = pytest.importorskip("torch")
    import token_reference
    r = np.random.default_rng(9)
    lens, G, H, K, V = [5, 0, 7], 2, 4, 3, 6
    T = sum(lens)
    q, k, v, do = (r.standard_normal((T, n, d)) for n, d in ((G, K), (G, K), (H, V), (H, V)))
    g, st, dl = -r.random((T, H)), r.standard_normal((3, H, K, V)), r.standard_normal((3, H, K, V))
    t = [torch.from_numpy(x) for x in (q, k, v, g)]
    for s, d in ((st, dl), (None, None)):
        s_, d_ = (None if x is None else torch.from_numpy(x) for x in (s, d))
        for a, b in zip(token_reference.attention(*t, lens, s_, 0.3), tokens.linear_attention(q, k, v, g, lens, s, 0.3)):
            np.testing.assert_allclose(a.numpy(), b, rtol=1e-12, atol=1e-12)
        for a, b in zip(token_reference.attention_backward(*t, torch.from_numpy(do), lens, s_, d_, 0.3),
                        tokens.linear_attention_backward(q, k, v, g, do, lens, s, d, 0.3)):
            np.testing.assert_allclose(a.numpy(), b, rtol=1e-12, atol=1e-12)
