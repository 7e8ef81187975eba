"""Pins of the delta rule's oracle (oracle/delta.py): closed forms, the triangular system of the errors, splits of a
sequence, the rotation, and central differences."""
import numpy as np
import pytest

from oracle import delta, tokens


def _inputs(seed, lens, G, H, K, V):
    r = np.random.default_rng(seed)
    T = sum(lens)
    return (r.standard_normal((T, G, K)), r.standard_normal((T, G, K)), r.standard_normal((T, H, V)),
            -r.exponential(0.5, (T, H)), r.uniform(0, 1, (T, H)), r.standard_normal((len(lens), H, K, V)))


def test_orthonormal_keys_are_linear_attention():
    """Keys orthogonal to each other and to the state: nothing to replace, beta v is added."""
    K = 5
    q, _, v, g, b, _ = _inputs(0, [K], 1, 2, K, 3)
    k = np.eye(K)[:, None]
    o, last = delta.delta_rule(q, k, v, g, b, [K], scale=0.5)
    want_o, want = tokens.linear_attention(q, k, v * b[..., None], g, [K], scale=0.5)
    np.testing.assert_allclose(o, want_o, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(last, want, rtol=1e-12, atol=1e-13)


def test_unit_key_with_beta_one_stores_the_value_and_beta_zero_only_decays():
    q, k, v, g, _, st = _inputs(1, [1], 1, 1, 4, 3)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    _, last = delta.delta_rule(q, k, v, g, np.ones((1, 1)), [1], st)
    np.testing.assert_allclose(k[0, 0] @ last[0, 0], v[0, 0], rtol=1e-12)
    _, last = delta.delta_rule(q, k, v, g, np.zeros((1, 1)), [1], st)
    np.testing.assert_allclose(last, np.exp(g[0, 0]) * st, rtol=1e-12)


def test_errors_solve_the_triangular_system():
    n = 7
    q, k, v, g, b, st = _inputs(2, [n], 1, 1, 3, 2)
    _, last = delta.delta_rule(q, k, v, g, b, [n], st)
    k, G, b = k[:, 0], np.cumsum(g[:, 0]), b[:, 0]
    L = np.tril(np.exp(G[:, None] - G) * (k @ k.T), -1)
    E = np.linalg.solve(np.eye(n) + L * b, v[:, 0] - np.exp(G)[:, None] * (k @ st[0, 0]))
    want = np.exp(G[-1]) * st[0, 0] + (k * (np.exp(G[-1] - G) * b)[:, None]).T @ E
    np.testing.assert_allclose(last[0, 0], want, rtol=1e-11, atol=1e-12)


def test_continues_from_a_state_and_steps_equal_prompts():
    q, k, v, g, b, st = _inputs(3, [5, 0, 3], 2, 4, 3, 2)
    o, last = delta.delta_rule(q, k, v, g, b, [5, 0, 3], st, 0.7)
    np.testing.assert_array_equal(last[1], st[1])
    _, mid = delta.delta_rule(q[:2], k[:2], v[:2], g[:2], b[:2], [2], st[:1], 0.7)
    o2, end = delta.delta_rule(q[2:5], k[2:5], v[2:5], g[2:5], b[2:5], [3], mid, 0.7)
    np.testing.assert_allclose(o2, o[2:5], rtol=1e-12)
    np.testing.assert_allclose(end[0], last[0], rtol=1e-12)
    so, cache = delta.delta_rule_step(q, k, v, g, b, st, [0] * 5 + [2] * 3, 0.7)
    np.testing.assert_allclose(so, o, rtol=1e-12)
    np.testing.assert_allclose(cache, last, rtol=1e-12)
    so, cache = delta.delta_rule_step(q[:2], k[:2], v[:2], g[:2], b[:2], st, [-1, 3], 0.7)
    assert not so.any()
    np.testing.assert_array_equal(cache, st)


@pytest.mark.parametrize("lens", [[1], [4, 0, 3]])
def test_gradients_by_central_differences(lens):
    ins = list(_inputs(4, lens, 2, 4, 3, 2))
    r = np.random.default_rng(5)
    do, dl = r.standard_normal(ins[2].shape), r.standard_normal(ins[5].shape)

    def loss(q, k, v, g, b, st):
        o, last = delta.delta_rule(q, k, v, g, b, lens, st, 0.6)
        return (o * do).sum() + (last * dl).sum()

    q, k, v, g, b, st = ins
    grads = delta.delta_rule_backward(q, k, v, g, b, do, lens, st, dl, 0.6)
    for i, d in enumerate(grads):
        u = r.standard_normal(d.shape)
        vals = []
        for e in (1e-5, -1e-5):
            arg = list(ins)
            arg[i] = ins[i] + e * u
            vals.append(loss(*arg))
        np.testing.assert_allclose((d * u).sum(), (vals[0] - vals[1]) / 2e-5, rtol=1e-6, atol=1e-7)


def test_terms_bound_the_outputs():
    q, k, v, g, b, st = _inputs(6, [9, 3], 1, 2, 3, 4)
    o, last = delta.delta_rule(q, k, v, g, b, [9, 3], st, 0.5)
    terms, mass = delta.delta_rule_terms(q, k, v, g, b, [9, 3], st, 0.5, chunk=4)
    assert np.all(np.abs(o) <= terms * (1 + 1e-12))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    _, last = delta.delta_rule(q, k, v, g, b, [9, 3], st, 0.5)
    _, mass = delta.delta_rule_terms(q, k, v, g, b, [9, 3], st, 0.5, chunk=4)
    assert np.all(np.linalg.norm(last, axis=2) <= mass * (1 + 1e-12))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_the_distance_alone(interleaved):
    r = np.random.default_rng(7)
    rot, D = 6, 8
    rate = 10.0 ** -np.arange(rot // 2)
    table = np.concatenate([np.cos(np.arange(50)[:, None] * rate), np.sin(np.arange(50)[:, None] * rate)], -1)
    x, y = r.standard_normal((2, 1, 1, D))
    dots = [(delta.rotate(x, table, [p], interleaved) * delta.rotate(y, table, [p + 5], interleaved)).sum()
            for p in (0, 11, 44)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)
    z = delta.rotate(x, table, [7], interleaved)
    np.testing.assert_allclose(delta.rotate(z, table, [7], interleaved, back=True), x, rtol=1e-12)
    np.testing.assert_array_equal(z[..., rot:], x[..., rot:])
    first = [0, 1] if interleaved else [0, 3]
    np.testing.assert_allclose(z[0, 0, first[0]], x[0, 0, first[0]] * np.cos(7) - x[0, 0, first[1]] * np.sin(7))


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_by_central_differences(interleaved):
    r = np.random.default_rng(8)
    T, H, D, rot = 3, 2, 7, 4
    x, dy, w = r.standard_normal((T, H, D)), r.standard_normal((T, H, D)), r.uniform(0.5, 1.5, D)
    angle = r.uniform(0, 6, (10, rot // 2))
    table, pos = np.concatenate([np.cos(angle), np.sin(angle)], -1), [3, 0, 9]
    dx, dw = delta.head_norm_backward(x, dy, w, table, pos, interleaved, 1e-3)
    f = lambda x, w: (delta.head_norm(x, w, table, pos, interleaved, 1e-3) * dy).sum()  # noqa: E731
    u, z = r.standard_normal(x.shape), r.standard_normal(D)
    np.testing.assert_allclose((dx * u).sum(), (f(x + 1e-5 * u, w) - f(x - 1e-5 * u, w)) / 2e-5, rtol=1e-7)
    np.testing.assert_allclose((dw * z).sum(), (f(x, w + 1e-5 * z) - f(x, w - 1e-5 * z)) / 2e-5, rtol=1e-7)
