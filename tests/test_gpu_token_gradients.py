"""Gradients of the token-sequence operators along themselves, and chained through norm and attention.

Differences.  Along the unit vector u of a gradient the loss changes by |gradient| per unit: a step that moves the
point by 2^-9 of its size changes it by so much times (1 + O(2^-18)), the third derivative's share (the loss is a
polynomial of the point and exponentials of the decays times sums of order 1), and fp32's rounding of the outputs,
2^-24 of each of their terms at random, is under 1e-4 of that change.  So 1e-3 of |gradient| holds, and not for
a gradient whose error along itself is a few parts in a thousand: a factor, or a missing term.  u is the gradient's
direction with as much of a random one added.

Chain.  The gradients that arrive at the norm are off by at most (c + 3 C) |.|: c the attention's bound for fp32, and
C = 64 2^-24 the norm's for each of the up to three factors of a term that the norm's output is; these errors pass the
norm's gradient, whose own bound is C times its terms.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import token_reference

C = 64 * 2.0 ** -24
EPS = 1e-5


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _normal(*shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _along(loss, x, grad, seed):
    """(difference quotient, gradient's product) along grad with noise of its size, for a step of 2^-9 of x's size."""
    u = grad.double() / grad.double().norm()
    n = _normal(*x.shape, seed=seed).double()
    u = u + n / n.norm()
    u /= u.norm()
    step = 2.0 ** -9 * float(x.double().norm())
    points = [(x.double() + s * step * u).to(x.dtype) for s in (1, -1)]
    size = float(((points[0].double() - points[1].double()) * u).sum())  # what the rounded points are apart
    return (loss(points[0]) - loss(points[1])) / size, float((grad.double() * u).sum())


def _check(name, num, got, grad):
    size = float(grad.double().norm())
    print(f"[gradients] {name}: {got:.6f} {num:.6f} of {size:.6f}", flush=True)
    assert abs(num - got) <= 1e-3 * size, name


def _attention_inputs(S, L, G, H, K, V):
    q, k, v, do = (_normal(S, L, n, d, seed=i) for i, (n, d) in enumerate(((G, K), (G, K), (H, V), (H, V))))
    g = -torch.exp(_normal(S, L, H, seed=5) - 1.5)
    return q, k, v, g, do, _normal(S, H, K, V, seed=6), _normal(S, H, K, V, seed=7)


@pytest.mark.parametrize("shape", [(1, 150, 2, 4, 20, 24), (1, 700, 1, 2, 64, 130)], ids=lambda s: "-".join(map(str, s)))
def test_attention_along_its_gradients(shape):
    ss2d = _lib()
    q, k, v, g, do, st, dl = _attention_inputs(*shape)
    args = dict(q=q, k=k, v=v, log_decay=g, state=st)
    scale = shape[4] ** -0.5
    grads = ss2d.linear_attention_backward(q, k, v, g, do, state=st, dfinal_state=dl, scale=scale)

    def loss(name, x):
        o, last = ss2d.linear_attention(**dict(args, **{name: x}), scale=scale, final_state=True)
        return float((o.double() * do.double()).sum() + (last.double() * dl.double()).sum())

    for i, (name, x) in enumerate(args.items()):
        grad = grads["d" + name]
        num, got = _along(lambda p: loss(name, p), x, grad, seed=10 + i)
        _check(name, num, got, grad)


@pytest.mark.parametrize("dim", [59, 414, 2048])
def test_norm_along_its_gradients(dim):
    ss2d = _lib()
    x, res, dy, dr = (_normal(200, dim, seed=20 + i) for i in range(4))
    w = 1 + 0.3 * _normal(dim, seed=24)
    y, r = ss2d.rms_norm(x, w, residual=res, eps=EPS)
    grads = ss2d.rms_norm_backward(r, w, dy, dresidual=dr, eps=EPS)

    def loss(x, w):
        y, r = ss2d.rms_norm(x, w, residual=res, eps=EPS)
        return float((y.double() * dy.double()).sum() + (r.double() * dr.double()).sum())

    _check("x", *_along(lambda p: loss(p, w), x, grads["dx"], seed=25), grads["dx"])
    _check("weight", *_along(lambda p: loss(x, p), w, grads["dweight"], seed=26), grads["dweight"])


def test_chained_gradients_match_the_definition():
    """loss = sum(o do), o = attention(split(norm(x + res))): the kernels' chain against the definitions' in 64 bits,
    element by element."""
    ss2d = _lib()
    S, L, G, H, K, V = 2, 150, 2, 6, 16, 32
    width = 2 * G * K + H * V
    x, res = (_normal(S, L, width, seed=30 + i) for i in range(2))
    w = 1 + 0.3 * _normal(width, seed=32)
    g, do = -torch.exp(_normal(S, L, H, seed=33) - 1.5), _normal(S, L, H, V, seed=34)

    def split(y):
        q, k, v = y.split([G * K, G * K, H * V], -1)
        return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))

    y, total = ss2d.rms_norm(x, w, residual=res, eps=EPS)
    a = ss2d.linear_attention_backward(*split(y), g, do, scale=0.25)
    dy = torch.cat([a["dq"].flatten(-2), a["dk"].flatten(-2), a["dv"].flatten(-2)], -1)
    n = ss2d.rms_norm_backward(total, w, dy, eps=EPS)
    torch.cuda.synchronize()

    def flat(t):
        return t.reshape(S * L, *t.shape[2:])

    # the definitions in 64 bits, and the same on absolute values
    r = x.double() + res.double()
    rstd = 1 / (r.square().mean(-1, keepdim=True) + EPS).sqrt()
    xhat = r * rstd
    exact = xhat * w.double()

    def attention(y, do):
        grads = token_reference.attention_backward(*(flat(t) for t in split(y)), flat(g), flat(do), [L] * S, scale=0.25)
        return torch.cat([t.flatten(1) for t in grads[:3]], -1).view(S, L, width), grads[3].view(S, L, H)

    dy_ref, dg_ref = attention(exact, do)
    dy_abs, dg_abs = attention(exact.abs(), do.abs())
    gy = dy_ref * w.double()
    dx_ref = rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
    dw_ref = (dy_ref * xhat).sum((0, 1))

    def terms(d):  # the norm's gradient on absolute values
        gy = d * w.double().abs()
        return rstd * (gy + xhat.abs() * (gy * xhat.abs()).mean(-1, keepdim=True))

    c = (L / 8 + 256 + K + V) * 2.0 ** -24 + 3 * C
    bound = terms(c * dy_abs) + C * terms(dy_abs)
    assert bool(((n["dx"].double() - dx_ref).abs() <= bound).all())
    bound = ((c + C + (S * L + 64) * 2.0 ** -24) * dy_abs * xhat.abs()).sum((0, 1))
    assert bool(((n["dweight"].double() - dw_ref).abs() <= bound).all())
    own = 0.25 * (split(exact)[0] * split(exact)[1]).abs().sum(-1).repeat_interleave(H // G, -1) * (do * split(exact)[2]).abs().sum(-1)
    near = torch.nn.functional.max_pool1d((dg_abs + own).transpose(1, 2), 127, stride=1, padding=63).transpose(1, 2)
    assert bool(((a["dlog_decay"].double() - dg_ref).abs() <= 2 * c * near).all())
