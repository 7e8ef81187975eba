"""The token-sequence operators run together, as a layer of a language model uses them:
residual and norm into 8 bits, the projection to queries, keys and values, linear
attention over a packed batch of prompts, norm and projection back, then single tokens
on the kept states.  Every stage is held to the float64 oracle on the values that really
entered it, with the tolerance of its own test; and the gradients of a norm before the
attention to differences of the two forwards.
"""
import numpy as np
import pytest

from oracle import tokens
from test_gpu_attention import _dev, _host, bounds, check
from test_gpu_matmul_fp8 import _check as check_product
from test_gpu_norm import C, EPS

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, G, H, K, V = 192, 2, 6, 16, 32  # 192 channels: six heads of 32 values, keys of 16 shared by three heads
WIDTH = 2 * G * K + H * V


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _weights(rng, n, k):
    q = tokens.round_e4m3(np.clip(rng.standard_normal((n, k)) * 100, -448, 448)).astype(np.float32)
    s = (np.exp(rng.normal(0, 0.3, (-(-n // 128), -(-k // 128)))) / (100 * np.sqrt(k))).astype(np.float32)
    return torch.from_numpy(q).cuda().to(torch.float8_e4m3fn), torch.from_numpy(s).cuda()


class Layer:
    def __init__(self):
        r = np.random.default_rng(41)
        self.w_in, self.s_in = _weights(r, WIDTH, D)
        self.w_out, self.s_out = _weights(r, D, H * V)
        self.norm1, self.norm2 = (_dev(r.uniform(0.5, 1.5, n).astype(np.float32)) for n in (D, H * V))
        self.decay = -np.exp(r.uniform(-4, 0, H)).astype(np.float32)

    def project(self, x, residual):
        """Checked: residual, norm in 8 bits, projection; returns q, k, v views and the new residual."""
        ss2d = _lib()
        y, s, res = ss2d.rms_norm_fp8(x, self.norm1, residual=residual, eps=EPS)
        ry, _ = tokens.rms_norm(_host(x), _host(self.norm1), _host(residual), EPS)
        per = np.repeat(_host(s), 128, 1)[:, :D]
        err = np.abs(_host(y) * per - ry)
        assert np.all(err <= np.maximum(np.abs(ry) * 2.0 ** -4, per * 2.0 ** -10) * (1 + 1e-4) + C * np.abs(ry))
        row = ss2d.matmul_fp8(y, s, self.w_in, self.s_in)
        check_product(row, (_host(y), _host(s), _host(self.w_in), _host(self.s_in)), "bf16", "projection in")
        q, k, v = row.split([G * K, G * K, H * V], -1)
        return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V)), res

    def out(self, o):
        ss2d = _lib()
        y, s = ss2d.rms_norm_fp8(o.flatten(-2), self.norm2, eps=EPS)
        out = ss2d.matmul_fp8(y, s, self.w_out, self.s_out)
        check_product(out, (_host(y), _host(s), _host(self.w_out), _host(self.s_out)), "bf16", "projection out")
        return out


def test_prompts_then_single_tokens():
    ss2d = _lib()
    layer = Layer()
    r = np.random.default_rng(42)
    lens = [70, 0, 1, 333]
    T = sum(lens)
    x, res = (_dev(r.standard_normal((T, D)).astype(np.float32), "bf16") for _ in range(2))
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    q, k, v, _ = layer.project(x, res)
    g = _dev(layer.decay).expand(T, H)
    scale = K ** -0.5
    o, last = ss2d.linear_attention(q, k, v, g, cu_seqlens=cu, scale=scale, final_state=True)
    args = [_host(t) for t in (q, k, v)] + [np.broadcast_to(layer.decay, (T, H))]
    ref_o, ref_s = tokens.linear_attention(*args, lens, None, scale)
    to, ts = bounds(*args, None, lens, scale, "bf16", ref_o)
    check("prompt o", _host(o), ref_o, to)
    check("prompt state", _host(last), ref_s, ts)
    assert layer.out(o).shape == (T, D)
    # the prompts' states move into a cache with free slots between, then five tokens each, one row padding
    cache = torch.zeros(9, H, K, V, device="cuda")
    slots = torch.tensor([4, 0, 7, 2], dtype=torch.int32).cuda()
    cache[slots.long()] = last
    index = torch.cat([slots, torch.tensor([-1], dtype=torch.int32).cuda()])
    for n in range(5):
        x, res = (_dev(r.standard_normal((5, D)).astype(np.float32), "bf16") for _ in range(2))
        q, k, v, _ = layer.project(x, res)
        before = _host(cache)
        g1 = _dev(layer.decay).expand(5, H).contiguous()
        o = ss2d.linear_attention_step(q, k, v, g1, cache, index, scale=scale)
        args = [_host(t) for t in (q, k, v)] + [np.broadcast_to(layer.decay, (5, H))]
        idx = index.cpu().numpy()
        ref_o, ref_s = tokens.linear_attention_step(*args, before, idx, scale)
        abs_o, abs_s = tokens.linear_attention_step(*(np.abs(a) for a in args[:3]), args[3], np.abs(before), idx, scale)
        check(f"token {n} o", _host(o), ref_o, (K + 16) * 2.0 ** -24 * abs_o + 2.0 ** -8 * np.abs(ref_o) + 1e-37)
        check(f"token {n} state", _host(cache), ref_s, 8 * 2.0 ** -24 * abs_s + 1e-37)
        assert layer.out(o).shape == (5, D)


def test_gradients_through_norm_and_attention():
    """loss = sum(o do), o = attention(split(norm(x + res))): the chained gradients against central differences of the
    chained forwards along random directions, in fp32."""
    ss2d = _lib()
    r = np.random.default_rng(43)
    S, L = 2, 150
    x, res = (_dev(r.standard_normal((S, L, WIDTH)).astype(np.float32)) for _ in range(2))
    w = _dev(r.uniform(0.5, 1.5, WIDTH).astype(np.float32))
    g = _dev(-np.exp(r.uniform(-4, 0, (S, L, H))).astype(np.float32))
    do = _dev(r.standard_normal((S, L, H, V)).astype(np.float32))

    def split(y):
        q, k, v = y.split([G * K, G * K, H * V], -1)
        return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))

    def forward(x, w, g):
        y, total = ss2d.rms_norm(x, w, residual=res, eps=EPS)
        return ss2d.linear_attention(*split(y), g, scale=0.25), y, total

    _, y, total = forward(x, w, g)
    a = ss2d.linear_attention_backward(*split(y), g, do, scale=0.25)
    dy = torch.cat([a["dq"].flatten(-2), a["dk"].flatten(-2), a["dv"].flatten(-2)], -1)
    n = ss2d.rms_norm_backward(total, w, dy, eps=EPS)
    for name, at, grad in (("x", 0, n["dx"]), ("weight", 1, n["dweight"]), ("decay", 2, a["dlog_decay"])):
        base = [x, w, g]
        u = _dev(r.standard_normal(base[at].shape).astype(np.float32))
        vals = []
        for e in (2e-3, -2e-3):
            arg = list(base)
            arg[at] = base[at] + e * u
            vals.append(float((forward(*arg)[0].double() * do.double()).sum()))
        num, got = (vals[0] - vals[1]) / 4e-3, float((grad.double() * u.double()).sum())
        size = float(grad.double().norm() * u.double().norm())
        print(f"[layer] d{name}: {got:.6f} {num:.6f}", flush=True)
        # the step's square times the third derivative, and fp32 rounding of the loss over the step
        assert abs(got - num) <= 2e-3 * size
