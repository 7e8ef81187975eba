"""The token-sequence operators in numpy float64.  TEST INFRASTRUCTURE ONLY: only
the test suite may import this module.  The HIP library never calls it and shares
no code with it.

Linear attention with a decay per head, token by token (S sequences as a list of
lengths, tokens packed one sequence after another):
    h_t = exp(g_t) h_{t-1} + k_t v_t',   o_t = scale h_t' q_t;
its gradients by the chain rule along the same recurrence; the root-mean-square
norm with the residual's addition, its 8-bit form and its gradients; the 8-bit
matrix product with a scale per block of 128.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
BLOCK = 128


def _f64(*xs):
    return [None if x is None else np.asarray(x, dtype=np.float64) for x in xs]


def linear_attention(q, k, v, g, lens, state=None, scale=1.0):
    """q, k (T,G,K), v (T,H,V), g (T,H), state (S,H,K,V) or None -> o (T,H,V), final states."""
    q, k, v, g, state = _f64(q, k, v, g, state)
    H, V = v.shape[1:]
    K = q.shape[2]
    rep = H // q.shape[1]
    o = np.zeros_like(v)
    last = np.zeros((len(lens), H, K, V)) if state is None else state.copy()
    t = 0
    for s, n in enumerate(lens):
        for _ in range(n):
            qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
            last[s] = np.exp(g[t])[:, None, None] * last[s] + kt[:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", qt, last[s])
            t += 1
    return o, last


def linear_attention_backward(q, k, v, g, do, lens, state=None, dlast=None, scale=1.0):
    """Gradients dq, dk, dv, dg, dstate of sum(o do) + sum(last dlast)."""
    q, k, v, g, do, state, dlast = _f64(q, k, v, g, do, state, dlast)
    H, V = v.shape[1:]
    G, K = q.shape[1:]
    rep = H // G
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g)
    dstate = np.zeros((len(lens), H, K, V))
    t0 = 0
    for s, n in enumerate(lens):
        h = [np.zeros((H, K, V)) if state is None else state[s]]
        for t in range(t0, t0 + n):
            kt = np.repeat(k[t], rep, 0)
            h.append(np.exp(g[t])[:, None, None] * h[-1] + kt[:, :, None] * v[t][:, None, :])
        d = np.zeros((H, K, V)) if dlast is None else dlast[s].copy()
        for i in range(n - 1, -1, -1):
            t = t0 + i
            qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
            d = d + scale * qt[:, :, None] * do[t][:, None, :]
            dq[t] = (scale * np.einsum("hkv,hv->hk", h[i + 1], do[t])).reshape(G, rep, K).sum(1)
            dk[t] = np.einsum("hkv,hv->hk", d, v[t]).reshape(G, rep, K).sum(1)
            dv[t] = np.einsum("hkv,hk->hv", d, kt)
            a = np.exp(g[t])
            dg[t] = a * np.einsum("hkv,hkv->h", d, h[i])
            d = a[:, None, None] * d
        dstate[s] = d
        t0 += n
    return dq, dk, dv, dg, dstate


def linear_attention_step(q, k, v, g, state, index, scale=1.0):
    """One token per row, rows in order; returns o (B,H,V) and the new cache."""
    q, k, v, g, state = _f64(q, k, v, g, state)
    state = state.copy()
    rep = v.shape[1] // q.shape[1]
    o = np.zeros_like(v)
    for b, s in enumerate(index):
        if 0 <= s < len(state):
            qt, kt = np.repeat(q[b], rep, 0), np.repeat(k[b], rep, 0)
            state[s] = np.exp(g[b])[:, None, None] * state[s] + kt[:, :, None] * v[b][:, None, :]
            o[b] = scale * np.einsum("hk,hkv->hv", qt, state[s])
    return o, state


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, r), both unrounded."""
    x, weight, residual = _f64(x, weight, residual)
    r = x if residual is None else x + residual
    y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * weight), r


def rms_norm_backward(r, weight, dy, dresidual=None, eps=1e-6):
    """(dx, dweight)."""
    r, weight, dy, dresidual = _f64(r, weight, dy, dresidual)
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    xhat = r * rstd
    gy = dy if weight is None else dy * weight
    dx = rstd * (gy - xhat * (gy * xhat).mean(-1, keepdims=True))
    return (dx if dresidual is None else dx + dresidual), (dy * xhat).reshape(-1, r.shape[-1]).sum(0)


def block_scales(y):
    """Scales (..., ceil(dim/128)) of the 8-bit form."""
    y = np.asarray(y, dtype=np.float64)
    m = [np.abs(y[..., i:i + BLOCK]).max(-1) for i in range(0, y.shape[-1], BLOCK)]
    return np.maximum(np.stack(m, -1) / E4M3_MAX, SCALE_MIN)


def round_e4m3(x):
    """Nearest e4m3 value, ties to even: 3 bits of mantissa, exponents -6..8, steps of 2^-9 below 2^-6."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)  # |x| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX)


def matmul_fp8(a, a_scales, b, b_scales):
    a, a_scales, b, b_scales = _f64(a, a_scales, b, b_scales)
    K, N = a.shape[1], b.shape[0]
    A = a * np.repeat(a_scales, BLOCK, 1)[:, :K]
    Bm = b * np.repeat(np.repeat(b_scales, BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    return A @ Bm.T
