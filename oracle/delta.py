"""The gated delta rule and the norms of its queries and keys in numpy float64.  TEST INFRASTRUCTURE ONLY: only the test
suite may import this module.  The HIP library never calls it and shares no code with it.

The delta rule token by token (S sequences as a list of lengths, tokens packed one sequence after another):
    h_t = a_t h_{t-1} + b_t k_t (v_t - a_t h_{t-1}' k_t)',   o_t = scale h_t' q_t,   a = exp(g), b = beta;
its gradients by the chain rule along the same recurrence; the root-mean-square norm of each head's query or key with
the rotation of pairs of channels by a position's angles, and its gradients.
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, dtype=np.float64) for x in xs]


def delta_rule(q, k, v, g, beta, lens, state=None, scale=1.0):
    """q, k (T,G,K), v (T,H,V), g, beta (T,H), state (S,H,K,V) or None -> o (T,H,V), final states."""
    q, k, v, g, beta, state = _f64(q, k, v, g, beta, state)
    H, V = v.shape[1:]
    K = q.shape[2]
    rep = H // q.shape[1]
    o = np.zeros_like(v)
    last = np.zeros((len(lens), H, K, V)) if state is None else state.copy()
    t = 0
    for s, n in enumerate(lens):
        h = last[s]
        for _ in range(n):
            qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
            h = np.exp(g[t])[:, None, None] * h
            e = v[t] - np.einsum("hk,hkv->hv", kt, h)
            h = h + kt[:, :, None] * (beta[t][:, None] * e)[:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", qt, h)
            t += 1
        last[s] = h
    return o, last


def delta_rule_backward(q, k, v, g, beta, do, lens, state=None, dlast=None, scale=1.0):
    """Gradients dq, dk, dv, dg, dbeta, dstate of sum(o do) + sum(last dlast)."""
    q, k, v, g, beta, do, state, dlast = _f64(q, k, v, g, beta, do, state, dlast)
    H, V = v.shape[1:]
    G, K = q.shape[1:]
    rep = H // G
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dstate = np.zeros((len(lens), H, K, V))
    t0 = 0
    for s, n in enumerate(lens):
        h = np.zeros((H, K, V)) if state is None else state[s]
        kept, errors, after = [], [], []
        for t in range(t0, t0 + n):
            kt = np.repeat(k[t], rep, 0)
            kept.append(np.exp(g[t])[:, None, None] * h)
            errors.append(v[t] - np.einsum("hk,hkv->hv", kt, kept[-1]))
            h = kept[-1] + kt[:, :, None] * (beta[t][:, None] * errors[-1])[:, None, :]
            after.append(h)
        d = np.zeros((H, K, V)) if dlast is None else dlast[s].copy()
        for i in range(n - 1, -1, -1):
            t = t0 + i
            qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
            d = d + scale * qt[:, :, None] * do[t][:, None, :]
            dq[t] = (scale * np.einsum("hkv,hv->hk", after[i], do[t])).reshape(G, rep, K).sum(1)
            du = np.einsum("hk,hkv->hv", kt, d)
            db[t] = (du * errors[i]).sum(-1)
            dv[t] = beta[t][:, None] * du
            dkt = np.einsum("hkv,hv->hk", d, beta[t][:, None] * errors[i]) - np.einsum("hkv,hv->hk", kept[i], dv[t])
            dk[t] = dkt.reshape(G, rep, K).sum(1)
            d = d - kt[:, :, None] * dv[t][:, None, :]
            dg[t] = (d * kept[i]).sum((-1, -2))
            d = np.exp(g[t])[:, None, None] * d
        dstate[s] = d
        t0 += n
    return dq, dk, dv, dg, db, dstate


def delta_rule_step(q, k, v, g, beta, state, index, scale=1.0):
    """One token per row, rows in order; returns o (B,H,V) and the new cache."""
    q, k, v, g, beta, state = _f64(q, k, v, g, beta, state)
    state = state.copy()
    o = np.zeros_like(v)
    for b, s in enumerate(index):
        if 0 <= s < len(state):
            at = slice(b, b + 1)
            o[at], state[s:s + 1] = delta_rule(q[at], k[at], v[at], g[at], beta[at], [1], state[s:s + 1], scale)
    return o, state


def delta_rule_terms(q, k, v, g, beta, lens, state=None, scale=1.0, chunk=64):
    """The sizes of what the chunks of delta_rule add up, every term by its absolute value:
    outputs (T,H,V): scale |q|' B, B the state at the chunk's start and the decayed |k| |u| since;
    mass (S,H,V): what has entered a column of the state, |k| beta (|v| + a |h| |k|) in 2-norms, decayed since."""
    q, k, v, g, beta, state = _f64(q, k, v, g, beta, state)
    H, V = v.shape[1:]
    K = q.shape[2]
    rep = H // q.shape[1]
    terms = np.zeros_like(v)
    mass = np.zeros((len(lens), H, V))
    t = 0
    for s, n in enumerate(lens):
        h = np.zeros((H, K, V)) if state is None else state[s]
        mass[s] = np.linalg.norm(h, axis=1)
        for i in range(n):
            if i % chunk == 0:
                B = np.abs(h)
            qt, kt, a = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0), np.exp(g[t])
            h = a[:, None, None] * h
            e = v[t] - np.einsum("hk,hkv->hv", kt, h)
            size = np.linalg.norm(kt, axis=-1)[:, None]
            mass[s] = a[:, None] * mass[s] + size * beta[t][:, None] * (np.abs(v[t]) + np.linalg.norm(h, axis=1) * size)
            u = beta[t][:, None] * e
            h = h + kt[:, :, None] * u[:, None, :]
            B = a[:, None, None] * B + np.abs(kt)[:, :, None] * np.abs(u)[:, None, :]
            terms[t] = abs(scale) * np.einsum("hk,hkv->hv", np.abs(qt), B)
            t += 1
    return terms, mass


def _pairs(rotated, interleaved):
    i = np.arange(rotated // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotated // 2)


def rotate(y, table, positions, interleaved=False, back=False):
    """y (T,heads,D): pairs of the first table.shape[1] channels turned by the angles of each token's table row."""
    y, table = _f64(y, table)
    rot = table.shape[1]
    a, b = _pairs(rot, interleaved)
    at = table[np.clip(positions, 0, len(table) - 1)][:, None]
    c, s = at[..., :rot // 2], at[..., rot // 2:] * (-1 if back else 1)
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def head_norm(x, weight=None, table=None, positions=None, interleaved=False, eps=1e-6):
    """x (T,heads,D) normed over D, weighted, turned."""
    x, weight = _f64(x, weight)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y if weight is None else y * weight
    return y if table is None else rotate(y, table, positions, interleaved)


def head_norm_backward(x, dy, weight=None, table=None, positions=None, interleaved=False, eps=1e-6):
    """(dx, dweight)."""
    x, dy, weight = _f64(x, dy, weight)
    if table is not None:
        dy = rotate(dy, table, positions, interleaved, back=True)
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    gy = dy if weight is None else dy * weight
    return rstd * (gy - xhat * (gy * xhat).mean(-1, keepdims=True)), (dy * xhat).sum((0, 1))
