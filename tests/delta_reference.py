"""Inputs and tolerances of the delta rule's GPU tests, beside the oracle in oracle/delta.py.

Roundings.  A chunk's values reach an output, or the state, by sums of at most n = K + V + 64 terms, each rounded to
fp32 a few times (half a step, 2^-24, each).  Errors that enter a state of unit keys and beta in [0, 1] do not grow
after that: each token's map a (1 - beta k k') shrinks them.  So
  element by element  an fp32 result is off by at most 2 n 2^-24 of the absolute values of its terms
                      (oracle.delta.delta_rule_terms: `terms` of a chunk, `mass` of all that entered a state);
  in the 2-norm       the roundings' signs are independent, so their squares add: 2 sqrt(n) 2^-24 of the terms' norm,
                      over all tokens for results of fp32.
For bf16 an output adds its own rounding, 2^-8 of itself, and three roundings to bf16 of what its terms are made of
(masked products, states, replaced values), 2^-8 of the terms each.
"""
import numpy as np

from oracle import delta
import ss2d_inputs


def values(a, dtype):
    a = np.asarray(a, dtype=np.float32)
    return ss2d_inputs.round_to_bf16(a) if dtype == "bf16" else a


def unit(a):
    return a / np.maximum(np.linalg.norm(a, axis=-1, keepdims=True), 1e-6)


def make(lens, G, H, K, V, dtype, seed, decay="mixed", keys="random", state=True):
    r = np.random.default_rng(seed)
    T = sum(lens)
    q, v = values(r.standard_normal((T, G, K)), dtype), values(r.standard_normal((T, H, V)), dtype)
    k = unit(r.standard_normal((T, G, K)))
    b = r.uniform(0, 1, (T, H)).astype(np.float32)
    if keys == "same":  # one key for all tokens, replaced outright: the hardest triangular system
        k = np.broadcast_to(k[:1], k.shape).copy()
        b[:] = 1
    elif keys == "zero":  # beta of 0 and 1, keys of 0 among others
        b[r.random((T, H)) < 0.3] = 0
        b[r.random((T, H)) < 0.3] = 1
        k[r.random(T) < 0.3] = 0
    k = values(k * (1 - 2.0 ** -8 if dtype == "bf16" else 1), dtype)  # not over 1 when rounded
    g = {"mixed": -np.exp(r.uniform(np.log(1e-3), np.log(2.0), (T, H))), "none": np.zeros((T, H)),
         "strong": -r.uniform(5, 60, (T, H)), "far": -np.exp(r.uniform(-3, 0, (T, H)))}[decay].astype(np.float32)
    if decay == "far":  # tokens that forget everything, by the type's lowest value and by -Inf
        g[r.random((T, H)) < 0.05] = np.finfo(np.float32).min
        g[r.random((T, H)) < 0.05] = -np.inf
    st = r.standard_normal((len(lens), H, K, V)).astype(np.float32) if state else None
    return q, k, v, g, b, st


def check(name, got, ref, terms, n, bf16=False):
    """got against ref, off by the roundings above of `terms` (broadcast to ref)."""
    terms = np.broadcast_to(terms, ref.shape)
    err = np.abs(got - ref)
    tol = 2 * n * 2.0 ** -24 * terms + 1e-37
    whole = 2 * np.sqrt(n) * 2.0 ** -24 * np.linalg.norm(terms)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + 3 * terms)
        whole += 2.0 ** -8 * (np.linalg.norm(ref) + np.linalg.norm(terms))
    worst = float(np.max(err / tol)) if err.size else 0.0
    norm = float(np.linalg.norm(err))
    rel = norm / max(float(np.linalg.norm(ref)), 1e-300)
    print(f"[delta] {name}: error / tolerance {worst:.3f}, of the norm {norm / (whole + 1e-37):.3f}, relative {rel:.2e}",
          flush=True)
    assert np.all(err <= tol), (name, worst, np.argwhere(~(err <= tol))[:5].tolist())
    assert norm <= whole + 1e-37, (name, norm / whole)


def check_forward(name, o, last, args, lens, scale, dtype, chunk=None):
    """o (T,H,V) and the final states (or None) of args = (q, k, v, g, b, st)."""
    q, k, v, g, b, st = args
    n = q.shape[2] + v.shape[2] + 64
    ref_o, ref_s = delta.delta_rule(q, k, v, g, b, lens, st, scale)
    terms, mass = delta.delta_rule_terms(q, k, v, g, b, lens, st, scale, chunk or (64 if dtype == "bf16" else 32))
    # what is in the state before a chunk has its own errors, in every direction
    over = abs(scale) * np.repeat(np.linalg.norm(q, axis=-1), v.shape[1] // q.shape[1], 1)
    per = np.concatenate([np.broadcast_to(mass[s], (n_,) + mass.shape[1:]) for s, n_ in enumerate(lens)]
                         or [mass[:0]])
    largest = np.maximum(per, np.abs(terms))
    check(name + " o", o, ref_o, terms + over[..., None] * largest if dtype == "f32" else terms, n, dtype == "bf16")
    if last is not None:
        check(name + " state", last, ref_s, mass[:, :, None], n)


def gradient_terms(q, k, v, g, b, do, lens, st, dl, scale, chunk):
    """Absolute values of the terms of dq, dk (per head), dv, dg, db, the chunk's tokens and the states around it."""
    q, k, v, g, b, do = (np.asarray(x, np.float64) for x in (q, k, v, g, b, do))
    H, V = v.shape[1:]
    G, K = q.shape[1:]
    rep = H // G
    tq, tk, tv = np.zeros((len(q), H, K)), np.zeros((len(q), H, K)), np.zeros_like(v)
    tg, tb = np.zeros_like(g), np.zeros_like(b)
    t0 = 0
    for s, n in enumerate(lens):
        hs = [np.zeros((H, K, V)) if st is None else np.asarray(st[s], np.float64)]
        B, e, kept = [], [], []
        for i in range(n):
            t = t0 + i
            kt, a = np.repeat(k[t], rep, 0), np.exp(g[t])[:, None, None]
            kept.append(a * hs[-1])
            e.append(v[t] - np.einsum("hk,hkv->hv", kt, kept[-1]))
            before = np.abs(hs[-1]) if i % chunk == 0 else B[-1]
            B.append(a * before + np.abs(kt)[:, :, None] * np.abs(b[t][:, None] * e[-1])[:, None, :])
            hs.append(kept[-1] + kt[:, :, None] * (b[t][:, None] * e[-1])[:, None, :])
        d = np.zeros((H, K, V)) if dl is None else np.asarray(dl[s], np.float64)
        for i in range(n - 1, -1, -1):
            t = t0 + i
            qt, kt, a = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0), np.exp(g[t])[:, None, None]
            if i % chunk == chunk - 1 or i == n - 1:
                D, sums = np.abs(d), (np.abs(d) * np.abs(hs[i + 1])).sum((-1, -2))
            d = d + scale * qt[:, :, None] * do[t][:, None, :]
            D = D + abs(scale) * np.abs(qt)[:, :, None] * np.abs(do[t])[:, None, :]
            dz = b[t][:, None] * np.einsum("hk,hkv->hv", kt, d)
            tq[t] = abs(scale) * np.einsum("hkv,hv->hk", B[i], np.abs(do[t]))
            tk[t] = np.einsum("hkv,hv->hk", D, np.abs(b[t][:, None] * e[i])) + np.einsum("hkv,hv->hk", B[i], np.abs(dz))
            tv[t] = b[t][:, None] * np.einsum("hkv,hk->hv", D, np.abs(kt))
            tb[t] = (np.einsum("hkv,hk->hv", D, np.abs(kt)) * (np.abs(e[i]) + np.einsum("hkv,hk->hv", np.abs(kept[i]), np.abs(kt)))).sum(-1)
            sums = sums + (np.abs(qt) * tq[t]).sum(-1) + (tv[t] * np.abs(v[t])).sum(-1)
            tg[t] = sums
            d = a * (d - kt[:, :, None] * dz[:, None, :])
            D = a * (D + np.abs(kt)[:, :, None] * np.abs(dz)[:, None, :])
        t0 += n
    group = lambda x: x.reshape(len(q), G, rep, K).sum(2)  # noqa: E731
    return group(tq), group(tk), tv, tg, tb


def check_gradients(name, got, args, do, lens, dl, scale, dtype):
    """got: dq, dk, dv, dg, db, dstate (or None) as arrays."""
    q, k, v, g, b, st = args
    H, V = v.shape[1:]
    K = q.shape[2]
    n = K + V + 64
    ref = delta.delta_rule_backward(q, k, v, g, b, do, lens, st, dl, scale)
    terms = gradient_terms(q, k, v, g, b, do, lens, st, dl, scale, 64 if dtype == "bf16" else 32)
    bf16 = dtype == "bf16"
    for i, what in enumerate(("dq", "dk", "dv", "dlog_decay", "dbeta")):
        # the states and their gradients before and behind a chunk have errors of their own, as large again
        check(f"{name} {what}", got[i], ref[i], 2 * terms[i], n, bf16 and i < 3)
    if got[5] is not None:
        # the mass of the state's gradient: the same recurrence backwards, keys in place of themselves, q do' entering
        mass = np.zeros((len(lens), H, V))
        t = 0
        for s, m in enumerate(lens):
            mass[s] = 0 if dl is None else np.linalg.norm(dl[s], axis=1)
            for i in range(t + m - 1, t - 1, -1):
                size = np.linalg.norm(np.repeat(np.asarray(q[i], np.float64), H // q.shape[1], 0), axis=-1)[:, None]
                new = abs(scale) * size * np.abs(do[i])
                mass[s] = np.exp(np.asarray(g[i], np.float64))[:, None] * (mass[s] + 2 * new)
            t += m
        full = np.exp(np.asarray(g, np.float64))
        assert np.isfinite(full).all()
        check(f"{name} dstate", got[5], ref[5], mass[:, :, None], n)
