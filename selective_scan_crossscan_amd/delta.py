"""The gated delta rule and the norms of its queries and keys (include/ss2d_delta_rule.h) on torch tensors.

Token-sequence operators beside those of tokens.py: linear attention whose state replaces what it holds for a key
(prompts, gradients, single tokens over a cache of states), and the root-mean-square norm of each head's query and key
with the rotation by the token's position in the same pass (and its gradients).  Streams, allocation and graph capture
as in tokens.py; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import lib
from .tokens import _attention_sizes, _call, _code, _empty, _on_stream, _ptr, _require, _workspace

_DELTA_SIZES = ctypes.c_int64 * 24  # ss2d_delta_sizes: linear attention's 21, beta's three strides
_QK_SIZES = ctypes.c_int64 * 19     # ss2d_qk_sizes: seven sizes, four times three strides


# ------------------------------------------------------------------ delta rule
def _delta_sizes(q, k, v, log_decay, beta, cu_seqlens, do=None):
    sizes, lead, S, G, H, K, V, code = _attention_sizes(q, k, v, log_decay, cu_seqlens, do)
    _require(v, ("beta", beta, torch.float32, lead + (H,), False))
    sb = beta.stride()
    return _DELTA_SIZES(*sizes, *((0,) + sb if cu_seqlens is not None else sb)), lead, S, G, H, K, V, code


def delta_rule(q, k, v, log_decay, beta, state=None, cu_seqlens=None, scale: float = 1.0, final_state: bool = False,
               out=None, stream=None):
    """The gated delta rule over prompts (ss2d_delta_rule), causal:
    h_t = exp(g_t) h_{t-1} + beta_t k_t (v_t - exp(g_t) h_{t-1}' k_t)', o_t = scale h_t' q_t.

    q, k (S,L,G,K), v (S,L,H,V): float32 or bfloat16, H a multiple of G; log_decay (g, usually <= 0) and beta (usually
    0..1) (S,L,H) float32.  Keys are meant to have unit length (qk_norm with a weight of K**-0.5); where
    beta |k|^2 is over 2 the state grows.  Packed sequences, strides, sizes, padding and state as in linear_attention.
    Returns o (v's shape, contiguous), and with final_state also the states after the last tokens (S,H,K,V) float32.
    """
    if stream is not None:
        return _on_stream(stream, v.device, delta_rule, q, k, v, log_decay, beta, state, cu_seqlens, scale,
                          final_state, out)
    sizes, lead, S, G, H, K, V, code = _delta_sizes(q, k, v, log_decay, beta, cu_seqlens)
    device = v.device
    if state is not None:
        _require(v, ("state", state, torch.float32, (S, H, K, V), True))
    if out is None:
        out = _empty(v)
    else:
        _require(v, ("out", out, v.dtype, v.shape, True))
    last = torch.empty((S, H, K, V), dtype=torch.float32, device=device) if final_state else None
    L = lib()
    nbytes = L.ss2d_delta_rule_workspace(sizes, 0 if cu_seqlens is None else 1, code)
    ws, at = _workspace(nbytes, device)
    _call(L.ss2d_delta_rule, device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(),
          _ptr(state), _ptr(cu_seqlens), out.data_ptr(), _ptr(last), sizes, scale, code, at, nbytes)
    return (out, last) if final_state else out


def delta_rule_backward(q, k, v, log_decay, beta, do, state=None, dfinal_state=None, cu_seqlens=None,
                        scale: float = 1.0, stream=None) -> dict:
    """Gradients of delta_rule (ss2d_delta_rule_backward): do the gradient of o (v's shape and dtype, any strides with a
    dense last axis), dfinal_state that of the final states (S,H,K,V) float32 or None.

    Returns dq, dk, dv (shapes and dtypes of q, k, v, contiguous), dlog_decay and dbeta (float32, one value per token and
    head) and, with a state, dstate.  Values of packed tokens in no sequence are undefined.
    """
    if stream is not None:
        return _on_stream(stream, v.device, delta_rule_backward, q, k, v, log_decay, beta, do, state, dfinal_state,
                          cu_seqlens, scale)
    sizes, lead, S, G, H, K, V, code = _delta_sizes(q, k, v, log_decay, beta, cu_seqlens, do)
    device = v.device
    for name, t in (("state", state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _require(v, (name, t, torch.float32, (S, H, K, V), True))
    out = {"dq": _empty(q), "dk": _empty(k), "dv": _empty(v)}
    for name in ("dlog_decay", "dbeta"):
        out[name] = torch.empty(lead + (H,), dtype=torch.float32, device=device)
    if state is not None:
        out["dstate"] = torch.empty((S, H, K, V), dtype=torch.float32, device=device)
    L = lib()
    nbytes = L.ss2d_delta_rule_backward_workspace(sizes, 0 if cu_seqlens is None else 1, code)
    ws, at = _workspace(nbytes, device)
    _call(L.ss2d_delta_rule_backward, device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          beta.data_ptr(), _ptr(state), _ptr(cu_seqlens), do.data_ptr(), _ptr(dfinal_state), out["dq"].data_ptr(),
          out["dk"].data_ptr(), out["dv"].data_ptr(), out["dlog_decay"].data_ptr(), out["dbeta"].data_ptr(),
          _ptr(out.get("dstate")), sizes, scale, code, at, nbytes)
    return out


def delta_rule_step(q, k, v, log_decay, beta, state, state_index=None, scale: float = 1.0, out=None, stream=None):
    """One token per row over a cache of states, updated in place (ss2d_delta_rule_step).

    q, k (B,G,K), v (B,H,V): float32 or bfloat16, rows any stride apart, dense inside; log_decay, beta (B,H) float32;
    state (slots,H,K,V) float32; state_index (B,) int32: each row's slot (None: row i has slot i).  A row with an index
    outside 0..slots-1 is padding (output 0, no state touched); rows of one slot are its consecutive tokens.
    Returns o (B,H,V) in v's dtype.
    """
    if stream is not None:
        return _on_stream(stream, v.device, delta_rule_step, q, k, v, log_decay, beta, state, state_index, scale, out)
    if v.dim() != 3 or q.dim() != 3 or state.dim() != 4:
        raise ValueError("q, k must be (B,G,K), v (B,H,V), state (slots,H,K,V)")
    code, dtype = _code(v), v.dtype
    B, H, V = v.shape
    qshape, cache = q.shape, state.shape
    G, K = qshape[1:]
    _require(v, ("v", v, dtype, None, False), ("q", q, dtype, (B, G, K), False), ("k", k, dtype, qshape, False),
             ("log_decay", log_decay, torch.float32, (B, H), True), ("beta", beta, torch.float32, (B, H), True),
             ("state", state, torch.float32, (cache[0], H, K, V), True))
    if G < 1 or H % G != 0:
        raise ValueError("the heads of v must be a multiple of those of q and k")
    if state_index is not None:
        _require(v, ("state_index", state_index, torch.int32, (B,), True))
    rows = [x.stride() for x in (q, k, v)]
    for name, st, n, d in (("q", rows[0], G, K), ("k", rows[1], G, K), ("v", rows[2], H, V)):
        if (n > 1 and st[1] != d) or (d > 1 and st[2] != 1):
            raise ValueError(f"{name} must be dense inside a row")
    if out is None:
        out = _empty(v)
    else:
        _require(v, ("out", out, dtype, (B, H, V), True))
    _call(lib().ss2d_delta_rule_step, v.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          beta.data_ptr(), state.data_ptr(), _ptr(state_index), out.data_ptr(), B, cache[0], G, H, K, V, rows[0][0],
          rows[1][0], rows[2][0], scale, code)
    return out


# ------------------------------------------------------------------ norms of queries and keys
def rotation_table(positions: int, rotated: int, base: float = 10000.0, device="cuda"):
    """A table for qk_norm: row p holds the cosines, then the sines, of p base^(-2 i / rotated), i < rotated / 2, formed
    in float64 and rounded once to float32; (positions, rotated)."""
    if positions < 1 or rotated < 2 or rotated % 2:
        raise ValueError("positions must be at least 1, rotated even and at least 2")
    rate = base ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device=device) / rotated)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def _three(x):
    """Strides of sequence, token and head."""
    s = x.stride()
    return (0, s[0], s[1]) if len(s) == 3 else s[:3]


def _qk_inputs(q, k, q_weight, k_weight, rotation, positions, others):
    """Checked (sizes without the strides, code); others: (name, tensor, q or k) of the same shapes and dtype."""
    n = q.dim()
    if n not in (3, 4) or k.dim() != n:
        raise ValueError("q and k must be (T, heads, dim) or (S, L, heads, dim)")
    code, dtype = _code(q), q.dtype
    lead, (Hq, D), Hk = q.shape[:-2], q.shape[-2:], k.shape[-2]
    items = [("q", q, dtype, None, False), ("k", k, dtype, lead + (Hk, D), False)]
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            items.append((name, w, torch.float32, (D,), True))
    rows = rot = 0
    if rotation is not None:
        items.append(("rotation", rotation, torch.float32, None, True))
        if rotation.dim() != 2:
            raise ValueError("rotation must be (positions, rotated)")
        rows, rot = rotation.shape
        if rot < 2 or rot % 2 or rot > D or rows < 1:
            raise ValueError("rotation must have an even number of columns, 2 to dim, and at least one row")
        if positions is not None:
            items.append(("positions", positions, torch.int32, lead, True))
    elif positions is not None:
        raise ValueError("positions without a rotation table")
    items += [(name, x, dtype, like.shape, False) for name, x, like in others]
    _require(q, *items)
    if D > 1 and any(x.stride(-1) != 1 for x in [q, k] + [x for _, x, _ in others]):
        raise ValueError("the last axis of queries, keys and their outputs must be dense")
    return ((1,) if n == 3 else ()) + tuple(lead) + (Hq, Hk, D, rot, rows), code


def qk_norm(q, k, q_weight=None, k_weight=None, rotation=None, positions=None, interleaved: bool = False,
            eps: float = 1e-6, out=None, stream=None):
    """Root-mean-square norm of each head's query and key, then the rotation by the token's position (ss2d_qk_norm):
    y = R(x / sqrt(mean(x^2) + eps) * weight).

    q (...,Hq,D), k (...,Hk,D), leading axes (T,) or (S,L): float32 or bfloat16, any strides with a dense last axis;
    q_weight, k_weight (D,) float32 or None (1); a weight of D**-0.5 gives unit length.  rotation (positions, rotated)
    float32: a position's cosines, then its sines (rotation_table), the first `rotated` channels of a head turn; None:
    no rotation.  positions: int32 of the leading axes (clamped to the table), or None: the token's number in its
    sequence.  interleaved: channels 2i and 2i+1 are a pair instead of i and i + rotated/2.  D <= 256.
    out: a pair of tensors for the results, any strides with a dense last axis; q and k themselves too.
    Returns (q, k) normed and rotated.
    """
    if stream is not None:
        if out is not None:
            for x in out:
                x.record_stream(stream)
        return _on_stream(stream, q.device, qk_norm, q, k, q_weight, k_weight, rotation, positions, interleaved, eps,
                          out)
    if out is None:
        out = _empty(q), _empty(k)
    sizes, code = _qk_inputs(q, k, q_weight, k_weight, rotation, positions, (("out[0]", out[0], q), ("out[1]", out[1], k)))
    sizes = _QK_SIZES(*sizes, *_three(q), *_three(k), *_three(out[0]), *_three(out[1]))
    _call(lib().ss2d_qk_norm, q.device, q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(rotation),
          _ptr(positions), out[0].data_ptr(), out[1].data_ptr(), sizes, eps, 1 if interleaved else 0, code)
    return out[0], out[1]


def qk_norm_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, rotation=None, positions=None,
                     interleaved: bool = False, eps: float = 1e-6, stream=None) -> dict:
    """Gradients of qk_norm (ss2d_qk_norm_backward): q, k its inputs, dq_out, dk_out the gradients of its outputs (same
    shapes and dtype, any strides with a dense last axis).  Returns dq, dk (contiguous) and, for each weight given,
    dq_weight, dk_weight (D,) float32."""
    if stream is not None:
        return _on_stream(stream, q.device, qk_norm_backward, q, k, dq_out, dk_out, q_weight, k_weight, rotation,
                          positions, interleaved, eps)
    sizes, code = _qk_inputs(q, k, q_weight, k_weight, rotation, positions, (("dq_out", dq_out, q), ("dk_out", dk_out, k)))
    sizes = _QK_SIZES(*sizes, *_three(q), *_three(k), *_three(dq_out), *_three(dk_out))
    out = {"dq": _empty(q), "dk": _empty(k)}
    for name, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        if w is not None:
            out[name] = _empty(w)
    L = lib()
    nbytes, at = 0, None
    if len(out) > 2:
        nbytes = L.ss2d_qk_norm_backward_workspace(sizes, code)
        ws, at = _workspace(nbytes, q.device)
    _call(L.ss2d_qk_norm_backward, q.device, q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight),
          _ptr(rotation), _ptr(positions), dq_out.data_ptr(), dk_out.data_ptr(), out["dq"].data_ptr(),
          out["dk"].data_ptr(), _ptr(out.get("dq_weight")), _ptr(out.get("dk_weight")), sizes, eps,
          1 if interleaved else 0, code, at, nbytes)
    return out
