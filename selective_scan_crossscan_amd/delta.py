"""The gated delta rule and the norms of its queries and keys (include/ss2d_delta_rule.h) on torch tensors.

Token-sequence operators beside those of tokens.py: linear attention whose state replaces what it holds for a key
(prompts, gradients, single tokens over a cache of states), and the root-mean-square norm of each head's query and key
with the rotation by the token's position in the same pass (and its gradients).  Streams, allocation and graph capture
as in tokens.py; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import check, lib
from .tokens import _call, _code, _empty, _on_stream, _ptr, _require, _workspace

_DELTA_SIZES = ctypes.c_int64 * 24  # ss2d_delta_sizes: linear attention's 21, beta's three strides
_QK_SIZES = ctypes.c_int64 * 19     # ss2d_qk_sizes: seven sizes, four times three strides


# ------------------------------------------------------------------ delta rule
@functools.lru_cache(maxsize=1024)
def _delta_plan(q, k, v, g, b, do, cu, code):
    """Sizes for the C ABI, bytes of workspace and the states' shape, from the shapes and strides of the tensors; kept, as a
    layer calls with the same ones again and again (4 us of a short prompt's 19 on the host otherwise).  do: None for the forward."""
    (qs, qt), (ks, kt), (vs, vt), (gs, gt), (bs, bt) = q, k, v, g, b
    packed = cu is not None
    n = 3 if packed else 4
    if len(vs) != n or len(qs) != n or len(ks) != n:
        raise ValueError("q, k, v must be (T, heads, dim) with cu_seqlens, else (S, L, heads, dim)")
    lead, (G, K), (H, V) = tuple(vs[:-2]), qs[-2:], vs[-2:]
    ds, dt = (vs, vt) if do is None else do
    for name, have, want in (("q", qs, lead + (G, K)), ("k", ks, lead + (G, K)), ("log_decay", gs, lead + (H,)),
                             ("beta", bs, lead + (H,)), ("do", ds, tuple(vs))):
        if have != want:
            raise ValueError(f"{name} must be {want}")
    if G < 1 or H % G != 0:
        raise ValueError("the heads of v must be a multiple of those of q and k")
    if packed and (len(cu) != 1 or cu[0] < 2):
        raise ValueError("cu_seqlens must be (sequences + 1,)")
    if (K > 1 and (qt[-1] != 1 or kt[-1] != 1)) or (V > 1 and (vt[-1] != 1 or dt[-1] != 1)):
        raise ValueError("the last axis of q, k, v and do must be dense")
    S, T = (cu[0] - 1, lead[0]) if packed else (lead[0], lead[0] * lead[1])
    three = (lambda t: (0,) + t[:2]) if packed else (lambda t: t[:3])
    sizes = _DELTA_SIZES(S, T, G, H, K, V, *three(qt), *three(kt), *three(vt), *three(gt), *three(dt), *three(bt))
    L = lib()
    need = (L.ss2d_delta_rule_workspace if do is None else L.ss2d_delta_rule_backward_workspace)(sizes, int(packed), code)
    if need < 0:
        check(int(need))
    return sizes, need, (S, H, K, V)


def _delta_inputs(q, k, v, log_decay, beta, cu_seqlens, do, states):
    """Checked plan and code; states: (name, tensor or None) of the states' shape."""
    code, dtype = _code(v), v.dtype
    plan = _delta_plan((q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride()),
                       (log_decay.shape, log_decay.stride()), (beta.shape, beta.stride()),
                       None if do is None else (do.shape, do.stride()),
                       None if cu_seqlens is None else cu_seqlens.shape, code)
    items = [("v", v, dtype, None, False), ("q", q, dtype, None, False), ("k", k, dtype, None, False),
             ("log_decay", log_decay, torch.float32, None, False), ("beta", beta, torch.float32, None, False)]
    if cu_seqlens is not None:
        items.append(("cu_seqlens", cu_seqlens, torch.int32, None, True))
    if do is not None:
        items.append(("do", do, dtype, None, False))
    for name, t in states:
        if t is not None:
            items.append((name, t, torch.float32, plan[2], True))
    _require(v, *items)
    return plan, code


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
    (sizes, nbytes, shape), code = _delta_inputs(q, k, v, log_decay, beta, cu_seqlens, None, (("state", state),))
    device = v.device
    if out is None:
        out = _empty(v)
    else:
        _require(v, ("out", out, v.dtype, v.shape, True))
    last = torch.empty(shape, dtype=torch.float32, device=device) if final_state else None
    ws, at = _workspace(nbytes, device)
    L = lib()
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
    (sizes, nbytes, shape), code = _delta_inputs(q, k, v, log_decay, beta, cu_seqlens, do,
                                                 (("state", state), ("dfinal_state", dfinal_state)))
    device = v.device
    out = {"dq": _empty(q), "dk": _empty(k), "dv": _empty(v), "dlog_decay": _empty(log_decay), "dbeta": _empty(beta)}
    if state is not None:
        out["dstate"] = torch.empty(shape, dtype=torch.float32, device=device)
    ws, at = _workspace(nbytes, device)
    L = lib()
    _call(L.ss2d_delta_rule_backward, device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          beta.data_ptr(), _ptr(state), _ptr(cu_seqlens), do.data_ptr(), _ptr(dfinal_state), out["dq"].data_ptr(),
          out["dk"].data_ptr(), out["dv"].data_ptr(), out["dlog_decay"].data_ptr(), out["dbeta"].data_ptr(),
          _ptr(out.get("dstate")), sizes, scale, code, at, nbytes)
    return out


@functools.lru_cache(maxsize=1024)
def _step_sizes(q, k, v, cache):
    """Rows, slots, groups, heads, key and value sizes and the rows' strides for the C ABI."""
    (qs, qt), (ks, kt), (vs, vt) = q, k, v
    if len(vs) != 3 or len(qs) != 3 or len(cache) != 4:
        raise ValueError("q, k must be (B,G,K), v (B,H,V), state (slots,H,K,V)")
    (B, H, V), (G, K) = vs, qs[1:]
    for name, have, want in (("q", qs, (B, G, K)), ("k", ks, (B, G, K)), ("state", cache, (cache[0], H, K, V))):
        if have != want:
            raise ValueError(f"{name} must be {want}")
    if G < 1 or H % G != 0:
        raise ValueError("the heads of v must be a multiple of those of q and k")
    for name, st, n, d in (("q", qt, G, K), ("k", kt, G, K), ("v", vt, H, V)):
        if (n > 1 and st[1] != d) or (d > 1 and st[2] != 1):
            raise ValueError(f"{name} must be dense inside a row")
    return B, cache[0], G, H, K, V, qt[0], kt[0], vt[0]


def delta_rule_step(q, k, v, log_decay, beta, state, state_index=None, scale: float = 1.0, out=None, stream=None):
    """One token per row over a cache of states, updated in place (ss2d_delta_rule_step).

    q, k (B,G,K), v (B,H,V): float32 or bfloat16, rows any stride apart, dense inside; log_decay, beta (B,H) float32;
    state (slots,H,K,V) float32; state_index (B,) int32: each row's slot (None: row i has slot i).  A row with an index
    outside 0..slots-1 is padding (output 0, no state touched); rows of one slot are its consecutive tokens.
    Returns o (B,H,V) in v's dtype.
    """
    if stream is not None:
        return _on_stream(stream, v.device, delta_rule_step, q, k, v, log_decay, beta, state, state_index, scale, out)
    code, dtype = _code(v), v.dtype
    sizes = _step_sizes((q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride()), state.shape)
    rates = v.shape[:2]
    items = [("v", v, dtype, None, False), ("q", q, dtype, None, False), ("k", k, dtype, None, False),
             ("log_decay", log_decay, torch.float32, rates, True), ("beta", beta, torch.float32, rates, True),
             ("state", state, torch.float32, None, True)]
    if state_index is not None:
        items.append(("state_index", state_index, torch.int32, rates[:1], True))
    if out is not None:
        items.append(("out", out, dtype, v.shape, True))
    _require(v, *items)
    if out is None:
        out = _empty(v)
    _call(lib().ss2d_delta_rule_step, v.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          beta.data_ptr(), state.data_ptr(), _ptr(state_index), out.data_ptr(), *sizes, scale, code)
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


@functools.lru_cache(maxsize=1024)
def _qk_sizes(q, k, to_q, to_k, table, positions):
    """Sizes for the C ABI from the shapes and strides of queries, keys and their outputs (None: dense), the table's and
    the positions' shapes; kept, as for the delta rule."""
    (qs, qt), (ks, kt) = q, k
    n = len(qs)
    if n not in (3, 4) or len(ks) != n:
        raise ValueError("q and k must be (T, heads, dim) or (S, L, heads, dim)")
    lead, (Hq, D), Hk = tuple(qs[:-2]), qs[-2:], ks[-2]
    if tuple(ks) != lead + (Hk, D):
        raise ValueError(f"k must be {lead + (Hk, D)}")
    strides = [qt, kt]
    for name, to, shape in (("queries", to_q, tuple(qs)), ("keys", to_k, tuple(ks))):
        if to is None:
            t = [1]
            for m in shape[:0:-1]:
                t.append(t[-1] * m)
            to = shape, tuple(t[::-1])
        if tuple(to[0]) != shape:
            raise ValueError(f"the {name}' outputs must be {shape}")
        strides.append(to[1])
    if D > 1 and any(t[-1] != 1 for t in strides):
        raise ValueError("the last axis of queries, keys and their outputs must be dense")
    rows = rot = 0
    if table is not None:
        if len(table) != 2:
            raise ValueError("rotation must be (positions, rotated)")
        rows, rot = table
        if rot < 2 or rot % 2 or rot > D or rows < 1:
            raise ValueError("rotation must have an even number of columns, 2 to dim, and at least one row")
        if positions is not None and tuple(positions) != lead:
            raise ValueError(f"positions must be {lead}")
    elif positions is not None:
        raise ValueError("positions without a rotation table")
    first = (1,) + lead if n == 3 else lead
    return _QK_SIZES(*first, Hq, Hk, D, rot, rows, *(x for t in strides for x in ((0,) + t[:2] if n == 3 else t[:3])))


def _qk_inputs(q, k, q_weight, k_weight, rotation, positions, to_q, to_k):
    """Checked (sizes, code); to_q, to_k: the outputs, or their gradients, or None for dense ones."""
    code, dtype = _code(q), q.dtype
    sizes = _qk_sizes((q.shape, q.stride()), (k.shape, k.stride()), None if to_q is None else (to_q.shape, to_q.stride()),
                      None if to_k is None else (to_k.shape, to_k.stride()), None if rotation is None else rotation.shape,
                      None if positions is None else positions.shape)
    items = [("q", q, dtype, None, False), ("k", k, dtype, None, False)]
    D = (q.shape[-1],)
    if q_weight is not None:
        items.append(("q_weight", q_weight, torch.float32, D, True))
    if k_weight is not None:
        items.append(("k_weight", k_weight, torch.float32, D, True))
    if rotation is not None:
        items.append(("rotation", rotation, torch.float32, None, True))
    if positions is not None:
        items.append(("positions", positions, torch.int32, None, True))
    if to_q is not None:
        items.append(("the queries' outputs", to_q, dtype, None, False))
        items.append(("the keys' outputs", to_k, dtype, None, False))
    _require(q, *items)
    return sizes, code


def qk_norm(q, k, q_weight=None, k_weight=None, rotation=None, positions=None, interleaved: bool = False,
            eps: float = 1e-6, out=None, stream=None):
    """Root-mean-square norm of each head's query and key, then the rotation by the token's position (ss2d_qk_norm):
    y = R(x / sqrt(mean(x^2) + eps) * weight).

    q (...,Hq,D), k (...,Hk,D), leading axes (T,) or (S,L): float32 or bfloat16, any strides with a dense last axis;
    q_weight, k_weight (D,) float32 or None (1); a weight of D**-0.5 gives unit length.  rotation (positions, rotated)
    float32: a position's cosines, then its sines (rotation_table), the first `rotated` channels of a head turn; None:
    no rotation.  positions: int32 of the leading axes (clamped to the table), or None: the token's number in its
    sequence.  interleaved: channels 2i and 2i+1 are a pair instead of i and i + rotated/2.  D <= 256.
    out: a pair of tensors for the results, any strides with a dense last axis that leave their elements apart; q and k
    themselves too, also as slices of one tensor in any layout that leaves the two no address in common.
    Returns (q, k) normed and rotated.
    """
    if stream is not None:
        if out is not None:
            for x in out:
                x.record_stream(stream)
        return _on_stream(stream, q.device, qk_norm, q, k, q_weight, k_weight, rotation, positions, interleaved, eps,
                          out)
    to_q, to_k = (None, None) if out is None else out
    sizes, code = _qk_inputs(q, k, q_weight, k_weight, rotation, positions, to_q, to_k)
    if out is None:
        to_q, to_k = _empty(q), _empty(k)
    _call(lib().ss2d_qk_norm, q.device, q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(rotation),
          _ptr(positions), to_q.data_ptr(), to_k.data_ptr(), sizes, eps, 1 if interleaved else 0, code)
    return to_q, to_k


def qk_norm_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, rotation=None, positions=None,
                     interleaved: bool = False, eps: float = 1e-6, stream=None) -> dict:
    """Gradients of qk_norm (ss2d_qk_norm_backward): q, k its inputs, dq_out, dk_out the gradients of its outputs (same
    shapes and dtype, any strides with a dense last axis).  Returns dq, dk (contiguous) and, for each weight given,
    dq_weight, dk_weight (D,) float32."""
    if stream is not None:
        return _on_stream(stream, q.device, qk_norm_backward, q, k, dq_out, dk_out, q_weight, k_weight, rotation,
                          positions, interleaved, eps)
    sizes, code = _qk_inputs(q, k, q_weight, k_weight, rotation, positions, dq_out, dk_out)
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
