"""Token-sequence operators of libss2d.so (include/ss2d_tokens.h) on torch tensors.

Linear attention with a decay per head (prompts, gradients, single tokens over a
cache of states), the root-mean-square norm with the residual's addition (storage
type or 8 bits with scales, gradients) and the 8-bit matrix product with a scale
per block of 128.  As in the rest of the package the binding only checks and
marshals arguments, and there is no CPU fallback.

Every function runs on `stream`, or on the current stream of the tensors' device,
and allocates its outputs and workspace from torch's allocator on that stream, so
it can run under torch.cuda.graph.  With `stream` the caller orders the streams
(wait_stream, events) where one uses what the other wrote; the tensors' memory is
kept from others until both are done with it.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import SS2D_BF16, SS2D_F32, check, lib

_CODES = {torch.float32: SS2D_F32, torch.bfloat16: SS2D_BF16}
_SIZES = ctypes.c_int64 * 21  # ss2d_attention_sizes: six sizes, five times three strides


def _code(x) -> int:
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    return code


def _require(first, *items):
    """Each item (name, tensor, dtype, shape, dense) is a GPU tensor on `first`'s device of that dtype and shape (None: not
    checked), contiguous if dense.  One cheap condition per tensor: a single token's call has six of them."""
    index = first.get_device()
    for name, x, dtype, shape, dense in items:
        if (x.dtype is not dtype or x.get_device() != index or (shape is not None and x.shape != shape)
                or (dense and not x.is_contiguous()) or index < 0):
            if not x.is_cuda or not first.is_cuda:
                raise ValueError("all tensors must be on the GPU (no CPU fallback)")
            if x.device != first.device:
                raise ValueError("all tensors must be on the same device")
            if x.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}")
            if shape is not None and x.shape != shape:
                raise ValueError(f"{name} must be {tuple(shape)}")
            raise ValueError(f"{name} must be contiguous")


def _call(fn, device, *args):
    """fn(*args, current stream) with `device` current; raises on a status code."""
    index = device.index
    # the raw handle: torch.cuda.current_stream builds a Stream object around it, 2 us of a call's 10
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != 0:
        check(rc)


def _on_stream(stream, device, fn, *args):
    """fn(*args) with `stream` current.  Tensors that go in and come out are marked as used by both streams, so that the
    allocator gives their memory to no one before either stream is done with it, however soon the caller lets them go."""
    if stream.device != device:
        raise ValueError("stream must belong to the tensors' device")
    caller = torch.cuda.current_stream(device)
    for x in args:
        if isinstance(x, torch.Tensor) and x.is_cuda:
            x.record_stream(stream)
    with torch.cuda.stream(stream):
        out = fn(*args)
    for x in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
        x.record_stream(caller)
    return out


def _ptr(x):
    return None if x is None else x.data_ptr()


def _empty(x):
    """A contiguous tensor of x's shape and dtype beside it."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _workspace(bytes_, device):
    """(tensor or None, address) of a workspace; a negative size is a status code."""
    if bytes_ < 0:
        check(int(bytes_))
    if bytes_ == 0:
        return None, None
    w = torch.empty(bytes_, dtype=torch.uint8, device=device)
    return w, w.data_ptr()


# ------------------------------------------------------------------ linear attention
def _attention_sizes(q, k, v, log_decay, cu_seqlens, do=None):
    """Checked (sizes array, lead, S, G, H, K, V, code)."""
    packed = cu_seqlens is not None
    n = 3 if packed else 4
    if v.dim() != n or q.dim() != n or k.dim() != n:
        raise ValueError("q, k, v must be (T, heads, dim) with cu_seqlens, else (S, L, heads, dim)")
    code, dtype = _code(v), v.dtype
    shape, qshape = v.shape, q.shape
    H, V, G, K = shape[-2], shape[-1], qshape[-2], qshape[-1]
    lead = (shape[0],) if packed else (shape[0], shape[1])
    items = [("v", v, dtype, None, False), ("q", q, dtype, lead + (G, K), False), ("k", k, dtype, qshape, False),
             ("log_decay", log_decay, torch.float32, lead + (H,), False)]
    if packed:
        items.append(("cu_seqlens", cu_seqlens, torch.int32, None, True))
    if do is not None:
        items.append(("do", do, dtype, shape, False))
    _require(v, *items)
    if G < 1 or H % G != 0:
        raise ValueError("the heads of v must be a multiple of those of q and k")
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must be (sequences + 1,)")
        S, T = cu_seqlens.shape[0] - 1, lead[0]
    else:
        S, T = lead[0], lead[0] * lead[1]
    sq, sk, sv, sg = q.stride(), k.stride(), v.stride(), log_decay.stride()
    sd = sv if do is None else do.stride()
    if (K > 1 and (sq[-1] != 1 or sk[-1] != 1)) or (V > 1 and (sv[-1] != 1 or sd[-1] != 1)):
        raise ValueError("the last axis of q, k, v and do must be dense")
    if packed:
        sizes = _SIZES(S, T, G, H, K, V, 0, sq[0], sq[1], 0, sk[0], sk[1], 0, sv[0], sv[1], 0, sg[0], sg[1],
                       0, sd[0], sd[1])
    else:
        sizes = _SIZES(S, T, G, H, K, V, sq[0], sq[1], sq[2], sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], *sg,
                       sd[0], sd[1], sd[2])
    return sizes, lead, S, G, H, K, V, code


def linear_attention(q, k, v, log_decay, state=None, cu_seqlens=None, scale: float = 1.0, final_state: bool = False,
                     out=None, stream=None):
    """Linear attention with a decay per head over prompts (ss2d_linear_attention):
    h_t = exp(g_t) h_{t-1} + k_t v_t', o_t = scale h_t' q_t, causal.

    q, k (S,L,G,K), v (S,L,H,V): float32 or bfloat16, H a multiple of G; log_decay (S,L,H) float32 (g, usually <= 0).
    With cu_seqlens (S+1,) int32 on the device the sequences are packed: q, k (T,G,K), v (T,H,V), log_decay (T,H),
    sequence s being tokens cu_seqlens[s]..cu_seqlens[s+1]-1; outputs of tokens in no sequence are left as they were.
    Any strides with a dense last axis (slices of one projection's output, expanded decays); K <= 256, V <= 1024.
    A padded batch's padding has to be finite: tokens are taken in chunks, in which NaN reaches the ones before it.
    state (S,H,K,V) float32: the states to start from (None: 0).
    Returns o (v's shape, contiguous), and with final_state also the states after the last tokens (S,H,K,V) float32.
    """
    if stream is not None:
        return _on_stream(stream, v.device, linear_attention, q, k, v, log_decay, state, cu_seqlens, scale,
                          final_state, out)
    sizes, lead, S, G, H, K, V, code = _attention_sizes(q, k, v, log_decay, cu_seqlens)
    device = v.device
    if state is not None:
        _require(v, ("state", state, torch.float32, (S, H, K, V), True))
    if out is None:
        out = _empty(v)
    else:
        _require(v, ("out", out, v.dtype, v.shape, True))
    last = torch.empty((S, H, K, V), dtype=torch.float32, device=device) if final_state else None
    L = lib()
    nbytes = L.ss2d_linear_attention_workspace(sizes, 0 if cu_seqlens is None else 1, code)
    ws, at = _workspace(nbytes, device)
    _call(L.ss2d_linear_attention, device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          _ptr(state), _ptr(cu_seqlens), out.data_ptr(), _ptr(last), sizes, scale, code, at, nbytes)
    return (out, last) if final_state else out


def linear_attention_backward(q, k, v, log_decay, do, state=None, dfinal_state=None, cu_seqlens=None,
                              scale: float = 1.0, stream=None) -> dict:
    """Gradients of linear_attention (ss2d_linear_attention_backward): do the gradient of o (v's shape and dtype, any
    strides with a dense last axis), dfinal_state that of the final states (S,H,K,V) float32 or None.

    Returns dq, dk, dv (shapes and dtypes of q, k, v, contiguous), dlog_decay (float32, one value per token and head)
    and, with a state, dstate.  Values of packed tokens in no sequence are undefined.
    """
    if stream is not None:
        return _on_stream(stream, v.device, linear_attention_backward, q, k, v, log_decay, do, state, dfinal_state,
                          cu_seqlens, scale)
    sizes, lead, S, G, H, K, V, code = _attention_sizes(q, k, v, log_decay, cu_seqlens, do)
    device = v.device
    out = {"dq": _empty(q), "dk": _empty(q), "dv": _empty(v),
           "dlog_decay": torch.empty(lead + (H,), dtype=torch.float32, device=device)}
    for name, t in (("state", state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _require(v, (name, t, torch.float32, (S, H, K, V), True))
    if state is not None:
        out["dstate"] = torch.empty((S, H, K, V), dtype=torch.float32, device=device)
    L = lib()
    nbytes = L.ss2d_linear_attention_backward_workspace(sizes, 0 if cu_seqlens is None else 1, code)
    ws, at = _workspace(nbytes, device)
    _call(L.ss2d_linear_attention_backward, device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          _ptr(state), _ptr(cu_seqlens), do.data_ptr(), _ptr(dfinal_state), out["dq"].data_ptr(),
          out["dk"].data_ptr(), out["dv"].data_ptr(), out["dlog_decay"].data_ptr(), _ptr(out.get("dstate")), sizes,
          scale, code, at, nbytes)
    return out


def linear_attention_step(q, k, v, log_decay, state, state_index=None, scale: float = 1.0, out=None, stream=None):
    """One token per row over a cache of states, updated in place (ss2d_linear_attention_step).

    q, k (B,G,K), v (B,H,V): float32 or bfloat16, rows any stride apart, dense inside; log_decay (B,H) float32.
    state (slots,H,K,V) float32.  state_index (B,) int32: each row's slot (None: row i has slot i).  A row with an index
    outside 0..slots-1 is padding (output 0, no state touched); rows of one slot are its consecutive tokens.
    Returns o (B,H,V) in v's dtype.
    """
    if stream is not None:
        return _on_stream(stream, v.device, linear_attention_step, q, k, v, log_decay, state, state_index, scale, out)
    if v.dim() != 3 or q.dim() != 3 or state.dim() != 4:
        raise ValueError("q, k must be (B,G,K), v (B,H,V), state (slots,H,K,V)")
    code, dtype = _code(v), v.dtype
    B, H, V = v.shape
    qshape, cache = q.shape, state.shape
    G, K = qshape[1:]
    _require(v, ("v", v, dtype, None, False), ("q", q, dtype, (B, G, K), False), ("k", k, dtype, qshape, False),
             ("log_decay", log_decay, torch.float32, (B, H), True),
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
    _call(lib().ss2d_linear_attention_step, v.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          state.data_ptr(), _ptr(state_index), out.data_ptr(), B, cache[0], G, H, K, V, rows[0][0], rows[1][0],
          rows[2][0], scale, code)
    return out


# ------------------------------------------------------------------ norm
def _norm_inputs(x, weight, others):
    code, device = _code(x), x.device
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., dim)")
    shape = x.shape
    dim = shape[-1]
    _require(x, ("x", x, x.dtype, None, True), *[(name, t, x.dtype, shape, True) for name, t in others if t is not None])
    if weight is not None:
        _require(x, ("weight", weight, torch.float32, (dim,), True))
    return code, device, x.numel() // dim, dim


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, out=None, residual_out=None, stream=None):
    """Root-mean-square norm over the last axis, with the residual's addition (ss2d_rms_norm):
    r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight.

    x, residual (...,dim): float32 or bfloat16; weight (dim,) float32 or None.  out and residual_out may be x or residual.
    Returns y, or (y, r) when a residual is given.
    """
    if stream is not None:
        return _on_stream(stream, x.device, rms_norm, x, weight, residual, eps, out, residual_out)
    code, device, rows, dim = _norm_inputs(x, weight, (("residual", residual), ("out", out),
                                                       ("residual_out", residual_out)))
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    _call(lib().ss2d_rms_norm, device, x.data_ptr(), _ptr(residual), _ptr(weight), eps, _ptr(residual_out),
          out.data_ptr(), None, rows, dim, code)
    return out if residual is None else (out, residual_out)


def rms_norm_fp8(x, weight=None, residual=None, eps: float = 1e-6, residual_out=None, stream=None):
    """rms_norm with y in 8 bits: returns (y float8_e4m3fn (...,dim), scales float32 (...,ceil(dim/128))) and, when a
    residual is given, r as a third; y times its block's scale is the norm's output (the left operand of matmul_fp8)."""
    if stream is not None:
        return _on_stream(stream, x.device, rms_norm_fp8, x, weight, residual, eps, residual_out)
    code, device, rows, dim = _norm_inputs(x, weight, (("residual", residual), ("residual_out", residual_out)))
    y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scales = torch.empty(x.shape[:-1] + ((dim + 127) // 128,), dtype=torch.float32, device=device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    _call(lib().ss2d_rms_norm, device, x.data_ptr(), _ptr(residual), _ptr(weight), eps, _ptr(residual_out),
          y.data_ptr(), scales.data_ptr(), rows, dim, code)
    return (y, scales) if residual is None else (y, scales, residual_out)


def rms_norm_backward(r, weight, dy, dresidual=None, eps: float = 1e-6, stream=None) -> dict:
    """Gradients of rms_norm (ss2d_rms_norm_backward): r the normalised sum (rms_norm's second output, or x),
    dy the gradient of y, dresidual that of r's other use or None.  Returns dx (the gradient of x and of the
    residual alike, r's dtype) and, with a weight, dweight (dim,) float32."""
    if stream is not None:
        return _on_stream(stream, r.device, rms_norm_backward, r, weight, dy, dresidual, eps)
    code, device, rows, dim = _norm_inputs(r, weight, (("dy", dy), ("dresidual", dresidual)))
    dx = torch.empty_like(r)
    L = lib()
    dweight = ws = at = None
    nbytes = 0
    if weight is not None:
        dweight = torch.empty((dim,), dtype=torch.float32, device=device)
        nbytes = L.ss2d_rms_norm_backward_workspace(rows, dim, code)
        ws, at = _workspace(nbytes, device)
    _call(L.ss2d_rms_norm_backward, device, r.data_ptr(), _ptr(weight), dy.data_ptr(), _ptr(dresidual), eps,
          dx.data_ptr(), _ptr(dweight), rows, dim, code, at, nbytes)
    return {"dx": dx} if weight is None else {"dx": dx, "dweight": dweight}


# ------------------------------------------------------------------ 8-bit matrix product
def matmul_fp8(a, a_scales, b, b_scales, out_dtype=torch.bfloat16, out=None, stream=None):
    """a b' in 8 bits (ss2d_matmul_fp8): a (...,K), b (N,K) float8_e4m3fn with a scale per 128 inner indices,
    a_scales (...,ceil(K/128)) for every row of a, b_scales (ceil(N/128),ceil(K/128)) for blocks of 128 x 128 of b,
    float32, as rms_norm_fp8 and block-quantised weights give them.  All contiguous.
    Returns (...,N) in out_dtype (float32 or bfloat16), or in `out` and its dtype if given.
    """
    if stream is not None:
        return _on_stream(stream, a.device, matmul_fp8, a, a_scales, b, b_scales, out_dtype, out)
    if a.dim() < 1 or b.dim() != 2:
        raise ValueError("a must be (...,K) and b (N,K)")
    N, K = b.shape
    lead = a.shape[:-1]
    blocks = (K + 127) // 128
    _require(a, ("a", a, torch.float8_e4m3fn, lead + (K,), True), ("b", b, torch.float8_e4m3fn, None, True),
             ("a_scales", a_scales, torch.float32, lead + (blocks,), True),
             ("b_scales", b_scales, torch.float32, ((N + 127) // 128, blocks), True))
    if out is None:
        out = torch.empty(lead + (N,), dtype=out_dtype, device=a.device)
    else:
        _require(a, ("out", out, out.dtype, lead + (N,), True))
    M = 1
    for n in lead:
        M *= n
    _call(lib().ss2d_matmul_fp8, a.device, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(),
          out.data_ptr(), M, N, K, _code(out))
    return out
