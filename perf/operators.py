"""Measured cases of the token-sequence operators: linear attention with a decay per head (prompts, its
gradients, single tokens over a state cache), the root-mean-square norm with the residual's addition (16/32-bit
output, 8-bit output with scales, gradients), and the 8-bit matrix product with a scale per block of 128.

`own` False computes each operator in its plain form, in elementary torch operations; True calls the library.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # chunk of the plain linear attention
BLOCK = 128  # channels per scale of the 8-bit values
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # A chat turn's few short prompts, one of a single token, continuing from kept states: latency counts.
        dict(name="attention_short", op="attention", dtype="bf16", lens="1,37,70", G=4, H=4, K=64, V=64, packed=True),
        # A serving batch packed without padding: one long document beside ragged prompts and an empty one.
        dict(name="attention_long", op="attention", dtype="bf16", lens="32768,4097,0,1023,255,1", G=16, H=16, K=128,
             V=128, packed=True),
        # The tokens of 56 x 56 feature maps, 192 channels as 6 heads of 32 that share keys of 16 states, fp32.
        dict(name="attention_map_f32", op="attention", dtype="f32", lens="3136,3136,3136,3136", G=1, H=6, K=16, V=32,
             packed=False),
        # A training step's layer: two sequences of 4096 tokens, 16 heads of 128.
        dict(name="attention_grad", op="attention_grad", dtype="bf16", lens="4096,4096", G=16, H=16, K=128, V=128,
             packed=False),
        # Odd sizes in fp32, one group of keys and queries shared by all heads.
        dict(name="attention_grad_odd_f32", op="attention_grad", dtype="f32", lens="777,300,63", G=1, H=5, K=24, V=40,
             packed=True),
        # One user's next token.
        dict(name="step_one", op="step", dtype="bf16", rows=1, slots=4, G=16, H=16, K=128, V=128),
        # A full decoding batch over a state cache.
        dict(name="step_batch", op="step", dtype="bf16", rows=192, slots=256, G=16, H=16, K=128, V=128),
        # Decoding: a few rows, the residual added, 8-bit output for the next projection.
        dict(name="norm_decode_fp8", op="norm_fp8", dtype="bf16", rows=4, D=4096),
        # A training batch: 16384 tokens with the residual added.
        dict(name="norm_train", op="norm", dtype="bf16", rows=16384, D=2048),
        # Its gradients, with a gradient that arrives through the residual too.
        dict(name="norm_grad", op="norm_grad", dtype="bf16", rows=16384, D=2048),
        # Decoding: three rows against a projection's weights.
        dict(name="matmul_decode", op="matmul", dtype="bf16", M=3, N=6144, K=4096),
        # A prompt's projection, an odd count of rows.
        dict(name="matmul_prompt", op="matmul", dtype="bf16", M=5001, N=4096, K=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_grad", "step", "norm_fp8", "norm", "norm_grad", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("attention", "attention_grad", "step"):
        H = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
        G = rng.choice([g for g in range(1, H + 1) if H % g == 0] + [H])
        K = rng.choice([16, 32, 48, 64, 100, 128, 128, 192, 256, rng.randint(1, 256)])
        V = rng.choice([32, 40, 64, 64, 96, 128, 128, 256, rng.randint(1, 320)])
        case = dict(op=op, dtype=dtype, G=G, H=H, K=K, V=V)
        if op == "step":
            rows = _log_int(rng, 1, max(1, min(256, (192 * 16 * 128 * 128) // (H * K * V))))
            case.update(rows=rows, slots=rows + rng.randint(0, 64))
            return case
        most = 32768 if op == "attention" else 8192
        most = min(most, (most * 16 * 128 * 128) // (H * max(K, 32) * max(V, 32)))
        most = max(16, min(most, 500_000_000 // (4 * (G * K + H * V) * (2 if dtype == "bf16" else 4))))
        if rng.random() < 0.5:
            lens = [_log_int(rng, 1, most)]
            left = most - lens[0]
            while len(lens) < rng.randint(1, 12) and left > 0:
                lens.append(rng.choice([0, 1, _log_int(rng, 1, left)]))
                left -= lens[-1]
            rng.shuffle(lens)
            case["packed"] = True
        else:
            count = _log_int(rng, 1, 16)
            lens = [_log_int(rng, 1, max(1, most // count))] * count
            case["packed"] = False
        case["lens"] = ",".join(str(n) for n in lens)
        return case
    if op.startswith("norm"):
        D = rng.choice([_log_int(rng, 32, 8192), 8 * _log_int(rng, 4, 1024), 128 * rng.randint(1, 64)])
        rows = _log_int(rng, 1, max(1, (1 << (25 if dtype == "bf16" else 24)) // D))
        return dict(op=op, dtype=dtype, rows=rows, D=D)
    K = rng.choice([128 * rng.randint(1, 40), 16 * _log_int(rng, 1, 320), _log_int(rng, 1, 4096)])
    N = rng.choice([_log_int(rng, 16, 8192), 128 * rng.randint(1, 48)])
    M = _log_int(rng, 1, max(1, min(16384, (1 << 36) // (K * N))))
    return dict(op=op, dtype=dtype, M=M, N=N, K=K)


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    s = {"op": case["op"], "case": dict(case)}
    if case["op"] in ("attention", "attention_grad", "step"):
        G, H, K, V = case["G"], case["H"], case["K"], case["V"]
        s["scale"] = K ** -0.5
        # a head's rate spans slow (a memory of thousands of tokens) to fast; each token's step varies around it
        rate = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(500.0) + math.log(1e-3))
        if case["op"] == "step":
            rows, slots = case["rows"], case["slots"]
            s["q"], s["k"], s["v"] = (normal(rows, n, d).to(dtype) for n, d in ((G, K), (G, K), (H, V)))
            s["g"] = -rate * torch.nn.functional.softplus(normal(rows, H) + 0.5)
            s["state"] = normal(slots, H, K, V)
            s["index"] = torch.randperm(slots, generator=gen, device=dev)[:rows].to(torch.int32)
            return s
        lens = _lens(case)
        s["lens"] = np.asarray(lens, dtype=np.int64)
        T = sum(lens)
        lead = (T,) if case["packed"] else (len(lens), lens[0])
        # queries, keys and values as one projection leaves them: three ranges of a row
        row = normal(*lead, 2 * G * K + H * V).to(dtype)
        s["q"] = row[..., :G * K].unflatten(-1, (G, K))
        s["k"] = row[..., G * K:2 * G * K].unflatten(-1, (G, K))
        s["v"] = row[..., 2 * G * K:].unflatten(-1, (H, V))
        s["g"] = -rate * torch.nn.functional.softplus(normal(*lead, H) + 0.5)
        s["state"] = normal(len(lens), H, K, V)
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
        if case["op"] == "attention_grad":
            s["do"] = normal(*lead, H, V).to(dtype)
            s["dstate"] = normal(len(lens), H, K, V, std=0.1)
        return s
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        s["dtype"] = dtype
        s["a"] = normal(M, K, std=100.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["b"] = normal(N, K, std=100.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["sa"] = torch.exp(normal(M, kb, std=0.5)) / 100.0
        s["sb"] = torch.exp(normal(-(-N // BLOCK), kb, std=0.5)) * (0.01 / math.sqrt(K))
        return s
    rows, D = case["rows"], case["D"]
    # a residual stream: channels of their own scale, a few of them large
    spread = torch.exp(normal(D, std=0.7))
    s["x"] = (normal(rows, D) * spread).to(dtype)
    s["w"] = 1.0 + normal(D, std=0.2)
    s["eps"] = 1e-6
    if case["op"] == "norm_grad":
        s["dy"], s["dr"] = normal(rows, D).to(dtype), normal(rows, D).to(dtype)
    else:
        s["r"] = (normal(rows, D) * spread).to(dtype)
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import selective_scan_crossscan_amd as ss2d

    op = s["op"]
    if op == "attention":
        o, last = ss2d.linear_attention(s["q"], s["k"], s["v"], s["g"], state=s["state"], cu_seqlens=s["cu"],
                                        scale=s["scale"], final_state=True)
        return {"o": o, "state": last}
    if op == "attention_grad":
        return ss2d.linear_attention_backward(s["q"], s["k"], s["v"], s["g"], s["do"], state=s["state"],
                                              dfinal_state=s["dstate"], cu_seqlens=s["cu"], scale=s["scale"])
    if op == "step":
        o = ss2d.linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], state_index=s["index"],
                                       scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "norm":
        y, r = ss2d.rms_norm(s["x"], s["w"], residual=s["r"], eps=s["eps"])
        return {"y": y, "r": r}
    if op == "norm_fp8":
        y, scales, r = ss2d.rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=s["eps"])
        return {"y": y, "scales": scales, "r": r}
    if op == "norm_grad":
        return ss2d.rms_norm_backward(s["x"], s["w"], s["dy"], dresidual=s["dr"], eps=s["eps"])
    return ss2d.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=s["dtype"])


def _plain(s):
    op = s["op"]
    if op == "attention":
        dtype = s["v"].dtype
        o, last = _plain_attention(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["state"], s)
        return {"o": o.to(dtype), "state": last}
    if op == "attention_grad":
        leaves = [s[n].float().detach().requires_grad_() for n in ("q", "k", "v", "g", "state")]
        o, last = _plain_attention(*leaves, s)
        grads = torch.autograd.grad([o, last], leaves, [s["do"].float(), s["dstate"]])
        dtype = s["v"].dtype
        return {"dq": grads[0].to(dtype), "dk": grads[1].to(dtype), "dv": grads[2].to(dtype), "dlog_decay": grads[3],
                "dstate": grads[4]}
    if op == "step":
        H, dtype, at = s["v"].shape[1], s["v"].dtype, s["index"].long()
        q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1) for n in ("q", "k"))
        h = s["state"][at] * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
        s["state"][at] = h
        return {"o": ((q[..., None] * h).sum(-2) * s["scale"]).to(dtype), "state": s["state"]}
    if op == "matmul":
        K = s["a"].shape[1]
        a = s["a"].float() * s["sa"].repeat_interleave(BLOCK, 1)[:, :K]
        b = s["b"].float() * s["sb"].repeat_interleave(BLOCK, 0)[:s["b"].shape[0]].repeat_interleave(BLOCK, 1)[:, :K]
        return (a @ b.t()).to(s["dtype"])
    dtype = s["x"].dtype
    if op == "norm_grad":
        x, dy = s["x"].float(), s["dy"].float()
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        xhat, gy = x * rstd, dy * s["w"]
        dx = s["dr"].float() + rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
        return {"dx": dx.to(dtype), "dweight": (dy * xhat).sum(0)}
    r = s["x"].float() + s["r"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + s["eps"]) * s["w"]
    if op == "norm":
        return {"y": y.to(dtype), "r": r.to(dtype)}
    rows, D = y.shape
    blocks = torch.nn.functional.pad(y, (0, -D % BLOCK)).unflatten(-1, (-1, BLOCK))
    scales = (blocks.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    values = (blocks / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :D]
    return {"y": values.to(torch.float8_e4m3fn), "scales": scales, "r": r.to(dtype)}


def _plain_attention(q, k, v, g, state, s):
    """o, final state of h_t = exp(g_t) h_{t-1} + k_t v_t', o_t = scale h_t' q_t, in chunks: inside a chunk as a
    masked product of queries and keys, between chunks through the chunks' states. Decays are summed in 64 bits."""
    lens, dev = s["lens"], q.device
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = -(-lens // CHUNK)  # chunks of each sequence
    first = np.cumsum(n) - n
    seq = np.repeat(np.arange(len(lens)), n)
    at = cu[seq] + (np.arange(n.sum()) - first[seq]) * CHUNK
    idx = at[:, None] + np.arange(CHUNK)
    valid = torch.from_numpy(idx < cu[seq + 1][:, None]).to(dev)
    idx = torch.from_numpy(np.minimum(idx, cu[-1] - 1)).to(dev)
    last, has = torch.from_numpy(np.maximum(first + n - 1, 0)).to(dev), torch.from_numpy(n > 0).to(dev)
    seq_t, first_t = torch.from_numpy(seq).to(dev), torch.from_numpy(np.minimum(first, max(0, n.sum() - 1))).to(dev)
    H, lead = v.shape[-2], v.shape[:-2]
    rep = H // q.shape[-2]

    def chunked(x):  # (chunks, H, CHUNK, dim), zeros behind the sequence's end
        x = x.reshape(-1, *x.shape[len(lead):])[idx]
        return torch.where(valid[..., None, None], x, x.new_zeros(())).transpose(1, 2)

    qc, kc, vc = chunked(q.repeat_interleave(rep, -2)), chunked(k.repeat_interleave(rep, -2)), chunked(v)
    G = torch.cumsum(chunked(g[..., None].double())[..., 0], -1)  # (chunks, H, CHUNK)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~tri, -math.inf)).float()
    o = ((qc @ kc.transpose(-1, -2)) * decay) @ vc
    total = G[..., -1]
    U = (kc * torch.exp(total[..., None] - G).float()[..., None]).transpose(-1, -2) @ vc  # (chunks, H, K, V)
    P = torch.cumsum(total, 0)  # decay up to a chunk's end; before - first's - inside one sequence only
    before = P - total
    c = torch.arange(len(seq), device=dev)
    earlier = (seq_t[:, None] == seq_t[None, :]) & (c[:, None] > c[None, :])
    between = (before.t()[:, :, None] - P.t()[:, None, :]).masked_fill(~earlier, -math.inf)  # (H, chunk, from chunk)
    Uh = U.transpose(0, 1).flatten(2)  # (H, chunks, K V)
    start = (torch.exp(between).float() @ Uh).unflatten(-1, U.shape[-2:]).transpose(0, 1)
    start = start + torch.exp(before - before[first_t][seq_t]).float()[..., None, None] * state[seq_t]
    o = o + torch.exp(G).float()[..., None] * (qc @ start)
    inside = (seq_t[None, :] == torch.arange(len(lens), device=dev)[:, None])
    to_end = (P[last].t()[:, :, None] - P.t()[:, None, :]).masked_fill(~inside, -math.inf)  # (H, sequence, chunk)
    final = (torch.exp(to_end).float() @ Uh).unflatten(-1, U.shape[-2:]).transpose(0, 1)
    whole = torch.where(has[:, None], P[last] - before[first_t], P.new_zeros(()))
    final = final + torch.exp(whole).float()[..., None, None] * state
    o = (o * s["scale"]).transpose(1, 2)[valid]
    return o.reshape(*lead, H, -1), final


# ----------------------------------------------------------------------------- the least work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("attention", "attention_grad", "step"):
        G, H, K, V = case["G"], case["H"], case["K"], case["V"]
        T = case["rows"] if op == "step" else sum(_lens(case))
        S = case["rows"] if op == "step" else len(_lens(case))
        qk, vo, g, st = 2 * T * G * K * e, T * H * V * e, T * H * 4, S * H * K * V * 4
        if op == "attention_grad":  # q, k, v, do in, dq, dk, dv out; states h and dh, three products with them
            return {"bytes": 2 * qk + 3 * vo + 2 * g + 3 * st, "flops": 10 * T * H * K * V}
        return {"bytes": qk + 2 * vo + g + 2 * st, "flops": 4 * T * H * K * V}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        return {"bytes": M * K + N * K + (M + -(-N // BLOCK)) * kb * 4 + M * N * e, "flops": 2 * M * N * K}
    n, D = case["rows"] * case["D"], case["D"]
    if op == "norm":
        return {"bytes": 4 * n * e + 4 * D, "flops": 5 * n}
    if op == "norm_fp8":
        return {"bytes": 3 * n * e + n + case["rows"] * -(-D // BLOCK) * 4 + 4 * D, "flops": 7 * n}
    return {"bytes": 4 * n * e + 8 * D, "flops": 10 * n}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("attention", "attention_grad"):
            return _exact_attention(s)
        if op == "step":
            at = s["index"].long()
            rep = s["v"].shape[1] // s["q"].shape[1]
            cache = s["state"].double()
            new = cache[at] * s["g"].double().exp()[:, :, None, None]
            new += torch.einsum("bhk,bhv->bhkv", s["k"].double().repeat_interleave(rep, 1), s["v"].double())
            cache[at] = new
            o = torch.einsum("bhk,bhkv->bhv", s["q"].double().repeat_interleave(rep, 1), new)
            return {"o": o * s["scale"], "state": cache}
        if op == "matmul":
            M, N = s["a"].shape[0], s["b"].shape[0]
            out = torch.zeros(M, N, dtype=torch.float64, device=s["a"].device)
            for i in range(s["sa"].shape[1]):  # block by block of the inner dimension
                cols = slice(i * BLOCK, (i + 1) * BLOCK)
                part = torch.mm(s["a"][:, cols].double(), s["b"][:, cols].double().t())
                out += part * s["sa"][:, i].double()[:, None] * s["sb"][:, i].double().repeat_interleave(BLOCK)[:N]
            return out
        x, w = s["x"].double(), s["w"].double()
        if op == "norm_grad":
            D = x.shape[1]
            m = (x ** 2).sum(1, keepdim=True) / D + s["eps"]
            dy = s["dy"].double()
            dot = (dy * w * x).sum(1, keepdim=True)
            dx = s["dr"].double() + dy * w / m.sqrt() - x * dot / (D * m ** 1.5)
            return {"dx": dx, "dweight": (dy * x / m.sqrt()).sum(0)}
        r = x + s["r"].double()
        y = r / ((r ** 2).mean(1, keepdim=True) + s["eps"]).sqrt() * w
        if op == "norm":
            return {"y": y, "r": r}
        rows, D = y.shape
        scales = torch.stack([y[:, i:i + BLOCK].abs().amax(1) for i in range(0, D, BLOCK)], 1) / E4M3_MAX
        scales = scales.clamp_min(SCALE_MIN)
        values = y / scales.repeat_interleave(BLOCK, 1)[:, :D]
        return {"y": values.float().to(torch.float8_e4m3fn).double(), "scales": scales, "r": r}


def _exact_attention(s):
    """The recurrence token by token, all sequences at once (shorter ones rest at their ends)."""
    lens = [int(n) for n in s["lens"]]
    S, L = len(lens), max(lens)
    H = s["v"].shape[-2]
    rep = H // s["q"].shape[-2]
    cu = [sum(lens[:i]) for i in range(S)]

    def padded(x):  # (tokens, ...) -> (L, S, ...), zeros behind a sequence's end
        out = torch.zeros(L, S, *x.shape[1:], dtype=torch.float64, device=x.device)
        for i in range(S):
            out[:lens[i], i] = x[cu[i]:cu[i] + lens[i]].double()
        return out

    flat = {n: s[n].reshape(-1, *s[n].shape[-2:]) for n in ("q", "k", "v")}
    q, k = (padded(flat[n].repeat_interleave(rep, 1)) for n in ("q", "k"))
    v = padded(flat["v"])
    a = torch.exp(padded(s["g"].reshape(-1, H, 1))[..., 0])[..., None, None]  # 1 behind the end
    h = s["state"].double()

    def whole(x, shape):  # back from (L, S, ...) to the tokens' layout
        return torch.cat([x[:lens[i], i] for i in range(S)]).reshape(shape)

    if s["op"] == "attention":
        o = torch.zeros_like(v)
        for t in range(L):
            h = torch.addcmul(h * a[t], k[t][..., None], v[t][..., None, :])
            o[t] = torch.matmul(q[t][..., None, :], h)[..., 0, :]
        return {"o": whole(o, s["v"].shape) * s["scale"], "state": h}
    scale = s["scale"]
    do = padded(s["do"].reshape(-1, *s["do"].shape[-2:])) * scale
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(L):
        h = torch.addcmul(h * a[t], k[t][..., None], v[t][..., None, :])
        dq[t] = torch.matmul(h, do[t][..., None])[..., 0]
    d = s["dstate"].double()
    at_end = (h * d).sum((-1, -2))  # what the final state's gradient sees of all decays, per sequence and head
    for t in range(L - 1, -1, -1):
        d = torch.addcmul(d, q[t][..., None], do[t][..., None, :])
        dk[t] = torch.matmul(d, v[t][..., None])[..., 0]
        dv[t] = torch.matmul(k[t][..., None, :], d)[..., 0, :]
        d = d * a[t]
    # a decay acts on every later output and the final state, through every earlier key
    flow = ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(0).cumsum(0).flip(0) + at_end

    def grouped(x):
        return x.unflatten(2, (-1, rep)).sum(3)

    return {"dq": whole(grouped(dq), s["q"].shape), "dk": whole(grouped(dk), s["k"].shape),
            "dv": whole(dv, s["v"].shape), "dlog_decay": whole(flow, s["g"].shape), "dstate": d}
