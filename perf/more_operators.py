"""Measured cases of the gated delta rule (prompts, its gradients, single tokens over a state cache) and of the norms
of queries and keys for each head with the position rotation in the same pass (and their gradients).

`own` False computes each operator in its plain form, in elementary torch operations; True calls the library.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # chunk of the plain delta rule
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # A chat turn's few short prompts, one of a single token, continuing from kept states: latency counts.
        dict(name="delta_short", op="delta", dtype="bf16", lens="1,37,70", G=4, H=4, K=64, V=64, packed=True),
        # A training batch's forward: 16 sequences of 2048 tokens, 16 heads of 128.
        dict(name="delta_batch", op="delta", dtype="bf16", lens=",".join(["2048"] * 16), G=16, H=16, K=128, V=128,
             packed=False),
        # A serving batch packed without padding: one long document beside ragged prompts and an empty one, pairs of
        # value heads sharing a key.
        dict(name="delta_long", op="delta", dtype="bf16", lens="32768,4097,0,1023,255,1", G=8, H=16, K=128, V=128,
             packed=True),
        # The tokens of 56 x 56 feature maps, 192 channels as 6 heads of 32 that share keys of 16 states, fp32.
        dict(name="delta_map_f32", op="delta", dtype="f32", lens="3136,3136,3136,3136", G=1, H=6, K=16, V=32,
             packed=False),
        # A training step's layer: two sequences of 4096 tokens, 16 heads of 128.
        dict(name="delta_grad", op="delta_grad", dtype="bf16", lens="4096,4096", G=16, H=16, K=128, V=128,
             packed=False),
        # Odd sizes in fp32, one group of keys and queries shared by all heads.
        dict(name="delta_grad_odd_f32", op="delta_grad", dtype="f32", lens="777,300,63", G=1, H=5, K=24, V=40,
             packed=True),
        # One user's next token.
        dict(name="step_one", op="step", dtype="bf16", rows=1, slots=4, G=16, H=16, K=128, V=128),
        # A full decoding batch over a state cache, pairs of value heads sharing a key.
        dict(name="step_batch", op="step", dtype="bf16", rows=192, slots=256, G=8, H=16, K=128, V=128),
        # Decoding: eight rows at positions of their own, 16 query heads and 4 key heads.
        dict(name="qk_decode", op="qk", dtype="bf16", T=8, Hq=16, Hk=4, D=128, rot=128, interleaved=False, far=32768),
        # A prompt or training batch: 16384 tokens, 16 heads each.
        dict(name="qk_prompt", op="qk", dtype="bf16", T=16384, Hq=16, Hk=16, D=128, rot=128, interleaved=False,
             far=32768),
        # Its gradients.
        dict(name="qk_grad", op="qk_grad", dtype="bf16", T=16384, Hq=16, Hk=16, D=128, rot=128, interleaved=False,
             far=32768),
        # Odd sizes in fp32: heads of 24 of which 10 channels rotate, in neighbouring pairs, one key head.
        dict(name="qk_grad_odd_f32", op="qk_grad", dtype="f32", T=4097, Hq=5, Hk=1, D=24, rot=10, interleaved=True,
             far=4097),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_grad", "step", "qk", "qk_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk", "qk_grad"):
        D = rng.choice([24, 32, 64, 64, 96, 128, 128, 256, rng.randint(1, 256)])
        Hk = rng.choice([1, 2, 4, 5, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 3, 4])
        most = (1 << (26 if dtype == "bf16" else 25)) // (D * (Hq + Hk))
        rot = rng.choice([D // 2 * 2, D // 2 * 2, D // 4 * 2, 0])
        T = _log_int(rng, 1, max(1, min(32768, most)))
        return dict(op=op, dtype=dtype, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, interleaved=rng.random() < 0.3,
                    far=max(1, T, rng.choice([1024, 8192, 65536])))
    H = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    G = rng.choice([g for g in range(1, H + 1) if H % g == 0] + [H])
    K = rng.choice([16, 32, 48, 64, 100, 128, 128, 192, 256, rng.randint(1, 256)])
    V = rng.choice([32, 40, 64, 64, 96, 128, 128, 256, rng.randint(1, 320)])
    case = dict(op=op, dtype=dtype, G=G, H=H, K=K, V=V)
    if op == "step":
        rows = _log_int(rng, 1, max(1, min(256, (192 * 16 * 128 * 128) // (H * K * V))))
        case.update(rows=rows, slots=rows + rng.randint(0, 64))
        return case
    most = 32768 if op == "delta" else 8192
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
    if case["op"] in ("qk", "qk_grad"):
        T, Hq, Hk, D, rot = (case[n] for n in ("T", "Hq", "Hk", "D", "rot"))
        # queries and keys as one projection leaves them: two ranges of a row, the values' behind them
        row = (normal(T, (Hq + 2 * Hk) * D) * torch.exp(normal(T, 1, std=0.5))).to(dtype)
        s["q"] = row[:, :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = row[:, Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["wq"], s["wk"] = 1.0 + normal(D, std=0.2), 1.0 + normal(D, std=0.2)
        s["eps"], s["interleaved"], s["table"], s["positions"] = 1e-6, case["interleaved"], None, None
        if rot:
            # the table of all positions that a program keeps, and where these tokens stand: a packed batch's
            # positions, each prompt counting from a place of its own
            rate = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
            angle = torch.arange(case["far"], dtype=torch.float64, device=dev)[:, None] * rate
            s["table"] = torch.cat([angle.cos(), angle.sin()], -1).float()
            start = torch.randint(0, case["far"], (-(-T // 256),), generator=gen, device=dev)
            at = start.repeat_interleave(256)[:T] + torch.arange(T, device=dev) % 256
            s["positions"] = (at % case["far"]).to(torch.int32)
        if case["op"] == "qk_grad":
            s["dq"], s["dk"] = normal(T, Hq, D).to(dtype), normal(T, Hk, D).to(dtype)
        return s
    G, H, K, V = case["G"], case["H"], case["K"], case["V"]
    s["scale"] = K ** -0.5
    # a head's rate spans slow (a memory of thousands of tokens) to fast; each token's step varies around it
    rate = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(500.0) + math.log(1e-3))

    def unit(x):  # queries and keys come normalised
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dtype)

    if case["op"] == "step":
        rows, slots = case["rows"], case["slots"]
        s["q"], s["k"] = unit(normal(rows, G, K)) * K ** 0.5, unit(normal(rows, G, K))
        s["v"] = normal(rows, H, V).to(dtype)
        s["g"] = -rate * torch.nn.functional.softplus(normal(rows, H) + 0.5)
        s["beta"] = torch.sigmoid(normal(rows, H))
        s["state"] = normal(slots, H, K, V)
        s["index"] = torch.randperm(slots, generator=gen, device=dev)[:rows].to(torch.int32)
        return s
    lens = _lens(case)
    s["lens"] = np.asarray(lens, dtype=np.int64)
    T = sum(lens)
    lead = (T,) if case["packed"] else (len(lens), lens[0])
    s["q"], s["k"] = unit(normal(*lead, G, K)) * K ** 0.5, unit(normal(*lead, G, K))
    # values as a projection of several leaves them: a range of a row
    s["v"] = normal(*lead, H * V + 64).to(dtype)[..., :H * V].unflatten(-1, (H, V))
    s["g"] = -rate * torch.nn.functional.softplus(normal(*lead, H) + 0.5)
    s["beta"] = torch.sigmoid(normal(*lead, H))
    s["state"] = normal(len(lens), H, K, V)
    s["cu"] = None
    if case["packed"]:
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    if case["op"] == "delta_grad":
        s["do"] = normal(*lead, H, V).to(dtype)
        s["dstate"] = normal(len(lens), H, K, V, std=0.1)
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import selective_scan_crossscan_amd as ss2d

    op = s["op"]
    if op == "delta":
        o, last = ss2d.delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], cu_seqlens=s["cu"],
                                  scale=s["scale"], final_state=True)
        return {"o": o, "state": last}
    if op == "delta_grad":
        return ss2d.delta_rule_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], state=s["state"],
                                        dfinal_state=s["dstate"], cu_seqlens=s["cu"], scale=s["scale"])
    if op == "step":
        o = ss2d.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], state_index=s["index"],
                                 scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "qk":
        q, k = ss2d.qk_norm(s["q"], s["k"], s["wq"], s["wk"], rotation=s["table"], positions=s["positions"],
                            interleaved=s["interleaved"], eps=s["eps"])
        return {"q": q, "k": k}
    return ss2d.qk_norm_backward(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], rotation=s["table"],
                                 positions=s["positions"], interleaved=s["interleaved"], eps=s["eps"])


def _plain(s):
    op = s["op"]
    if op == "delta":
        dtype = s["v"].dtype
        o, last = _plain_delta(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["state"], s)
        return {"o": o.to(dtype), "state": last}
    if op == "delta_grad":
        leaves = [s[n].float().detach().requires_grad_() for n in ("q", "k", "v", "g", "beta", "state")]
        o, last = _plain_delta(*leaves, s)
        grads = torch.autograd.grad([o, last], leaves, [s["do"].float(), s["dstate"]])
        dtype = s["v"].dtype
        return {"dq": grads[0].to(dtype), "dk": grads[1].to(dtype), "dv": grads[2].to(dtype), "dlog_decay": grads[3],
                "dbeta": grads[4], "dstate": grads[5]}
    if op == "step":
        H, dtype, at = s["v"].shape[1], s["v"].dtype, s["index"].long()
        q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1) for n in ("q", "k"))
        h = s["state"][at] * torch.exp(s["g"])[..., None, None]
        e = s["v"].float() - (k[..., None] * h).sum(-2)
        h = h + k[..., None] * (s["beta"][..., None] * e)[..., None, :]
        s["state"][at] = h
        return {"o": ((q[..., None] * h).sum(-2) * s["scale"]).to(dtype), "state": s["state"]}
    dtype = s["q"].dtype
    if op == "qk":
        return {n: _plain_rotate(_plain_norm(s[n], s["eps"]) * s["w" + n], s, 1.0).to(dtype) for n in ("q", "k")}
    out = {}
    for n in ("q", "k"):
        dy = _plain_rotate(s["d" + n].float(), s, -1.0)
        xhat, gy = _plain_norm(s[n], s["eps"]), dy * s["w" + n]
        rstd = torch.rsqrt(s[n].float().square().mean(-1, keepdim=True) + s["eps"])
        out["d" + n] = (rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))).to(dtype)
        out["d%s_weight" % n] = (dy * xhat).sum((0, 1))
    return out


def _plain_norm(x, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)


def _plain_rotate(y, s, sign):
    """Pairs of channels turned by the token's angles (sign -1: back); y (T, heads, D) fp32."""
    if s["table"] is None:
        return y
    rot = s["table"].shape[1]
    cos, sin = s["table"][s["positions"].long()][:, None].split(rot // 2, -1)
    sin = sin * sign
    x = y[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
    axis = -1 if s["interleaved"] else -2
    a, b = x.unbind(axis)
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], axis).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_delta(q, k, v, g, beta, state, s):
    """o, final state of h_t = exp(g_t) h_{t-1} + beta_t k_t (v_t - exp(g_t) h_{t-1}' k_t)', o_t = scale h_t' q_t, in
    chunks: inside a chunk the triangular system of the tokens' errors is inverted, by halves; the chunks follow each
    other, all sequences' and heads' at once. Decays are summed in 64 bits."""
    lens, dev = s["lens"], q.device
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = -(-lens // CHUNK)  # chunks of each sequence
    seq = np.repeat(np.arange(len(lens)), n)
    num = np.arange(n.sum()) - (np.cumsum(n) - n)[seq]  # a chunk's number in its sequence
    order = np.argsort(-n, kind="stable")  # sequences, the longest first
    place = np.argsort(order, kind="stable")
    by = np.lexsort((place[seq], num))  # chunks: all first ones, all second ones, ...
    seq, num = seq[by], num[by]
    counts = np.bincount(num).tolist()  # sequences that have a first, a second, ... chunk
    idx = (cu[seq] + num * CHUNK)[:, None] + np.arange(CHUNK)
    valid = torch.from_numpy(idx < cu[seq + 1][:, None]).to(dev)
    idx = torch.from_numpy(np.minimum(idx, cu[-1] - 1)).to(dev)
    H, lead = v.shape[-2], v.shape[:-2]
    rep = H // q.shape[-2]

    def chunked(x):  # (chunks, H, CHUNK, dim), zeros behind the sequence's end
        x = x.reshape(-1, *x.shape[len(lead):])[idx]
        return torch.where(valid[..., None, None], x, x.new_zeros(())).transpose(1, 2)

    qc, kc, vc = chunked(q.repeat_interleave(rep, -2)), chunked(k.repeat_interleave(rep, -2)), chunked(v)
    b = chunked(beta[..., None])
    G = torch.cumsum(chunked(g[..., None].double())[..., 0], -1)  # (chunks, H, CHUNK)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~tri, -math.inf)).float()
    T = _plain_inverse((kc @ kc.transpose(-1, -2)) * decay * b.transpose(-1, -2))
    since = torch.exp(G).float()[..., None]
    W, E, P = T @ (kc * since), T @ vc, (qc @ kc.transpose(-1, -2)) * decay
    left = kc * torch.exp(G[..., -1:] - G).float()[..., None]
    h, outs, ends = state[torch.from_numpy(order).to(dev)], [], []
    for W, E, P, q, l, b, f in zip(*(x.split(counts) for x in (W, E, P, qc * since, left, b, since[..., -1:, :]))):
        ends.append(h[len(b):])  # sequences that ended before
        h = h[:len(b)]
        u = b * (E - W @ h)
        outs.append(q @ h + P @ u)
        h = f * h + l.transpose(-1, -2) @ u
    last = torch.cat([h] + ends[::-1])[torch.from_numpy(place).to(dev)]
    o = torch.cat(outs).transpose(1, 2)
    back = torch.zeros(int(cu[-1]), dtype=torch.int64, device=dev)
    back[idx[valid]] = torch.arange(idx.numel(), device=dev)[valid.flatten()]  # where a token's output is
    return (o.flatten(0, 1)[back] * s["scale"]).reshape(*lead, H, -1), last


def _plain_inverse(A):
    """(1 + the strictly lower part of A)^-1, by halves: two inverted blocks of a pair give the pair's."""
    n = A.shape[-1]
    inv = torch.eye(n, device=A.device).expand(A.shape)
    row = torch.arange(n, device=A.device)
    size = 1
    while size < n:
        below = (row[:, None] // (2 * size) == row // (2 * size)) & (row[:, None] // size > row // size)
        inv = inv - inv @ torch.where(below, A, A.new_zeros(())) @ inv
        size *= 2
    return inv


# ----------------------------------------------------------------------------- the least work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("qk", "qk_grad"):
        rows, D = case["T"] * (case["Hq"] + case["Hk"]), case["D"]
        turn = case["T"] * (case["rot"] * 4 + 4) if case["rot"] else 0
        if op == "qk":
            return {"bytes": 2 * rows * D * e + turn + 8 * D, "flops": 7 * rows * D}
        return {"bytes": 3 * rows * D * e + turn + 16 * D, "flops": 14 * rows * D}
    G, H, K, V = case["G"], case["H"], case["K"], case["V"]
    T = case["rows"] if op == "step" else sum(_lens(case))
    S = case["rows"] if op == "step" else len(_lens(case))
    qk, vo, g, st = 2 * T * G * K * e, T * H * V * e, 2 * T * H * 4, S * H * K * V * 4
    if op == "delta_grad":  # q, k, v, do in, dq, dk, dv out; the states' two products again, six of their gradients
        return {"bytes": 2 * qk + 3 * vo + 2 * g + 3 * st, "flops": 16 * T * H * K * V}
    return {"bytes": qk + 2 * vo + g + 2 * st, "flops": 6 * T * H * K * V}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("delta", "delta_grad"):
            return _exact_delta(s)
        if op == "step":
            at = s["index"].long()
            rep = s["v"].shape[1] // s["q"].shape[1]
            q, k = (s[n].double().repeat_interleave(rep, 1) for n in ("q", "k"))
            cache = s["state"].double()
            h = cache[at] * s["g"].double().exp()[:, :, None, None]
            e = s["v"].double() - torch.einsum("bhk,bhkv->bhv", k, h)
            h += torch.einsum("bhk,bhv->bhkv", k, e * s["beta"].double()[..., None])
            cache[at] = h
            return {"o": torch.einsum("bhk,bhkv->bhv", q, h) * s["scale"], "state": cache}
        out = {}
        for n in ("q", "k"):
            x, w = s[n].double(), s["w" + n].double()
            D = x.shape[-1]
            m = (x ** 2).sum(-1, keepdim=True) / D + s["eps"]
            if op == "qk":
                out[n] = _exact_turn(x / m.sqrt() * w, s, False)
                continue
            dy = _exact_turn(s["d" + n].double(), s, True)
            dot = (dy * w * x).sum(-1, keepdim=True)
            out["d" + n] = dy * w / m.sqrt() - x * dot / (D * m ** 1.5)
            out["d%s_weight" % n] = (dy * x / m.sqrt()).sum((0, 1))
        return out


def _exact_turn(y, s, back):
    if s["table"] is None:
        return y
    rot = s["table"].shape[1]
    at = s["table"].double()[s["positions"].long()]
    turn = torch.complex(at[:, :rot // 2], -at[:, rot // 2:] if back else at[:, rot // 2:])[:, None]
    first = torch.arange(0, rot, 2, device=y.device) if s["interleaved"] else torch.arange(rot // 2, device=y.device)
    second = first + (1 if s["interleaved"] else rot // 2)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_delta(s):
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
    a = torch.exp(padded(s["g"].reshape(-1, H, 1)))[..., None]  # 1 behind the end
    b = padded(s["beta"].reshape(-1, H, 1))
    h = s["state"].double()
    scale = s["scale"]

    def whole(x, shape):  # back from (L, S, ...) to the tokens' layout
        return torch.cat([x[:lens[i], i] for i in range(S)]).reshape(shape)

    def seen(x, h):  # h' x
        return torch.matmul(x[..., None, :], h)[..., 0, :]

    if s["op"] == "delta":
        o = torch.zeros_like(v)
        for t in range(L):
            h = h * a[t]
            h = torch.addcmul(h, k[t][..., None], (b[t] * (v[t] - seen(k[t], h)))[..., None, :])
            o[t] = seen(q[t], h)
        return {"o": whole(o, s["v"].shape) * scale, "state": h}
    do = padded(s["do"].reshape(-1, *s["do"].shape[-2:])) * scale
    kept = torch.zeros(L, *h.shape, dtype=torch.float64, device=h.device)  # decayed, before a token's own part
    error = torch.zeros_like(v)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(b), torch.zeros_like(b)
    for t in range(L):
        kept[t] = h * a[t]
        error[t] = v[t] - seen(k[t], kept[t])
        h = torch.addcmul(kept[t], k[t][..., None], (b[t] * error[t])[..., None, :])
        dq[t] = torch.matmul(h, do[t][..., None])[..., 0]
    d = s["dstate"].double()
    for t in range(L - 1, -1, -1):
        d = torch.addcmul(d, q[t][..., None], do[t][..., None, :])
        du = seen(k[t], d)
        db[t] = (du * error[t]).sum(-1, keepdim=True)
        dv[t] = b[t] * du
        dk[t] = torch.matmul(d, (b[t] * error[t])[..., None])[..., 0] - torch.matmul(kept[t], dv[t][..., None])[..., 0]
        d = torch.addcmul(d, k[t][..., None], dv[t][..., None, :], value=-1.0)
        dg[t] = (d * kept[t]).sum((-1, -2))[..., None]
        d = d * a[t]

    def grouped(x):
        return x.unflatten(2, (-1, rep)).sum(3)

    return {"dq": whole(grouped(dq), s["q"].shape), "dk": whole(grouped(dk), s["k"].shape),
            "dv": whole(dv, s["v"].shape), "dlog_decay": whole(dg, s["g"].shape), "dbeta": whole(db, s["g"].shape),
            "dstate": d}
