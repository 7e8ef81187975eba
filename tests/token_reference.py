"""Linear attention with a decay per head and its gradients in torch float64, token by token and on the inputs' device:
for sizes that oracle/tokens.py, which says the same in numpy and pins this one, would take minutes for."""
import torch


def attention(q, k, v, g, lens, state=None, scale=1.0):
    """q, k (T,G,K), v (T,H,V), g (T,H), state (S,H,K,V) or None -> o (T,H,V), final states."""
    q, k, v, a = q.double(), k.double(), v.double(), g.double().exp()
    H, V = v.shape[1:]
    rep, K = H // q.shape[1], q.shape[2]
    last = torch.zeros(len(lens), H, K, V, dtype=torch.float64, device=v.device) if state is None else state.double().clone()
    o = torch.zeros_like(v)
    t = 0
    for s, n in enumerate(lens):
        h = last[s]
        for _ in range(n):
            h = h * a[t][:, None, None] + k[t].repeat_interleave(rep, 0)[:, :, None] * v[t][:, None, :]
            o[t] = (q[t].repeat_interleave(rep, 0)[:, :, None] * h).sum(1) * scale
            t += 1
        last[s] = h
    return o, last


def attention_backward(q, k, v, g, do, lens, state=None, dlast=None, scale=1.0):
    """dq, dk, dv, dg, dstate of sum(o do) + sum(last dlast)."""
    q, k, v, do, a = q.double(), k.double(), v.double(), do.double(), g.double().exp()
    H, V = v.shape[1:]
    G, K = q.shape[1:]
    rep = H // G
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, a))
    dstate = torch.zeros(len(lens), H, K, V, dtype=torch.float64, device=v.device)
    t0 = 0
    for s, n in enumerate(lens):
        h = torch.zeros(n + 1, H, K, V, dtype=torch.float64, device=v.device)
        if state is not None:
            h[0] = state[s]
        for i in range(n):
            t = t0 + i
            h[i + 1] = h[i] * a[t][:, None, None] + k[t].repeat_interleave(rep, 0)[:, :, None] * v[t][:, None, :]
        d = torch.zeros_like(h[0]) if dlast is None else dlast[s].double().clone()
        for i in range(n - 1, -1, -1):
            t = t0 + i
            d = d + scale * q[t].repeat_interleave(rep, 0)[:, :, None] * do[t][:, None, :]
            dq[t] = scale * (h[i + 1] * do[t][:, None, :]).sum(-1).view(G, rep, K).sum(1)
            dk[t] = (d * v[t][:, None, :]).sum(-1).view(G, rep, K).sum(1)
            dv[t] = (d * k[t].repeat_interleave(rep, 0)[:, :, None]).sum(1)
            dg[t] = a[t] * (d * h[i]).sum((-1, -2))
            d = a[t][:, None, None] * d
        dstate[s] = d
        t0 += n
    return dq, dk, dv, dg, dstate
