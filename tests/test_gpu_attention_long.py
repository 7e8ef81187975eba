"""Linear attention and its gradients on sequences long enough for every kernel that long prompts and
training steps run: tiles of 128 value columns for each padded key size, whole sequences and sequences in
segments, equal lengths and packed ones, shared keys; against a float64 reference on the GPU (which the
oracle pins).

Tolerances.  With |.| the operator on absolute values, fp32 results of T tokens are off by at most c |.|:
c = (T/8 + 128 + K) 2^-24 for outputs and states (per 64 tokens the state takes one product and at most eight
accumulations, each half a step of 2^-23; a term is a sum over K, a decay and two products), (T/8 + 256 + K + V)
2^-24 for gradients.  In bf16 an output adds its own rounding, 2^-8 of itself, and 2^-8 (1 + 2^-8) |.|: its terms
from inside a chunk pass a masked score rounded to bf16, those from the state before a chunk a state rounded to
bf16, each term one of the two.  dq and dk likewise have a rounded score in the chunk's terms only, dv both.  A
decay's gradient subtracts two sums of one chunk's terms, at most 64 of each token's |q||k||do||v|: its |.| is
taken as twice the largest within 64 tokens.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import token_reference

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def make(lens, G, H, K, V, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    q, k, v, do = (normal(T, n, d).to(DT[dtype]) for n, d in ((G, K), (G, K), (H, V), (H, V)))
    g = -torch.exp(torch.rand(T, H, generator=gen, device="cuda") * 7.6 - 6.9)  # 1e-3 .. 2
    return q, k, v, g, do, normal(len(lens), H, K, V), normal(len(lens), H, K, V)


def check(name, got, ref, tol):
    err = (got.double() - ref).abs()
    worst = float((err / tol).max())
    print(f"[long attention] {name}: worst error / tolerance {worst:.3f}", flush=True)
    assert bool((err <= tol).all()), (name, worst)


def shaped(x, lens, equal):
    """The call's layout: (S, L, ...) for equal lengths."""
    return x.view(len(lens), lens[0], *x.shape[1:]) if equal else x


def offsets(lens, equal):
    return None if equal else torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()


# lens, G, H, K, V, equal lengths: key sizes padded to 32, 64, 128 and 256, whole and ragged tiles, in segments and whole
FORWARD = [
    ([1290, 0, 70], 4, 64, 128, 128, False),
    ([1501], 64, 64, 128, 128, False),
    ([301] * 5, 2, 64, 128, 128, True),
    ([1400], 2, 64, 100, 120, True),
    ([1333, 1, 200], 2, 64, 60, 128, False),
    ([1500], 1, 64, 64, 97, True),
    ([700, 800], 4, 64, 32, 128, False),
    ([1300, 100], 1, 64, 200, 100, False),
    ([300] * 5, 2, 64, 256, 128, True),
    ([1500], 2, 40, 128, 200, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_prompts(case, dtype):
    lens, G, H, K, V, equal = case
    print(f"[case] long attention {case} {dtype}", flush=True)
    q, k, v, g, _, st, _ = make(lens, G, H, K, V, dtype, seed=K + V)
    scale = K ** -0.5
    o, last = _lib().linear_attention(*(shaped(x, lens, equal) for x in (q, k, v, g)), state=st,
                                      cu_seqlens=offsets(lens, equal), scale=scale, final_state=True)
    torch.cuda.synchronize()
    ref_o, ref_s = token_reference.attention(q, k, v, g, lens, st, scale)
    o_abs, s_abs = token_reference.attention(q.abs(), k.abs(), v.abs(), g, lens, st.abs(), scale)
    c = (max(lens) / 8 + 128 + K) * 2.0 ** -24
    to = c * o_abs + 1e-37
    if dtype == "bf16":
        to = to + 2.0 ** -8 * ref_o.abs() + 2.0 ** -8 * (1 + 2.0 ** -8) * o_abs
    check("o", o.reshape(ref_o.shape), ref_o, to)
    check("state", last, ref_s, c * s_abs + 1e-37)


# tiles of 128 value columns for every padded key size over several segments, equal lengths, shared keys, several tiles
BACKWARD = [
    ([1500, 1500], 8, 8, 128, 128, True),
    ([700, 0, 333, 64], 8, 8, 128, 128, False),
    ([900, 65], 2, 8, 128, 128, False),
    ([640], 1, 2, 100, 127, True),
    ([900, 1], 2, 2, 64, 128, False),
    ([800], 2, 4, 32, 100, True),
    ([600, 200], 1, 2, 200, 128, False),
    ([600], 1, 2, 128, 256, True),
    ([900], 4, 4, 64, 64, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gradients(case, dtype):
    lens, G, H, K, V, equal = case
    print(f"[case] long attention gradients {case} {dtype}", flush=True)
    q, k, v, g, do, st, dl = make(lens, G, H, K, V, dtype, seed=K + V + 1)
    scale = K ** -0.5
    out = _lib().linear_attention_backward(*(shaped(x, lens, equal) for x in (q, k, v, g, do)), state=st,
                                           dfinal_state=dl, cu_seqlens=offsets(lens, equal), scale=scale)
    torch.cuda.synchronize()
    ref = token_reference.attention_backward(q, k, v, g, do, lens, st, dl, scale)
    mag = token_reference.attention_backward(q.abs(), k.abs(), v.abs(), g, do.abs(), lens, st.abs(), dl.abs(), scale)
    c = (max(lens) / 8 + 256 + K + V) * 2.0 ** -24
    for name, r, m in zip(("dq", "dk", "dv", "dlog_decay", "dstate"), ref, mag):
        if name == "dlog_decay":
            rep = H // G
            own = scale * ((q.double() * k.double()).abs().sum(-1).repeat_interleave(rep, 1)
                           * (do.double() * v.double()).abs().sum(-1))
            near = torch.nn.functional.max_pool1d((m + own).t()[None], 127, stride=1, padding=63)[0].t()
            tol = c * 2 * near + 1e-37
        else:
            tol = c * m + 1e-37
            if dtype == "bf16" and name != "dstate":
                tol = tol + 2.0 ** -8 * r.abs() + 2.0 ** -8 * (1 + 2.0 ** -8) * m
        check(name, out[name].reshape(r.shape), r, tol)
