"""Wrong offsets of packed sequences, given to the C entries with guard values around everything that is written:
clamped on the device, so whatever the results are, nothing outside the outputs and the workspace changes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T, S, G, H, K, V = 700, 4, 1, 2, 24, 72
GUARD = 1 << 14
WRONG = [[0, 2 ** 31 - 1, 5, 700, 9], [-5, 600, 50, 700, 700], [700, 0, 700, 0, 700], [-2 ** 31, -1, -1, 3, 2 ** 31 - 1],
         [650, 640, 630, 620, 610], [0, 700, 0, 700, 0], [10, 11, 12, 13, 9000]]


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


class Guarded:
    """A range of bytes between guards of 16 KiB."""

    def __init__(self, nbytes):
        self.n = nbytes
        self.all = torch.full((2 * GUARD + (nbytes + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda")
        self.at = self.all.data_ptr() + GUARD

    def unharmed(self):
        return bool((self.all[:GUARD] == 0xA5).all()) and bool((self.all[GUARD + self.n:] == 0xA5).all())


@pytest.mark.parametrize("wrong", WRONG, ids=lambda w: ",".join(map(str, w)))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wrong_offsets_write_nothing_outside(dtype, wrong):
    print(f"[case] guards {dtype} {wrong}", flush=True)
    ss2d = _lib()
    from selective_scan_crossscan_amd import tokens
    kind, e = (torch.float32, 4) if dtype == "f32" else (torch.bfloat16, 2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(T, n, d, generator=gen, device="cuda").to(kind) for n, d in ((G, K), (G, K), (H, V), (H, V)))
    g = -torch.rand(T, H, generator=gen, device="cuda")
    st, dl = (torch.randn(S, H, K, V, generator=gen, device="cuda") for _ in range(2))
    cu = torch.tensor(np.array(wrong, dtype=np.int32)).cuda()
    sizes, *_, code = tokens._attention_sizes(q, k, v, g, cu, do)
    stream = torch.cuda.current_stream().cuda_stream
    L = ss2d.lib()
    states = S * H * K * V * 4

    n = L.ss2d_linear_attention_workspace(sizes, 1, code)
    o, last, ws = Guarded(T * H * V * e), Guarded(states), Guarded(n)
    rc = L.ss2d_linear_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), st.data_ptr(), cu.data_ptr(),
                                 o.at, last.at, sizes, 1.0, code, ws.at, n, stream)
    torch.cuda.synchronize()
    assert rc == 0 and n > 0 and all(x.unharmed() for x in (o, last, ws))

    n = L.ss2d_linear_attention_backward_workspace(sizes, 1, code)
    out = [Guarded(b) for b in (T * G * K * e, T * G * K * e, T * H * V * e, T * H * 4, states, n)]
    rc = L.ss2d_linear_attention_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), st.data_ptr(),
                                          cu.data_ptr(), do.data_ptr(), dl.data_ptr(), *(x.at for x in out[:5]), sizes,
                                          1.0, code, out[5].at, n, stream)
    torch.cuda.synchronize()
    assert rc == 0 and all(x.unharmed() for x in out)
