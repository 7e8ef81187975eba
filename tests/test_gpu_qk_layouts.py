"""Norms of queries and keys over their inputs (ss2d_qk_norm with q_out q and k_out k), both slices of one tensor in the
layouts that models use: the same values as into new tensors, and nothing else of the tensor changed."""
import pytest

from test_gpu_delta import DT, _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

S, T, H, D = 2, 37, 6, 40
LAYOUTS = {
    "per head": ((S, T, H, 3, D), lambda x: (x[..., 0, :], x[..., 1, :])),
    "packed, per head": ((T, H, 3, D), lambda x: (x[..., 0, :], x[..., 1, :])),
    "planes": ((S, 3, T, H, D), lambda x: (x[:, 0], x[:, 1])),
    "heads first": ((S, 3 * H, T, D), lambda x: (x[:, :H].transpose(1, 2), x[:, H:H + 2].transpose(1, 2))),
    "sequences inside": ((T, S, 3, H, D), lambda x: (x[:, :, 0].transpose(0, 1), x[:, :, 1].transpose(0, 1))),
    "one token": ((S, 1, H, 3, D), lambda x: (x[..., 0, :], x[..., 1, :])),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_norms_over_their_inputs(name, dtype):
    ss2d = _lib()
    shape, slices = LAYOUTS[name]
    x = torch.randn(shape, device="cuda").to(DT[dtype])
    kw = dict(q_weight=torch.rand(D, device="cuda"), k_weight=torch.rand(D, device="cuda"),
              rotation=ss2d.rotation_table(T, 32))
    want = x.clone()
    for part, y in zip(slices(want), ss2d.qk_norm(*slices(x), **kw)):
        part.copy_(y)
    q, k = slices(x)
    got = ss2d.qk_norm(q, k, out=(q, k), **kw)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k
    assert torch.equal(x, want) and not torch.equal(x, torch.zeros_like(x))


def test_sides_that_share_addresses_are_refused():
    ss2d = _lib()
    x = torch.randn(T, H, 3, D, device="cuda")
    q, k = x[..., 0, :], x[..., 1, :]
    for out in ((k, q), (q, q), (x.view(T, 3 * H, D)[:, :H], k)):
        with pytest.raises(ss2d.SS2DError):
            ss2d.qk_norm(q, k, out=out)
