"""The token-sequence operators on a stream given by the caller: inputs let go right after the call,
and outputs let go while the caller's stream still has them to read, keep their memory until then."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _lib():
    import selective_scan_crossscan_amd as ss2d
    return ss2d


def _inputs(op, seed):
    """Tensors of a call of some 30 MB, each in a block of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op.startswith("linear_attention"):
        if op.endswith("step"):
            return [normal(64, 8, 128).to(BF) for _ in range(3)] + [-normal(64, 8).abs(), normal(64, 8, 128, 128)]
        x = [normal(2, 2048, 8, 128).to(BF) for _ in range(3)] + [-normal(2, 2048, 8).abs()]
        return x + [normal(2, 2048, 8, 128).to(BF)] if op.endswith("backward") else x
    if op == "matmul_fp8":
        return [normal(4096, 4096).to(F8), normal(4096, 32).abs(), normal(2048, 4096).to(F8), normal(16, 32).abs()]
    x = [normal(4096, 2048).to(BF), normal(2048)]
    return x + [normal(4096, 2048).to(BF)] if op == "rms_norm_backward" else x


def _outputs(out):
    out = list(out.values()) if isinstance(out, dict) else out if isinstance(out, tuple) else [out]
    return [x.view(torch.uint8) if x.dtype == F8 else x for x in out]


def _busy():
    """Some milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=BF, device="cuda")
    for _ in range(8):
        a = torch.mm(a, a)


OPS = ["linear_attention", "linear_attention_backward", "linear_attention_step", "rms_norm", "rms_norm_fp8",
       "rms_norm_backward", "matmul_fp8"]


@pytest.mark.parametrize("op", OPS)
def test_inputs_and_outputs_outlive_their_names(op):
    fn = getattr(_lib(), op)
    want = _outputs(fn(*_inputs(op, 1)))
    side = torch.cuda.Stream()
    _busy()
    with torch.cuda.stream(side):
        _busy()
    torch.cuda.synchronize()
    for _ in range(3):
        other = _inputs(op, 2)
        x = _inputs(op, 1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _busy()
        out = fn(*x, stream=side)
        sizes = [t.numel() * t.element_size() for t in x]
        del x
        spoilt = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]  # before `side` gets to the call
        torch.cuda.current_stream().wait_stream(side)
        _busy()
        got = [t.clone() for t in _outputs(out)]
        del out
        second = fn(*other, stream=side)  # writes at once, while this stream is busy
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del spoilt, second


def test_a_stream_may_be_captured():
    """The call with `stream` inside a capture of that stream, replayed with eager work between."""
    ss2d = _lib()
    x = _inputs("linear_attention", 3)
    want = ss2d.linear_attention(*x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o = ss2d.linear_attention(*x, stream=side)
    for _ in range(3):
        o.zero_()
        ss2d.linear_attention(*_inputs("linear_attention", 4))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
