"""C-ABI contract of the token-sequence operators (include/ss2d_tokens.h), checked on the
CPU: bad arguments get their documented codes before the device is touched.  Addresses
are fake and never dereferenced; calls that pass validation report SS2D_ERR_NO_DEVICE (-7)
here, and those tests are skipped where a device exists."""
import ctypes
import math
import os
import re

import pytest

import selective_scan_crossscan_amd as ss2d

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, ALIAS, ALIGN, NO_DEVICE, WORKSPACE = -1, -2, -4, -5, -6, -7, -10
FAKE = 1 << 40
STEP = 1 << 34


def _no_device_here():
    try:
        import torch
        return torch.cuda.device_count() == 0
    except Exception:
        return True


needs_no_device = pytest.mark.skipif(not _no_device_here(), reason="a valid call would launch kernels on fake addresses")


def at(i):
    return FAKE + i * STEP


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ss2d_tokens.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(ss2d_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(["ss2d_linear_attention", "ss2d_linear_attention_workspace", "ss2d_linear_attention_backward",
                            "ss2d_linear_attention_backward_workspace", "ss2d_linear_attention_step", "ss2d_rms_norm",
                            "ss2d_rms_norm_backward", "ss2d_rms_norm_backward_workspace", "ss2d_matmul_fp8"])
    lib = ctypes.CDLL(ss2d.library_path())
    assert all(hasattr(lib, n) for n in names)


def test_header_is_plain_c(tmp_path):
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    src = tmp_path / "t.c"
    src.write_text('#include "ss2d_tokens.h"\nint main(void) { return sizeof(ss2d_attention_sizes) == 21 * 8 ? 0 : 1; }\n')
    exe = tmp_path / "t"
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-o",
                           str(exe), str(src)])
    assert subprocess.call([str(exe)]) == 0


def test_workspace_status_has_a_text():
    assert "workspace" in ss2d.status_string(WORKSPACE)


# ------------------------------------------------------------------ linear attention
def sizes(S=2, T=200, G=2, H=4, K=16, V=24, **strides):
    z = {"q": (T // S * G * K, G * K, K), "k": (T // S * G * K, G * K, K), "v": (T // S * H * V, H * V, V),
         "g": (T // S * H, H, 1), "do": (T // S * H * V, H * V, V)}
    z.update(strides)
    return (ctypes.c_int64 * 21)(S, T, G, H, K, V, *z["q"], *z["k"], *z["v"], *z["g"], *z["do"])


def resized(**kw):
    """The usual strides with other sizes."""
    z = sizes()
    for i, n in enumerate(("S", "T", "G", "H", "K", "V")):
        z[i] = kw.get(n, z[i])
    return z


def forward(z=None, dtype=0, cu=None, ws=at(20), nbytes=1 << 33, state_in=at(5), **ptr):
    p = {"q": at(1), "k": at(2), "v": at(3), "g": at(4), "o": at(6), "state_out": at(7)}
    p.update(ptr)
    return ss2d.lib().ss2d_linear_attention(p["q"], p["k"], p["v"], p["g"], state_in, cu, p["o"], p["state_out"],
                                            sizes() if z is None else z, 1.0, dtype, ws, nbytes, None)


def backward(z=None, dtype=0, cu=None, ws=at(20), nbytes=1 << 33, **ptr):
    names = ("q", "k", "v", "g", "state_in", "cu", "do", "dstate_out", "dq", "dk", "dv", "dg", "dstate_in")
    p = {n: at(i + 1) for i, n in enumerate(names)}
    p["cu"] = cu
    p.update(ptr)
    return ss2d.lib().ss2d_linear_attention_backward(*(p[n] for n in names), sizes() if z is None else z, 1.0, dtype, ws,
                                                     nbytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_refusals(call):
    for name in ("q", "k", "v", "g"):
        assert call(**{name: None}) == NULL
    assert call(z=ctypes.POINTER(ctypes.c_int64)()) == NULL
    for bad in (dict(S=0), dict(T=0), dict(S=3, T=200), dict(G=0), dict(G=3, H=4), dict(H=0, G=1), dict(K=0), dict(K=257),
                dict(V=0), dict(V=1025), dict(T=1 << 31, S=1)):
        assert call(z=resized(**bad)) == SHAPE, bad
    assert call(z=sizes(q=(-1, 32, 16))) == SHAPE
    assert call(z=sizes(v=(1 << 62, 1 << 62, 24))) == SHAPE
    assert call(z=sizes(v=(1 << 40, 1 << 24, 24))) == SHAPE  # the device multiplies strides of 24 bits
    assert call(z=sizes(q=(1 << 40, 1 << 24, 16))) == SHAPE
    assert call(dtype=2) == DTYPE
    assert call(q=at(1) + 2) == ALIGN
    assert call(g=at(4) + 1) == ALIGN
    assert call(q=at(1) + 1, dtype=1) == ALIGN


def test_attention_alias_rules():
    assert forward(o=at(3)) == ALIAS
    assert forward(o=at(3) + 200 * 4 * 24 * 4 - 4) == ALIAS   # the last value of v
    assert forward(state_out=at(5) + 4) == ALIAS              # partly state_in
    assert forward(state_out=at(6)) == ALIAS
    assert forward(o=at(30), cu=at(30)) == ALIAS
    for out in ("dq", "dk", "dv", "dg", "dstate_in"):
        assert backward(**{out: at(3)}) == ALIAS
    assert backward(dq=at(10)) == ALIAS                        # dk's address
    assert backward(dstate_in=at(5)) == ALIAS


def test_attention_workspace_rules():
    lib = ss2d.lib()
    z = sizes(S=1, T=5000, G=1, H=1, K=16, V=16)
    need = lib.ss2d_linear_attention_workspace(z, 0, 0)
    assert need > 0 and lib.ss2d_linear_attention_workspace(sizes(), 0, 0) == 0
    assert forward(z=z, ws=None, nbytes=need) == WORKSPACE
    assert forward(z=z, nbytes=need - 1) == WORKSPACE
    assert forward(z=z, ws=at(20) + 8, nbytes=need) == WORKSPACE
    assert forward(z=z, ws=at(3)) == ALIAS
    assert lib.ss2d_linear_attention_workspace(sizes(K=300), 0, 0) == SHAPE
    assert lib.ss2d_linear_attention_workspace(sizes(), 0, 5) == DTYPE
    assert lib.ss2d_linear_attention_workspace(None, 0, 0) == NULL
    for name in ("ss2d_linear_attention_workspace", "ss2d_linear_attention_backward_workspace"):  # no such grid
        assert getattr(lib, name)(sizes(S=1 << 20, T=1 << 30, G=1, H=65536, K=256, V=1024), 1, 1) == SHAPE
        assert getattr(lib, name)(sizes(S=1 << 24, T=1 << 24, G=1, H=65536, K=256, V=1024), 0, 0) == SHAPE
    need = lib.ss2d_linear_attention_backward_workspace(sizes(), 0, 0)
    assert need > 0
    assert backward(nbytes=need - 1) == WORKSPACE and backward(ws=None) == WORKSPACE
    assert backward(ws=at(9)) == ALIAS


@needs_no_device
def test_valid_attention_reaches_the_device():
    assert forward() == NO_DEVICE
    assert forward(ws=None, nbytes=0, state_in=None, state_out=None) == NO_DEVICE
    assert forward(state_out=at(5)) == NO_DEVICE               # state_in itself
    assert forward(cu=at(31), dtype=1) == NO_DEVICE
    assert forward(z=sizes(g=(0, 0, 1))) == NO_DEVICE          # one decay per head
    assert backward() == NO_DEVICE
    assert backward(cu=at(31), state_in=None, dstate_out=None, dstate_in=None) == NO_DEVICE


def step(dtype=0, rows=3, slots=5, G=2, H=4, K=16, V=24, q_row=None, index=at(6), **ptr):
    p = {"q": at(1), "k": at(2), "v": at(3), "g": at(4), "state": at(5), "o": at(7)}
    p.update(ptr)
    q_row = G * K if q_row is None else q_row
    return ss2d.lib().ss2d_linear_attention_step(p["q"], p["k"], p["v"], p["g"], p["state"], index, p["o"], rows, slots, G,
                                                 H, K, V, q_row, G * K, H * V, 1.0, dtype, None)


def test_step_refusals():
    for name in ("q", "k", "v", "g", "state", "o"):
        assert step(**{name: None}) == NULL
    for bad in (dict(rows=0), dict(rows=65536), dict(slots=0), dict(rows=6, index=None), dict(G=3), dict(K=257),
                dict(V=1025), dict(H=0), dict(q_row=-1), dict(slots=1 << 40)):
        assert step(**bad) == SHAPE, bad
    assert step(dtype=-1) == DTYPE
    assert step(o=at(3)) == ALIAS and step(o=at(5)) == ALIAS and step(state=at(1)) == ALIAS and step(o=at(6)) == ALIAS
    assert step(state=at(5) + 2) == ALIGN and step(v=at(3) + 1, dtype=1) == ALIGN


@needs_no_device
def test_valid_step_reaches_the_device():
    assert step() == NO_DEVICE and step(index=None) == NO_DEVICE and step(q_row=0, dtype=1) == NO_DEVICE


# ------------------------------------------------------------------ norm
def norm(x=at(1), residual=at(2), weight=at(3), eps=1e-6, residual_out=at(4), y=at(5), scales=None, rows=7, dim=300,
         dtype=0):
    return ss2d.lib().ss2d_rms_norm(x, residual, weight, eps, residual_out, y, scales, rows, dim, dtype, None)


def norm_backward(r=at(1), weight=at(2), dy=at(3), dr=at(4), eps=1e-6, dx=at(5), dw=at(6), rows=7, dim=300, dtype=0,
                  ws=at(7), nbytes=1 << 30):
    return ss2d.lib().ss2d_rms_norm_backward(r, weight, dy, dr, eps, dx, dw, rows, dim, dtype, ws, nbytes, None)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_refusals(call):
    for bad in (dict(rows=0), dict(rows=1 << 31), dict(dim=0), dict(dim=16385), dict(eps=-1.0), dict(eps=math.nan),
                dict(eps=math.inf)):
        assert call(**bad) == SHAPE, bad
    assert call(dtype=7) == DTYPE
    assert call(weight=at(3) + 2) == ALIGN


def test_norm_pointer_rules():
    assert norm(x=None) == NULL and norm(y=None) == NULL
    assert norm(y=at(1) + 4) == ALIAS and norm(residual_out=at(2) + 4) == ALIAS and norm(y=at(4)) == ALIAS
    assert norm(y=at(3)) == ALIAS and norm(scales=at(1)) == ALIAS and norm(scales=at(6), y=at(1)) == ALIAS
    assert norm(x=at(1) + 1, dtype=1) == ALIGN and norm(scales=at(6) + 2) == ALIGN
    assert norm_backward(r=None) == NULL and norm_backward(dy=None) == NULL and norm_backward(dx=None) == NULL
    assert norm_backward(dx=at(1)) == ALIAS and norm_backward(dx=at(3) + 4) == ALIAS and norm_backward(dw=at(3)) == ALIAS
    need = ss2d.lib().ss2d_rms_norm_backward_workspace(7, 300, 0)
    assert need == 7 * 300 * 4
    assert norm_backward(nbytes=need - 1) == WORKSPACE and norm_backward(ws=None) == WORKSPACE
    assert norm_backward(ws=at(5)) == ALIAS
    assert ss2d.lib().ss2d_rms_norm_backward_workspace(0, 300, 0) == SHAPE


@needs_no_device
def test_valid_norm_reaches_the_device():
    assert norm() == NO_DEVICE and norm(residual=None, weight=None, residual_out=None, eps=0.0) == NO_DEVICE
    assert norm(y=at(1), residual_out=at(2)) == NO_DEVICE      # in place
    assert norm(y=at(5) + 1, scales=at(6)) == NO_DEVICE        # 8 bits: any address
    assert norm_backward() == NO_DEVICE and norm_backward(dw=None, ws=None, nbytes=0) == NO_DEVICE
    assert norm_backward(dx=at(3)) == NO_DEVICE and norm_backward(dx=at(4)) == NO_DEVICE


# ------------------------------------------------------------------ product
def matmul(a=at(1), sa=at(2), b=at(3), sb=at(4), out=at(5), m=5, n=300, k=200, dtype=1):
    return ss2d.lib().ss2d_matmul_fp8(a, sa, b, sb, out, m, n, k, dtype, None)


def test_matmul_refusals():
    for name in ("a", "sa", "b", "sb", "out"):
        assert matmul(**{name: None}) == NULL
    for bad in (dict(m=0), dict(n=0), dict(k=0), dict(m=(1 << 30) + 1), dict(k=(1 << 20) + 1), dict(m=1 << 30, n=1 << 30)):
        assert matmul(**bad) == SHAPE, bad
    assert matmul(dtype=2) == DTYPE
    assert matmul(out=at(1)) == ALIAS and matmul(out=at(4)) == ALIAS
    assert matmul(out=at(5) + 1) == ALIGN and matmul(sa=at(2) + 2) == ALIGN


@needs_no_device
def test_valid_matmul_reaches_the_device():
    assert matmul() == NO_DEVICE and matmul(a=at(1) + 1, b=at(3) + 3, dtype=0) == NO_DEVICE


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    for f in (lambda: ss2d.rms_norm(x), lambda: ss2d.rms_norm_fp8(x), lambda: ss2d.rms_norm_backward(x, None, x),
              lambda: ss2d.linear_attention(*[torch.zeros(1, 4, 1, 8)] * 3, torch.zeros(1, 4, 1)),
              lambda: ss2d.linear_attention_step(*[torch.zeros(2, 1, 8)] * 3, torch.zeros(2, 1), torch.zeros(2, 1, 8, 8)),
              lambda: ss2d.matmul_fp8(x.to(torch.float8_e4m3fn), torch.ones(2, 1), x.to(torch.float8_e4m3fn),
                                      torch.ones(1, 1))):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        ss2d.rms_norm(x.half())
    with pytest.raises(ValueError):
        ss2d.linear_attention(x, x, x, x)
    with pytest.raises(AttributeError):
        ss2d.no_such_operator


def test_step_rows_may_lie_any_distance_apart():
    """Only prompts limit the distance of tokens to 24 bits."""
    assert step(o=at(3), q_row=1 << 24) == ALIAS  # past the checks of sizes
    assert step(o=at(3), q_row=1 << 30) == ALIAS
    assert step(o=at(3), q_row=1 << 62) == SHAPE


@needs_no_device
def test_step_far_rows_reach_the_device():
    assert step(q_row=1 << 24, q=at(100)) == NO_DEVICE


@pytest.mark.parametrize("torch_there", [False, True])
def test_everything_imports_with_and_without_torch(torch_there):
    import subprocess
    import sys
    if torch_there:
        pytest.importorskip("torch")
    code = ("import sys\n" + ("" if torch_there else "sys.modules['torch'] = None\n")
            + "from selective_scan_crossscan_amd import *\nassert version() > 0 and ss2d_forward\n"
            + f"assert ('rms_norm' in dir()) == {torch_there}")
    subprocess.check_call([sys.executable, "-c", code], cwd=ROOT)


@needs_no_device
def test_norm_takes_any_finite_eps():
    for eps in (0.0, 2e30, 3.4e38):
        assert norm(eps=eps) == NO_DEVICE and norm_backward(eps=eps) == NO_DEVICE
