"""C-ABI contract of the delta rule and of the query and key norms (include/ss2d_delta_rule.h), checked on the CPU: bad
arguments get their documented codes before the device is touched.  Addresses are fake and never dereferenced; calls
that pass validation report SS2D_ERR_NO_DEVICE (-7) here, and those tests are skipped where a device exists."""
import ctypes
import math
import os
import re

import pytest

import selective_scan_crossscan_amd as ss2d
from test_abi_tokens import ALIAS, ALIGN, DTYPE, NO_DEVICE, NULL, ROOT, SHAPE, WORKSPACE, at, needs_no_device


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ss2d_delta_rule.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(ss2d_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(["ss2d_delta_rule", "ss2d_delta_rule_workspace", "ss2d_delta_rule_backward",
                            "ss2d_delta_rule_backward_workspace", "ss2d_delta_rule_step", "ss2d_qk_norm",
                            "ss2d_qk_norm_backward", "ss2d_qk_norm_backward_workspace"])
    lib = ctypes.CDLL(ss2d.library_path())
    assert all(hasattr(lib, n) for n in names)


def test_header_is_plain_c(tmp_path):
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    src = tmp_path / "t.c"
    src.write_text('#include "ss2d_delta_rule.h"\nint main(void) { return sizeof(ss2d_delta_sizes) == 24 * 8 && '
                   'sizeof(ss2d_qk_sizes) == 19 * 8 ? 0 : 1; }\n')
    exe = tmp_path / "t"
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-o",
                           str(exe), str(src)])
    assert subprocess.call([str(exe)]) == 0


# ------------------------------------------------------------------ delta rule
def sizes(S=2, T=200, G=2, H=4, K=16, V=24, **strides):
    z = {"q": (T // S * G * K, G * K, K), "k": (T // S * G * K, G * K, K), "v": (T // S * H * V, H * V, V),
         "g": (T // S * H, H, 1), "do": (T // S * H * V, H * V, V), "b": (T // S * H, H, 1)}
    z.update(strides)
    return (ctypes.c_int64 * 24)(S, T, G, H, K, V, *z["q"], *z["k"], *z["v"], *z["g"], *z["do"], *z["b"])


def resized(**kw):
    """The usual strides with other sizes."""
    z = sizes()
    for i, n in enumerate(("S", "T", "G", "H", "K", "V")):
        z[i] = kw.get(n, z[i])
    return z


def forward(z=None, dtype=0, cu=None, ws=at(20), nbytes=1 << 33, state_in=at(5), **ptr):
    p = {"q": at(1), "k": at(2), "v": at(3), "g": at(4), "b": at(8), "o": at(6), "state_out": at(7)}
    p.update(ptr)
    return ss2d.lib().ss2d_delta_rule(p["q"], p["k"], p["v"], p["g"], p["b"], state_in, cu, p["o"], p["state_out"],
                                      sizes() if z is None else z, 1.0, dtype, ws, nbytes, None)


def backward(z=None, dtype=0, cu=None, ws=at(20), nbytes=1 << 33, **ptr):
    names = ("q", "k", "v", "g", "b", "state_in", "cu", "do", "dstate_out", "dq", "dk", "dv", "dg", "db", "dstate_in")
    p = {n: at(i + 1) for i, n in enumerate(names)}
    p["cu"] = cu
    p.update(ptr)
    return ss2d.lib().ss2d_delta_rule_backward(*(p[n] for n in names), sizes() if z is None else z, 1.0, dtype, ws,
                                               nbytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_delta_refusals(call):
    for name in ("q", "k", "v", "g", "b"):
        assert call(**{name: None}) == NULL
    assert call(z=ctypes.POINTER(ctypes.c_int64)()) == NULL
    for bad in (dict(S=0), dict(T=0), dict(S=3, T=200), dict(G=0), dict(G=3, H=4), dict(H=0, G=1), dict(K=0), dict(K=257),
                dict(V=0), dict(V=1025), dict(T=1 << 31, S=1)):
        assert call(z=resized(**bad)) == SHAPE, bad
    assert call(z=sizes(q=(-1, 32, 16))) == SHAPE
    assert call(z=sizes(b=(-1, 4, 1))) == SHAPE
    assert call(z=sizes(v=(1 << 62, 1 << 62, 24))) == SHAPE
    assert call(z=sizes(v=(1 << 40, 1 << 24, 24))) == SHAPE  # the device multiplies strides of 24 bits
    # 2^31 tokens times heads in chunks are over the most workgroups
    assert call(z=sizes(S=1 << 20, T=1 << 20, G=1, H=2048, K=16, V=16)) == SHAPE
    assert call(dtype=2) == DTYPE
    assert call(q=at(1) + 2) == ALIGN
    assert call(g=at(4) + 1) == ALIGN
    assert call(b=at(28) + 2) == ALIGN
    assert call(q=at(1) + 1, dtype=1) == ALIGN


def test_delta_alias_rules():
    assert forward(o=at(3)) == ALIAS
    assert forward(o=at(8)) == ALIAS
    assert forward(o=at(3) + 200 * 4 * 24 * 4 - 4) == ALIAS   # the last value of v
    assert forward(state_out=at(5) + 4) == ALIAS              # partly state_in
    assert forward(state_out=at(6)) == ALIAS
    assert forward(ws=at(8)) == ALIAS
    assert forward(o=at(30), cu=at(30)) == ALIAS
    for out in ("dq", "dk", "dv", "dg", "db", "dstate_in"):
        assert backward(**{out: at(5)}) == ALIAS
    assert backward(dq=at(30), dk=at(30)) == ALIAS
    assert backward(db=at(30), dg=at(30) + 4) == ALIAS


@pytest.mark.parametrize("name,call", [("ss2d_delta_rule_workspace", forward),
                                       ("ss2d_delta_rule_backward_workspace", backward)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_delta_workspace(name, call, dtype):
    need = getattr(ss2d.lib(), name)(sizes(), 0, dtype)
    assert need > 0
    assert call(dtype=dtype, nbytes=need - 1) == WORKSPACE
    assert call(dtype=dtype, ws=None) == WORKSPACE
    assert call(dtype=dtype, ws=at(20) + 8) == WORKSPACE
    assert getattr(ss2d.lib(), name)(resized(K=0), 0, dtype) == SHAPE
    assert getattr(ss2d.lib(), name)(sizes(), 0, 7) == DTYPE
    assert getattr(ss2d.lib(), name)(ctypes.POINTER(ctypes.c_int64)(), 0, 0) == NULL
    # room for any packing of the same tokens
    assert getattr(ss2d.lib(), name)(resized(S=7), 1, dtype) > 0


@needs_no_device
@pytest.mark.parametrize("call", [forward, backward])
def test_valid_delta_calls_reach_the_device(call):
    for dtype in (0, 1):
        assert call(dtype=dtype) == NO_DEVICE
        assert call(dtype=dtype, cu=at(21)) == NO_DEVICE
    assert call(z=sizes(g=(0, 0, 1), b=(0, 0, 0))) == NO_DEVICE
    assert call(state_in=None) == NO_DEVICE
    assert forward(state_out=at(5)) == NO_DEVICE
    assert forward(state_out=None) == NO_DEVICE


def step(rows=8, slots=16, G=2, H=4, K=16, V=24, dtype=0, index=at(9), **ptr):
    p = {"q": at(1), "k": at(2), "v": at(3), "g": at(4), "b": at(5), "state": at(6), "o": at(7)}
    p.update(ptr)
    return ss2d.lib().ss2d_delta_rule_step(p["q"], p["k"], p["v"], p["g"], p["b"], p["state"], index, p["o"], rows,
                                           slots, G, H, K, V, G * K, G * K, H * V, 1.0, dtype, None)


def test_step_refusals():
    for name in ("q", "k", "v", "g", "b", "state", "o"):
        assert step(**{name: None}) == NULL
    for bad in (dict(rows=0), dict(rows=65536), dict(slots=0), dict(rows=17, index=None), dict(G=3), dict(K=0),
                dict(K=257), dict(V=0), dict(V=1025), dict(H=0)):
        assert step(**bad) == SHAPE, bad
    assert step(dtype=2) == DTYPE
    for a, b in (("b", "state"), ("b", "o"), ("state", "o"), ("q", "o"), ("v", "state")):
        assert step(**{a: at(30), b: at(30)}) == ALIAS
    assert step(b=at(5) + 1) == ALIGN
    assert step(state=at(6) + 2) == ALIGN


# ------------------------------------------------------------------ query and key norms
def qk_sizes(S=2, T=50, Hq=4, Hk=2, D=16, rot=8, rows=64, **strides):
    z = {n: (T * h * D, h * D, D) for n, h in (("q", Hq), ("k", Hk), ("qo", Hq), ("ko", Hk))}
    z.update(strides)
    return (ctypes.c_int64 * 19)(S, T, Hq, Hk, D, rot, rows, *z["q"], *z["k"], *z["qo"], *z["ko"])


def norm(z=None, dtype=0, eps=1e-6, wq=at(3), wk=at(4), table=at(5), pos=at(6), **ptr):
    p = {"q": at(1), "k": at(2), "qo": at(7), "ko": at(8)}
    p.update(ptr)
    return ss2d.lib().ss2d_qk_norm(p["q"], p["k"], wq, wk, table, pos, p["qo"], p["ko"], qk_sizes() if z is None else z,
                                   eps, 0, dtype, None)


def norm_back(z=None, dtype=0, eps=1e-6, wq=at(3), wk=at(4), table=at(5), pos=at(6), ws=at(20), nbytes=1 << 33, **ptr):
    p = {"q": at(1), "k": at(2), "qo": at(7), "ko": at(8), "dq": at(9), "dk": at(10), "dwq": at(11), "dwk": at(12)}
    p.update(ptr)
    return ss2d.lib().ss2d_qk_norm_backward(p["q"], p["k"], wq, wk, table, pos, p["qo"], p["ko"], p["dq"], p["dk"],
                                            p["dwq"], p["dwk"], qk_sizes() if z is None else z, eps, 0, dtype, ws,
                                            nbytes, None)


@pytest.mark.parametrize("call", [norm, norm_back])
def test_norm_refusals(call):
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: None}) == NULL
    assert call(z=ctypes.POINTER(ctypes.c_int64)()) == NULL
    for bad in (dict(S=0), dict(T=0), dict(Hq=0), dict(Hk=0), dict(D=0), dict(D=257), dict(rot=7), dict(rot=18),
                dict(rot=-2), dict(rot=0), dict(rows=0), dict(S=1 << 20, T=1 << 20), dict(q=(-1, 64, 16)),
                dict(k=(1 << 62, 1 << 62, 16))):
        assert call(z=qk_sizes(**bad)) == SHAPE, bad
    assert call(table=None) == SHAPE
    for eps in (-1e-6, math.inf, math.nan):
        assert call(eps=eps) == SHAPE
    assert call(dtype=3) == DTYPE
    assert call(q=at(1) + 2) == ALIGN
    assert call(wk=at(4) + 2) == ALIGN
    assert call(pos=at(6) + 1) == ALIGN
    assert call(qo=at(7) + 1, dtype=1) == ALIGN


def test_norm_outputs_lie_apart_and_over_their_own_inputs_alone():
    row = 6 * 16  # queries and keys as slices of one row
    both = dict(q=(50 * row, row, 16), k=(50 * row, row, 16))
    z = qk_sizes(**both, qo=both["q"], ko=both["k"])
    for bad in ((0, 64, 16), (50 * 64, 64, 8), (50 * 64, 0, 16), (64, 64, 16)):
        assert norm(z=qk_sizes(qo=bad)) == SHAPE
    q, k = at(1), at(1) + 4 * 16 * 4
    assert norm(z=z, q=q, k=k, qo=k, ko=q) == ALIAS           # each over the other's input
    assert norm(z=z, q=q, k=k, qo=q + 4, ko=k) == ALIAS       # partly its own
    assert norm(z=z, q=q, k=q, qo=q, ko=k) == ALIAS           # keys that are queries
    assert norm(z=qk_sizes(**both), q=q, k=k, qo=q, ko=k) == ALIAS  # other strides than its own
    assert norm(qo=at(30), ko=at(30)) == ALIAS
    for other in (at(3), at(4), at(5), at(6)):
        assert norm(qo=other) == ALIAS
    for out in ("dq", "dk", "dwq", "dwk"):
        for other in (at(1), at(2), at(3), at(5), at(6), at(7), at(8)):
            assert norm_back(**{out: other}) == ALIAS
    assert norm_back(dq=at(30), dk=at(30)) == ALIAS
    assert norm_back(wq=None) == NULL                          # a gradient without its weight


def test_norm_workspace():
    need = ss2d.lib().ss2d_qk_norm_backward_workspace(qk_sizes(), 0)
    assert need > 0
    assert norm_back(nbytes=need - 1) == WORKSPACE
    assert norm_back(ws=None) == WORKSPACE
    assert norm_back(ws=at(20) + 4) == WORKSPACE
    assert ss2d.lib().ss2d_qk_norm_backward_workspace(qk_sizes(D=0), 0) == SHAPE
    assert ss2d.lib().ss2d_qk_norm_backward_workspace(ctypes.POINTER(ctypes.c_int64)(), 0) == NULL


@needs_no_device
def test_valid_norm_calls_reach_the_device():
    row = 6 * 16
    both = dict(q=(50 * row, row, 16), k=(50 * row, row, 16))
    q, k = at(1), at(1) + 4 * 16 * 4
    assert norm(z=qk_sizes(**both, qo=both["q"], ko=both["k"]), q=q, k=k, qo=q, ko=k) == NO_DEVICE
    for dtype in (0, 1):
        assert norm(dtype=dtype) == NO_DEVICE
        assert norm_back(dtype=dtype) == NO_DEVICE
    assert norm(pos=None, wq=None, wk=None) == NO_DEVICE
    assert norm(z=qk_sizes(rot=0, rows=0), table=None, pos=None) == NO_DEVICE
    assert norm_back(dwq=None, dwk=None, ws=None, nbytes=0) == NO_DEVICE
    assert norm_back(z=qk_sizes(qo=(0, 0, 16), ko=(0, 0, 0))) == NO_DEVICE


# ------------------------------------------------------------------ the binding
def test_binding_refuses_cpu_tensors_and_bad_tables():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 5, 2, 16)
    with pytest.raises(ValueError, match="GPU"):
        ss2d.delta_rule(x, x, x, x[..., 0], x[..., 0])
    with pytest.raises(ValueError, match="GPU"):
        ss2d.qk_norm(x, x)
    for bad in ((0, 4), (4, 3), (4, 0)):
        with pytest.raises(ValueError):
            ss2d.rotation_table(*bad, device="cpu")
    t = ss2d.rotation_table(9, 4, base=100.0, device="cpu")
    assert t.shape == (9, 4) and t.dtype == torch.float32
    assert abs(float(t[7, 1]) - math.cos(0.7)) < 1e-7 and abs(float(t[7, 3]) - math.sin(0.7)) < 1e-7
