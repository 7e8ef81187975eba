"""Build libss2d.so (HIP, gfx950 only) in-tree with hipcc."""
from __future__ import annotations

import os
import re
import shutil
import struct
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libss2d.so")
# The kernel templates (ss2d_kernels.h) are instantiated in one unit per storage
# type and steps per lane, compiled in parallel.
SOURCES = ["ss2d_api.hip", "ss2d_plan.hip", "ss2d_f32_t16.hip", "ss2d_f32_t8.hip", "ss2d_bf16_t16.hip",
           "ss2d_bf16_t8.hip", "ss2d_peaks.hip", "ss2d_project.hip",
           "ss2d_epilogue.hip", "ss2d_backward.hip", "ss2d_tokens_api.hip", "ss2d_norm.hip",
           "ss2d_attention_step.hip", "ss2d_attention.hip", "ss2d_attention_state.hip",
           "ss2d_attention_backward.hip", "ss2d_matmul_fp8.hip", "ss2d_delta_api.hip", "ss2d_delta_systems.hip",
           "ss2d_delta.hip", "ss2d_delta_backward.hip", "ss2d_delta_step.hip", "ss2d_qk_norm.hip"]

# -packed-fp32-ops: no packed FP32 instructions are generated (plain VALU only).
HIPCC_FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libss2d.so)")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{out}")
    if verbose and out.strip():
        print(out)


def vector_spills(path: str) -> dict:
    """Kernel (mangled name) -> vector registers spilled to memory, of all gfx950 kernels in a library or object that hipcc
    built, from the metadata beside their code."""
    tool = next((c for c in (os.path.join(os.path.dirname(os.path.realpath(hipcc())), "..", "llvm", "bin", "llvm-readelf"),
                             "/opt/rocm/llvm/bin/llvm-readelf", shutil.which("llvm-readelf")) if c and os.path.exists(c)), None)
    if tool is None:
        raise RuntimeError("llvm-readelf not found (it comes with ROCm's compiler)")
    with open(path, "rb") as f:
        data = f.read()
    out = {}
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        entry = at + len(magic) + 8
        for _ in range(struct.unpack_from("<Q", data, entry - 8)[0]):
            begin, size, length = struct.unpack_from("<QQQ", data, entry)
            name = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if name.endswith(b"gfx950"):
                with tempfile.NamedTemporaryFile() as code:
                    code.write(data[at + begin:at + begin + size])
                    code.flush()
                    notes = subprocess.run([tool, "--notes", code.name], capture_output=True, text=True, check=True).stdout
                # one kernel's fields are in the order of their names
                for kernel, scratch, spilled in re.findall(
                        r"^ +\.name: +(\S+)\n(?:(?! +\.name:).*\n)*? +\.private_segment_fixed_size: (\d+)\n"
                        r"(?:(?! +\.name:).*\n)*? +\.vgpr_spill_count: (\d+)", notes, flags=re.M):
                    out[kernel] = max(out.get(kernel, 0), int(spilled), 1 if int(scratch) else 0)
        at = data.find(magic, at + 1)
    return out


def check_registers(path: str) -> None:
    """Kernels of the delta rule must keep all vector registers.  Compiled with too few, those of 256 keys stored some to
    memory while only part of a wave's threads were active and read them back for all: wrong results, and addresses out of
    range."""
    spills = vector_spills(path)
    if not spills:
        raise RuntimeError(f"no kernels' metadata found in {path}")
    bad = {k: n for k, n in spills.items() if n and "delta_" in k}
    if bad:
        raise RuntimeError(f"spilled vector registers where none may be: {bad}")


def build(verbose: bool = False, jobs: int = 0) -> str:
    """Compile every HIP source into selective_scan_crossscan_amd/libss2d.so; returns its path."""
    tag = f".tmp{os.getpid()}"
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(CSRC, src.replace(".hip", ".o")) + tag
        objs.append(obj)
        cmds.append([hipcc(), *HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, os.path.join(CSRC, src)])
    jobs = jobs or min(len(cmds), os.cpu_count() or 1)
    try:
        with ThreadPoolExecutor(max_workers=jobs) as ex:
            for f in [ex.submit(_run, c, verbose) for c in cmds]:
                f.result()
        tmp = LIB + tag
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
        check_registers(tmp)
        os.replace(tmp, LIB)
    finally:
        for o in objs + [LIB + tag]:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
