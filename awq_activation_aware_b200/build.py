"""Builds libawq.so (the C-ABI library) in-tree for sm_100a.

    python -m awq_activation_aware_b200.build [--verbose]

nvcc cross-compiles without a GPU.  The CUDA runtime is linked statically so
the library does not depend on which libcudart another package has loaded.
"""
from __future__ import annotations

import os
import subprocess
import sys
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
LIB = PKG / "libawq.so"
SOURCES = [CSRC / "awq_abi.cu", CSRC / "awq_kv_abi.cu"]
DEPS = SOURCES + [CSRC / n for n in ("awq_kernels.cuh", "awq_device.cuh", "awq_host.h", "awq_kv.cuh", "awq_kv_decode.cuh",
                                     "awq_kv_prefill.cuh")] + [ROOT / "include" / "awq.h"]

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-fmad=false",          # no implicit multiply-add contraction: every FMA in the code is explicit
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-v",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = Path(cand) / "bin" / "nvcc"
    return str(p) if p.exists() else "nvcc"


def needs_build() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    return any(d.stat().st_mtime > t for d in DEPS)


def build(force: bool = False, verbose: bool = False) -> Path:
    if not force and not needs_build():
        return LIB
    tmp = LIB.with_suffix(f".so.tmp{os.getpid()}")
    objs = [PKG / f"{src.stem}.tmp{os.getpid()}.o" for src in SOURCES]
    cmds = [[nvcc(), *NVCC_FLAGS, "-I", str(ROOT / "include"), "-I", str(CSRC), "-c", "-o", str(obj), str(src)]
            for src, obj in zip(SOURCES, objs)]
    # the units compile side by side
    procs = [subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for cmd in cmds]
    log, code = "", 0
    for cmd, proc in zip(cmds, procs):
        out = proc.communicate()[0]
        log += " ".join(cmd) + "\n" + out
        code = code or proc.returncode
    if code == 0:
        cmd = [nvcc(), *LINK_FLAGS, "-o", str(tmp), *map(str, objs)]
        res = subprocess.run(cmd, capture_output=True, text=True)
        log += " ".join(cmd) + "\n" + res.stdout + res.stderr
        code = res.returncode
    for obj in objs:
        obj.unlink(missing_ok=True)
    (PKG / "build.log").write_text(log)
    if code != 0:
        sys.stderr.write(log)
        raise RuntimeError(f"nvcc failed ({code}); see {PKG / 'build.log'}")
    if verbose:
        sys.stdout.write(log)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
