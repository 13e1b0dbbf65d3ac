"""Build the HIP library libsgemm_f32.so in-tree for gfx950 with hipcc, and, where torch is
installed, the host extension _torch_calls.so that the tensor layer calls it through. The C ABI needs
the library alone.

    python -m fp32_gemm_f32_amd.build           # build
    python -m fp32_gemm_f32_amd.build --asm     # also write the gfx950 assembly

The resource usage of every kernel (VGPRs, AGPRs, LDS, occupancy) is written to
fp32_gemm_f32_amd/_build/resource_usage.txt from the compiler's own report.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libsgemm_f32.so")
BUILD_DIR = os.path.join(PKG, "_build")
# Translation units and whether their MFMA accumulators are held in VGPRs (see flags()).
# The one-wave-per-SIMD kernel keeps 256 accumulators per lane in AGPRs, so it is compiled
# on its own, without that option. The 8-bit product goes without it too: with it the compiler
# gave the few-rows kernel an accumulator whose registers its load addresses overwrote.
SOURCES = [(os.path.join(CSRC, "sgemm_f32.hip"), True),
           (os.path.join(CSRC, "sgemm_regpanel.hip"), False),
           (os.path.join(CSRC, "sgemm_persist.hip"), False),
           (os.path.join(CSRC, "gemm_i8.hip"), False),
           (os.path.join(CSRC, "token_logprobs.hip"), True),
           (os.path.join(CSRC, "gemm_mx4.hip"), False),
           (os.path.join(CSRC, "beam_search.hip"), True)]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the library)")


def flags(vgpr_form: bool = True) -> list[str]:
    f = [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        # packed FP32 instructions stay off: the compiler must not form them from float2
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-command-line-argument",
        f"-I{INCLUDE}", f"-I{CSRC}",
    ]
    if vgpr_form:
        # MFMA accumulators stay in VGPRs (every kernel of the unit fits in 256 registers);
        # left to its heuristics the register allocator moves them between AGPRs and VGPRs
        # on each iteration of the persistent stream-K tile loop
        f += ["-mllvm", "-amdgpu-mfma-vgpr-form"]
    return f


def build(asm: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    report = os.path.join(BUILD_DIR, "resource_usage.txt")
    objs = [os.path.join(BUILD_DIR, os.path.basename(src) + ".o") for src, _ in SOURCES]

    def compile_unit(unit):
        (src, vgpr_form), obj = unit
        cmd = [hipcc(), *flags(vgpr_form), "-c", src, "-o", obj, "-Rpass-analysis=kernel-resource-usage"]
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.run(cmd, capture_output=True, text=True)

    # the units side by side: the largest takes most of the time
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        done = list(pool.map(compile_unit, zip(SOURCES, objs)))
    with open(report, "w") as f:
        f.write("".join(r.stderr for r in done))
    for (src, _), r in zip(SOURCES, done):
        if r.returncode != 0:
            sys.stderr.write(r.stderr[-8000:])
            raise RuntimeError(f"hipcc failed ({r.returncode}) on {src}; see {report}")
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *objs, "-o", OUT + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr[-8000:])
        raise RuntimeError(f"hipcc link failed ({r.returncode})")
    check_symbols(OUT + ".tmp")
    os.replace(OUT + ".tmp", OUT)
    build_calls(verbose)
    if asm:
        assemble()
    return OUT


def build_calls(verbose: bool = False) -> str | None:
    """Build the extension module _torch_calls (host code) against the library and torch; None where
    there is no torch, and so no tensor layer to serve."""
    import sysconfig

    try:
        import torch
    except ImportError:
        print("torch is not installed: built without _torch_calls, which the tensor layer needs",
              file=sys.stderr)
        return None
    from torch.utils.cpp_extension import include_paths, library_paths

    out = os.path.join(PKG, "_torch_calls.so")
    includes = [INCLUDE, *include_paths(), "/opt/rocm/include", sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{i}" for i in includes), os.path.join(CSRC, "torch_calls.cpp"), "-o", out + ".tmp",
           *(f"-L{l}" for l in library_paths()), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip",
           "-lc10", "-lc10_hip", f"-L{PKG}", f"-l:{os.path.basename(OUT)}", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr[-8000:])
        raise RuntimeError(f"g++ failed ({r.returncode}) on torch_calls.cpp")
    os.replace(out + ".tmp", out)
    return out


def check_symbols(lib: str) -> None:
    """Fail on any undefined symbol of the library's own namespace. The compiler can drop a
    kernel template's host stub without a diagnostic (and exit 0); the library then fails
    to load only where it is used, so the build refuses it here."""
    nm = shutil.which("nm") or "/opt/rocm/llvm/bin/llvm-nm"
    r = subprocess.run([nm, "-D", "--undefined-only", lib], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nm failed on {lib}: {r.stderr[-2000:]}")
    missing = [l.split()[-1] for l in r.stdout.splitlines() if "_ZN5sgemm" in l]
    if missing:
        raise RuntimeError("library has undefined kernel symbols (host stubs not emitted): " +
                           ", ".join(missing[:8]))


def assemble(out: str | None = None) -> str:
    """Write the gfx950 assembly of the library's device code (same flags as the build),
    all translation units into one file."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    s = out or os.path.join(BUILD_DIR, "sgemm_f32.s")
    parts = []
    for src, vgpr_form in SOURCES:
        part = s + "." + os.path.basename(src) + ".s"
        subprocess.run([hipcc(), *flags(vgpr_form), "--cuda-device-only", "-S", src, "-o", part],
                       check=True)
        with open(part) as f:
            parts.append(f.read())
        os.remove(part)
    with open(s, "w") as f:
        f.write("\n".join(parts))
    return s


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--asm", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(asm=a.asm, verbose=a.verbose))


if __name__ == "__main__":
    main()
