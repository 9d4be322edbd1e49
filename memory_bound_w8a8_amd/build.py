"""Build libfp8bq.so in-tree with hipcc for gfx950.

    python -m memory_bound_w8a8_amd.build

Each .hip source under csrc/ is compiled to an object in _build/ (in
parallel), then linked into memory_bound_w8a8_amd/libfp8bq.so. Beside it the
Python module _binding.so is built from binding.cpp (host code only, against
the installed torch) and linked to that library; where that fails, the error
is raised with libfp8bq.so in place, which needs hipcc alone. The compile always
runs (no up-to-date check) so that a stale library is never shipped.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8bq.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = "gfx950"
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep the compiler from forming packed-fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # unroll the chunk loops in full even where in-kernel quantisation makes
    # them long: a partly rolled loop indexes the register arrays at run time,
    # which puts them in scratch memory
    "-mllvm", "-pragma-unroll-threshold=1000000",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]
# MFMA results in ordinary VGPRs: the per-group scale FMAs read them directly
# instead of copying each out of an accumulation register. Not for the int8
# product, whose sums stay in the accumulation registers (256 per wave).
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=true"]
ACC_FORM_SOURCES = {"gemm_i8.hip"}


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm required to build libfp8bq.so)")


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass warns about the device-only target feature; drop that noise
    out = "\n".join(ln for ln in proc.stdout.splitlines() if "packed-fp32-ops" not in ln)
    if proc.returncode != 0:
        raise RuntimeError(f"command failed ({proc.returncode}): {' '.join(cmd)}\n{out}")
    return out


def _binding_compile(obj):
    import torch
    from torch.utils import cpp_extension

    includes = [f"-I{p}" for p in cpp_extension.include_paths()]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", abi, f"-I{INCLUDE}", *includes,
            f"-I{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def _binding_link(obj, out):
    from torch.utils import cpp_extension

    return ["g++", "-shared", "-fPIC", obj, "-o", out, *[f"-L{p}" for p in cpp_extension.library_paths()],
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", f"-L{PKG}", "-l:libfp8bq.so", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False) -> str:
    def say(out):
        if verbose and out.strip():
            print(out)

    hipcc = _hipcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(f for f in os.listdir(CSRC) if f.endswith(".hip"))
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in sources]
    form = lambda s: [] if s in ACC_FORM_SOURCES else VGPR_FORM  # noqa: E731
    cmds = [[hipcc, *HIPCC_FLAGS, *form(s), "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(sources, objs)]
    binding_obj = os.path.join(BUILD, "binding.o")
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(cmds) + 1)) as ex:
        binding = ex.submit(lambda: _run(_binding_compile(binding_obj)))
        for out in ex.map(_run, cmds):
            say(out)
    tmp = LIB + ".tmp"
    say(_run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]))
    os.replace(tmp, LIB)
    # The library is there; the module needs more (g++, torch's headers). One of
    # an earlier build does not outlive a failure.
    try:
        say(binding.result())
        tmp = BINDING + ".tmp"
        say(_run(_binding_link(binding_obj, tmp)))
    except Exception:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        raise
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    path = build(verbose="-v" in sys.argv)
    print(path)
