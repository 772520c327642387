"""Build libq4amd.so in-tree for gfx950 with hipcc.

    python -m q4_weight_only_amd.build [--library] [-v]

Each .hip source is compiled to an object in parallel, then linked into
q4_weight_only_amd/libq4amd.so (written to a temporary name and renamed, so a
concurrent reader never sees a half-written library).  That takes hipcc alone;
the decoder operators' Python binding, _q4decoder.so, is linked after it and
takes a C++ compiler and torch's and Python's headers (--library leaves it out).
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libq4amd.so")
BINDING = os.path.join(PKG, "_q4decoder.so")     # the decoder operators' Python binding

SOURCES = ("q4_0_format.hip", "q4_1_format.hip", "q4_0_linear.hip", "q4_0_measure.hip", "q4_0_abi.hip",
           "q4_kv_append.hip", "q4_kv_attention.hip", "q4_rmsnorm.hip", "q4_logits.hip", "q4_decoder_abi.hip",
           "q4_beam.hip", "q4_kv_pages.hip", "q4_kv_select.hip", "q4_kv_blocks.hip", "q4_search_abi.hip")
ARCH = "gfx950"

COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # Packed fp32 VALU ops stay off: every fp32 op is issued one lane value
    # at a time.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in VGPRs: the per-block fp32 rescale reads them directly
    # instead of copying each one out of an AGPR first.
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    # Up to 12 leading scalar kernel arguments arrive preloaded in SGPRs, so a
    # decode launch's first loads do not wait on a fetch of its arguments.
    "-mllvm", "-amdgpu-kernarg-preload-count=12",
    "-Wall",
    "-Wextra",
    "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (expected /opt/rocm/bin/hipcc)")


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # the host pass of hipcc does not know the packed-fp32 target feature and
    # says so; that note is harmless and filtered out
    out = "\n".join(l for l in proc.stdout.splitlines() if "packed-fp32-ops" not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"command failed ({proc.returncode}): {' '.join(cmd)}\n{out}")
    return out


BUILD_INFO = os.path.join(BUILD_DIR, "build_info.json")


def _write_build_info() -> None:
    """Record the source revision the library was built from (reports read
    it where no git checkout exists)."""
    import json

    def git(*args):
        try:
            return subprocess.run(["git", *args], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.DEVNULL,
                                  text=True, timeout=30).stdout.strip()
        except (OSError, subprocess.SubprocessError):
            return ""
    info = {"git_rev": git("rev-parse", "HEAD") or None,
            "dirty": bool(git("status", "--porcelain", "--untracked-files=no"))}
    with open(BUILD_INFO, "w") as f:
        json.dump(info, f)


def _binding_command(out: str):
    """The C++ compiler's line for the decoder operators' binding (host code
    against torch's and Python's headers)."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_hipcc())))
    flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-unknown-pragmas", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__=1",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    dirs = [f"-I{INCLUDE}", *(f"-isystem{d}" for d in (
        os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
        os.path.join(rocm, "include"), sysconfig.get_paths()["include"]))]
    libs = [f"-L{PKG}", "-l:libq4amd.so", "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu",
            "-ltorch_hip", "-lc10", "-lc10_hip"]
    src = os.path.join(CSRC, "decoder_binding.cpp")
    return ([shutil.which("g++") or "c++", *flags, *dirs, "-c", src, "-o", os.path.join(BUILD_DIR, "decoder_binding.o")],
            [shutil.which("g++") or "c++", "-shared", "-o", out, os.path.join(BUILD_DIR, "decoder_binding.o"), *libs])


def build(verbose: bool = False, binding: bool = True) -> str:
    """Compile every HIP source for gfx950 and link libq4amd.so, which takes
    hipcc alone, then (unless `binding` is false) the Python binding of the
    decoder operators on top of it, which takes the C++ compiler and torch's and
    Python's headers; return the library's path.  Where the binding cannot be
    built, the library is in place before that is raised."""
    hipcc = _hipcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        cmds.append([hipcc, *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])

    def show(out):
        # compiler warnings are always shown; other output only when asked
        shown = out if verbose else "\n".join(l for l in out.splitlines() if "warning:" in l)
        if shown.strip():
            print(shown)

    def compile_binding():
        compile_cmd, link_cmd = _binding_command(binding_tmp)
        return _run(compile_cmd), link_cmd

    binding_tmp = BINDING + f".tmp{os.getpid()}"
    with ThreadPoolExecutor(max_workers=len(cmds) + 1) as ex:
        # beside the HIP sources; its failure is looked at when the library is there
        pending = ex.submit(compile_binding) if binding else None
        for out in ex.map(_run, cmds):
            show(out)
    _write_build_info()
    tmp = LIB + f".tmp{os.getpid()}"
    _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    if binding:
        try:
            out, link_cmd = pending.result()
            show(out)
            _run(link_cmd)
            os.replace(binding_tmp, BINDING)
        except Exception as e:
            if os.path.exists(BINDING):      # of another build: not to be used with this library
                os.remove(BINDING)
            raise RuntimeError(f"{LIB} is built (the C ABI and the linears); the decoder operators' Python binding is not: "
                               f"{e}") from e
    return LIB


if __name__ == "__main__":
    path = build(verbose="-v" in sys.argv, binding="--library" not in sys.argv)
    print(path)
