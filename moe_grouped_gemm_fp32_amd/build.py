"""Ahead-of-time build of libfp8gemm.so for gfx950 (hipcc, in-tree), and of the native half
of the layer operators' Python binding (_layer_call.so, host code).

Every kernel variant is a template instance compiled once here; the host code
picks one per call. Packed-FP32 VALU instructions are disabled for all device code.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", "fp8gemm.hip"), os.path.join(PKG, "csrc_layer", "fp8layer.hip")]
LIB = os.path.join(PKG, "libfp8gemm.so")
CALL_SRC = os.path.join(PKG, "csrc_layer", "binding.cpp")
CALL = os.path.join(PKG, "_layer_call.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         # MFMA results in VGPRs: the FP32 promotion FMAs read them directly
         "-mllvm", "-amdgpu-mfma-vgpr-form",
         "-I", os.path.join(ROOT, "include")]


def sources() -> list:
    """Every file that the library is built from."""
    return [f for d in ("csrc", "csrc_layer") for f in sorted(glob.glob(os.path.join(PKG, d, "*")))] + \
        sorted(glob.glob(os.path.join(ROOT, "include", "*.h"))) + [os.path.abspath(__file__)]


def _call_command() -> list:
    """Compiles the layer operators' Python calls: host code against the interpreter's, torch's
    and the HIP runtime's headers. The library itself is bound when it is loaded."""
    from torch.utils.cpp_extension import include_paths, library_paths
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    headers = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
            "-I", os.path.join(ROOT, "include"), *(x for h in headers for x in ("-isystem", h)), CALL_SRC,
            *("-L" + d for d in library_paths()), "-lc10", "-ltorch_cpu", "-ltorch_python"]


def _compile(out: str, extra: list, verbose: bool, beside: dict = {}) -> str:
    """One object per source, compiled side by side, linked into `out`; `beside`: further
    files and the commands, up to -o, that make them. What could be made is there when another
    file's failure is raised."""
    tmp = out + ".tmp%d" % os.getpid()
    objs = ["%s.%d.o" % (tmp, i) for i in range(len(SRCS))]
    more = {path: path + ".tmp%d" % os.getpid() for path in beside}
    steps = [[hipcc(), *FLAGS, *extra, "-c", src, "-o", obj] for src, obj in zip(SRCS, objs)]
    steps += [[*cmd, "-o", more[path]] for path, cmd in beside.items()]
    link = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *extra, *objs, "-o", tmp]

    def start(cmd):
        try:
            return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        except OSError as e:  # no such compiler
            return e

    def finish(p):
        """A command's output if it failed, else None."""
        if isinstance(p, OSError):
            return f"{p}\n"
        said = p.communicate()[0]
        return said if p.returncode != 0 else None

    try:
        if verbose:
            print("\n".join("[build] " + " ".join(c) for c in [*steps, link]), flush=True)
        failed = [finish(p) for p in [start(c) for c in steps]]
        parts = failed[:len(objs)]
        if not any(f is not None for f in parts):
            parts.append(finish(start(link)))
        results = [(out, tmp, parts)] + [(path, made, [f]) for (path, made), f in zip(more.items(), failed[len(objs):])]
        missing = []
        for path, made, errors in results:
            if all(f is None for f in errors):
                os.replace(made, path)
            else:
                sys.stderr.write("".join(f for f in errors if f))
                missing.append(os.path.basename(path))
        if missing:
            raise RuntimeError("the compiler failed building " + ", ".join(missing))
    finally:
        for f in (*objs, tmp, *more.values()):
            if os.path.exists(f):
                os.remove(f)
    return out


def build_library(verbose: bool = True) -> str:
    """Compile libfp8gemm.so next to this file (always rebuilds). Returns its path. The C
    interface alone: hipcc is all that it needs."""
    return _compile(LIB, [], verbose)


def build(verbose: bool = True) -> str:
    """Compile libfp8gemm.so and _layer_call.so next to this file (always rebuilds). Returns the
    library's path. Where the binding cannot be built (no torch or Python headers, no host
    compiler), the library is built all the same before that is raised."""
    try:
        beside = {CALL: _call_command()}
    except Exception as e:
        build_library(verbose)
        raise RuntimeError(f"{os.path.basename(CALL)} cannot be built: {e}") from e
    return _compile(LIB, [], verbose, beside)


# Host-sanitizer build: the same library with its host code (argument checks, planner,
# plan cache, workspace and scratch bookkeeping) instrumented by AddressSanitizer and
# UndefinedBehaviorSanitizer, every finding fatal. The device code is built as usual
# (GPU sanitizers are not used). Load it with the sanitizer runtime preloaded
# (sanitizer_runtime()) and FP8GEMM_LIBRARY pointing at it; it is for host-only checks.
LIB_HOSTSAN = os.path.join(PKG, "libfp8gemm_hostsan.so")
HOSTSAN_FLAGS = ["-Xarch_host", "-g", "-Xarch_host", "-fsanitize=address,undefined",
                 "-Xarch_host", "-fno-sanitize-recover=undefined",
                 "-Xarch_host", "-fno-omit-frame-pointer", "-shared-libasan"]


def sanitizer_runtime() -> str:
    """Path of the shared AddressSanitizer runtime of hipcc's clang (for LD_PRELOAD)."""
    clang = os.path.join(os.path.dirname(os.path.realpath(hipcc())), "..", "llvm", "bin", "clang")
    if not os.path.exists(clang):
        clang = shutil.which("clang") or clang
    res = subprocess.run([clang, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True)
    path = res.stdout.strip()
    if res.returncode != 0 or not os.path.isabs(path) or not os.path.exists(path):
        raise RuntimeError("the AddressSanitizer runtime of hipcc's clang was not found")
    return path


def build_host_sanitized(verbose: bool = True, force: bool = False) -> str:
    """Compile libfp8gemm_hostsan.so next to this file unless it is newer than every
    source. Returns its path."""
    if not force and os.path.exists(LIB_HOSTSAN) and \
            os.path.getmtime(LIB_HOSTSAN) > max(os.path.getmtime(s) for s in sources()):
        return LIB_HOSTSAN
    return _compile(LIB_HOSTSAN, HOSTSAN_FLAGS, verbose)


if __name__ == "__main__":
    if "--host-sanitizers" in sys.argv[1:]:
        build_host_sanitized(force=True)
    elif "--library" in sys.argv[1:]:
        build_library()
    else:
        build()
