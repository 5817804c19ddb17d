"""Build libfattn.so in-tree with nvcc for sm_103a only.

    python -m tiled_attention_forward_gb300.build [--force]

Each translation unit under csrc/ is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -lineinfo -O3``, then linked into
``tiled_attention_forward_gb300/libfattn.so`` (CUDA runtime linked
statically; the driver API is reached through the runtime's entry-point
query, so the library does not link libcuda).  The Python marshalling of the
serving calls, ``_fattn_binding.so``, is compiled against torch's headers and
linked to that library.  No host-architecture flags are used, so the same
command builds on x86_64 and aarch64.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfattn.so")
BINDING = os.path.join(PKG, "_fattn_binding.so")
SOURCES = ["fattn_api.cu", "fwd_tc.cu", "fwd_ffma.cu", "fwd_unfused.cu", "bwd_tc.cu",
           "fwd_packed.cu", "cache_append.cu", "decode.cu", "fwd_rows.cu", "decode_shared.cu",
           "decode_cross.cu", "bwd_cross.cu", "rotate.cu"]
HEADERS = ["internal.h", "sm103_ptx.cuh", "fwd_tc_kernel.cuh", "bwd_tc_kernel.cuh", "decode_kernel.cuh",
           "tma_4d.cuh", "bwd_cross_dq.cuh", "bwd_cross_dkv.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I" + INCLUDE, "-I" + CSRC]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfattn")


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "fattn.h")]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [s] + hdrs):
            jobs.append([cc] + NVCC_FLAGS + ["-c", s, "-o", obj])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed for %s" % cmd[-3])
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        link = [cc] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(link) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


def build_binding(force=False, verbose=False):
    """The marshalling of the serving calls (csrc/binding.cpp), against this
    interpreter's and torch's headers."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "binding.cpp")
    # Rebuilt also for another torch or interpreter than it was built against.
    stamp = os.path.join(BUILD, "binding.txt")
    what = "%s %s" % (torch.__version__, sys.version)
    same = os.path.exists(stamp) and open(stamp).read() == what
    if same and not force and not _stale(BINDING, [src, os.path.join(INCLUDE, "fattn.h")]):
        return
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
           "-I" + INCLUDE, "-I" + os.path.join(t, "include"),
           "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"), "-I" + cuda,
           "-I" + sysconfig.get_paths()["include"], src, "-o", tmp, "-L" + PKG, "-lfattn",
           "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(t, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("the compiler failed for binding.cpp")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(what)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
