"""Build libfp8q.so (the C-ABI library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8q.so")
BINDING = os.path.join(HERE, "_kv4_binding.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = ["fp8q.cu", "kv4.cu"]
# What each source file is made of; the public header belongs to both.
PARTS = {
    "fp8q.cu": ["fp8q.cu", "ptx.cuh", "quant.cuh", "gemm_prefill.cuh", "gemm_decode.cuh", "gemv_w8a16.cuh",
                "calib.cuh", "sched.cuh", "host.cuh"],
    "kv4.cu": ["kv4.cu", "ptx.cuh", "rope.cuh", "kv4.cuh", "kv4_list.cuh", "kv4_attention.cuh", "kv4_prefill.cuh", "host.cuh"],
}
DEPS = sorted({d for parts in PARTS.values() for d in parts})


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def flags(verbose: bool = False) -> list:
    f = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _older(out: str, deps: list) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = [os.path.join(CSRC, d) for d in deps] + [os.path.join(ROOT, "include", "fp8q.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def stale(lib: str = LIB) -> bool:
    return _older(lib, DEPS)


# Test build for the failure-detection tests: waits give up after 2 ms instead
# of 4 s, and a test-only switch makes one decode CTA withhold a release.  It
# is a separate file; the product library never contains the switch.
TEST_LIB = os.path.join(HERE, "libfp8q_testhooks.so")
TEST_FLAGS = ["-DFP8Q_TEST_HOOKS", "-DFP8Q_WAIT_LIMIT_NS=2000000ull"]


def _compile(out: str, extra: list, force: bool, verbose: bool) -> str:
    if not force and not stale(out):
        return out
    # one object per source file, side by side; those that are up to date are kept
    os.makedirs(OBJ, exist_ok=True)
    name = os.path.splitext(os.path.basename(out))[0]
    compile_flags = [f for f in flags(verbose) if f != "-shared"]
    objects, running = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, f"{name}.{os.path.splitext(src)[0]}.o")
        objects.append(obj)
        if force or _older(obj, PARTS[src]):
            cmd = [nvcc()] + compile_flags + extra + ["-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
            running.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = ""
    for obj, p in running:
        said, _ = p.communicate()
        if p.returncode != 0:
            failed += said
        else:
            os.replace(obj + ".tmp", obj)
            if verbose:
                sys.stderr.write(said)
    if failed:
        raise RuntimeError("nvcc failed:\n" + failed)
    r = subprocess.run([nvcc()] + flags() + objects + ["-o", out + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    os.replace(out + ".tmp", out)
    return out


def build_binding(force: bool = False) -> str:
    """_kv4_binding.so: the operand checks and calls of the KV-cache entry points in C++ (g++, torch's headers)."""
    if not force and not _older(BINDING, ["binding.cpp"]):
        return BINDING
    import sysconfig

    import torch
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    t = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for path in (os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
                 sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp", "-L", os.path.join(t, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + r.stdout + r.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    _compile(LIB, [], force, verbose)
    build_binding(force)
    return LIB


def build_test_hooks(force: bool = False) -> str:
    """The test build (libfp8q_testhooks.so) -- for tests only."""
    return _compile(TEST_LIB, TEST_FLAGS, force, False)


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
