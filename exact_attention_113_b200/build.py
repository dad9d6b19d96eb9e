"""Build libfa.so (the C ABI of include/fa.h) for sm_100a with nvcc, and its
compiled torch binding with g++.

The library is built in-tree, at exact_attention_113_b200/lib/libfa.so, and
links the CUDA runtime statically; it reaches the driver's tensor-map encoder
through cudaGetDriverEntryPoint, so it loads on a machine without a GPU.

    python -m exact_attention_113_b200.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa.so")
# translation units, compiled at the same time: training and contiguous
# decoding; attention over a paged cache; page tables, norm and rotation
SOURCES = [os.path.join(CSRC, f) for f in ("fa_api.cu", "fa_paged_api.cu", "fa_serve_api.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("sm100.cuh", "fa_fwd_kernel.cuh",
                                                     "fa_bwd_kernel.cuh",
                                                     "fa_decode_kernel.cuh",
                                                     "fa_paged_kernel.cuh",
                                                     "fa_plan_kernel.cuh",
                                                     "fa_rope_kernel.cuh",
                                                     "fa_serve_host.h")] + [
    os.path.join(INCLUDE, "fa.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in DEPENDS)


# The forward launches 384 threads and re-splits its registers with
# setmaxnreg (2 warpgroups x 224 + 1 x 56 = 384 x 168); the backward 768
# for D <= 64 (4 x 80 + 104 + 56 = 768 x 80) and 512 above (2 x 144 + 168 +
# 56 = 512 x 128).  A split is only valid when every instance is compiled at
# exactly its launch allocation (registers per thread).
LAUNCH_REGS = {"fa_fwd_kernel": 168, "fa_bwd_kernel": 128}
# the paged forward's split is the forward's
PAGED_LAUNCH_REGS = {"fa_paged_kernel": 168}


def launch_regs(name: str, tag: str) -> int:
    """The launch allocation of one instance (its mangled name): the
    backward's depends on its head dim, the first template argument."""
    if tag == "fa_bwd_kernel":
        m = re.search(r"fa_bwd_kernelILi(\d+)E", name)
        if m and int(m.group(1)) <= 64:
            return 80
    return {**LAUNCH_REGS, **PAGED_LAUNCH_REGS}[tag]


def check_register_counts(ptxas_log: str, want: dict = LAUNCH_REGS) -> dict:
    """Parse `ptxas -v` output; require `want` for every instance of each
    setmaxnreg kernel (by default the forward's and the backward's)."""
    counts, current = {}, None
    for line in ptxas_log.splitlines():
        m = re.search(r"Function properties for (\S+)", line)
        if m:
            current = m.group(1)
            continue
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            current = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and current and any(tag in current for tag in want):
            counts[current] = int(m.group(1))
    for tag in want:
        if not any(tag in k for k in counts):
            raise RuntimeError(f"no register counts found for {tag}")
    bad = {k: v for k, v in counts.items()
           for tag in want if tag in k and v != launch_regs(k, tag)}
    if bad:
        raise RuntimeError(f"register counts differ from the launch allocation "
                           f"{want}: {bad}; the setmaxnreg split would not match")
    return counts


# The watchdog test library: the same sources with the test hook compiled in
# (FA_TEST_HOOKS: the forward kernel's K producer can withhold one copy) and a
# 10 ms device wait limit, fp16 head dims 64 and 128 only.  Never libfa.so.
TESTHOOKS_PATH = os.path.join(LIB_DIR, "libfa_testhooks.so")
TESTHOOKS_FLAGS = ["-DFA_TEST_HOOKS", "-DFA_WAIT_LIMIT_NS=10000000ull"]


# The compiled torch binding of the serving entries: plain C++ against torch's
# headers, linked to libfa.so beside it; torch's own libraries are in the
# process before it is imported.  It is bound to the torch and the Python that
# it was compiled against, so both are in its name: another torch does not load
# it, and has its own built.
BINDING_SOURCE = os.path.join(CSRC, "fa_torch.cpp")


def binding_path() -> str:
    import torch
    return os.path.join(LIB_DIR, f"_fa_torch.torch-{torch.__version__}"
                                 f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False, verbose: bool = False) -> str | None:
    """Path of the binding; None where there is no torch to bind to (the C
    library does not need it)."""
    try:
        path = binding_path()
    except ImportError:
        sys.stderr.write("no torch: libfa.so without its torch binding\n")
        return None
    depends = [BINDING_SOURCE, os.path.join(INCLUDE, "fa.h")]
    if not force and os.path.exists(path) and \
            all(os.path.getmtime(p) <= os.path.getmtime(path) for p in depends):
        return path
    import torch
    from torch.utils import cpp_extension
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = path + f".tmp{os.getpid()}"
    dirs = cpp_extension.include_paths() + [sysconfig.get_paths()["include"],
                                            os.path.join(cuda, "include"), INCLUDE]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in dirs), "-o", tmp, BINDING_SOURCE, f"-L{LIB_DIR}", "-l:libfa.so",
           "-Wl,-rpath,$ORIGIN", *(f"-L{d}" for d in cpp_extension.library_paths()),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0 or verbose:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError("g++ failed building the torch binding")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, testhooks: bool = False) -> str:
    path = TESTHOOKS_PATH if testhooks else LIB_PATH
    if not force and not is_stale(path):
        if not testhooks:
            build_binding(verbose=verbose)
        return path
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    sources = SOURCES[:2] if testhooks else SOURCES   # (the kernels with bounded waits)
    objects = [f"{tmp}.{i}.o" for i in range(len(sources))]

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("nvcc failed building libfa.so")
        if verbose:
            sys.stderr.write(res.stdout + res.stderr)
        return res.stdout + res.stderr

    def compile_one(src, obj):
        return run([nvcc(), "-Xptxas=-v", *NVCC_FLAGS, *(TESTHOOKS_FLAGS if testhooks else []),
                    "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src])

    try:
        with concurrent.futures.ThreadPoolExecutor(len(sources)) as pool:
            logs = list(pool.map(compile_one, sources, objects))
        check_register_counts(logs[0])
        check_register_counts(logs[1], PAGED_LAUNCH_REGS)
        run([nvcc(), *LINK_FLAGS, "-o", tmp, *objects])
        os.replace(tmp, path)
    finally:
        for f in objects + [tmp]:
            if os.path.exists(f):
                os.remove(f)
    if not testhooks:
        build_binding(force, verbose)
    return path


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv,
                testhooks="--testhooks" in sys.argv))
