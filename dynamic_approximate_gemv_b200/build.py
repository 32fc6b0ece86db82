"""Builds libeffort.so in-tree with nvcc for sm_100a (B200).

Run as ``python -m dynamic_approximate_gemv_b200.build``; ``__graft_entry__``
calls :func:`build`.  Device code is compiled without fast-math and with
denormals kept, so the selection products round exactly as the C ABI states.
"""
import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libeffort.so")
LIB_DEBUG = os.path.join(HERE, "libeffort_debug.so")
BINDING = os.path.join(HERE, "_effort_torch.so")  # csrc/torch_binding.cpp
SOURCES = ["api.cu", "prep.cu", "effort.cu", "dense.cu", "noalloc.cu",
           "api_ffn.cu", "norm.cu", "fp8.cu", "fp8_tc.cu", "tensor_map.cu", "moe.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xptxas", "-v",
]


def needs_build():
    built = (LIB, LIB_DEBUG, BINDING)
    if not all(os.path.exists(p) for p in built):
        return True
    t = min(os.path.getmtime(p) for p in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(HERE, "..", "include", "effort.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = " ".join(cmd) + "\n" + res.stdout + res.stderr
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + log[-8000:])
    return log


def _compile(out, extra):
    """Compiles every source to an object (side by side) and links `out`."""
    objs = os.path.join(HERE, "_build", os.path.basename(out) + ".o.d")
    os.makedirs(objs, exist_ok=True)
    flags = [NVCC] + [f for f in FLAGS if f != "-shared"] + extra + ["-I" + os.path.join(HERE, "..", "include")]
    pairs = [(os.path.join(CSRC, s), os.path.join(objs, s + ".o")) for s in SOURCES]
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers += [os.path.join(HERE, "..", "include", "effort.h"), __file__]
    newest = max(os.path.getmtime(h) for h in headers)
    todo = [(src, o) for src, o in pairs
            if not os.path.exists(o) or os.path.getmtime(o) < max(newest, os.path.getmtime(src))]

    def one(p):
        log = _run(flags + ["-c", "-o", p[1] + ".tmp", p[0]])
        os.replace(p[1] + ".tmp", p[1])
        return log

    with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 4) as pool:
        logs = list(pool.map(one, todo))
    logs.append(_run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", out + ".tmp"]
                      + [o for _, o in pairs]))
    os.replace(out + ".tmp", out)
    log = "".join(logs)
    with open(os.path.join(HERE, "build.log"), "a") as f:
        f.write(log)
    return log


def _compile_binding(out):
    """The binding of the feed-forward operators to torch tensors: host code only."""
    src = os.path.join(CSRC, "torch_binding.cpp")
    deps = (src, os.path.join(HERE, "..", "include", "effort.h"), __file__)
    if os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(d) for d in deps):
        os.utime(out)
        return ""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(NVCC), "..", "include")]
    libs = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-isystem" + i for i in inc), src, "-L" + libs, "-Wl,-rpath," + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-o", out + ".tmp"]
    log = _run(cmd)
    os.replace(out + ".tmp", out)
    return log


def build(force=False, verbose=False):
    """Compile the CUDA sources into libeffort.so (release) and
    libeffort_debug.so (-DEFFORT_DEBUG: kernels bounds-check the indices they
    take from data and report violations through the status word), and the
    feed-forward operators' binding to torch into _effort_torch.so, next to
    this file."""
    if not force and not needs_build():
        return LIB
    if force:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        for lib in (LIB, LIB_DEBUG):
            for s in SOURCES:
                o = os.path.join(HERE, "_build", os.path.basename(lib) + ".o.d", s + ".o")
                if os.path.exists(o):
                    os.remove(o)
    with open(os.path.join(HERE, "build.log"), "w"):
        pass
    log = _compile_binding(BINDING)
    log += _compile(LIB, [])
    log += _compile(LIB_DEBUG, ["-DEFFORT_DEBUG"])
    if verbose:
        print(log)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
