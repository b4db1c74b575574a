"""Build the gfx950 HIP library in-tree: quantized_linear_attention_amd/libstq.so,
and the binding's compiled checks beside it, _tensor.so."""
import os
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = [os.path.join(PKG, "csrc", f) for f in ("stq.hip", "attn.hip", "attn_long.hip", "alloc.cpp")]
DEPS = SRC + [os.path.join(PKG, "csrc", f) for f in ("stq_device.h", "attn_device.h")] + [os.path.join(ROOT, "include", "stq.h")]
LIB = os.path.join(PKG, "libstq.so")
TENSOR_SRC, TENSOR_LIB = os.path.join(PKG, "csrc", "tensor.cpp"), os.path.join(PKG, "_tensor.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # every floating-point contraction in the kernels is an explicit fma
    "-ffp-contract=off",
    # no packed fp32 VALU ops (v_pk_{add,mul,fma}_f32) anywhere
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, out, verbose):
    tmp = out + ".tmp%d" % os.getpid()
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("%s failed (%d)" % (os.path.basename(cmd[0]), r.returncode))
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, out)


def _current(out, deps):
    return os.path.exists(out) and all(os.path.getmtime(out) >= os.path.getmtime(d) for d in deps)


def build(force=True, verbose=False):
    """Compile libstq.so and _tensor.so (always when force=True), the sources side by side."""
    from concurrent.futures import ThreadPoolExecutor
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor() as pool:
        jobs, link = [], None
        if force or not _current(LIB, DEPS):
            objects = [os.path.join(tmp, os.path.basename(f) + ".o") for f in SRC]
            jobs = [pool.submit(_run, [HIPCC] + FLAGS + ["-c", f], o, verbose) for f, o in zip(SRC, objects)]
            link = [HIPCC] + FLAGS[:1] + ["-shared", "-fPIC"] + objects
        if force or not _current(TENSOR_LIB, [TENSOR_SRC]):
            from torch.utils.cpp_extension import include_paths, library_paths
            inc = include_paths() + [sysconfig.get_paths()["include"]]
            jobs.append(pool.submit(_run, [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared"] +
                                    ["-I" + d for d in inc] + [TENSOR_SRC] + ["-L" + d for d in library_paths()] +
                                    ["-ltorch_python", "-ltorch_cpu", "-lc10"], TENSOR_LIB, verbose))
        for j in jobs:
            j.result()
        if link:
            _run(link, LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=False))
