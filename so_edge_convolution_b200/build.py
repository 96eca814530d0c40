"""Build libso2conv.so in-tree with nvcc for sm_100a.

The library is one shared object with a C ABI (include/so2conv.h and so2model.h).  It is
linked against the static CUDA runtime and does not link libcuda, so it loads
(and reports its symbols) on a machine without a GPU.

    python -m so_edge_convolution_b200.build [--force] [--verbose]
"""

import argparse
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libso2conv.so")
# translation units, compiled in parallel and linked into one shared object
SOURCES = ["so2conv_api.cu", "so2conv_dbl_terms.cu"] + [
    os.path.join("model", f) for f in ("dropout.cu", "embed.cu", "mix.cu", "route.cu")]
OBJDIR = os.path.join(HERE, "_build")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]
LINK_FLAGS = ["-shared", "-cudart", "static"]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(d, f) for d in (CSRC, os.path.join(CSRC, "model"))
             for f in os.listdir(d) if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(ROOT, "include", f) for f in ("so2conv.h", "so2model.h")]
    return files


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force=False, verbose=False, extra=()):
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(OBJDIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        objs.append(obj)
        procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                      text=True))
    failed = False
    for src, pr in zip(SOURCES, procs):
        out = pr.communicate()[0]
        if pr.returncode != 0:
            failed = True
            sys.stderr.write(f"--- {src}\n" + out)
        elif verbose and out:
            sys.stderr.write(out)
    if failed:
        raise RuntimeError("nvcc failed building libso2conv.so")
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", *LINK_FLAGS, *objs, "-o", LIB]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed linking libso2conv.so")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true",
                    help="print registers / spills / shared memory per kernel")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra=extra))
