"""Build libtiles.so in-tree with nvcc for sm_103a (no cmake), and the compiled
half of the Python binding (_calls.so, against the installed PyTorch).

    python -m tile_size_decision_gb300.build [-v] [--force]

Each translation unit compiles in parallel into ``_build/``; the GEMM source
compiles once per (tile width, CTAs per MMA).  Objects newer than every source and header
are reused.  The shared library links the CUDA runtime statically and looks
up the driver at run time, so it loads on machines without a GPU.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtiles.so")
CALLS = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
          "--expt-relaxed-constexpr"]
GEMM_VARIANTS = ((64, 1), (128, 1), (192, 1), (256, 1), (128, 2), (256, 2))


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libtiles")
    return path


def units():
    """(source, object, extra flags) of every translation unit."""
    out = [
        ("planner.cpp", "planner.o", []),
        ("api.cu", "api.o", []),
        ("conv_sm103a.cu", "conv_sm103a.o", []),
        ("conv_tma_sm103a.cu", "conv_tma_sm103a.o", []),
        ("host_pipeline.cu", "host_pipeline.o", []),
        ("norm_sm103a.cu", "norm_sm103a.o", []),
        ("layernorm_sm103a.cu", "layernorm_sm103a.o", []),
        ("route_sm103a.cu", "route_sm103a.o", []),
        ("clip_sm103a.cu", "clip_sm103a.o", []),
        ("stream_sm103a.cu", "stream_sm103a.o", []),
        ("pair_sm103a.cu", "pair_sm103a.o", []),
        ("pair8_sm103a.cu", "pair8_sm103a.o", []),
        ("product_api.cu", "product_api.o", []),
        ("launch_util.cu", "launch_util.o", []),
    ]
    for bn, cg in GEMM_VARIANTS:
        out.append(("gemm_sm103a.cu", f"gemm_bn{bn}_cg{cg}.o",
                    [f"-DTILES_GEMM_BN={bn}", f"-DTILES_GEMM_CG={cg}"]))
    return out


def _headers_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, obj: str, extra: list, force: bool, verbose: bool) -> str:
    src_path = os.path.join(CSRC, src)
    obj_path = os.path.join(BUILD, obj)
    if not force and os.path.exists(obj_path):
        newest = max(os.path.getmtime(src_path), _headers_mtime())
        if os.path.getmtime(obj_path) >= newest:
            return obj_path
    cmd = [nvcc(), *ARCH, *COMMON, *extra, "-c", src_path, "-o", obj_path]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src} ({obj}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)
    return obj_path


def build_calls(force: bool = False, verbose: bool = False) -> str | None:
    """Compile the compiled calls (csrc/torch_calls.cpp); None without a PyTorch
    for CUDA, whose headers and libraries they need."""
    spec = importlib.util.find_spec("torch")
    torch = os.path.dirname(spec.origin) if spec is not None and spec.origin else None
    if torch is None or not os.path.exists(os.path.join(torch, "lib", "libtorch_cuda.so")):
        return None
    src = os.path.join(CSRC, "torch_calls.cpp")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(INCLUDE, "tiles.h"),
                                               os.path.join(torch, "version.py")))
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= newest:
        return CALLS
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-o", tmp, src,
           "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_calls.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS)
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every unit, link libtiles.so and the compiled calls; return
    libtiles.so's path.  Where the compiled calls do not compile (another
    PyTorch's headers, say) the library is there all the same: the package's
    functions then marshal their arguments in Python."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(units()) + 1, max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(build_calls, force, verbose)
        futs = [ex.submit(_compile, s, o, e, force, verbose) for s, o, e in units()]
        objs = [f.result() for f in futs]
    if force or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
               "-ldl", "-lpthread", "-lrt"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    try:
        got = calls.result()
    except (OSError, RuntimeError) as e:
        got = None
        warnings.warn(f"the compiled calls were not built: {e}")
    if got is None and os.path.exists(CALLS):
        os.remove(CALLS)                 # of other sources, or for another PyTorch
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("-v", "--verbose", action="store_true", help="print commands and ptxas usage")
    ap.add_argument("--force", action="store_true", help="rebuild every unit")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
