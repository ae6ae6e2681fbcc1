"""Build libscout.so, libscoutgen.so and the native binding in-tree with nvcc for sm_103a.

    python -m block_sparse_kv_pred_gb300.build

Each translation unit compiles in its own process; the objects are linked into
shared libraries next to this file.  No CMake, no torch extension machinery.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
          "-Xcompiler", "-pthread", "-I" + os.path.join(ROOT, "include")]

LIBS = {
    "libscout.so": [os.path.join(PKG, "csrc", f) for f in
                    ("api.cu", "digest.cu", "score_topk.cu", "sparse_attn.cu", "merge.cu", "predict_q.cu",
                     "recall.cu", "lists.cu", "tables.cu", "append8.cu", "digest8.cu", "sparse_attn8.cu",
                     "cpu_attend.cpp")],
    "libscoutgen.so": [os.path.join(PKG, "workload", "gen.cu")],
}
# the native part of the Python binding: plain C++ against PyTorch's and Python's headers
BINDING = os.path.join(PKG, "csrc", "binding.cpp")


def _binding_flags() -> tuple[list[str], list[str]]:
    import torch

    t = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    libs = ["-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L" + PKG, "-lscout", "-Xlinker", "-rpath=$ORIGIN"]
    return [f for d in inc for f in ("-I", d)], libs


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [nvcc(), *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def lib_path(name: str) -> str:
    return os.path.join(PKG, name)


def _link(name: str, objs: list[str], libs: list[str]) -> str:
    target = lib_path(name)
    tmp = target + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, *libs, "-lcudart", "-Xcompiler", "-pthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed for {name}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, target)
    return target


def _binding_object() -> tuple[str, list[str]]:
    flags, libs = _binding_flags()
    return _compile(BINDING, flags), libs


def build(verbose: bool = False, extra: list[str] | None = None) -> dict[str, str]:
    """The libraries, then the native binding: where PyTorch's headers are missing, or do not fit, it raises
    with the libraries in place."""
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    out = {}
    srcs = [s for v in LIBS.values() for s in v]
    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as ex:
        binding = ex.submit(_binding_object)
        objs = {s: ex.submit(_compile, s, extra) for s in srcs}
        for name, lib_srcs in LIBS.items():
            out[name] = _link(name, [objs[s].result() for s in lib_srcs], [])
        obj, libs = binding.result()
    out["_binding.so"] = _link("_binding.so", [obj], libs)
    if verbose:
        for target in out.values():
            print("built", target)
    return out


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
