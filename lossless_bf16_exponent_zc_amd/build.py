"""Build libzc.so (HIP, gfx950) in-tree with hipcc, and with the host compiler
zc_experts_binding.so, the module that calls the expert operators from Python.

Flags:
  -O3 --offload-arch=gfx950      MI355X code objects only
  -ffp-contract=off              the fp64 moments and the fp32 reduce must be
                                 separately rounded adds/multiplies
  -fno-gpu-flush-denormals-to-zero   subnormal BF16 values are data
  -Xclang -target-feature -Xclang -packed-fp32-ops   no packed fp32 ops
  -Wall -Werror                  also what the optimizer says it could not do
                                 (a loop that a pragma asks it to unroll)
"""
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libzc.so")
BINDING = os.path.join(HERE, "zc_experts_binding.so")
SOURCES = ["zc_api.hip", "zc_sigma.hip", "zc_encode.hip", "zc_decode.hip", "zc_finish.hip",
           "zc_experts_api.hip", "zc_route.hip", "zc_rows.hip", "zc_blocks.hip", "zc_product.hip", "zc_choose.hip", "zc_orthogonalize.hip"]

INCLUDE = os.path.join(os.path.dirname(HERE), "include")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["-std=c++17", "-O3", "-fPIC", "--offload-arch=gfx950",
         "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Werror", "-Wno-unused-result", "-I" + INCLUDE]


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _build_binding() -> None:
    import torch

    at = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-I" + os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"), "-isystem", os.path.join(at, "include"),
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "zc_experts_binding.cpp"), "-o", BINDING + ".tmp",
           "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the expert operators' binding failed:\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(lambda s: _compile(s, list(extra)), SOURCES))
        binding.result()
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", LIB + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=[a for a in sys.argv[1:] if a.startswith("-")])
