"""The host's choice between a product's forms, from fme_launch.h as it is, so that a test knows which form its sizes take."""
import ctypes
import functools
import os
import subprocess

from fp8_moe_expert_gb300 import build as fme_build

BUILD = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build")
SOURCE = """
#include "fme_launch.h"
extern "C" int few_halves(int64_t m, int64_t n, int64_t k, int32_t e, int sms) { return fme::bf16_few_halves(m, n, k, e, sms); }
extern "C" int gemv_share(int swiglu, int64_t m, int64_t n, int64_t k, int32_t e, int sms) {
  return fme::gemv_share(fme::gemv_units(swiglu != 0, m, n, k, e), k, sms);
}
"""


@functools.lru_cache(None)
def _lib():
    os.makedirs(BUILD, exist_ok=True)
    src, out = os.path.join(BUILD, f"rules_{os.getpid()}.cpp"), os.path.join(BUILD, f"librules_{os.getpid()}.so")
    try:
        with open(src, "w") as f:
            f.write(SOURCE)
        res = subprocess.run([fme_build.nvcc(), "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", fme_build.CSRC, "-I",
                              os.path.join(fme_build.ROOT, "include"), src, "-o", out], capture_output=True, text=True)
        assert res.returncode == 0, res.stdout + res.stderr
        lib = ctypes.CDLL(out)
    finally:
        for path in (src, out):
            if os.path.exists(path):
                os.remove(path)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.few_halves.argtypes = [i64, i64, i64, i32, i32]
    lib.gemv_share.argtypes = [i32, i64, i64, i64, i32, i32]
    return lib


def few_halves(m, n, k, experts, sms):
    """The bf16 forward: 0 for tiles, or the blocks of 64 of k in a stage of the form for few rows."""
    return _lib().few_halves(m, n, k, experts, sms)


def gemv_share(swiglu, m, n, k, experts, sms):
    """Warps that share a unit of the products with NVFP4 weights."""
    return _lib().gemv_share(int(swiglu), m, n, k, experts, sms)
