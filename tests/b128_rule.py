"""The rule that chooses a kernel for a grouped product in blocks of 128, asked
of the library's own source (csrc/b128_rule.hpp, plain C++), built for the host."""

import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = ("few16", "few32", "few64", "narrow", "wide")
CUS = 256

SOURCE = """
#include "b128_rule.hpp"
extern "C" int product(int64_t El, int64_t M, int64_t N, int cus) { return moe::b128::product_kernel(El, M, N, cus); }
extern "C" int gradient(int64_t El, int64_t K, int64_t N, int cus) { return moe::b128::gradient_kernel(El, K, N, cus); }
"""


def compiler():
    return shutil.which("g++")


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "rule.so")
        subprocess.run([compiler(), "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "moe_fp8_grouped_amd", "csrc"),
                        "-x", "c++", "-", "-o", out], input=SOURCE, text=True, check=True)
        lib = ctypes.CDLL(out)
    for f in (lib.product, lib.gradient):
        f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
    return lib


def product_kernel(El, M, N, cus=CUS):
    return KERNELS[_lib().product(El, M, N, cus)]


def gradient_kernel(El, K, N, cus=CUS):
    return KERNELS[_lib().gradient(El, K, N, cus)]
