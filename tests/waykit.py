"""The host's rules of the 8-bit products, from the source itself: which way a
product's rows take (experts_launch.h), so that a test can state the kernels
that it means to run."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

SOURCE = """
#include "experts_launch.h"
using namespace experts;
extern "C" int way(int64_t rows, int count, int planes, int n, int k, int offsets) {
  const int blocks = red_blocks(k);
  const Way w = way_of(rows, count, planes * column_tiles(n), blocks, offsets != 0);
  return is_fused(w, rows, count, blocks, offsets != 0) ? -1 : (int)w;
}
"""
NAMES = {-1: "fused", 0: "brief", 1: "apart", 2: "together", 3: "few"}


@functools.lru_cache(maxsize=None)
def _library():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "way.cpp"), os.path.join(d, "way.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                            "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
                            "-I", os.path.join(ROOT, "latent_projection_top_amd", "csrc"), src, "-o", lib],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr)
        fn = ctypes.CDLL(lib).way
    fn.argtypes, fn.restype = [ctypes.c_int64] + [ctypes.c_int] * 5, ctypes.c_int
    return fn


def way(planes: int, rows: int, k: int, n: int, experts: int = 1, offsets: bool = False) -> str:
    """"fused", "brief", "few", "together" or "apart"."""
    return NAMES[_library()(rows, experts, planes, n, k, int(offsets))]


def way_of_counts(planes: int, counts, k: int, n: int, spare: int = 0) -> str:
    return way(planes, sum(counts) + spare, k, n, len(counts), True)


def heights(counts) -> set[int]:
    """Rows that the tile kernel's bodies for these experts' tiles have (those
    of more than 32 rows, on ways with tiles)."""
    out = set()
    for n in counts:
        if n <= 32:
            continue
        high = (n + 255) // 256
        height = min(((n + high - 1) // high + 31) // 32 * 32, 256)
        for t in range(high):
            rows = min(height, n - t * height)
            least = 64 if high == 1 else 192
            out.add(max(least, min(256, (rows + 63) // 64 * 64)))
    return out
