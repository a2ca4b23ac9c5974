"""How the accounting of the cache's pages walks through the counts: every page is looked at once and none outside, up to the
most pages that are accepted.  The arithmetic is the kernels' own (csrc/paged_pool_walk.h, compiled here for the host)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "video_diffusion_transformer_sage_gb300", "csrc")
WARPS = 8 * 32

SOURCE = r"""
#include "paged_pool_walk.h"
using namespace sage;
// Pages that warp `warp` looks at, or -1: one outside its part, one out of order, or more steps than there are.
extern "C" long long walk(uint32_t n_pages, int warp, int warps) {
  const PoolPart part = pool_part(n_pages, warp, warps);
  if (part.from > part.to || part.to > n_pages) return -1;
  long long seen = 0, steps = 0;
  uint64_t at = part.from;
  for (uint32_t p0 = part.from; p0 < part.to; p0 += kPoolStep) {
    if (++steps > (static_cast<long long>(part.to) - part.from + kPoolStep - 1) / kPoolStep) return -1;
    for (int k = 0; k < kPoolKept; ++k)
      for (int lane = 0; lane < 32; ++lane) {
        const uint32_t p = pool_four(p0, k, lane);
        if (p >= part.to) continue;
        const int n = pool_four_whole(p, part.to) ? 4 : 0;
        for (uint64_t j = 0; j < 4; ++j)
          if (n == 4 || p + j < part.to) {
            if (p + j != at || p + j >= part.to) return -1;
            ++at;
            ++seen;
          }
      }
  }
  return seen;
}
extern "C" uint32_t bound(uint32_t n_pages, int warp, int warps, int upper) {
  const PoolPart part = pool_part(n_pages, warp, warps);
  return upper ? part.to : part.from;
}
"""


@pytest.fixture(scope="module")
def W(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    tmp = tmp_path_factory.mktemp("walk")
    (tmp / "w.cpp").write_text(SOURCE)
    lib = str(tmp / "w.so")
    subprocess.run([gxx, "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-shared", "-fPIC", "-I", CSRC,
                    str(tmp / "w.cpp"), "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.walk.restype, so.walk.argtypes = ctypes.c_longlong, [ctypes.c_uint32, ctypes.c_int, ctypes.c_int]
    so.bound.restype, so.bound.argtypes = ctypes.c_uint32, [ctypes.c_uint32] + [ctypes.c_int] * 3
    return so


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("n", [1, 3, 4, 127, 128, 129, 2047, 2048, 2049, 32768 * 16 - 1, 32768 * 16 + 1, 9_000_001])
def test_every_page_once(W, n):
    assert sum(W.walk(n, w, WARPS) for w in range(WARPS)) == n
    assert [W.bound(n, w, WARPS, 1) for w in range(WARPS)][:-1] == [W.bound(n, w, WARPS, 0) for w in range(1, WARPS)]


@pytest.mark.parametrize("n", [TOP, TOP - 1, TOP - 3, TOP - 127, TOP - 2047, TOP - 2048, TOP - 2049, 2 ** 30 + 5])
def test_the_last_pages_of_the_largest_pools(W, n):
    """The last warp's steps end behind 2^31 there."""
    assert W.bound(n, 0, WARPS, 0) == 0 and W.bound(n, WARPS - 1, WARPS, 1) == n
    for w in (0, 1, 100, WARPS - 2, WARPS - 1):
        assert W.walk(n, w, WARPS) == W.bound(n, w, WARPS, 1) - W.bound(n, w, WARPS, 0) > 0


def test_the_kernels_walk_by_it():
    text = open(os.path.join(CSRC, "paged_pool.cu")).read()
    assert text.count("for (uint32_t p0 = part.from; p0 < part.to") == 2 and "int p0" not in text.replace("uint32_t p0", "")
