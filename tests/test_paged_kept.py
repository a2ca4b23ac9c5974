"""How sage_paged_compact orders the items of a long list: which of them an item waits for (csrc/paged_kept.h, which the kernel
uses, compiled here for the host), and what puts their numbers in order, read from the kernel's source."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "video_diffusion_transformer_sage_gb300", "csrc")
SOURCE = os.path.join(CSRC, "paged_move.cu")

HOST = r"""
#include "paged_kept.h"
using namespace sage;
extern "C" int search(const int* keep, int n, long long place) {
  return kept_search(n, [&](int lo, int step, int m) {
    int below = 0;
    for (int lane = 0; lane < 32; ++lane) {
      const int at = kept_part_end(lo, step, m, lane);
      if (at < 0 || at >= n) return -1000000;   // outside the list
      below += keep[at] < place;
    }
    return below;
  });
}
extern "C" void wait(int i0, int count, int tokens, int from, uint32_t* out) {
  const KeptWait w = kept_wait(i0, count, tokens, from);
  out[0] = w.near;
  out[1] = w.far;
}
"""


@pytest.fixture(scope="module")
def K(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    tmp = tmp_path_factory.mktemp("kept")
    (tmp / "k.cpp").write_text(HOST)
    lib = str(tmp / "k.so")
    subprocess.run([gxx, "-O1", "-shared", "-fPIC", "-I", CSRC, str(tmp / "k.cpp"), "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.search.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_longlong]
    return so


def _list(r, n, first, gap):
    """n ascending positions, each from its new place on."""
    out, at = [], first - 1
    for i in range(n):
        at += 1 if r.random() > gap else r.randint(1, 1 + int(3 / gap))
        out.append(at)
    return out


def test_the_search_finds_the_first_entry_not_below(K):
    r = random.Random(1)
    for n in list(range(0, 70)) + [100, 1000, 1023, 1024, 1025, 1056, 1057, 4000, 33000]:
        keep = _list(r, n, r.randint(0, 50), r.choice([0.02, 0.3, 1.0]))
        raw = (ctypes.c_int * max(n, 1))(*keep)
        places = [0, keep[0] if keep else 5, keep[-1] if keep else 5, keep[-1] + 1 if keep else 5, 2 ** 40]
        for place in places + [r.randint(0, (keep[-1] if keep else 0) + 3) for _ in range(60)]:
            want = next((i for i, x in enumerate(keep) if x >= place), n)
            assert K.search(raw, n, place) == want, (n, place)


@pytest.mark.parametrize("tokens", [1, 3, 12, 256])
def test_an_item_waits_for_those_that_stand_in_its_new_places(K, tokens):
    """Against every entry looked at.  (The kernel waits for the items of as many entries as it has tokens, which in a list with
    gaps may be one more.)"""
    r = random.Random(tokens)
    waits = 0
    for _ in range(40):
        n, first = r.randint(1, 40 * tokens if tokens < 256 else 1500), r.randint(0, 300)
        keep = _list(r, n, first, r.choice([0.005, 0.05, 0.3, 1.0]))
        raw, out = (ctypes.c_int * n)(*keep), (ctypes.c_uint32 * 2)()
        for i0 in range(0, n, tokens):
            count = min(tokens, n - i0)
            start = K.search(raw, i0, first + i0) if i0 else 0
            K.wait(i0, count, tokens, start, out)
            near, far = int(out[0]), int(out[1])
            named = set(range(i0 // tokens - far, i0 // tokens - near + 1)) if far else set()
            # in the item itself all is read before anything is written
            there = {i // tokens for i in range(i0) if first + i0 <= keep[i] < first + i0 + count}
            assert named >= there and len(named) <= 2 and all(0 <= x < i0 // tokens for x in named), (i0, named, there)
            assert not there or min(named) == min(there)
            waits += bool(there)
    assert waits > 20


def test_the_rings_numbers_have_an_order():
    """An item's number is put behind a fence of the GPU's scope that comes after its rows were read, a writer goes on behind
    one that comes after it saw the numbers, and bulk stores behind a fence between the proxies."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert "fence.acq_rel.gpu" in text and "fence.proxy.async.global" in text
    kernel = text[text.index("paged_compact_long_kernel(const"):]
    assert "volatile uint16_t" not in kernel and "*at" not in kernel and not re.search(r"ring\[", kernel)
    read, fence, put, go = (kernel.index(x) for x in ("wait(full, k, B) &&", "fence_gpu();", "ring_put(", "pass(go, k, B)"))
    assert read < fence < put < go and kernel.count("ring_put(") == 1
    late = kernel[put:go]
    assert late.index("clear()") < late.index("fence_gpu();")
    write = kernel[kernel.index("bulk_store(") - 250:kernel.index("bulk_store(")]
    assert "fence_proxy_async_global();" in write
