"""Host-side checks of the page entry points: the header and the library agree, and bad arguments are refused before
anything is launched (fake device pointers are never followed on these paths)."""
import ctypes

import pytest
import torch

import test_paged_abi as base
import video_diffusion_transformer_sage_gb300 as sage
from test_paged_abi import BAD_BATCH, BAD_CACHE, _batch, _kv
from video_diffusion_transformer_sage_gb300 import _lib

BY = ctypes.byref
L = base.L


def _pool(**kw):
    f = dict(refs=4096, n_pages=100, page_table=4096, n_rows=6, max_pages=9, table_stride=9, page_size=16)
    f.update(kw)
    return _lib.SagePagedPoolC(**f)


def _release(L, pool=None, lo=None, hi=4096, status=4096):
    return L.sage_paged_release(BY(pool or _pool()), lo, hi, status, None)


def _reserve(L, pool=None, lo=None, hi=4096, ok=None, ws=4096, nbytes=1 << 30):
    return L.sage_paged_reserve(BY(pool or _pool()), lo, hi, ok, ws, nbytes, None)


def _fork(L, pool=None, src=4096, dst=4096, tokens=4096, n=2, out=(4096,) * 4, ws=4096, nbytes=1 << 30):
    return L.sage_paged_fork(BY(pool or _pool()), src, dst, tokens, n, *out, ws, nbytes, None)


def _copy(L, kv=None, src=4096, dst=4096, tokens=None, n=3, status=4096):
    return L.sage_paged_copy(BY(kv or _kv()), src, dst, tokens, n, status, None)


def _compact(L, kv=None, batch=None, first=4096, keep=4096, most=4, stride=4, n_keep=4096, ws=4096, nbytes=4096):
    return L.sage_paged_compact(BY(kv or _kv()), BY(batch or _batch()), first, keep, most, stride, n_keep, ws, nbytes, None)


def test_header_and_library(L):
    names = sage.header_functions(_lib.POOL_HEADER)
    assert set(names) == {"sage_paged_pool_workspace_bytes", "sage_paged_release", "sage_paged_reserve", "sage_paged_fork",
                          "sage_paged_copy", "sage_paged_compact"}
    for n in names:
        assert hasattr(L, n) and (hasattr(sage, n) or n.endswith("_bytes"))
    assert ctypes.sizeof(_lib.SagePagedPoolC) == 7 * 8


def test_workspace_bytes(L):
    f = L.sage_paged_pool_workspace_bytes
    assert f(1, 1) > 256 and f(512, 400000) >= 256 + 4 * 400512
    assert f(0, 5) == 0 and f(5, 0) == 0 and f(65537, 5) == 0 and f(5, 1 << 31) == 0


BAD_POOL = [(dict(refs=None), 1), (dict(page_table=None), 1), (dict(n_pages=0), 1), (dict(n_rows=0), 1), (dict(max_pages=0), 1),
            (dict(table_stride=8), 1), (dict(table_stride=-9), 1), (dict(page_size=12), 3), (dict(page_size=4), 3),
            (dict(page_size=2048), 3), (dict(n_pages=1 << 31), 3), (dict(n_rows=65537), 3),
            (dict(max_pages=1 << 27, table_stride=1 << 27), 3), (dict(refs=4104), 2), (dict(page_table=4097), 2)]


@pytest.mark.parametrize("fields,code", BAD_POOL, ids=lambda x: str(x))
def test_bad_pool(L, fields, code):
    assert _release(L, pool=_pool(**fields)) == code
    assert _reserve(L, pool=_pool(**fields)) == code
    assert _fork(L, pool=_pool(**fields)) == code


def test_accounting_refusals(L):
    need = int(L.sage_paged_pool_workspace_bytes(6, 100))
    assert L.sage_paged_release(None, None, 4096, 4096, None) == 1
    assert _release(L, hi=None) == 1 and _release(L, status=None) == 1
    assert _release(L, lo=4097) == 2 and _release(L, hi=4098) == 2 and _release(L, status=4098) == 2
    assert _reserve(L, hi=None) == 1 and _reserve(L, lo=4097) == 2 and _reserve(L, ok=4097) == 2
    for call in (_reserve, _fork):
        assert call(L, ws=None) == 4 and call(L, nbytes=need - 1) == 4 and call(L, ws=4096 + 16) == 2
    assert _fork(L, n=-1) == 1 and _fork(L, n=7) == 1 and _fork(L, src=None) == 1 and _fork(L, dst=None) == 1
    assert _fork(L, tokens=None) == 1 and _fork(L, src=4097) == 2
    for i in range(4):
        assert _fork(L, out=[None if i == k else 4096 for k in range(4)]) == 1
        assert _fork(L, out=[4098 if i == k else 4096 for k in range(4)]) == 2
    assert _fork(L, n=0, src=None, dst=None, tokens=None, out=(None,) * 4) == 0


@pytest.mark.parametrize("fields,code", BAD_CACHE, ids=lambda x: str(x))
def test_bad_cache(L, fields, code):
    assert _copy(L, kv=_kv(**fields)) == code
    assert _compact(L, kv=_kv(**fields)) == code


@pytest.mark.parametrize("fields,code", BAD_BATCH, ids=lambda x: str(x))
def test_bad_batch(L, fields, code):
    assert _compact(L, batch=_batch(**fields)) == code


def test_move_refusals(L):
    assert _copy(L, src=None) == 1 and _copy(L, dst=None) == 1 and _copy(L, n=-1) == 1 and _copy(L, status=None) == 1
    assert _copy(L, n=(1 << 22) + 1) == 3
    assert _copy(L, src=4097) == 2 and _copy(L, tokens=4098) == 2 and _copy(L, status=4097) == 2
    assert _copy(L, n=0, src=None, dst=None) == 0
    assert _compact(L, first=None) == 1 and _compact(L, keep=None) == 1 and _compact(L, n_keep=None) == 1
    assert _compact(L, most=-1) == 1 and _compact(L, stride=3) == 1
    assert _compact(L, most=(1 << 30) + 1, stride=1 << 31) == 3
    assert _compact(L, first=4097) == 2 and _compact(L, keep=4098) == 2 and _compact(L, n_keep=4097) == 2
    assert _compact(L, ws=None) == 4 and _compact(L, nbytes=4095) == 4 and _compact(L, ws=4096 + 16) == 2
    assert _compact(L, most=0, keep=None) == 0
    assert _compact(L, batch=_batch(n_seqs=0), first=None, keep=None, n_keep=None) == 0
    big = _batch(n_seqs=65536)
    assert _compact(L, batch=big, most=1 << 20, stride=1 << 20) == 3      # over 2^31 items


def test_binding_refuses_before_any_call():
    """On CPU tensors: none of these reaches the library."""
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        sage.PagedPool(z(4), z(2, 3), 16)                              # not on a GPU
    with pytest.raises(ValueError):
        sage.PagedPool(z(4), z(3), 16)
    with pytest.raises(ValueError):
        sage.PagedPool(z(4), z(2, 0), 16)


@pytest.mark.parametrize("ctas,places,slots,buffers", [(1, 8, 8, 4), (3, 24, 8, 4), (7, 56, 8, 4), (4, 4, 8, 4), (5, 7, 3, 1)])
def test_the_order_of_long_lists_ends_and_overwrites_nothing(ctas, places, slots, buffers):
    """sage_paged_compact's items, drawn, read, announced and written by CTAs in any interleaving: no item waits for ever (also
    with fewer places in the ring than items in work), and none is written before the items that it names have been read."""
    import random
    for seed in range(25):
        r = random.Random(seed)
        units, runs = r.randint(1, 4), r.randint(1, 30)
        items = units * runs
        needs = [[i - d * units for d in range(1, r.randint(0, i // units) + 1)] for i in range(items)]
        ring = [0] * places
        turns = [[] for _ in range(ctas)]              # each CTA's items in the order drawn
        reads, writes, announced = [0] * ctas, [0] * ctas, [set() for _ in range(ctas)]
        drawn, was_read, was_written, idle = 0, set(), set(), 0
        while len(was_written) < items:
            idle += 1
            assert idle < 5000, "stuck"
            c, what = r.randrange(ctas), r.randrange(4)
            mine = turns[c]
            if what == 0 and drawn < items and len(mine) - writes[c] < slots:
                mine.append(drawn)
                drawn += 1
            elif what == 1 and reads[c] < len(mine) and reads[c] - writes[c] < buffers:
                was_read.add(mine[reads[c]])
                reads[c] += 1
            elif what == 2:                            # any buffer that has been read, not in order
                open_ = [k for k in range(writes[c], reads[c]) if k not in announced[c]]
                if open_:
                    k = r.choice(open_)
                    if ring[mine[k] % places] >= mine[k] // places:
                        assert ring[mine[k] % places] == mine[k] // places
                        ring[mine[k] % places] += 1
                        announced[c].add(k)
                        idle = 0
            elif what == 3 and writes[c] in announced[c]:
                item = mine[writes[c]]
                if all(ring[n % places] >= n // places + 1 for n in needs[item]):
                    assert was_read >= set(needs[item])
                    was_written.add(item)
                    writes[c] += 1
                    idle = 0
