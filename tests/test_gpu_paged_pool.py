"""The pages of the paged K/V cache on the GPU: accounting against lists (tests/pool_ref.py), copies and kept tokens against
plain indexing, bit for bit."""
import random

import pytest
import torch

import pool_ref
import video_diffusion_transformer_sage_gb300 as sage

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------------------- accounting
def _world(r, rows, width, n_pages, page, used=0.4, filled=0.5):
    """A pool in order: rows with some pages each, a few shared, other pages held elsewhere, some never given out."""
    order = list(range(n_pages))
    r.shuffle(order)
    refs, table = [0] * n_pages, []
    for _ in range(rows):
        n = r.randint(0, int(width * filled))
        row = [order.pop() if order and r.random() < 0.95 else -1 for _ in range(n)]
        if table and r.random() < 0.3:
            row[:1] = table[-1][:1]
        table.append((row + [-1] * width)[:width])
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    for p in order[:int(len(order) * used)]:
        refs[p] = r.choice([1, 1, 2, -1])
    return refs, table


def _both(refs, table, page, pad=3):
    """(GPU pool, list pool, the wide buffer around the table)."""
    wide = torch.full((len(table), len(table[0]) + pad), -9, dtype=torch.int32, device="cuda")
    wide[:, :len(table[0])] = _i32(table)
    return sage.PagedPool(_i32(refs), wide[:, :len(table[0])], page), pool_ref.Pool(refs, table, page), wide


def _same(gpu, ref, wide):
    assert gpu.refs.tolist() == ref.refs
    assert gpu.page_table.tolist() == ref.table
    assert bool((wide[:, len(ref.table[0]):] == -9).all())
    code, where = sage.sage_check_device_status(gpu.status)
    assert (where in ref.bad if ref.bad else (code, where) == (0, 0)), (code, where, ref.bad)
    ref.bad.clear()


WORLDS = [(1, 1, 1, 8), (1, 5, 40, 16), (3, 40, 129, 8), (20, 7, 1000, 32), (33, 33, 1500, 64), (300, 20, 9001, 16),
          (5, 3000, 20000, 16), (40, 64, 300001, 128)]


@pytest.mark.parametrize("rows,width,n_pages,page", WORLDS)
def test_accounting_of_many_turns(rows, width, n_pages, page):
    r = random.Random(rows * 7 + width)
    gpu, ref, wide = _both(*_world(r, rows, width, n_pages, page), page)
    for turn in range(8):
        hi = [r.choice([0, r.randint(0, width * page), width * page, r.randint(0, 3 * page)]) for _ in range(rows)]
        lo = [r.choice([0, 0, r.randint(0, width * page)]) for _ in range(rows)]
        if turn % 3 == 2:
            sage.sage_paged_release(gpu, _i32(hi), _i32(lo))
            ref.release(lo, hi)
        else:
            none = turn % 2
            ok = sage.sage_paged_reserve(gpu, _i32(hi), None if none else _i32(lo))
            assert ok.tolist() == ref.reserve([0] * rows if none else lo, hi)
        _same(gpu, ref, wide)
        if rows > 1:
            n = r.randint(1, max(1, rows // 2))
            src, dst = [r.randrange(rows) for _ in range(n)], r.sample(range(rows), n)
            if turn % 2:      # rows that may be had: empty ones, and sources that are no children
                empty = [x for x in dst if x not in src]
                gone = [0 if x in empty else 2 ** 31 - 1 for x in range(rows)]
                sage.sage_paged_release(gpu, _i32(gone))
                ref.release([0] * rows, gone)
                _same(gpu, ref, wide)
            tokens = [r.choice([0, page, r.randint(0, width * page), r.randint(0, 2 * page)]) for _ in range(n)]
            tokens = [min(t, width * page) for t in tokens]
            got = sage.sage_paged_fork(gpu, _i32(src), _i32(dst), _i32(tokens))
            assert [x.tolist() for x in got] == ref.fork(src, dst, tokens)
            _same(gpu, ref, wide)


def test_reserve_until_the_pages_run_out():
    """A row that misses none is served whatever the others want; the first that cannot be ends it for all behind it."""
    refs, table = [1, 0, 0, 1, 0, 0], [[0, -1, -1, -1], [3, -1, -1, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]]
    gpu, ref, wide = _both(refs, table, 8)
    hi = [17, 8, 24, 8]
    ok = sage.sage_paged_reserve(gpu, _i32(hi))
    assert ok.tolist() == ref.reserve([0] * 4, hi) == [1, 1, 0, 0]
    assert gpu.page_table.tolist()[0] == [0, 1, 2, -1]
    _same(gpu, ref, wide)


def test_reserve_behind_a_window():
    """Entries before lo stay without a page."""
    gpu, ref, wide = _both([0] * 9, [[-1] * 6, [-1] * 6], 16)
    lo, hi = [33, 16], [96, 17]
    assert sage.sage_paged_reserve(gpu, _i32(hi), _i32(lo)).tolist() == ref.reserve(lo, hi) == [1, 1]
    assert gpu.page_table.tolist() == [[-1, -1, 0, 1, 2, 3], [-1, 4, -1, -1, -1, -1]]
    _same(gpu, ref, wide)


def test_numbers_out_of_range():
    big, low = 2 ** 31 - 1, -2 ** 31
    gpu, ref, wide = _both([0] * 50, [[-1] * 4 for _ in range(3)], 8)
    assert sage.sage_paged_reserve(gpu, _i32([big, low, 9]), _i32([low, 0, big])).tolist() == [1, 1, 1]
    ref.reserve([low, 0, big], [big, low, 9])
    assert ref.bad == {17}
    _same(gpu, ref, wide)
    for a, b, n in (([0], [7], [8]), ([-1], [1], [8]), ([2], [2], [8]), ([big], [low], [8]), ([0], [1], [big]), ([1], [2], [-5])):
        got = sage.sage_paged_fork(gpu, _i32(a), _i32(b), _i32(n))
        assert [x.tolist() for x in got] == ref.fork(a, b, n)
        assert ref.bad
        _same(gpu, ref, wide)
    # pages that do not exist, pages that nobody holds
    gpu, ref, wide = _both([0, 1, 0, -3, 2], [[1, 5, 2, big], [3, 0, 1, 4], [4, 4, 4, -7]], 8)
    sage.sage_paged_release(gpu, _i32([8, 0, 0]), _i32([0, 0, 0]))
    ref.release([0] * 3, [8, 0, 0])
    assert ref.bad == {16, 24} and ref.refs == [0, 0, 0, -3, 0]
    _same(gpu, ref, wide)


def test_fork_of_rows_with_missing_pages_and_of_rows_named_twice():
    gpu, ref, wide = _both([1, 1, 0, 0, 0, 0, 0, 0], [[0, 99, 1], [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3], 8)
    src, dst, n = [0, 0, 1, 0, 0], [1, 1, 2, 3, 4], [20, 8, 8, 12, 24]
    got = sage.sage_paged_fork(gpu, _i32(src), _i32(dst), _i32(n))
    want = ref.fork(src, dst, n)
    assert [x.tolist() for x in got] == want and want[3] == [1, 0, 0, 1, 1] and ref.bad == {16, 25}
    _same(gpu, ref, wide)


def test_fork_until_the_pages_run_out():
    gpu, ref, wide = _both([1, 1, 0, 0], [[0, 1]] + [[-1, -1] for _ in range(5)], 8)
    src, dst, n = [0] * 5, [5, 4, 3, 2, 1], [12, 8, 3, 9, 16]
    got = sage.sage_paged_fork(gpu, _i32(src), _i32(dst), _i32(n))
    want = ref.fork(src, dst, n)
    assert [x.tolist() for x in got] == want and want[3] == [1, 1, 1, 0, 1]
    _same(gpu, ref, wide)


def test_accounting_in_a_graph_and_on_another_stream():
    """Captured once, replayed with other lengths; scratch and outputs made on the given stream."""
    r = random.Random(5)
    refs, table = _world(r, 12, 30, 2000, 16)
    gpu, ref, wide = _both(refs, table, 16)
    hi, keep, ok = _i32([0] * 12), _i32([2 ** 31 - 1] * 12), torch.zeros(12, dtype=torch.int32, device="cuda")
    gpu.status
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.sage_paged_release(gpu, keep)
        sage.sage_paged_reserve(gpu, hi, ok=ok)
    for _ in range(4):
        k, h = ([r.randint(0, 480) for _ in range(12)] for _ in range(2))
        keep.copy_(_i32(k)), hi.copy_(_i32(h))
        graph.replay()
        ref.release([0] * 12, k)
        assert ok.tolist() == ref.reserve([0] * 12, h)
        _same(gpu, ref, wide)
    side = torch.cuda.Stream()
    busy = torch.randn((6000, 6000), device="cuda")
    fresh, ref, wide = _both(ref.refs, ref.table, 16)
    torch.cuda.synchronize()
    for _ in range(8):
        busy = busy @ busy * 1e-4
    h = [480] * 12
    h_dev = _i32(h)
    torch.cuda.synchronize()
    for _ in range(8):
        busy = busy @ busy * 1e-4
    ok = sage.sage_paged_reserve(fresh, h_dev, stream=side)
    side.synchronize()
    assert ok.tolist() == ref.reserve([0] * 12, h)
    _same(fresh, ref, wide)
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------------------- copies
LAYOUTS = [("bf16", "nhd"), ("bf16", "hnd"), ("bf16", "kv"), ("e4m3", "nhd"), ("e4m3", "hnd")]


def _cache(n_pages, page, hkv, d, fmt, layout, seed=0):
    """A cache of random bytes (NaN codes among them): (PagedKV, pages as bytes [n_pages, page, hkv, row] views)."""
    g = torch.Generator("cuda").manual_seed(seed)
    dt, e = (torch.float8_e4m3fn, 1) if fmt == "e4m3" else (torch.bfloat16, 2)
    if layout == "kv":      # K and V side by side in one buffer, heads before slots, with room between rows
        raw = torch.randint(0, 256, (n_pages, 2, hkv, page, d * e + 16), generator=g, device="cuda", dtype=torch.uint8)
        kv = [raw[:, i, :, :, :d * e].permute(0, 2, 1, 3) for i in range(2)]
    else:
        shape = (n_pages, hkv, page, d * e) if layout == "hnd" else (n_pages, page, hkv, d * e)
        kv = [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        if layout == "hnd":
            kv = [x.permute(0, 2, 1, 3) for x in kv]
    scale = [torch.ones(hkv, device="cuda") for _ in range(2)] if fmt == "e4m3" else [None, None]
    return sage.PagedKV(kv[0].view(dt), kv[1].view(dt), *scale), kv


@pytest.mark.parametrize("fmt,layout", LAYOUTS)
@pytest.mark.parametrize("page,hkv,d", [(8, 1, 64), (16, 3, 128), (64, 8, 128), (256, 5, 64), (1024, 2, 128)])
def test_copy(fmt, layout, page, hkv, d):
    r = random.Random(page + hkv)
    n_pages = 23
    cache, kv = _cache(n_pages, page, hkv, d, fmt, layout, seed=page)
    for tokens in ([r.randint(0, page) for _ in range(8)], None):
        order = r.sample(range(n_pages), n_pages)
        src, dst = [r.choice(order[8:]) for _ in range(8)], order[:8]
        src[1], dst[2] = -1, -1
        src[3] = dst[3]                      # a page to itself
        want = [x.clone() for x in kv]
        for w in want:
            for i, (a, b) in enumerate(zip(src, dst)):
                if a >= 0 and b >= 0:
                    n = page if tokens is None else tokens[i]
                    w[b, :n] = w[a, :n]
        sage.sage_paged_copy(cache, _i32(src), _i32(dst), None if tokens is None else _i32(tokens))
        assert all(torch.equal(a, b) for a, b in zip(kv, want))
    assert sage.sage_check_device_status(cache.status) == (0, 0)


def test_copy_numbers_out_of_range():
    cache, kv = _cache(6, 8, 2, 64, "bf16", "nhd")
    before = [x.clone() for x in kv]
    for src, dst, n, where in (([6], [0], [8], 16), ([0], [6], [8], 16), ([-2], [1], [8], 16), ([1], [2 ** 31 - 1], None, 16),
                               ([0], [1], [-1], 17), ([2], [3], [9], 17)):
        sage.sage_paged_copy(cache, _i32(src), _i32(dst), None if n is None else _i32(n))
        assert sage.sage_check_device_status(cache.status) == (1, where)
    for x, b in zip(kv, before):
        b[3] = b[2]                          # the last one: cut to the page
        assert torch.equal(x, b)
    sage.sage_paged_copy(cache, _i32([]), _i32([]))


def test_copy_of_more_pages_than_a_grid_has():
    cache, kv = _cache(140001, 8, 1, 64, "e4m3", "nhd", seed=3)
    order = torch.randperm(140001, device="cuda").to(torch.int32)
    src, dst = order[:70000].contiguous(), order[70000:140000].contiguous()
    want = [x.clone() for x in kv]
    for w in want:
        w[dst.long()] = w[src.long()]
    sage.sage_paged_copy(cache, src, dst)
    assert all(torch.equal(a, b) for a, b in zip(kv, want))


# ----------------------------------------------------------------------------------------- kept tokens
def _table(r, kv_lens, page, extra=1):
    need = [-(-k // page) for k in kv_lens]
    n_pages = sum(need) + 2
    order = r.sample(range(n_pages), n_pages)
    width, at, table = max(need + [0]) + extra, 0, []
    for n in need:
        table.append(order[at:at + n] + [-7] * (width - n))
        at += n
    return table, n_pages


def _moved(kv, table, page, first, keep):
    """Plain: everything read, then written."""
    out = []
    for x in kv:
        w = x.clone()
        for b, ks in enumerate(keep):
            if not ks:
                continue
            t = torch.tensor(table[b], device="cuda")
            old, now = torch.tensor(ks, device="cuda"), torch.arange(first[b], first[b] + len(ks), device="cuda")
            w[t[now // page], now % page] = x[t[old // page], old % page]
        out.append(w)
    return out


def _padded(keep, room=0):
    most = max([len(k) for k in keep] + [1]) + room
    return _i32([k + [2 ** 31 - 1] * (most - len(k)) for k in keep])   # behind n_keep: not read


def _compact(cache, table, kv_lens, first, keep, room=0, ws=None, stream=None):
    n = len(kv_lens)
    batch = sage.PagedBatch(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), _i32(kv_lens), _i32(table))
    sage.sage_paged_compact(cache, batch, _i32(first), _padded(keep, room), _i32([len(k) for k in keep]), ws=ws, stream=stream)


SHAPES = [
    # kv_lens, kept from there on (of how many), page, hkv, d
    ([9, 1, 40, 0, 33], 6, 8, 1, 64),
    ([70, 300, 64, 65] * 9, 9, 16, 8, 128),
    ([200, 1000], 200, 32, 3, 64),
    ([3000], 2500, 64, 8, 128),
    ([1500, 10, 2999, 0], 1400, 16, 5, 128),
    ([700, 650], 600, 1024, 56, 64),
]


@pytest.mark.parametrize("fmt,layout", LAYOUTS)
@pytest.mark.parametrize("kv_lens,most,page,hkv,d", SHAPES, ids=lambda x: str(x)[:16])
@pytest.mark.parametrize("kind", ["ascending", "runs", "near"])
def test_compact(fmt, layout, kv_lens, most, page, hkv, d, kind):
    r = random.Random(most + d)
    table, n_pages = _table(r, kv_lens, page)
    cache, kv = _cache(n_pages, page, hkv, d, fmt, layout, seed=most)
    first = [r.randint(0, k // 3) for k in kv_lens]
    keep = []
    for f, n in zip(first, kv_lens):
        if kind == "near":      # nearly all tokens kept: each place is still to be read by one just before
            gone = set(r.sample(range(f, n), min(n - f, 3)))
            keep.append([x for x in range(f, n) if x not in gone])
        elif kind == "ascending":
            keep.append(sorted(r.sample(range(f, n), r.randint(0, min(most, n - f)))))
        else:                   # runs of tokens: frames
            ks = []
            while len(ks) < most:
                at = (ks[-1] if ks else f) + r.choice([1, 1, 1, 17, n // 9 + 1])
                ks += range(at, min(at + r.randint(1, 2 * page), n))
                if at >= n:
                    break
            keep.append(ks[:most])
    want = _moved(kv, table, page, first, keep)
    ws = sage.paged_workspace(d)
    _compact(cache, table, kv_lens, first, keep, ws=ws)
    assert sage.sage_check_device_status(ws) == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(kv, want))
    assert not ws[256:sage._lib.PAGED_WS_HEADER].any()                    # the counters are back at zero


@pytest.mark.parametrize("hkv,layout", [(8, "nhd"), (56, "hnd")])
def test_compact_long_lists_again_and_again(hkv, layout):
    """Many items in flight that stand in each other's places; the last call's counters do not matter to the next."""
    n, page = 9000, 64
    r = random.Random(hkv)
    table, n_pages = _table(r, [n], page)
    cache, kv = _cache(n_pages, page, hkv, 128, "bf16", layout)
    ws = torch.zeros(sage._lib.PAGED_WS_HEADER, dtype=torch.uint8, device="cuda")
    for i in range(12):
        keep = sorted(r.sample(range(5, n), n - 5 - r.choice([1, 40, 3000])))
        want = _moved(kv, table, page, [5], [keep])
        _compact(cache, table, [n], [5], [keep], room=r.choice([0, 700]), ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(kv, want)), i
    assert sage.sage_check_device_status(ws) == (0, 0) and not ws.any()


def test_compact_numbers_out_of_range():
    page, n = 8, 30
    table = [[4, 1, 3, 0]]
    for keep, first, where in (([3, 4], [5], 23), ([9, 30], [2], 23), ([9, -1], [2], 23), ([9, 2 ** 31 - 1], [2], 23),
                               ([5, 7], [-1], 23), ([9, 9, 12], [2], 23), ([9, 7, 12], [2], 23), ([6, 28], [0], 16), ([25, 26], [6], 16)):
        cache, kv = _cache(5, page, 2, 64, "bf16", "nhd")
        t = [list(table[0])]
        if where == 16:
            t[0][3] = 5 if keep[0] == 6 else -1
        good = [(k, first[0] + i) for i, k in enumerate(keep) if first[0] + i >= 0 and first[0] + i <= k < n
                and (i == 0 or k > keep[i - 1])
                and 0 <= t[0][k // page] < 5]
        want = [x.clone() for x in kv]
        for w, x in zip(want, kv):
            for a, b in good:
                w[t[0][b // page], b % page] = x[t[0][a // page], a % page]
        ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
        _compact(cache, t, [n], first, [keep], ws=ws)
        assert sage.sage_check_device_status(ws) == (1, where)
        assert all(torch.equal(a, b) for a, b in zip(kv, want))
    # more than there is room for, fewer than none, a length above the table
    cache, kv = _cache(5, page, 2, 64, "bf16", "nhd")
    want = _moved(kv, table, page, [0], [[4, 9]])
    batch = sage.PagedBatch(_i32([0, 0]), _i32([500]), _i32(table))
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for n_keep in (3, 2 ** 31 - 1, -1):
        sage.sage_paged_compact(cache, batch, _i32([0]), _i32([[4, 9]]), _i32([n_keep]), ws=ws)
        assert sage.sage_check_device_status(ws) == (1, 17)
        assert all(torch.equal(a, b) for a, b in zip(kv, want))
        want = _moved(kv, table, page, [0], [[4, 9]]) if n_keep == 3 else want
    sage.sage_paged_compact(cache, batch, _i32([0]), _i32([[40, 9]]), _i32([2]), ws=ws)   # behind the table's last page
    assert sage.sage_check_device_status(ws) == (1, 23)


@pytest.mark.parametrize("most", [5, 700])
def test_values_that_are_the_keys_move_once(most):
    """One tensor for K and V."""
    r = random.Random(most)
    table, n_pages = _table(r, [900], 16)
    cache, kv = _cache(n_pages, 16, 2, 128, "bf16", "nhd")
    both = sage.PagedKV(cache.k_pages, cache.k_pages)
    for _ in range(5):
        keep = sorted(r.sample(range(3, 900), most))
        want = _moved(kv[:1], table, 16, [3], [keep])[0]
        _compact(both, table, [900], [3], [keep])
        assert torch.equal(kv[0], want)
    want[table[0][5]] = want[table[0][0]]
    sage.sage_paged_copy(both, _i32([table[0][0]]), _i32([table[0][5]]))
    assert torch.equal(kv[0], want)


def test_accounting_of_very_many_rows():
    """More rows than a grid has in one direction."""
    rows = 65536
    gpu = sage.PagedPool(torch.zeros(rows + 7, dtype=torch.int32, device="cuda"),
                         torch.full((rows, 2), -1, dtype=torch.int32, device="cuda"), 8)
    hi = torch.full((rows,), 8, dtype=torch.int32, device="cuda")
    assert bool(sage.sage_paged_reserve(gpu, hi).all())
    assert torch.equal(gpu.page_table[:, 0], torch.arange(rows, dtype=torch.int32, device="cuda"))
    hi[::2] = 0
    sage.sage_paged_release(gpu, hi)
    assert int(gpu.refs.sum()) == rows // 2 and bool((gpu.page_table[::2] == -1).all()) and bool((gpu.page_table[1::2, 0] >= 0).all())
    src = torch.arange(1, 2 * 20000, 2, dtype=torch.int32, device="cuda")
    lists = sage.sage_paged_fork(gpu, src, src - 1, torch.full_like(src, 8))
    assert bool(lists[3].all()) and torch.equal(gpu.page_table[0:40000:2, 0], gpu.page_table[1:40000:2, 0])
    assert sage.sage_check_device_status(gpu.status) == (0, 0)


def test_compact_nothing():
    cache, kv = _cache(5, 8, 2, 64, "bf16", "nhd")
    before = [x.clone() for x in kv]
    _compact(cache, [[4, 1, 3, 0]], [30], [7], [[]])
    none = sage.PagedBatch(_i32([0]), _i32([]), torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    sage.sage_paged_compact(cache, none, _i32([]), torch.zeros((0, 2), dtype=torch.int32, device="cuda"), _i32([]))
    batch = sage.PagedBatch(_i32([0, 0]), _i32([30]), _i32([[4, 1, 3, 0]]))
    sage.sage_paged_compact(cache, batch, _i32([0]), torch.zeros((1, 0), dtype=torch.int32, device="cuda"), _i32([0]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kv, before))


def test_compact_and_copy_over_offsets_past_32_bits():
    """A cache of more than 2^32 bytes a side, its pages at both ends in use."""
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (page * hkv * d * 2) + 40
    k = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache, kv = sage.PagedKV(k, v), [k, v]
    ends = [0, n_pages - 1, 1, n_pages - 2, 2, n_pages - 3]
    for x in kv:
        for p in ends:
            x[p].normal_()
    for most in (10, 1200):     # one item, and many
        keep = sorted(random.Random(most).sample(range(20, 1500), most))
        want = [torch.stack([x[ends[p // page], p % page] for p in keep]) for x in kv]
        _compact(cache, [ends], [1500], [7], [keep])
        for x, w in zip(kv, want):
            assert all(torch.equal(x[ends[(7 + i) // page], (7 + i) % page], w[i]) for i in range(most))
    sage.sage_paged_copy(cache, _i32([n_pages - 1, 0]), _i32([2, n_pages - 3]))
    for x in kv:
        assert torch.equal(x[2], x[n_pages - 1]) and torch.equal(x[n_pages - 3], x[0])


@pytest.mark.parametrize("most", [6, 900])
def test_compact_in_graphs_and_on_streams(most):
    """Two graphs that share a workspace, replayed with other lists; two calls at once on workspaces of their own."""
    r = random.Random(most)
    kv_lens, page = [1000, 990], 16
    table, n_pages = _table(r, kv_lens, page)
    cache, kv = _cache(n_pages, page, 8, 128, "bf16", "nhd")
    ws = sage.paged_workspace(128)
    batch = sage.PagedBatch(_i32([0, 0, 0]), _i32(kv_lens), _i32(table))
    first, n_keep = _i32([0, 0]), _i32([0, 0])
    keep = torch.zeros((2, most), dtype=torch.int32, device="cuda")
    sage.sage_paged_compact(cache, batch, first, keep, n_keep, ws=ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            sage.sage_paged_compact(cache, batch, first, keep, n_keep, ws=ws)
    for gr in graphs + graphs:
        ks = [sorted(r.sample(range(9, n), r.randint(1, most))) for n in kv_lens]
        first.copy_(_i32([9, 3])), n_keep.copy_(_i32([len(k) for k in ks]))
        keep.copy_(_padded(ks, most - max(map(len, ks))))
        want = _moved(kv, table, page, [9, 3], ks)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kv, want))
    caches = [_cache(n_pages, page, 8, 128, "bf16", "nhd", seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in caches]
    wants = [_moved(c[1], table, page, [9, 3], ks) for c in caches]
    torch.cuda.synchronize()
    busy = torch.randn((4000, 4000), device="cuda")
    for _ in range(6):
        busy = busy @ busy * 1e-4
    torch.cuda.current_stream().synchronize()
    first, n_keep, keep = _i32([9, 3]), _i32([len(k) for k in ks]), _padded(ks)
    torch.cuda.synchronize()
    for c, st in zip(caches, streams):
        sage.sage_paged_compact(c[0], batch, first, keep, n_keep, stream=st)
    torch.cuda.synchronize()
    for c, want in zip(caches, wants):
        assert all(torch.equal(a, b) for a, b in zip(c[1], want))


def test_a_workspace_with_an_unread_timeout_is_left_alone():
    """After an expired wait the calls on the block do no work until it has been read."""
    table, page = [[0, 1, 2, 3]], 8
    cache, kv = _cache(5, page, 2, 64, "bf16", "nhd")
    before = [x.clone() for x in kv]
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    sage.sage_debug_wait_timeout(ws, 1000)
    _compact(cache, table, [30], [0], [[4, 9]], ws=ws)
    assert sage.sage_check_device_status(ws)[0] == 6
    assert all(torch.equal(a, b) for a, b in zip(kv, before))
