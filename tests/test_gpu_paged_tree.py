"""Drafted trees over the paged K/V cache on the GPU: the ancestor bits, and attention of a tree over the cache, against the
definitions in 64 bits (tests/tree_ref.py; the error bounds are derived in tests/paged_ref.py)."""
import math
import random

import pytest
import torch

import paged_ref
import tree_ref
import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu


def _handles(p):
    return sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale), sage.PagedBatch(p.cu_q, p.kv_len, p.table)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _batch(q_lens, kv_lens):
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return sage.PagedBatch(_i32(cu), _i32(kv_lens), torch.zeros((len(q_lens), 1), dtype=torch.int32, device="cuda"))


def _bits(t):
    return t.contiguous().view(torch.int16)


# ----------------------------------------------------------------------------------------- the tree
TREES = [
    # q_lens, kv_lens, bushy, window
    ([1], [1], 1, 0),
    ([7, 0, 1, 33], [20, 5, 1, 40], 3, 0),
    ([32, 31, 64, 65, 1], [100, 31, 70, 65, 9], 2, 0),
    ([250] * 3, [300] * 3, 1, 0),
    ([100, 200], [5000, 200], 2, 3),
    ([40, 9], [41, 9], 1, 1),
    ([12, 6], [5, 0], 2, 0),                      # left padding
    ([3] * 300, list(range(3, 303)), 2, 0),
]


@pytest.mark.parametrize("q_lens,kv_lens,bushy,window", TREES, ids=lambda x: str(x)[:24])
def test_tree(q_lens, kv_lens, bushy, window):
    n, pad = sum(q_lens), 2
    parents = tree_ref.parents_of(q_lens, len(q_lens) + n, bushy)
    words = (max(q_lens) + 31) // 32 + 1
    mask = torch.full((n + pad, words + 3), -5, dtype=torch.int32, device="cuda")   # rows of a wider buffer
    depth, positions = (torch.full((n + pad,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    tree = sage.PagedTree(mask[:, :words], depth, positions)
    status = sage.status_block()
    got = sage.sage_paged_tree(_i32(parents + [0] * pad), _batch(q_lens, kv_lens), tree, status=status, window=window)
    assert got is tree and sage.sage_check_device_status(status) == (0, 0)
    seen, want = tree_ref.closure(q_lens, parents, window)
    assert torch.equal(mask[:, :words].cpu(), tree_ref.packed(seen, words, n + pad, -5))
    assert bool((mask[:, words:] == -5).all())
    assert depth.tolist() == want + [-5] * pad
    first = [max(0, k - q) for q, k in zip(q_lens, kv_lens) for _ in range(q)]
    assert positions.tolist() == [f + d for f, d in zip(first, want)] + [-5] * pad


def test_tree_of_more_tokens_than_shared_memory_holds():
    q_lens = [5000, 40]
    parents = [min(j - 1, max(-1, j - 1 - (j * j) % 90)) for j in range(5000)] + list(range(-1, 39))
    status = sage.status_block()
    tree = sage.sage_paged_tree(_i32(parents), _batch(q_lens, [6000, 40]), status=status, words=157)
    seen, depth = tree_ref.closure(q_lens, parents)
    assert torch.equal(tree.mask.cpu(), tree_ref.packed(seen, 157, 5040))
    assert tree.depth.tolist() == depth and sage.sage_check_device_status(status) == (0, 0)


def test_tree_without_depth_and_positions():
    parents = [-1, 0, 0, 1]
    tree = sage.PagedTree(torch.zeros((4, 1), dtype=torch.int32, device="cuda"))
    sage.sage_paged_tree(_i32(parents), _batch([4], [9]), tree, status=sage.status_block())
    assert tree.mask.flatten().tolist() == [0b1, 0b11, 0b101, 0b1011]


@pytest.mark.parametrize("bad", [(5, 5), (5, 6), (5, -2), (0, 0), (5, 2 ** 31 - 1), (5, -2 ** 31)])
def test_tree_bad_parents_are_recorded_and_taken_as_roots(bad):
    at, value = bad
    q_lens = [9]
    parents = tree_ref.parents_of(q_lens, 3)
    right = list(parents)
    parents[at], right[at] = value, -1
    status = sage.status_block()
    tree = sage.sage_paged_tree(_i32(parents), _batch(q_lens, [9]), status=status, words=1)
    assert sage.sage_check_device_status(status) == (1, 22) and sage.sage_check_device_status(status) == (0, 0)
    seen, depth = tree_ref.closure(q_lens, right)
    assert torch.equal(tree.mask.cpu(), tree_ref.packed(seen, 1, 9)) and tree.depth.tolist() == depth


def test_tree_of_more_tokens_than_words_is_recorded():
    q_lens, kv_lens = [40, 5], [50, 5]
    parents = tree_ref.parents_of(q_lens, 4, 1)
    status = sage.status_block()
    tree = sage.sage_paged_tree(_i32(parents), _batch(q_lens, kv_lens), status=status, words=1)
    assert sage.sage_check_device_status(status) == (1, 17)
    seen, depth = tree_ref.closure(q_lens, parents)
    assert torch.equal(tree.mask.cpu(), tree_ref.packed(seen, 1, 45)) and tree.depth.tolist() == depth


# ----------------------------------------------------------------------------------------- attention
ATTN = [
    # q_lens, kv_lens, hq, hkv, d, page, fmt, layout, window
    ([1], [1], 1, 1, 64, 8, "bf16", "nhd", 0),
    ([4], [4], 4, 1, 128, 8, "e4m3", "nhd", 0),                          # no cached text
    ([6, 8, 7], [300, 64, 71], 8, 2, 128, 16, "bf16", "nhd", 0),
    ([3, 0, 5], [1000, 9, 66], 24, 3, 64, 32, "bf16", "kv", 0),
    ([7, 2], [257, 2], 8, 4, 128, 64, "e4m3", "hnd", 0),
    ([4, 1], [777, 128], 12, 12, 64, 1024, "e4m3", "nhd", 0),
    ([15, 16], [500, 400], 4, 2, 128, 16, "bf16", "hnd", 0),             # 32 rows: two row tiles
    ([30, 31], [600, 130], 2, 2, 64, 8, "e4m3", "nhd", 0),
    ([16, 12], [900, 333], 8, 4, 128, 32, "e4m3", "kv", 0),
    ([9, 3], [4, 3], 4, 2, 64, 8, "bf16", "nhd", 0),                     # left padding
    ([8, 5, 3], [700, 90, 40], 8, 2, 128, 16, "bf16", "nhd", 100),
    ([5, 8], [2000, 64], 4, 1, 64, 32, "e4m3", "nhd", 6),
    ([33, 40], [500, 41], 1, 1, 128, 16, "bf16", "nhd", 0),              # the many-row kernel: one row tile
    ([64, 20, 1], [2003, 64, 900], 8, 2, 128, 64, "bf16", "nhd", 0),
    ([60, 0, 24], [1300, 9, 200], 24, 24, 64, 32, "e4m3", "nhd", 0),
    ([65, 50], [65, 190], 4, 2, 128, 64, "e4m3", "kv", 0),
    ([200, 130], [200, 1000], 7, 1, 128, 16, "bf16", "hnd", 0),          # units of two row tiles
    ([250, 129], [1111, 700], 6, 3, 64, 8, "bf16", "kv", 0),
    ([256], [900], 5, 5, 64, 16, "e4m3", "hnd", 0),
    ([150, 40], [700, 41], 10, 2, 128, 16, "bf16", "nhd", 130),
    ([190, 90], [800, 400], 8, 2, 128, 64, "e4m3", "nhd", 50),
    ([129, 70], [50, 0], 4, 2, 64, 16, "bf16", "nhd", 40),               # left padding in a wide tree
    ([300], [20000], 1, 1, 128, 64, "bf16", "nhd", 0),                   # the key axis split
    ([64], [9001], 8, 2, 64, 16, "e4m3", "nhd", 0),
    ([3], [30001], 8, 2, 128, 256, "bf16", "nhd", 0),
]


def _name(c):
    return f"q{max(c[0])}-kv{max(c[1])}-{c[2]}-{c[3]}-{c[4]}-p{c[5]}-{c[6]}-{c[7]}-w{c[8]}"


def _tree(q_lens, parents, rows, window=0, kind="tree", seed=0):
    """(who sees whom, depths, PagedTree).  "any": arbitrary bits, some rows and some tokens without any."""
    seen, depth = tree_ref.closure(q_lens, parents, window)
    if kind == "any":
        g = torch.Generator().manual_seed(seed)
        for m in seen:
            n = m.shape[0]
            m.copy_(torch.rand((n, n), generator=g) < 0.3)
            m[torch.rand(n, generator=g) < 0.3] = False
            m[:, torch.rand(n, generator=g) < 0.3] = False
    words = (max(q_lens + [1]) + 31) // 32
    mask = torch.full((rows, words + 1), -1, dtype=torch.int32, device="cuda")
    mask[:, :words] = tree_ref.packed(seen, words, rows, -1).cuda()
    return seen, depth, sage.PagedTree(mask[:, :words], _i32(depth + [10 ** 6] * (rows - len(depth))))


def _check(p, out, lse, ref, q=None):
    q = p.q if q is None else q
    tree_ref.check_attention(p, out, ref, q)
    # ln of the sum: score errors, and the rounded weights' 2^-8 (see paged_ref.attention_bound)
    empty = torch.isinf(ref[1])
    assert torch.equal(torch.isinf(lse[:p.n]), empty)
    lim = p.d * 2.0 ** -23 * ref[3] / math.sqrt(p.d) + 1.01 * 2.0 ** -8 + 1e-5 * (1 + ref[1].abs())
    lim = lim + tree_ref.score_slack(p, q, ref)
    assert ((lse[:p.n].double() - ref[1]).abs() <= lim)[~empty].all()


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("case", ATTN, ids=_name)
def test_attention(case, kind):
    """With "any", the new tokens that no row sees hold NaN, as the slots without a token do."""
    q_lens, kv_lens, hq, hkv, d, page, fmt, layout, window = case
    p = Problem(q_lens, kv_lens, hq, hkv, d, page, fmt, layout, seed=hq + sum(q_lens), pad_rows=2)
    seen, depth, tree = _tree(q_lens, tree_ref.parents_of(q_lens, 7 + sum(q_lens)), p.rows, window, kind, sum(kv_lens))
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        for i in range(max(0, n - kv), n):
            if not seen[b][:, i].any():
                pos = kv - n + i
                at = int(p.table[b, pos // page]), pos % page
                for pages in (p.k_pages, p.v_pages):
                    pages.view(torch.uint8)[at] = 0x7F if fmt == "e4m3" else 0xFF   # NaN in either type
    cache, batch = _handles(p)
    out = torch.full((p.rows, hq, d), -7.0, dtype=torch.bfloat16, device=p.dev)
    lse = torch.full((p.rows, hq), -7.0, dtype=torch.float32, device=p.dev)
    ws = sage.paged_workspace(d)
    got = sage.sage_paged_attn_tree(p.q, cache, batch, tree, window=window, out=out, lse=lse, ws=ws)
    assert got is out and sage.sage_check_device_status(ws) == (0, 0)
    _check(p, out, lse, tree_ref.attention(p, p.q, seen, depth, window))
    assert bool((out[p.n:] == -7.0).all()) and bool((lse[p.n:] == -7.0).all())
    assert not ws[256:sage._lib.PAGED_WS_HEADER].any()                    # the join counters are back at zero
    for _ in range(3):
        again = sage.sage_paged_attn_tree(p.q, cache, batch, tree, window=window, ws=ws)
        assert torch.equal(_bits(again[:p.n]), _bits(out[:p.n]))          # and the result does not vary


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("e4m3", 128), ("bf16", 64), ("e4m3", 64)])
@pytest.mark.parametrize("most", [8, 70])
def test_attention_of_many_trees_of_mixed_sizes(fmt, d, most):
    """More sequences than a warp has lanes, empty ones among them, ragged contexts."""
    r = random.Random(most + d)
    q_lens = [r.choice([0, 1, most // 2, most, r.randint(1, most)]) for _ in range(45)]
    kv_lens = [n + r.choice([0, 3, 64, 700, r.randint(0, 1500)]) for n in q_lens]
    p = Problem(q_lens, kv_lens, 8, 4, d, 32, fmt, seed=60 + d)
    seen, depth, tree = _tree(q_lens, tree_ref.parents_of(q_lens, most), p.rows)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(d)
    lse = torch.empty((p.rows, 8), dtype=torch.float32, device="cuda")
    out = sage.sage_paged_attn_tree(p.q, cache, batch, tree, lse=lse, ws=ws)
    _check(p, out, lse, tree_ref.attention(p, p.q, seen))
    for _ in range(5):
        assert torch.equal(_bits(sage.sage_paged_attn_tree(p.q, cache, batch, tree, ws=ws)), _bits(out))
    assert sage.sage_check_device_status(ws) == (0, 0)


@pytest.mark.parametrize("q_len,hq", [(6, 8), (80, 8)])
def test_a_chain_is_causal_attention(q_len, hq):
    p = Problem([q_len, q_len], [500, q_len + 3], hq, 2, 128, 16, seed=41)
    cache, batch = _handles(p)
    tree = sage.sage_paged_tree(_i32(list(range(-1, q_len - 1)) * 2), batch, status=cache.status, words=(q_len + 31) // 32)
    for window in (0, 3, 90):
        sage.sage_paged_tree(_i32(list(range(-1, q_len - 1)) * 2), batch, tree, status=cache.status, window=window)
        out = sage.sage_paged_attn_tree(p.q, cache, batch, tree, window=window)
        paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True, window))
    assert sage.sage_check_device_status(cache.status) == (0, 0)


@pytest.mark.parametrize("q_len", [5, 60])
def test_attention_new_tokens_behind_the_masks_words_are_seen_by_none(q_len):
    """One word for 40 and more tokens: those from 32 on count as unseen; a NaN there does no harm."""
    q_lens, kv_lens = [q_len, 45], [400, 60]
    p = Problem(q_lens, kv_lens, 4, 2, 64, 16, seed=43)
    seen, depth = tree_ref.closure(q_lens, tree_ref.parents_of(q_lens, 5))
    for m in seen:
        m[:, 32:] = False
    tree = sage.PagedTree(tree_ref.packed(seen, 1, p.rows).cuda())
    cache, batch = _handles(p)
    out = sage.sage_paged_attn_tree(p.q, cache, batch, tree)
    paged_ref.check_attention(p, out, tree_ref.attention(p, p.q, seen))


def test_attention_bits_of_tokens_that_do_not_exist_count_nothing():
    q_lens, kv_lens = [5, 40], [70, 300]
    p = Problem(q_lens, kv_lens, 8, 2, 128, 16, seed=44)
    seen, depth = tree_ref.closure(q_lens, tree_ref.parents_of(q_lens, 6))
    mask = tree_ref.packed(seen, 2, p.rows).cuda()
    mask[:5, 0] |= ~31                     # tokens 5 and up of a sequence of five
    mask[:5, 1] = -1
    cache, batch = _handles(p)
    out = sage.sage_paged_attn_tree(p.q, cache, batch, sage.PagedTree(mask))
    paged_ref.check_attention(p, out, tree_ref.attention(p, p.q, seen))


@pytest.mark.parametrize("q_len", [2, 90])
def test_attention_pages_before_the_window_may_be_gone(q_len):
    p = Problem([q_len], [900], 4, 2, 128, 16, seed=11)
    seen, depth, tree = _tree([q_len], tree_ref.parents_of([q_len], 8, 2), p.rows, 200)
    cache, batch = _handles(p)
    ref = tree_ref.attention(p, p.q, seen, depth, 200)
    first = (900 - q_len + 1 - 200) // 16
    p.table[0, :first] = -1
    ws = sage.paged_workspace(128)
    out = sage.sage_paged_attn_tree(p.q, cache, batch, tree, window=200, ws=ws)
    assert sage.sage_check_device_status(ws) == (0, 0)
    paged_ref.check_attention(p, out, ref)
    p.table[0, first + 4] = p.n_pages      # one that is read: its keys count as masked, and it is recorded
    sage.sage_paged_attn_tree(p.q, cache, batch, tree, window=200, out=out, ws=ws)
    assert sage.sage_check_device_status(ws) == (1, 16) and torch.isfinite(out.float()).all()


def test_attention_length_above_the_table_is_cut_and_recorded():
    p = Problem([3], [48], 2, 2, 64, 16, seed=12, extra_width=0)
    seen, depth, tree = _tree([3], [-1, 0, 0], p.rows)
    cache, batch = _handles(p)
    ref = tree_ref.attention(p, p.q, seen)
    p.kv_len[0] = 500
    ws = sage.paged_workspace(64)
    out = sage.sage_paged_attn_tree(p.q, cache, batch, tree, ws=ws)
    assert sage.sage_check_device_status(ws) == (1, 17)
    paged_ref.check_attention(p, out, ref)


@pytest.mark.parametrize("fmt,d", [("bf16", 64), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("q_len", [4, 50])
def test_attention_a_query_row_with_nan(q_len, fmt, d):
    """NaN in a row's q: NaN out, unless it sees no key; the other rows are as they were."""
    p = Problem([q_len], [300 + q_len], 4, 2, d, 16, fmt, seed=46)
    seen, depth, tree = _tree([q_len], tree_ref.parents_of([q_len], 9), p.rows)
    cache, batch = _handles(p)
    want = sage.sage_paged_attn_tree(p.q, cache, batch, tree)
    q = p.q.contiguous().clone()
    q[1, 2, 5] = float("nan")
    lse = torch.empty((p.n, 4), dtype=torch.float32, device="cuda")
    out = sage.sage_paged_attn_tree(q, cache, batch, tree, lse=lse)
    assert bool(out[1, 2].isnan().all()) and bool(lse[1, 2].isnan())
    out[1, 2], lse[1, 2] = want[1, 2], 0
    assert torch.equal(_bits(out), _bits(want)) and torch.isfinite(lse).all()


def test_attention_strided_views_and_expanded_query():
    q_lens = [5, 40]
    p = Problem(q_lens, [44, 300], 6, 2, 64, 16, seed=47)
    seen, depth, tree = _tree(q_lens, tree_ref.parents_of(q_lens, 10), p.rows)
    cache, batch = _handles(p)
    wide = torch.full((p.n, 2 * 6 * 64), -7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 6 * 64:].view(p.n, 6, 64)
    q = p.q[:, :1].expand(-1, 6, -1)
    sage.sage_paged_attn_tree(q, cache, batch, tree, sm_scale=0.3, out=out)
    paged_ref.check_attention(p, out, tree_ref.attention(p, q, seen, sm_scale=0.3), sm_scale=0.3)
    assert bool((wide[:, :6 * 64] == -7.0).all())


@pytest.mark.parametrize("q_len", [4, 70])
@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("e4m3", 128), ("e4m3", 64)])
def test_attention_of_rows_of_very_different_size(q_len, fmt, d):
    """Query rows scaled by 2^-90 .. 2^10, and the scores' scale with them; a head of zeros; rows with one channel far above
    the others."""
    p = Problem([q_len], [400], 4, 2, d, 16, fmt, seed=34)
    seen, depth, tree = _tree([q_len], tree_ref.parents_of([q_len], 12), p.rows)
    cache, batch = _handles(p)
    lse = torch.empty((p.rows, 4), dtype=torch.float32, device="cuda")
    for shift in (-90, 10):
        q = (p.q.float() * 2.0 ** shift).to(torch.bfloat16)
        sm = 2.0 ** -shift / math.sqrt(d)
        out = sage.sage_paged_attn_tree(q, cache, batch, tree, sm_scale=sm)
        tree_ref.check_attention(p, out, tree_ref.attention(p, q, seen, sm_scale=sm), q, sm_scale=sm)
    q = p.q.contiguous().clone()
    q[:, 1] = 0                       # uniform weights
    q[:, 2, 7] = 300.0
    q[:, 3, :-1] *= 2.0 ** -9
    out = sage.sage_paged_attn_tree(q, cache, batch, tree, lse=lse)
    _check(p, out, lse, tree_ref.attention(p, q, seen), q)


@pytest.mark.parametrize("q_len", [6, 48])
def test_graph_replay_after_trees_and_lengths_changed(q_len):
    """Tree and attention captured together; replayed with other parents, lengths and queries; two graphs that share the
    workspace one after the other."""
    hq, hkv, d, page = 8, 2, 128, 16
    p = Problem([q_len] * 2, [900, 640], hq, hkv, d, page, seed=48)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(d)
    q, parents = p.q.contiguous().clone(), _i32(tree_ref.parents_of(p.q_lens, 1))
    out = torch.zeros_like(q)
    tree = sage.sage_paged_tree(parents, batch, status=ws, words=2)
    sage.sage_paged_attn_tree(q, cache, batch, tree, out=out, ws=ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            sage.sage_paged_tree(parents, batch, tree, status=ws)
            sage.sage_paged_attn_tree(q, cache, batch, tree, out=out, ws=ws)
    for seed, kv in ((2, [900, 640]), (3, [q_len, 500]), (4, [333, 640])):
        new = tree_ref.parents_of(p.q_lens, seed)
        parents.copy_(_i32(new)), q.copy_(torch.randn(q.shape).to(torch.bfloat16)), p.kv_len.copy_(_i32(kv))
        p.kv_lens = kv
        want = tree_ref.attention(p, q, tree_ref.closure(p.q_lens, new)[0])
        for gr in graphs:
            out.zero_()
            gr.replay()
            torch.cuda.synchronize()
            paged_ref.check_attention(p, out, want)
    assert sage.sage_check_device_status(ws) == (0, 0)


def test_on_another_stream():
    """Buffers that the calls make belong to the given stream, while the current one is busy."""
    p = Problem([9, 40], [4000, 900], 8, 2, 128, 32, seed=49)
    parents = tree_ref.parents_of(p.q_lens, 11)
    cache, batch = _handles(p)
    ref = tree_ref.attention(p, p.q, tree_ref.closure(p.q_lens, parents)[0])
    parents, status = _i32(parents), sage.status_block()
    busy, side = torch.randn((6000, 6000), device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        for _ in range(8):
            busy = busy @ busy * 1e-4
        tree = sage.sage_paged_tree(parents, batch, status=status, words=2, stream=given)
        outs = [sage.sage_paged_attn_tree(p.q, cache, batch, tree, stream=given) for _ in range(3)]
        for _ in range(4):
            torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        for o in outs:
            paged_ref.check_attention(p, o, ref)
    torch.cuda.synchronize()
    assert sage.sage_check_device_status(status) == (0, 0)


def test_nothing_to_do():
    p = Problem([0], [30], 2, 2, 64, 8, seed=21)
    cache, batch = _handles(p)
    tree = sage.PagedTree(torch.zeros((0, 1), dtype=torch.int32, device="cuda"))
    assert tuple(sage.sage_paged_attn_tree(p.q, cache, batch, tree).shape) == (0, 2, 64)
    sage.sage_paged_tree(_i32([]), batch, tree, status=cache.status)
    none = sage.PagedBatch(_i32([0]), p.kv_len[:0], p.table[:0])
    p2 = Problem([2], [2], 2, 2, 64, 8, seed=21)
    out = torch.full_like(p2.q, -7.0)
    two = sage.PagedTree(torch.full((2, 1), 5, dtype=torch.int32, device="cuda"))
    sage.sage_paged_attn_tree(p2.q, cache, none, two, out=out)
    sage.sage_paged_tree(_i32([-1, 0]), none, two, status=cache.status)
    torch.cuda.synchronize()
    assert bool((out == -7.0).all()) and bool((two.mask == 5).all())
