"""The paged K/V cache on the GPU where its arithmetic or its records could go wrong."""
import math

import pytest
import torch

import paged_ref
import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu


def _handles(p):
    return sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale), sage.PagedBatch(p.cu_q, p.kv_len, p.table)


# new tokens, tokens in the cache: few rows and many, in one item and with the key axis split over the SMs
ROWS = [([1], [90]), ([1], [40000]), ([7], [30000]), ([65], [300]), ([65], [9001]), ([200], [6000])]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", ROWS, ids=lambda x: f"q{x[0][0]}-kv{x[1][0]}")
def test_a_query_row_of_no_numbers_gives_none(lens, fmt):
    """A NaN in a query row makes its output and its lse NaN, however the key axis is split; no other row changes."""
    p = Problem(*lens, 4, 2, 128, 64, fmt, seed=60)
    cache, batch = _handles(p)
    t, h = p.n - 1, 1
    q = p.q.contiguous().clone()
    lse = torch.zeros((p.n, 4), dtype=torch.float32, device=p.dev)
    clean_lse = torch.zeros_like(lse)
    clean = sage.sage_paged_attn(q, cache, batch, lse=clean_lse)
    assert bool(torch.isfinite(clean.float()).all()) and bool(torch.isfinite(clean_lse).all())
    q[t, h, 5] = float("nan")
    out = sage.sage_paged_attn(q, cache, batch, lse=lse)
    assert bool(out[t, h].isnan().all()) and bool(lse[t, h].isnan())
    out[t, h], lse[t, h] = clean[t, h], clean_lse[t, h]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,d,kv", [(1, 64, 60), (1, 128, 30), (9, 64, 60), (70, 64, 100), (70, 128, 100), (300, 128, 100)])
@pytest.mark.parametrize("low", [14, 22])
def test_weights_far_below_the_largest_keep_their_precision(q_len, d, kv, fmt, low):
    """A first key that takes nearly all the weight and has no value: what is left is the sum over keys whose weights are
    2^-low of the largest and less.  It keeps the bound of every other case."""
    p = Problem([q_len], [kv], 2, 2, d, 64, fmt, seed=61)
    page = int(p.table[0, 0]), int(p.table[0, 1]) if kv > 64 else 0
    k = torch.zeros((kv, 2, d), device=p.dev)
    # with q = 1, sm_scale = ln 2 and unit scales, the base-2 score of a key is the sum of its channels
    k[1:, :, :low // 2] = -2.0
    k[1:, :, d - 1] = -0.125 * (torch.arange(1, kv, device=p.dev) % 8)[:, None]
    for i in range(kv):
        p.k_pages[page[i // 64], i % 64] = k[i].to(p.k_pages.dtype)
    p.v_pages[page[0], 0] = torch.zeros((2, d), device=p.dev).to(p.v_pages.dtype)
    if fmt == "e4m3":
        p.k_scale.fill_(1.0)
    q = torch.ones((q_len, 2, d), dtype=torch.bfloat16, device=p.dev)
    cache, batch = _handles(p)
    lse = torch.zeros((q_len, 2), dtype=torch.float32, device=p.dev)
    out = sage.sage_paged_attn(q, cache, batch, sm_scale=math.log(2.0), causal=False, lse=lse)
    ref = paged_ref.attention(p, q, False, sm_scale=math.log(2.0))
    assert float(ref[0].abs().max()) < 2.0 ** (4 - low) * 64       # nothing but the small weights
    paged_ref.check_attention(p, out, ref, sm_scale=math.log(2.0))
    assert float((lse.double() - ref[1]).abs().max()) <= 1.01 * 2.0 ** -8


def test_a_timeout_replaces_a_bad_index_that_nobody_read():
    """After both, the caller learns of the timeout (whose remedy is to zero the workspace header), and calls until then
    do no work; a bad index after a timeout changes nothing."""
    p = Problem([2], [20], 2, 2, 64, 8, seed=62)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(64)
    want = sage.sage_paged_attn(p.q, cache, batch, ws=ws).clone()
    p.table.fill_(p.n_pages)
    sage.sage_paged_attn(p.q, cache, batch, ws=ws)
    sage.sage_debug_wait_timeout(ws, 1_000_000)
    out = torch.full_like(want, -7.0)
    sage.sage_paged_attn(p.q, cache, batch, out=out, ws=ws)
    sage.sage_paged_append(p.k, p.v, cache, batch, status=ws)          # a bad index again: nothing over the timeout
    assert sage.sage_check_device_status(ws) == (6, 10)
    assert bool((out == -7.0).all())
    assert sage.sage_check_device_status(ws) == (0, 0)
    p2 = Problem([2], [20], 2, 2, 64, 8, seed=62)
    cache, batch = _handles(p2)
    assert torch.equal(sage.sage_paged_attn(p2.q, cache, batch, ws=ws), want)


def test_a_record_is_not_erased_by_the_blocks_making():
    """The cache's status block is needed first by a call on a busy stream; a record of a call on another stream, which
    runs before that, stays."""
    p = Problem([2], [20], 2, 2, 64, 8, seed=63)
    busy, idle = torch.cuda.Stream(), torch.cuda.Stream()
    bad = sage.PagedBatch(p.cu_q, p.kv_len, torch.full_like(p.table, p.n_pages))
    work = torch.randn((6000, 6000), device="cuda")
    torch.cuda.synchronize()
    for given in (busy, busy.cuda_stream):
        cache, batch = _handles(p)
        with torch.cuda.stream(busy):
            for _ in range(8):
                work = work @ work * 1e-4
        sage.sage_paged_append(p.k, p.v, cache, batch, stream=given)
        sage.sage_paged_append(p.k, p.v, cache, bad, stream=idle)
        idle.synchronize()
        torch.cuda.synchronize()
        assert sage.sage_check_device_status(cache.status) == (1, 16)
        assert sage.sage_check_device_status(cache.status) == (0, 0)


def test_a_block_made_in_a_graph_capture_is_ready_and_keeps_its_records():
    """The first call of a cache is captured: the block is zeros before any replay, and replays do not erase what others
    recorded; a replay's own bad index is recorded."""
    p = Problem([2], [20], 2, 2, 64, 8, seed=64)
    warm, _ = _handles(p)
    cache, batch = _handles(p)
    sage.sage_paged_append(p.k, p.v, warm, batch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.sage_paged_append(p.k, p.v, cache, batch)
    assert sage.sage_check_device_status(cache.status) == (0, 0)
    bad = sage.PagedBatch(p.cu_q, p.kv_len, torch.full_like(p.table, -1))
    sage.sage_paged_append(p.k, p.v, cache, bad)
    graph.replay()
    assert sage.sage_check_device_status(cache.status) == (1, 16)
    before = p.k_pages.clone()
    p.k_pages.fill_(0)
    graph.replay()
    assert sage.sage_check_device_status(cache.status) == (0, 0)
    assert torch.equal(p.k_pages[int(p.table[0, 2]), 2:4], before[int(p.table[0, 2]), 2:4])
    p.table.fill_(p.n_pages)
    graph.replay()
    assert sage.sage_check_device_status(cache.status) == (1, 16)
