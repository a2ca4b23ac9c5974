"""The paged K/V cache on the GPU where its arithmetic or its records could go wrong."""
import pytest
import torch

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
