"""The paged K/V cache on the GPU where its arithmetic or its records could go wrong."""
import pytest
import torch

import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu


def _handles(p):
    return sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale), sage.PagedBatch(p.cu_q, p.kv_len, p.table)


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
