"""Host-side checks of the paged-cache entry points: the header and the library agree, and bad arguments are
refused before anything is launched (fake device pointers are never followed on these paths)."""
import ctypes

import pytest
import torch

import video_diffusion_transformer_sage_gb300 as sage
from video_diffusion_transformer_sage_gb300 import _lib

BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    from video_diffusion_transformer_sage_gb300 import build
    build.build()
    return sage.lib()


def _view(ptr=4096, n=8, h=4, d=128, st=512, sh=128):
    return _lib.SageView(ptr, n, h, d, st, sh)


def _kv(**kw):
    f = dict(k_pages=4096, v_pages=8192, n_pages=10, page_size=16, n_heads=4, head_dim=128, k_stride_page=8192,
             k_stride_token=512, k_stride_head=128, v_stride_page=8192, v_stride_token=512, v_stride_head=128,
             format=0, k_scale=None, v_scale=None)
    f.update(kw)
    return _lib.SagePagedKVC(**f)


def _batch(**kw):
    f = dict(n_seqs=2, cu_q=4096, kv_len=4096, page_table=4096, max_pages=4, table_stride=4)
    f.update(kw)
    return _lib.SagePagedBatchC(**f)


def _append(L, q=None, k=None, v=None, gq=None, gk=None, cos=None, sin=None, rows=0, positions=None, eps=1e-6, kv=None,
            batch=None, q_out=4096, ost=512, osh=128, status=4096):
    return L.sage_paged_append(BY(q) if q else None, BY(k or _view()), BY(v or _view()), gq, gk, cos, sin, rows, positions,
                               eps, BY(kv or _kv()), BY(batch or _batch()), q_out, ost, osh, status, None)


def _attn(L, q=None, kv=None, batch=None, sm=0.1, causal=1, window=0, out=4096, ost=1024, osh=128, lse=None, ws=4096,
          nbytes=1 << 30):
    return L.sage_paged_attn(BY(q or _view(h=8, st=1024)), BY(kv or _kv()), BY(batch or _batch()), sm, causal, window, out,
                             ost, osh, lse, ws, nbytes, None)


def test_header_and_library(L):
    names = sage.header_functions(_lib.PAGED_HEADER)
    assert set(names) == {"sage_paged_append", "sage_paged_attn", "sage_paged_workspace_bytes"}
    for n in names:
        assert hasattr(L, n)
    text = open(_lib.PAGED_HEADER).read()
    assert f"#define SAGE_PAGED_WS_HEADER {_lib.PAGED_WS_HEADER}" in text
    assert ctypes.sizeof(_lib.SagePagedKVC) == 15 * 8 and ctypes.sizeof(_lib.SagePagedBatchC) == 6 * 8


def test_workspace_bytes(L):
    for d in (64, 128):
        assert L.sage_paged_workspace_bytes(d) > _lib.PAGED_WS_HEADER
    assert L.sage_paged_workspace_bytes(96) == 0 and L.sage_paged_workspace_bytes(0) == 0


BAD_CACHE = [
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(n_pages=0), 1), (dict(n_heads=0), 1), (dict(format=2), 1),
    (dict(format=1), 1), (dict(format=1, k_scale=4096), 1), (dict(k_stride_token=0), 1), (dict(v_stride_page=-8192), 1),
    (dict(head_dim=96), 3), (dict(page_size=12), 3), (dict(page_size=4), 3), (dict(page_size=2048), 3),
    (dict(n_heads=5000), 3), (dict(n_pages=1 << 31), 3), (dict(k_stride_page=1 << 39), 3),
    (dict(k_pages=4104), 2), (dict(v_stride_head=132), 2), (dict(format=1, k_scale=4096, v_scale=4096, k_stride_head=72), 2),
    (dict(format=1, k_scale=4098, v_scale=4096), 2),
]
BAD_BATCH = [
    (dict(n_seqs=-1), 1), (dict(cu_q=None), 1), (dict(kv_len=None), 1), (dict(page_table=None), 1), (dict(max_pages=0), 1),
    (dict(table_stride=3), 1), (dict(table_stride=-4), 1), (dict(n_seqs=65537), 3),
    (dict(max_pages=1 << 27, table_stride=1 << 27), 3), (dict(cu_q=4098), 2), (dict(page_table=4097), 2),
]


@pytest.mark.parametrize("fields,code", BAD_CACHE, ids=lambda x: str(x))
def test_bad_cache(L, fields, code):
    assert _append(L, kv=_kv(**fields)) == code
    assert _attn(L, kv=_kv(**fields)) == code


@pytest.mark.parametrize("fields,code", BAD_BATCH, ids=lambda x: str(x))
def test_bad_batch(L, fields, code):
    assert _append(L, batch=_batch(**fields)) == code
    assert _attn(L, batch=_batch(**fields)) == code


def test_append_refusals(L):
    assert _append(L, k=_view(ptr=0)) == 1
    assert _append(L, v=_view(n=7)) == 1
    assert _append(L, v=_view(n=-1), k=_view(n=-1)) == 1
    assert _append(L, k=_view(h=2)) == 1                      # another head count than the cache's
    assert _append(L, k=_view(d=64)) == 1
    assert _append(L, k=_view(n=(1 << 22) + 1), v=_view(n=(1 << 22) + 1)) == 3
    assert _append(L, k=_view(ptr=4100)) == 2
    assert _append(L, v=_view(st=500)) == 2
    assert _append(L, k=_view(st=-512)) == 1
    q = _view(h=8, st=1024)
    assert _append(L, q=_view(n=9)) == 1
    assert _append(L, q=q, q_out=None) == 1
    assert _append(L, q=q, q_out=4104) == 2
    assert _append(L, q=q, ost=12) == 2
    assert _append(L, q=q, ost=0) == 1 and _append(L, q=q, osh=0) == 1      # rows that coincide
    assert _append(L, q=_view(n=1 << 20, h=2500), k=_view(n=1 << 20), v=_view(n=1 << 20)) == 3   # over 2^31 rows
    assert _append(L, q=_view(h=5000)) == 3
    assert _append(L, cos=4096) == 1 and _append(L, sin=4096) == 1
    assert _append(L, cos=4096, sin=4096, rows=0) == 1
    assert _append(L, cos=4100, sin=4096, rows=5) == 2
    assert _append(L, gk=4100) == 2
    assert _append(L, positions=4098) == 2
    for eps in (-1.0, float("nan"), float("inf")):
        assert _append(L, eps=eps) == 1
    assert _append(L, status=None) == 1
    assert L.sage_paged_append(None, None, BY(_view()), None, None, None, None, 0, None, 1e-6, BY(_kv()), BY(_batch()),
                               None, 0, 0, 4096, None) == 1
    assert L.sage_paged_append(None, BY(_view()), BY(_view()), None, None, None, None, 0, None, 1e-6, None, BY(_batch()),
                               None, 0, 0, 4096, None) == 1
    # nothing to do: no launch
    assert _append(L, k=_view(ptr=0, n=0), v=_view(ptr=0, n=0)) == 0
    assert _append(L, batch=_batch(n_seqs=0, cu_q=None, kv_len=None, page_table=None)) == 0


def test_attention_refusals(L):
    assert _attn(L, q=_view(ptr=0, h=8, st=1024)) == 1
    assert _attn(L, q=_view(h=6, st=768)) == 1                # not a multiple of the cache's heads
    assert _attn(L, q=_view(h=4 * 129)) == 3                  # over 128 query heads per K/V head
    assert _attn(L, q=_view(d=64)) == 1
    assert _attn(L, q=_view(ptr=4100, h=8)) == 2
    assert _attn(L, causal=2) == 1 and _attn(L, window=-1) == 1
    assert _attn(L, causal=0, window=5) == 1                  # a window needs causal attention
    for sm in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert _attn(L, sm=sm) == 1
    assert _attn(L, ost=0) == 1 and _attn(L, osh=0) == 1
    assert _attn(L, out=None) == 1 and _attn(L, out=4100) == 2 and _attn(L, osh=20) == 2 and _attn(L, ost=-8) == 1
    assert _attn(L, lse=4098) == 2
    need = int(L.sage_paged_workspace_bytes(128))
    assert _attn(L, ws=None) == 4 and _attn(L, nbytes=need - 1) == 4 and _attn(L, ws=4096 + 16) == 2
    assert L.sage_paged_attn(None, BY(_kv()), BY(_batch()), 0.1, 1, 0, 4096, 0, 0, None, 4096, need, None) == 1
    assert _attn(L, q=_view(ptr=0, n=0, h=8, st=1024)) == 0
    assert _attn(L, batch=_batch(n_seqs=0)) == 0


def test_binding_refuses_before_any_call():
    """On CPU tensors: none of these reaches the library."""
    z = torch.zeros
    pages = z(2, 8, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sage.PagedKV(pages, pages)                                     # not on a GPU
    with pytest.raises(ValueError):
        sage.PagedKV(pages, pages.float())
    with pytest.raises(ValueError):
        sage.PagedKV(pages.half(), pages.half())
    with pytest.raises(ValueError):
        sage.PagedKV(pages, pages, z(2), z(2))                         # scales without an 8-bit cache
    with pytest.raises(ValueError):
        sage.PagedBatch(z(3, dtype=torch.int32), z(2, dtype=torch.int32), z(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sage.PagedBatch(z(3, dtype=torch.int64), z(2, dtype=torch.int32), z(2, 4, dtype=torch.int32))
