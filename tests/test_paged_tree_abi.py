"""Host-side checks of the drafted-tree entry points: the header and the library agree, and bad arguments are refused before
anything is launched (fake device pointers are never followed on these paths)."""
import ctypes

import pytest
import torch

import test_paged_abi as base
import video_diffusion_transformer_sage_gb300 as sage
from test_paged_abi import BAD_BATCH, BAD_CACHE, _batch, _kv, _view
from video_diffusion_transformer_sage_gb300 import _lib

BY = ctypes.byref
L = base.L


def _tree(mask=4096, words=2, stride=2, depth=4096):
    return _lib.SagePagedTreeMaskC(mask, words, stride, depth)


def _build(L, batch=None, n=8, parents=4096, window=0, tree=None, positions=None, status=4096):
    return L.sage_paged_tree(BY(batch or _batch()), n, parents, window, BY(tree or _tree()), positions, status, None)


def _attn(L, q=None, kv=None, batch=None, tree=None, sm=0.1, window=0, out=4096, ost=1024, osh=128, lse=None, ws=4096,
          nbytes=1 << 30):
    return L.sage_paged_attn_tree(BY(q or _view(h=8, st=1024)), BY(kv or _kv()), BY(batch or _batch()), BY(tree or _tree()),
                                  sm, window, out, ost, osh, lse, ws, nbytes, None)


def test_header_and_library(L):
    names = sage.header_functions(_lib.TREE_HEADER)
    assert set(names) == {"sage_paged_tree", "sage_paged_attn_tree"}
    for n in names:
        assert hasattr(L, n) and hasattr(sage, n)
    assert ctypes.sizeof(_lib.SagePagedTreeMaskC) == 4 * 8


@pytest.mark.parametrize("fields,code", BAD_CACHE, ids=lambda x: str(x))
def test_bad_cache(L, fields, code):
    assert _attn(L, kv=_kv(**fields)) == code


@pytest.mark.parametrize("fields,code", BAD_BATCH, ids=lambda x: str(x))
def test_bad_batch(L, fields, code):
    assert _attn(L, batch=_batch(**fields)) == code
    if fields.get("max_pages") != 1 << 27:      # that table is too wide for its page size, which the tree does not know
        assert _build(L, batch=_batch(**fields)) == code


BAD_TREE = [(dict(mask=None), 1), (dict(words=0), 1), (dict(words=-1), 1), (dict(stride=1), 1), (dict(stride=-2), 1),
            (dict(words=65537, stride=65537), 3), (dict(stride=(1 << 31) + 1), 3), (dict(mask=4098), 2), (dict(depth=4097), 2)]


@pytest.mark.parametrize("fields,code", BAD_TREE, ids=lambda x: str(x))
def test_bad_tree(L, fields, code):
    assert _build(L, tree=_tree(**fields)) == code
    assert _attn(L, tree=_tree(**fields)) == code


def test_tree_refusals(L):
    assert _build(L, n=-1) == 1 and _build(L, parents=None) == 1 and _build(L, window=-1) == 1
    assert _build(L, status=None) == 1
    assert _build(L, n=(1 << 22) + 1) == 3
    assert _build(L, parents=4098) == 2 and _build(L, positions=4098) == 2 and _build(L, status=4097) == 2
    assert L.sage_paged_tree(None, 8, 4096, 0, BY(_tree()), None, 4096, None) == 1
    assert L.sage_paged_tree(BY(_batch()), 8, 4096, 0, None, None, 4096, None) == 1
    # nothing to do: no launch
    assert _build(L, n=0, parents=None, tree=_tree(mask=None)) == 0
    assert _build(L, batch=_batch(n_seqs=0, cu_q=None, kv_len=None, page_table=None)) == 0


def test_attention_refusals(L):
    assert _attn(L, q=_view(ptr=0, h=8, st=1024)) == 1
    assert _attn(L, q=_view(h=6, st=768)) == 1 and _attn(L, q=_view(h=4 * 129)) == 3 and _attn(L, q=_view(d=64)) == 1
    assert _attn(L, window=-1) == 1 and _attn(L, window=5, tree=_tree(depth=None)) == 1
    for sm in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert _attn(L, sm=sm) == 1
    assert _attn(L, ost=0) == 1 and _attn(L, osh=0) == 1
    assert _attn(L, out=None) == 1 and _attn(L, out=4100) == 2 and _attn(L, osh=20) == 2 and _attn(L, ost=-8) == 1
    assert _attn(L, lse=4098) == 2
    need = int(L.sage_paged_workspace_bytes(128))
    assert _attn(L, ws=None) == 4 and _attn(L, nbytes=need - 1) == 4 and _attn(L, ws=4096 + 16) == 2
    assert L.sage_paged_attn_tree(BY(_view(h=8, st=1024)), BY(_kv()), BY(_batch()), None, 0.1, 0, 4096, 1024, 128, None, 4096,
                                  1 << 30, None) == 1
    assert _attn(L, q=_view(ptr=0, n=0, h=8, st=1024), tree=_tree(mask=None, depth=None)) == 0
    assert _attn(L, batch=_batch(n_seqs=0)) == 0


def test_binding_refuses_before_any_call():
    """On CPU tensors: none of these reaches the library."""
    z = torch.zeros
    with pytest.raises(ValueError):
        sage.PagedTree(z(3, 1, dtype=torch.int32))                     # not on a GPU
    with pytest.raises(ValueError):
        sage.PagedTree(z(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        sage.PagedTree(z(3, 1, dtype=torch.int64))
