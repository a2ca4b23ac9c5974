"""q_out of sage_paged_append in q's own memory: only as q itself lies, since rows would be overwritten before they are
read otherwise.  Host-side checks: nothing is launched."""
import ctypes

import pytest

import video_diffusion_transformer_sage_gb300 as sage
from video_diffusion_transformer_sage_gb300 import _lib

BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    from video_diffusion_transformer_sage_gb300 import build
    build.build()
    return sage.lib()


# n, heads, q's token and head stride, q_out's
OTHER = [(8, 4, 512, 128, 128, 1024), (8, 4, 512, 128, 1024, 128), (8, 1, 512, 128, 1024, 128), (1, 4, 512, 128, 512, 256)]


@pytest.mark.parametrize("n,h,st,sh,ost,osh", OTHER)
def test_q_out_in_qs_memory_with_other_strides_is_refused(L, n, h, st, sh, ost, osh):
    kv = _lib.SagePagedKVC(4096, 8192, 10, 16, 4, 128, 8192, 512, 128, 8192, 512, 128, 0, None, None)
    batch = _lib.SagePagedBatchC(2, 4096, 4096, 4096, 4, 4)
    q, k = _lib.SageView(65536, n, h, 128, st, sh), _lib.SageView(4096, n, 4, 128, 512, 128)

    def call(q_out, seqs=batch):
        return L.sage_paged_append(BY(q), BY(k), BY(k), None, None, None, None, 0, None, 1e-6, BY(kv), BY(seqs), q_out, ost,
                                   osh, 4096, None)

    assert call(65536) == 1
    # with memory of its own it passes the checks (no sequences: nothing is launched)
    assert call(1 << 24, _lib.SagePagedBatchC(0, None, None, None, 0, 0)) == 0


def test_q_out_as_q_lies_is_taken(L):
    """Strides of a dimension with one element do not count."""
    kv = _lib.SagePagedKVC(4096, 8192, 10, 16, 4, 128, 8192, 512, 128, 8192, 512, 128, 0, None, None)
    none = _lib.SagePagedBatchC(0, None, None, None, 0, 0)
    for n, h, st, sh, ost, osh in ((8, 4, 512, 128, 512, 128), (1, 4, 512, 128, 64, 128), (8, 1, 512, 128, 512, 8)):
        q, k = _lib.SageView(65536, n, h, 128, st, sh), _lib.SageView(4096, n, 4, 128, 512, 128)
        assert L.sage_paged_append(BY(q), BY(k), BY(k), None, None, None, None, 0, None, 1e-6, BY(kv), BY(none), 65536, ost,
                                   osh, 4096, None) == 0
