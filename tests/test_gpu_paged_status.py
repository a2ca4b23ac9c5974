"""The status blocks that the handles of the paged cache make when they are first needed, whatever other streams do."""
import pytest
import torch

import video_diffusion_transformer_sage_gb300 as sage
from video_diffusion_transformer_sage_gb300 import _lib

pytestmark = pytest.mark.gpu

STREAMS = 40   # torch gives the same 32 streams out again and again


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache():
    pages = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    pages[0] = 1.0
    return sage.PagedKV(pages, pages.clone())


def test_the_stream_of_the_blocks_is_nobody_elses():
    cache = _cache()
    assert not cache.status.any()
    own = _lib._side_stream(0).cuda_stream
    for priority in (0, -1):
        assert own not in {torch.cuda.Stream(priority=priority).cuda_stream for _ in range(2 * STREAMS)}
    assert own != torch.cuda.default_stream().cuda_stream


def test_a_handles_first_call_in_a_capture_on_every_stream():
    """A cache's and a pool's first calls are captured, on each of torch's streams: the capture ends well, the blocks are zeros
    before any replay, and replays do not erase what was recorded."""
    warm, src, dst = _cache(), _i32([0]), _i32([1])
    sage.sage_paged_copy(warm, src, dst)
    sage.sage_paged_release(sage.PagedPool(_i32([1, 0]), _i32([[0, -1]]), 16), _i32([16]))
    for _ in range(STREAMS):
        cache, refs = _cache(), _i32([1, 0, 0, 2])
        pool, hi, stream, graph = sage.PagedPool(refs, _i32([[0, 3]]), 16), _i32([16]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            sage.sage_paged_copy(cache, src, dst)
            sage.sage_paged_release(pool, hi)
        assert sage.sage_check_device_status(cache.status) == sage.sage_check_device_status(pool.status) == (0, 0)
        sage.sage_paged_copy(cache, _i32([9]), dst)
        graph.replay()
        torch.cuda.synchronize()
        assert sage.sage_check_device_status(cache.status) == (1, 16)
        assert bool((cache.k_pages[1] == 1).all()) and refs.tolist() == [1, 0, 0, 1]
