"""Drafted trees over the paged cache on the GPU where their arithmetic could go wrong."""
import math

import pytest
import torch

import video_diffusion_transformer_sage_gb300 as sage

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("q_len", [3, 48, 200])                       # few rows, one row tile, two
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (128, 3, 3), (64, 8, 2), (64, 5, 5)])
@pytest.mark.parametrize("kind", ["normal", "outlier", "wide", "tiny", "huge"])
def test_scores_over_e4m3_keep_the_precision_of_the_plain_call(kind, d, hq, hkv, q_len):
    """Rows that see one key each, so that lse is the score.  "outlier": a channel 2^9 above the others whose K is zero, so that
    nothing of the row's largest value is in the score; "wide": channels over 24 powers of two; "tiny", "huge": the rows at the
    type's ends, with a channel of its largest value.

    What is allowed: fp32 sums of d products, d 2^-23 sum |q_c k_c|; q as fp16 times the row's power of two, half a step of whose
    subnormals is 2^-25 of the row's largest: 2^-25 max |q_c| sum |k_c|; and for lse itself, whose sum of one weight is
    2^7 by ex2 and back by log2 (2^-22 each), a few roundings of a number of |s| + 7: 2^-19 (2 + |s|)."""
    g = torch.Generator().manual_seed(d + q_len)
    page = 16
    n_pages = (q_len + page - 1) // page
    k = torch.randn((n_pages, page, hkv, d), generator=g) * 60
    q = torch.randn((q_len, hq, d), generator=g)
    if kind == "outlier":
        q[:, :, 5], k[..., 5] = 600.0, 0.0
    elif kind == "wide":
        q = torch.sign(q) * torch.exp2(-24 * torch.rand(q.shape, generator=g))
    elif kind == "tiny":
        q = q * 2.0 ** -118
    elif kind == "huge":
        q, k[..., 3] = q * 2.0 ** 120, 0.0
        q[:, :, 3] = torch.finfo(torch.bfloat16).max
    q, k = q.to(torch.bfloat16).cuda(), k.to(torch.float8_e4m3fn).cuda()
    v = torch.randn((n_pages, page, hkv, d), generator=g).to(torch.float8_e4m3fn).cuda()
    k_scale = torch.full((hkv,), 2.0 ** -6, device="cuda")
    cache = sage.PagedKV(k, v, k_scale, torch.ones(hkv, device="cuda"))
    batch = sage.PagedBatch(_i32([0, q_len]), _i32([q_len]), _i32([list(range(n_pages))]))
    bits = torch.zeros((q_len, (q_len + 31) // 32), dtype=torch.int64)
    for t in range(q_len):
        bits[t, t // 32] = 1 << (t % 32)
    tree = sage.PagedTree(torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).cuda())
    kd = k.view(-1, hkv, d)[:q_len].double().repeat_interleave(hq // hkv, 1) * 2.0 ** -6
    sm = {"tiny": 2.0 ** 118, "huge": 2.0 ** -120}.get(kind, 1.0) / math.sqrt(d)
    s = (q.double() * kd).sum(-1) * sm
    lim = d * 2.0 ** -23 * (q.double() * kd).abs().sum(-1) * sm
    lim += 2.0 ** -25 * q.double().abs().amax(-1) * kd.abs().sum(-1) * sm + 2.0 ** -19 * (2 + s.abs())
    lse, plain = (torch.zeros((q_len, hq), device="cuda") for _ in range(2))
    out = sage.sage_paged_attn_tree(q, cache, batch, tree, sm_scale=sm, lse=lse)
    assert bool(((lse.double() - s).abs() <= lim).all()), float(((lse.double() - s).abs() - lim).max())
    vd = v.view(-1, hkv, d)[:q_len].repeat_interleave(hq // hkv, 1)
    assert torch.equal(out.float(), vd.float())                       # one weight: V itself
    sage.sage_paged_attn(q, cache, batch, sm_scale=sm, window=1, lse=plain)
    assert bool(((plain.double() - s).abs() <= lim).all())


@pytest.mark.parametrize("kv_len,first", [(-2 ** 31, 0), (-2 ** 31 + 1, 0), (-1, 0), (2, 0), (300, 0), (301, 1), (2 ** 31 - 1, 2 ** 31 - 301)])
@pytest.mark.parametrize("window", [0, 2])
def test_positions_of_lengths_at_the_types_ends(kv_len, first, window):
    """A tree of 300 tokens, all children of the first: positions are max(0, kv_len - 300) + depth, whatever the length; small
    trees beside it."""
    status = sage.status_block()
    batch = sage.PagedBatch(_i32([0, 300, 303]), _i32([kv_len, kv_len]), _i32([[0], [0]]))
    parents = [-1] + [0] * 299 + [-1, -1, -1]
    tree = sage.sage_paged_tree(_i32(parents), batch, status=status, words=10, window=window)
    assert tree.depth.tolist() == [0] + [1] * 299 + [0] * 3
    second = max(0, kv_len - 3)
    assert tree.positions.tolist() == [first] + [first + 1] * 299 + [second] * 3
    assert sage.sage_check_device_status(status) == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_what_is_no_number_in_a_query_row_over_e4m3(value, d):
    """The kernel for many rows: such a row is NaN, the others as without it."""
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn((6, 16, 2, d), generator=g).to(torch.float8_e4m3fn).cuda() for _ in range(2))
    one = torch.ones(2, device="cuda")
    cache = sage.PagedKV(k, v, one, one)
    batch = sage.PagedBatch(_i32([0, 70]), _i32([90]), _i32([list(range(6))]))
    tree = sage.sage_paged_tree(_i32([-1] + [(j - 1) // 2 for j in range(1, 70)]), batch, status=cache.status, words=3)
    q = torch.randn((70, 2, d), generator=g).to(torch.bfloat16).cuda()
    want = sage.sage_paged_attn_tree(q, cache, batch, tree)
    q[33, 1, 7] = value
    lse = torch.zeros((70, 2), device="cuda")
    out = sage.sage_paged_attn_tree(q, cache, batch, tree, lse=lse)
    assert bool(out[33, 1].isnan().all()) and bool(lse[33, 1].isnan())
    out[33, 1], lse[33, 1] = want[33, 1], 0
    assert torch.equal(out, want) and bool(torch.isfinite(lse).all())
