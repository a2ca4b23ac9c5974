"""The paged K/V cache on the GPU: appending new tokens and attention over the cache, against the
definitions in 64 bits (tests/paged_ref.py, where the error bounds are derived)."""
import math

import pytest
import torch

import paged_ref
import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _handles(p):
    return sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale), sage.PagedBatch(p.cu_q, p.kv_len, p.table)


def _bits(t):
    return t.contiguous().view(torch.uint8 if t.dtype == torch.float8_e4m3fn else torch.int16)


# ----------------------------------------------------------------------------------------- append
APPEND = [
    # q_lens, kv_lens, hq, hkv, d, page, fmt, layout
    ([1], [1], 1, 1, 64, 8, "bf16", "nhd"),
    ([1] * 9, [1, 5, 16, 17, 300, 31, 32, 33, 64], 32, 8, 128, 16, "bf16", "nhd"),
    ([3, 0, 70, 1, 0], [3, 9, 200, 257, 0], 6, 2, 128, 32, "bf16", "hnd"),
    ([40, 33], [40, 133], 24, 24, 64, 64, "bf16", "kv"),
    ([5, 0, 129], [12, 4, 129], 7, 1, 64, 256, "e4m3", "nhd"),
    ([2, 19, 1], [100, 19, 64], 8, 4, 128, 8, "e4m3", "hnd"),
    ([1] * 70, list(range(1, 71)), 4, 2, 128, 1024, "e4m3", "kv"),
]


def _append_ref(p, gq, gk, cos, sin, rows=None):
    """(row, sequence, position, page, slot) of the placed tokens, and q, k, v in 64 bits."""
    placed = [(t, b, pos, int(p.table[b, pos // p.page]), pos % p.page)
              for t, b, pos in p.token_positions() if pos >= 0]
    idx = torch.tensor([x[0] for x in placed], device=p.dev)
    at = torch.tensor([x[2] if rows is None else rows[x[0]] for x in placed], device=p.dev)
    c, s = (None, None) if cos is None else (cos[at], sin[at])
    return (placed, idx, paged_ref.transform(p.q[idx], gq, c, s, EPS), paged_ref.transform(p.k[idx], gk, c, s, EPS),
            p.v[idx].double())


def _check_stored(p, pages, scale, placed, want, before, exact):
    got = torch.stack([pages[x[3], x[4]].double() for x in placed])
    if scale is None:
        # one rounding to bf16 (2^-8) of an fp32 value a few 2^-24 of the row's largest part off
        lim = torch.zeros_like(want) if exact else want.abs() * 2.0 ** -8 + 1e-6 * want.abs().amax(-1, keepdim=True)
    else:
        want = want / scale.double()[:, None]
        want = want.clamp(-448, 448)
        # one rounding to E4M3: 2^-4 of a normal value, half a step (2^-10) of a subnormal one
        lim = want.abs() * 2.0 ** -4 + 2.0 ** -10 + 1e-6 * want.abs().amax(-1, keepdim=True)
    assert ((got - want).abs() <= lim).all(), float(((got - want).abs() - lim).max())
    # every other slot as it was, bit for bit
    kept = torch.ones(pages.shape[:2], dtype=torch.bool, device=pages.device)
    for x in placed:
        kept[x[3], x[4]] = False
    assert torch.equal(_bits(pages)[kept], before[kept])


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[0])}x{c[2]}-{c[3]}-{c[4]}-{c[5]}-{c[6]}-{c[7]}")
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False), (False, False)])
def test_append(case, norm, rope):
    q_lens, kv_lens, hq, hkv, d, page, fmt, layout = case
    p = Problem(q_lens, kv_lens, hq, hkv, d, page, fmt, layout, seed=len(q_lens) + d, pad_rows=3)
    cache, batch = _handles(p)
    gq, gk = (p.gamma_q, p.gamma_k) if norm else (None, None)
    cos, sin = (p.cos, p.sin) if rope else (None, None)
    kb, vb = _bits(p.k_pages).clone(), _bits(p.v_pages).clone()
    q_out = torch.full((p.rows, hq, d), -7.0, dtype=torch.bfloat16, device=p.dev)
    assert sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, gamma_q=gq, gamma_k=gk, rope_cos=cos, rope_sin=sin,
                                  eps=EPS, q_out=q_out) is q_out
    assert sage.sage_check_device_status(cache.status) == (0, 0)
    placed, idx, q, k, v = _append_ref(p, gq, gk, cos, sin)
    lim = q.abs() * 2.0 ** -8 + 1e-6 * q.abs().amax(-1, keepdim=True)
    assert ((q_out[idx].double() - q).abs() <= lim).all()
    assert bool((q_out[p.n:] == -7.0).all())                    # rows behind the last sequence
    _check_stored(p, p.k_pages, p.k_scale, placed, k, kb, not norm and not rope)
    _check_stored(p, p.v_pages, p.v_scale, placed, v, vb, True)


def test_append_gives_the_bits_of_the_in_place_stage():
    """Norm and rotation as sage_qk_rmsnorm_rope does them, here with the table rows given."""
    p = Problem([37, 5], [37, 105], 6, 6, 128, 32, seed=4)
    cache, batch = _handles(p)
    gen = torch.Generator("cpu").manual_seed(1)
    rows = torch.randint(0, 105, (p.n,), generator=gen, dtype=torch.int32).to(p.dev)
    q_out = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, gamma_q=p.gamma_q, gamma_k=p.gamma_k,
                                   rope_cos=p.cos, rope_sin=p.sin, positions=rows, eps=EPS)
    q, k = p.q.clone(), p.k.clone()
    sage.sage_qk_rmsnorm_rope(q, k, p.gamma_q, p.gamma_k, p.cos[rows.long()].contiguous(),
                              p.sin[rows.long()].contiguous(), EPS)
    assert torch.equal(_bits(q_out), _bits(q))
    for t, b, pos in p.token_positions():
        pg = int(p.table[b, pos // p.page])
        assert torch.equal(p.k_pages[pg, pos % p.page], k[t])
        assert torch.equal(p.v_pages[pg, pos % p.page], p.v[t])


def test_append_q_in_place_and_without_q():
    p = Problem([6, 2], [6, 20], 4, 2, 64, 16, seed=5)
    cache, batch = _handles(p)
    want = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, gamma_q=p.gamma_q, gamma_k=p.gamma_k, rope_cos=p.cos,
                                  rope_sin=p.sin)
    kp, vp = p.k_pages.clone(), p.v_pages.clone()
    p.k_pages.zero_(), p.v_pages.zero_()
    assert sage.sage_paged_append(p.k, p.v, cache, batch, gamma_k=p.gamma_k, rope_cos=p.cos, rope_sin=p.sin) is None
    for t, b, pos in p.token_positions():
        pg = int(p.table[b, pos // p.page])
        assert torch.equal(p.k_pages[pg, pos % 16], kp[pg, pos % 16]) and torch.equal(p.v_pages[pg, pos % 16], vp[pg, pos % 16])
    sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, gamma_q=p.gamma_q, gamma_k=p.gamma_k, rope_cos=p.cos,
                           rope_sin=p.sin, q_out=p.q)
    assert torch.equal(p.q, want)


def test_append_left_padding():
    """Fewer tokens in the cache than rows: the first rows are padding, not stored, their q_out 0."""
    p = Problem([7, 4], [3, 0], 4, 2, 64, 8, seed=6)
    cache, batch = _handles(p)
    vb = _bits(p.v_pages).clone()
    q_out = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, rope_cos=p.cos, rope_sin=p.sin)
    assert sage.sage_check_device_status(cache.status) == (0, 0)
    placed, idx, q, k, v = _append_ref(p, None, None, p.cos, p.sin)
    assert [x[0] for x in placed] == [4, 5, 6]
    _check_stored(p, p.v_pages, None, placed, v, vb, True)
    assert not q_out[:4].any() and not q_out[7:].any() and q_out[4:7].any()


@pytest.mark.parametrize("what,where", [("page", 16), ("negative page", 16), ("length", 17), ("table row", 18)])
def test_append_bad_index_is_recorded_not_followed(what, where):
    p = Problem([2, 3, 2], [9, 11, 16], 2, 2, 64, 8, seed=7, extra_width=0)
    cache, batch = _handles(p)
    bad = {2, 3, 4}
    rows = None
    if what == "page":
        p.table[1, 1] = p.n_pages
    elif what == "negative page":
        p.table[1, 1] = -1
    elif what == "length":      # two pages of 8: positions 15 and up have no entry from the third token on
        p.kv_len[1] = 18        # positions 15, 16, 17
        bad = {3, 4}
    else:
        rows = torch.zeros(p.n, dtype=torch.int32, device=p.dev)
        rows[2:5] = p.cos.shape[0]
    if what == "length":
        p.table[1, 1] = 0 if int(p.table[1, 1]) < 0 else p.table[1, 1]
    kb = _bits(p.k_pages).clone()
    q_out = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, rope_cos=p.cos, rope_sin=p.sin, positions=rows) \
        if what != "length" else sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q)
    assert sage.sage_check_device_status(cache.status) == (1, where)
    assert sage.sage_check_device_status(cache.status) == (0, 0)          # read once, cleared
    kv = p.kv_len.tolist()
    stored = set()
    t = 0
    for b, n in enumerate(p.q_lens):
        for j in range(n):
            pos = kv[b] - n + j
            if t in bad:
                assert not q_out[t].any()
            else:
                assert q_out[t].any()
                stored.add((int(p.table[b, pos // 8]), pos % 8))
            t += 1
    changed = (_bits(p.k_pages) != kb).flatten(2).any(-1)
    assert {tuple(x) for x in changed.nonzero().tolist()} <= stored and len(stored) == 7 - len(bad)
    assert changed.sum() >= len(stored) - 1


def test_append_special_values_into_an_8_bit_cache():
    """Infinities saturate, NaN stays NaN, the largest code is 448, zeros keep their sign."""
    p = Problem([1, 1], [1, 1], 2, 2, 64, 8, "e4m3", seed=31)
    cache, batch = _handles(p)
    v = p.v.clone()
    s = p.v_scale.double()
    v[0, 0, :6] = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 1e30], dtype=torch.bfloat16)
    sage.sage_paged_append(p.k, v, cache, batch)
    got = p.v_pages[int(p.table[0, 0]), 0, 0]
    assert got[:2].double().tolist() == [448.0, -448.0] and bool(got[2].double().isnan())
    assert got.view(torch.uint8)[3:6].tolist() == [0x00, 0x80, 0x7E]
    want = (v[0, 0, 6:].double() / s[0]).clamp(-448, 448)
    assert ((got[6:].double() - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -10).all()


def test_append_nothing():
    p = Problem([0, 0], [0, 5], 2, 2, 64, 8, seed=8)
    cache, batch = _handles(p)
    before = _bits(p.k_pages).clone()
    q_out = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q)
    assert tuple(q_out.shape) == (0, 2, 64)
    none = sage.PagedBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), p.kv_len[:0], p.table[:0])
    p2 = Problem([2], [2], 2, 2, 64, 8, seed=8)
    sage.sage_paged_append(p2.k, p2.v, cache, none, q=p2.q)
    torch.cuda.synchronize()
    assert torch.equal(_bits(p.k_pages), before)


# ----------------------------------------------------------------------------------------- attention
ATTN = [
    # q_lens, kv_lens, hq, hkv, d, page, fmt, layout, causal, window
    ([1], [1], 1, 1, 64, 8, "bf16", "nhd", True, 0),
    ([1], [1], 8, 1, 128, 16, "e4m3", "nhd", False, 0),
    ([1, 1, 1, 1], [1, 63, 64, 65], 8, 2, 128, 16, "bf16", "nhd", True, 0),
    ([1] * 5, [127, 128, 129, 1000, 3], 32, 8, 128, 64, "bf16", "hnd", True, 0),
    ([1] * 40, [7 * i + 1 for i in range(40)], 4, 4, 64, 32, "bf16", "kv", True, 0),
    ([1, 0, 1], [5000, 17, 0], 7, 1, 128, 256, "bf16", "nhd", True, 0),
    ([1, 1], [3001, 777], 16, 2, 128, 8, "e4m3", "nhd", True, 0),
    ([1, 1, 1], [255, 256, 1025], 12, 12, 64, 1024, "e4m3", "hnd", True, 0),
    ([4, 5, 7], [300, 5, 133], 8, 4, 64, 16, "bf16", "nhd", True, 0),
    ([3, 4], [1111, 64], 24, 3, 128, 32, "bf16", "nhd", True, 0),
    ([8, 2], [500, 2], 16, 4, 64, 64, "e4m3", "kv", True, 0),
    ([3, 6], [700, 66], 5, 1, 128, 128, "e4m3", "nhd", True, 0),
    ([6, 1], [640, 90], 4, 2, 128, 16, "bf16", "nhd", False, 0),
    ([1, 1, 4], [900, 30, 333], 8, 2, 128, 16, "bf16", "nhd", True, 100),
    ([1, 3], [2000, 64], 4, 1, 64, 32, "e4m3", "nhd", True, 1),
    ([9, 3], [4, 3], 4, 2, 64, 8, "bf16", "nhd", True, 0),            # left padding
    ([9, 3], [4, 0], 4, 2, 128, 8, "e4m3", "nhd", True, 2),
    ([5, 2], [3, 0], 4, 2, 64, 8, "bf16", "nhd", False, 0),
    ([65], [2003], 8, 2, 128, 64, "bf16", "nhd", True, 0),
    ([130, 17], [130, 400], 6, 3, 64, 32, "bf16", "kv", True, 0),
    ([200, 1, 0, 77], [1300, 900, 3, 77], 7, 1, 128, 16, "bf16", "hnd", True, 0),
    ([150, 40], [700, 41], 10, 2, 128, 16, "bf16", "nhd", True, 130),
    ([257], [600], 3, 3, 128, 128, "bf16", "nhd", False, 0),
    ([190, 90], [800, 90], 8, 2, 128, 64, "e4m3", "nhd", True, 0),
    ([300], [1029], 5, 5, 64, 8, "e4m3", "hnd", False, 0),
    ([129, 300], [50, 300], 4, 2, 64, 16, "bf16", "nhd", True, 40),   # left padding in a long chunk
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"q{max(c[0])}-kv{max(c[1])}-{c[2]}-{c[3]}-{c[4]}-p{c[5]}-{c[6]}-{c[7]}-c{int(c[8])}-w{c[9]}")
def test_attention(case):
    q_lens, kv_lens, hq, hkv, d, page, fmt, layout, causal, window = case
    p = Problem(q_lens, kv_lens, hq, hkv, d, page, fmt, layout, seed=hq + sum(q_lens), pad_rows=2)
    cache, batch = _handles(p)
    out = torch.full((p.rows, hq, d), -7.0, dtype=torch.bfloat16, device=p.dev)
    lse = torch.full((p.rows, hq), -7.0, dtype=torch.float32, device=p.dev)
    ws = sage.paged_workspace(d)
    got = sage.sage_paged_attn(p.q, cache, batch, causal=causal, window=window, out=out, lse=lse, ws=ws)
    assert got is out
    assert sage.sage_check_device_status(ws) == (0, 0)
    ref = paged_ref.attention(p, p.q, causal, window)
    paged_ref.check_attention(p, out, ref)
    assert bool((out[p.n:] == -7.0).all()) and bool((lse[p.n:] == -7.0).all())
    # ln of the sum: score errors, and the rounded weights' 2^-8 (see attention_bound)
    empty = torch.isinf(ref[1])
    assert torch.equal(torch.isinf(lse[:p.n]), empty)
    lim = p.d * 2.0 ** -23 * ref[3] / math.sqrt(d) + 1.01 * 2.0 ** -8 + 1e-5 * (1 + ref[1].abs())
    assert ((lse[:p.n].double() - ref[1]).abs() <= lim)[~empty].all()
    assert not ws[256:sage._lib.PAGED_WS_HEADER].any()                    # the join counters are back at zero
    again = sage.sage_paged_attn(p.q, cache, batch, causal=causal, window=window, ws=ws)
    assert torch.equal(_bits(again[:p.n]), _bits(out[:p.n]))              # and the result does not vary


def test_attention_of_a_long_split_sequence():
    """One token over many pages: every SM takes a part, joined in the end."""
    p = Problem([1], [70001], 8, 2, 128, 256, seed=9)
    cache, batch = _handles(p)
    out = sage.sage_paged_attn(p.q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_of_a_long_ragged_batch(fmt):
    """Many key tiles and several units to each SM: the ring of stages goes round often, across units."""
    p = Problem([1] * 40, [700 + 61 * ((7 * i) % 40) for i in range(40)], 64, 8, 128, 64, fmt, seed=30)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(128)
    out = sage.sage_paged_attn(p.q, cache, batch, ws=ws)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))
    for _ in range(10):
        assert torch.equal(_bits(sage.sage_paged_attn(p.q, cache, batch, ws=ws)), _bits(out))
    assert sage.sage_check_device_status(ws) == (0, 0)


SPLIT = [
    # few units over many keys: the key axis of the many-row kernel is split and joined
    ([65], [9001], 8, 2, 128, 64, "bf16", True, 0),
    ([40], [7777], 8, 1, 128, 16, "e4m3", True, 0),
    ([300], [6000], 1, 1, 64, 32, "bf16", False, 0),
    ([129], [5000], 2, 2, 64, 8, "e4m3", True, 3000),
    ([128, 1], [8000, 70], 4, 2, 128, 256, "bf16", True, 2500),
]


@pytest.mark.parametrize("case", SPLIT, ids=lambda c: f"q{max(c[0])}-kv{max(c[1])}-{c[2]}-{c[3]}-{c[4]}-{c[6]}-w{c[8]}")
def test_attention_of_a_chunk_behind_a_long_context(case):
    q_lens, kv_lens, hq, hkv, d, page, fmt, causal, window = case
    p = Problem(q_lens, kv_lens, hq, hkv, d, page, fmt, seed=32 + hq)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(d)
    lse = torch.empty((p.n, hq), dtype=torch.float32, device="cuda")
    out = sage.sage_paged_attn(p.q, cache, batch, causal=causal, window=window, lse=lse, ws=ws)
    ref = paged_ref.attention(p, p.q, causal, window)
    paged_ref.check_attention(p, out, ref)
    lim = p.d * 2.0 ** -23 * ref[3] / math.sqrt(d) + 1.01 * 2.0 ** -8 + 1e-5 * (1 + ref[1].abs())
    assert ((lse.double() - ref[1]).abs() <= lim).all()
    assert torch.equal(_bits(sage.sage_paged_attn(p.q, cache, batch, causal=causal, window=window, ws=ws)), _bits(out))
    assert sage.sage_check_device_status(ws) == (0, 0)


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("e4m3", 64)])
def test_attention_of_many_sequences_of_mixed_lengths(fmt, d):
    """More sequences than a warp has lanes, prompts among single tokens and empty ones."""
    q_lens = [(1, 0, 90, 3, 260)[i % 5] for i in range(45)]
    kv_lens = [n + (37 * i) % 500 if n else 0 for i, n in enumerate(q_lens)]
    p = Problem(q_lens, kv_lens, 4, 2, d, 16, fmt, seed=33)
    cache, batch = _handles(p)
    out = sage.sage_paged_attn(p.q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_more_chunks_than_sms(fmt, d):
    """Several units to each SM, drawn as they end: of one row tile and of two, long and short, windows that begin
    behind the first page; whichever SM takes which, the result is the same, and the next call starts anew."""
    q_lens = [(70, 1, 0, 300, 33, 129, 256)[i % 7] for i in range(42)]
    kv_lens = [q + (0, 1500, 3, 640, 127)[i % 5] for i, q in enumerate(q_lens)]
    p = Problem(q_lens, kv_lens, 16, 8, d, 64, fmt, seed=50 + d)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(d)
    for window in (0, 200):
        out = sage.sage_paged_attn(p.q, cache, batch, window=window, ws=ws)
        paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True, window))
        for _ in range(8):
            assert torch.equal(_bits(sage.sage_paged_attn(p.q, cache, batch, window=window, ws=ws)[:p.n]), _bits(out[:p.n]))
    assert sage.sage_check_device_status(ws) == (0, 0)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_of_rows_of_very_different_size(q_len, fmt):
    """Query rows scaled by 2^-90 .. 2^10, and the scores' scale with them: relative accuracy is kept."""
    p = Problem([q_len], [400], 4, 2, 64, 16, fmt, seed=34)
    cache, batch = _handles(p)
    for shift in (-90, 10):
        q = (p.q.float() * 2.0 ** shift).to(torch.bfloat16)
        sm = 2.0 ** -shift / 8
        out = sage.sage_paged_attn(q, cache, batch, sm_scale=sm)
        paged_ref.check_attention(p, out, paged_ref.attention(p, q, True, sm_scale=sm), sm_scale=sm)
    q = p.q.contiguous().clone()
    q[:, 1] = 0                       # a head of zeros: uniform weights
    out = sage.sage_paged_attn(q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, q, True))


def test_attention_of_an_expanded_query():
    """One query row for all heads (stride 0)."""
    p = Problem([3, 60], [50, 200], 6, 2, 128, 16, seed=35)
    cache, batch = _handles(p)
    q = p.q[:, :1].expand(-1, 6, -1)
    out = sage.sage_paged_attn(q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, q, True))


def test_attention_shared_prefix_and_strided_views():
    """Sequences with a page in common; q a slice of the projection buffer, out a slice of a wider one."""
    p = Problem([3, 2, 4], [40, 70, 20], 6, 2, 64, 16, seed=10, share_first_page=True)
    cache, batch = _handles(p)
    wide = torch.full((p.n, 2 * 6 * 64), -7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 6 * 64:].view(p.n, 6, 64)
    sage.sage_paged_attn(p.q, cache, batch, sm_scale=0.3, out=out)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True, sm_scale=0.3), sm_scale=0.3)
    assert bool((wide[:, :6 * 64] == -7.0).all())


@pytest.mark.parametrize("q_len", [1, 150])
def test_attention_pages_before_the_window_may_be_gone(q_len):
    """Entries of pages that no key in the window lies on are not read; one that is read and out of range
    hides its keys and is recorded."""
    p = Problem([q_len], [900], 4, 2, 128, 16, seed=11)
    cache, batch = _handles(p)
    ref = paged_ref.attention(p, p.q, True, 200)
    first = (900 - q_len + 1 - 200) // 16
    p.table[0, :first] = -1
    ws = sage.paged_workspace(128)
    out = sage.sage_paged_attn(p.q, cache, batch, window=200, ws=ws)
    assert sage.sage_check_device_status(ws) == (0, 0)
    paged_ref.check_attention(p, out, ref)
    keep = int(p.table[0, first + 4])
    p.table[0, first + 4] = p.n_pages
    out = sage.sage_paged_attn(p.q, cache, batch, window=200, ws=ws)
    assert sage.sage_check_device_status(ws) == (1, 16)
    p.table[0, first + 4] = keep
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True, 200, hide_pages=[(0, first + 4)]))


def test_attention_length_above_the_table_is_cut_and_recorded():
    p = Problem([1], [48], 2, 2, 64, 16, seed=12, extra_width=0)
    cache, batch = _handles(p)
    ref = paged_ref.attention(p, p.q, True)
    p.kv_len[0] = 500
    ws = sage.paged_workspace(64)
    out = sage.sage_paged_attn(p.q, cache, batch, ws=ws)
    assert sage.sage_check_device_status(ws) == (1, 17)
    paged_ref.check_attention(p, out, ref)


def test_attention_large_scores_and_equal_keys():
    """Scores of some hundreds (the running maximum rises often) and all keys alike (uniform weights)."""
    p = Problem([2, 40], [600, 333], 4, 2, 128, 32, seed=13)
    p.q.mul_(16)
    cache, batch = _handles(p)
    out = sage.sage_paged_attn(p.q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))
    p.k_pages[p.used] = p.k_pages[p.used][0].clone()
    out = sage.sage_paged_attn(p.q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))


def test_attention_over_offsets_past_32_bits():
    """A cache of more than 2^32 bytes a side, its pages at both ends in use."""
    n_pages, page, d = (1 << 32) // (256 * 8 * 128 * 2) + 40, 256, 128
    k = torch.empty((n_pages, page, 8, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    p = Problem([1, 3], [600, 300], 16, 8, d, page, seed=14)
    far = {int(x): n_pages - 1 - 3 * i for i, x in enumerate(sorted({int(x) for x in p.table.flatten() if x >= 0}))}
    table = p.table.clone()
    for old, new in far.items():
        k[new], v[new] = p.k_pages[old], p.v_pages[old]
        table[p.table == old] = new
    cache, batch = sage.PagedKV(k, v), sage.PagedBatch(p.cu_q, p.kv_len, table)
    out = sage.sage_paged_attn(p.q, cache, batch)
    paged_ref.check_attention(p, out, paged_ref.attention(p, p.q, True))
    # and appended to there
    sage.sage_paged_append(p.k, p.v, cache, batch)
    for t, b, pos in p.token_positions():
        assert torch.equal(k[int(table[b, pos // page]), pos % page], p.k[t])


# ----------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("e4m3", 64)])
def test_generation_in_pieces(fmt, d):
    """A prompt, a chunk and single tokens of two sequences, appended and attended step by step: each
    step's attention against the cache's own contents, and the cache against all tokens at once."""
    hq, hkv, page = 6, 2, 16
    steps = [(70, 41), (9, 150), (1, 1), (1, 1), (3, 0)]
    total = [sum(x[b] for x in steps) for b in range(2)]
    p = Problem([0, 0], total, hq, hkv, d, page, fmt, seed=15)
    cache = sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale)
    ws, kv = sage.paged_workspace(d), [0, 0]
    gen = torch.Generator("cpu").manual_seed(3)
    seen_k = [[], []]
    for step in steps:
        kv = [a + b for a, b in zip(kv, step)]
        s = Problem(list(step), kv, hq, hkv, d, page, fmt, seed=100 + kv[0])
        s.table, s.k_pages, s.v_pages, s.k_scale, s.v_scale = p.table, p.k_pages, p.v_pages, p.k_scale, p.v_scale
        batch = sage.PagedBatch(s.cu_q, s.kv_len, p.table)
        q = sage.sage_paged_append(s.k, s.v, cache, batch, q=s.q, gamma_q=p.gamma_q, gamma_k=p.gamma_k, rope_cos=p.cos,
                                   rope_sin=p.sin, eps=EPS)
        out = sage.sage_paged_attn(q, cache, batch, ws=ws)
        paged_ref.check_attention(s, out, paged_ref.attention(s, q, True))
        for t, b, pos in s.token_positions():
            at = torch.tensor([pos], device="cuda")
            seen_k[b].append(paged_ref.transform(s.k[t:t + 1], p.gamma_k, p.cos[at], p.sin[at], EPS)[0])
    for b in range(2):
        key = torch.arange(total[b], device="cuda")
        got = p.values(p.k_pages, p.k_scale)[p.table[b].long()[key // page], key % page]
        want = torch.stack(seen_k[b])
        step = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -4
        sub = 0.0 if fmt == "bf16" else 2.0 ** -10 * float(p.k_scale.max())
        if fmt == "e4m3":
            top = 448 * p.k_scale.double()[:, None]
            want = torch.minimum(torch.maximum(want, -top), top)
        assert ((got - want).abs() <= step * want.abs() + sub + 1e-6 * want.abs().amax(-1, keepdim=True)).all()
    assert sage.sage_check_device_status(ws) == (0, 0) and sage.sage_check_device_status(cache.status) == (0, 0)


def test_whole_sequence_equals_dense_attention():
    """All tokens appended at once and attended without a mask: the framework's dense attention on
    the same values, both within their bounds of the exact one."""
    p = Problem([333], [333], 4, 4, 128, 64, seed=16)
    cache, batch = _handles(p)
    sage.sage_paged_append(p.k, p.v, cache, batch)
    out = sage.sage_paged_attn(p.q, cache, batch, causal=False)
    dense = sage.sage_attn_dense_bf16(p.q, p.k, p.v)
    ref = paged_ref.attention(p, p.q, False)
    paged_ref.check_attention(p, out, ref)
    paged_ref.check_attention(p, dense, ref)


@pytest.mark.parametrize("q_len", [1, 40])
def test_graph_replay_after_lengths_changed(q_len):
    """One captured pair of calls, replayed with other lengths, pages and inputs; two graphs that share the
    workspace replayed one after the other."""
    hq, hkv, d, page = 8, 2, 128, 16
    a = Problem([q_len, q_len], [300, 140], hq, hkv, d, page, seed=17)
    b = Problem([q_len, q_len], [90, 299], hq, hkv, d, page, seed=18)
    cache, batch = _handles(a)
    ws = sage.paged_workspace(d)
    q = a.q.contiguous().clone()
    out = torch.zeros_like(q)
    sage.sage_paged_attn(q, cache, batch, out=out, ws=ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            sage.sage_paged_attn(q, cache, batch, out=out, ws=ws)
    want_a, want_b = paged_ref.attention(a, a.q, True), paged_ref.attention(b, b.q, True)
    for gr in graphs:
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        paged_ref.check_attention(a, out, want_a)
    n = min(a.n_pages, b.n_pages)
    used = sorted({int(x) for x in b.table.flatten() if x >= 0})
    assert len(used) <= a.n_pages
    move = {old: i for i, old in enumerate(used)}
    table = torch.full_like(a.table, 0)
    for r in range(2):
        for i in range(min(b.table.shape[1], a.table.shape[1])):
            if int(b.table[r, i]) >= 0:
                table[r, i] = move[int(b.table[r, i])]
    for old, new in move.items():
        a.k_pages[new], a.v_pages[new] = b.k_pages[old], b.v_pages[old]
    a.table.copy_(table), a.kv_len.copy_(b.kv_len), q.copy_(b.q)
    for gr in graphs + graphs:
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        paged_ref.check_attention(b, out, want_b)
    assert n > 0 and sage.sage_check_device_status(ws) == (0, 0)


def test_on_another_stream():
    p = Problem([1, 5], [400, 77], 8, 2, 128, 32, seed=19)
    cache, batch = _handles(p)
    ws = sage.paged_workspace(128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, rope_cos=p.cos, rope_sin=p.sin)
        out = sage.sage_paged_attn(q, cache, batch, ws=ws)
    side.synchronize()
    paged_ref.check_attention(p, out, paged_ref.attention(p, q, True))
    out2 = sage.sage_paged_attn(q, cache, batch, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, out2)


def test_buffers_that_a_call_makes_belong_to_its_stream():
    """Output, status block and workspace made by a call on a given stream, while the current stream is busy: zeroed
    before the kernel, and not given away before it is done."""
    p = Problem([1, 5, 60], [4000, 77, 900], 8, 2, 128, 32, seed=23)
    cache, batch = _handles(p)
    ref_q = sage.sage_paged_append(p.k, p.v, *_handles(p), q=p.q, rope_cos=p.cos, rope_sin=p.sin)
    want = sage.sage_paged_attn(ref_q, cache, batch).clone()
    busy = torch.randn((6000, 6000), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        cache, batch = _handles(p)
        for _ in range(8):
            busy = busy @ busy * 1e-4
        q = sage.sage_paged_append(p.k, p.v, cache, batch, q=p.q, rope_cos=p.cos, rope_sin=p.sin, stream=given)
        outs = [sage.sage_paged_attn(q, cache, batch, stream=given) for _ in range(3)]
        for _ in range(4):
            torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")   # what was freed on the current stream
        side.synchronize()
        assert sage.sage_check_device_status(cache.status, stream=side) == (0, 0)
        assert torch.equal(_bits(q), _bits(ref_q))
        assert all(torch.equal(_bits(o), _bits(want)) for o in outs)
    torch.cuda.synchronize()


def test_two_calls_at_once_on_their_own_workspaces():
    ps = [Problem([1], [20000 + 999 * i], 8, 2, 128, 64, seed=20 + i) for i in range(2)]
    hs = [_handles(p) for p in ps]
    wss = [sage.paged_workspace(128) for _ in ps]
    want = [sage.sage_paged_attn(p.q, *h, ws=w).clone() for p, h, w in zip(ps, hs, wss)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(sage.sage_paged_attn(ps[i].q, *hs[i], ws=wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_attention_nothing():
    p = Problem([0], [30], 2, 2, 64, 8, seed=21)
    cache, batch = _handles(p)
    assert tuple(sage.sage_paged_attn(p.q, cache, batch).shape) == (0, 2, 64)
    none = sage.PagedBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), p.kv_len[:0], p.table[:0])
    p2 = Problem([2], [2], 2, 2, 64, 8, seed=21)
    out = torch.full_like(p2.q, -7.0)
    sage.sage_paged_attn(p2.q, cache, none, out=out)
    torch.cuda.synchronize()
    assert bool((out == -7.0).all())
