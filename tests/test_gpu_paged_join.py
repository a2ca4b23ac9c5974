"""Few query rows over the paged cache where one sequence's key tiles lie in more than 16 CTAs among other sequences':
its parts are joined in groups, beside units that begin where it ends."""
import math

import pytest
import torch

import paged_ref
import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu


def _lens(short, n, longs):
    """n sequences of `short` keys (a little more for some), with longs {index: keys} among them."""
    kv = [short + 3 * (i % 5) for i in range(n)]
    for at, keys in sorted(longs.items()):
        kv.insert(at, keys)
    return kv


# On 152 SMs these leave a last group of one part to groups of about the square root of 21, 31 or 43 parts, or
# have two such units next to each other; on any number of SMs they are long units among short ones.
CASES = [
    # keys, hq, hkv, d, page, fmt
    (_lens(1000, 63, {20: 70000}), 8, 4, 128, 64, "bf16"),
    (_lens(1000, 200, {0: 32032}), 1, 1, 128, 64, "bf16"),
    (_lens(1000, 200, {0: 33312}), 2, 1, 128, 128, "bf16"),
    (_lens(500, 160, {70: 30000}), 2, 2, 64, 32, "bf16"),
    (_lens(900, 170, {10: 60000, 12: 40000}), 3, 1, 128, 16, "bf16"),
    (_lens(1000, 180, {33: 50000, 90: 64000}), 4, 1, 128, 64, "e4m3"),
    (_lens(1500, 170, {5: 90000}), 1, 1, 64, 256, "e4m3"),
]


def _run(kv, hq, hkv, d, page, fmt, q_lens, seed):
    p = Problem(q_lens, kv, hq, hkv, d, page, fmt, seed=seed)
    cache, batch = sage.PagedKV(p.k_pages, p.v_pages, p.k_scale, p.v_scale), sage.PagedBatch(p.cu_q, p.kv_len, p.table)
    ws = sage.paged_workspace(d)
    ref = paged_ref.attention(p, p.q, True)
    lim = p.d * 2.0 ** -23 * ref[3] / math.sqrt(d) + 1.01 * 2.0 ** -8 + 1e-5 * (1 + ref[1].abs())
    first = None
    for _ in range(4):      # on one workspace: each call leaves it as it was
        out = torch.full((p.n, hq, d), float("nan"), dtype=torch.bfloat16, device=p.dev)
        lse = torch.full((p.n, hq), float("nan"), dtype=torch.float32, device=p.dev)
        sage.sage_paged_attn(p.q, cache, batch, out=out, lse=lse, ws=ws)
        paged_ref.check_attention(p, out, ref)
        assert bool(((lse.double() - ref[1]).abs() <= lim).all())
        assert not ws[256:sage._lib.PAGED_WS_HEADER].any()
        assert first is None or torch.equal(out, first)
        first = out
    assert sage.sage_check_device_status(ws) == (0, 0)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}seqs-max{max(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[5]}")
def test_one_long_sequence_among_many(case):
    kv, hq, hkv, d, page, fmt = case
    _run(kv, hq, hkv, d, page, fmt, [1] * len(kv), seed=len(kv))


@pytest.mark.parametrize("parts", range(17, 46, 2))
def test_every_odd_number_of_parts(parts):
    """The long unit about `parts` CTAs' share long, whatever the share is: one K/V head, 200 short sequences behind it."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    short, n = 16, 200                                   # tiles of 64 keys
    tiles = round(parts * short * n / (sms - parts))     # tiles / share = parts, share = (tiles + n short) / sms
    _run([tiles * 64 - 7] + [short * 64] * n, 1, 1, 128, 64, "bf16", [1] * (n + 1), seed=parts)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_prompt_among_single_tokens(fmt):
    """A mean of at most 32 rows with one sequence of many row tiles: units of one sequence in the hundreds."""
    q_lens = [1] * 70
    q_lens[31] = 150
    kv = [40 + 11 * i for i in range(70)]
    kv[31] = 3000
    _run(kv, 16, 2, 128, 32, fmt, q_lens, seed=8)
