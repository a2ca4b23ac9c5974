"""Trees of drafted tokens and attention of them over a paged cache, in 64 bits, from the definitions alone."""
import math
import random

import torch

import paged_ref
from paged_ref import Problem


def parents_of(q_lens, seed, bushy=3):
    """A forest for each sequence: token i's parent is one of the last few before it, or -1."""
    r, out = random.Random(seed), []
    for n in q_lens:
        b = r.randint(1, bushy)
        out += [min(j - 1, r.randint(max(-1, j // b - 3), max(0, j // b))) for j in range(n)]
    return out


def closure(q_lens, parents, window=0):
    """(who sees whom [n][n] for each sequence, depth of every row) from the parents."""
    seen, depth, at = [], [], 0
    for n in q_lens:
        m = torch.zeros((n, n), dtype=torch.bool)
        for t in range(n):
            i, d = t, 0
            while i >= 0:
                if not window or d < window:
                    m[t, i] = True
                i, d = parents[at + i], d + 1
            depth.append(d - 1)
        seen.append(m)
        at += n
    return seen, depth


def packed(seen, words, rows, fill=0):
    """The mask words [rows, words] of who sees whom; rows of no sequence keep `fill`."""
    out, at = torch.full((rows, words), fill, dtype=torch.int64), 0
    for m in seen:
        n = m.shape[0]
        wide = torch.zeros((n, max(words * 32, n)), dtype=torch.int64)
        wide[:, :n] = m
        out[at:at + n] = (wide[:, :words * 32].view(n, words, 32) << torch.arange(32)).sum(-1)
        at += n
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def score_slack(p: Problem, q, ref, sm_scale=None):
    """What the bounds of paged_ref.attention_bound grow by with an E4M3 cache and many rows, relative on a weight, [n, hq].

    There the kernel holds q as the sum of two E4M3 values times a power of two, the row's largest in [2^7, 2^8): the first is at
    most 2^-4 of the value off, the second represents that difference but for half a step of E4M3's smallest, 2^-10.  So a
    channel is at most 2^-10 off where the row's largest is at least 2^7: 2^-17 of it, and a score at most
    2^-17 max_c |q_c| sum_c |k_c| sm; a weight is a ratio of two exponentials: twice that."""
    if p.fmt != "e4m3":
        return torch.zeros_like(ref[1])
    sm = 1 / math.sqrt(p.d) if sm_scale is None else sm_scale
    k = torch.nan_to_num(p.values(p.k_pages, p.k_scale).abs()).sum(-1).amax((0, 1))        # [hkv], over all stored keys
    return 2 * 2.0 ** -17 * q[:p.n].double().abs().amax(-1) * k.repeat_interleave(p.hq // p.hkv) * sm


def check_attention(p: Problem, got, ref, q, sm_scale=None):
    off = (got[:p.n].double() - ref[0]).abs() - paged_ref.attention_bound(p, ref, sm_scale)
    off -= score_slack(p, q, ref, sm_scale)[..., None] * ref[2]
    assert torch.isfinite(got[:p.n].float()).all()
    assert float(off.max()) <= 0.0, (float(off.max()), [int(i) for i in torch.nonzero(off == off.max())[0]])


def attention(p: Problem, q, seen, depth=None, window=0, sm_scale=None):
    """As paged_ref.attention: (out, lse, sum_j w_j |v_j|, largest sum_c |q_c k_jc|)."""
    d, group = p.d, p.hq // p.hkv
    sm = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    kp, vp = p.values(p.k_pages, p.k_scale), p.values(p.v_pages, p.v_scale)
    dev = p.dev
    out = torch.zeros((p.n, p.hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((p.n, p.hq), -math.inf, dtype=torch.float64, device=dev)
    wv, unit = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, (n, kv) in enumerate(zip(p.q_lens, p.kv_lens)):
        if n == 0 or kv <= 0:
            t += n
            continue
        key = torch.arange(kv, device=dev)
        page = p.table[b].long()[key // p.page]
        prefix = kv - n
        see = (key < prefix).expand(n, kv).clone()
        if window:
            dep = torch.tensor(depth[t:t + n], device=dev)[:, None].clamp(0, n - 1)
            see &= key > prefix + dep - window
        new = seen[b].to(dev)
        see[:, max(prefix, 0):] |= new[:, max(prefix, 0) - prefix:]
        # what no row sees may hold anything
        used = see.any(0)
        page = torch.where(used, page, page[used][:1] if used.any() else page[:1])
        k, v = (torch.where(used[:, None, None], x[page, key % p.page], 0.0) for x in (kp, vp))
        some = see.any(-1)
        rows = torch.nonzero(some).squeeze(-1) + t
        for h in range(p.hq):
            kh, vh, qh = k[:, h // group], v[:, h // group], q[t:t + n, h].double()
            s = (qh @ kh.T * sm).masked_fill(~see, -math.inf)
            w = torch.softmax(s[some], -1)
            out[rows, h] = w @ vh
            wv[rows, h] = w @ vh.abs()
            lse[rows, h] = torch.logsumexp(s[some], -1)
            unit[rows, h] = (qh[some].abs() @ kh.abs().T).masked_fill(~see[some], 0).amax(-1)
        t += n
    return out, lse, wv, unit
