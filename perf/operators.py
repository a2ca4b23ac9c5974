"""Cases of the paged K/V cache operators: appending a batch's new tokens to the cache (with the
per-head RMSNorm and the rotation of Q and K on the way) and attention of new tokens over it.

`own` false: the plain form, elementary torch operations in fp32.  `own` true: the library.
Sequence lengths follow from the case alone; values, page order and weights from the seed.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------- the cases
def _append(name, n_seqs, q, kv, hq, hkv, d, page, fmt, norm=True):
    return {"name": name, "op": "append", "n_seqs": n_seqs, "q_min": q[0], "q_max": q[1], "kv_min": kv[0],
            "kv_max": kv[1], "hq": hq, "hkv": hkv, "d": d, "page": page, "fmt": fmt, "norm": norm, "lens": 1}


def _attn(name, n_seqs, q, kv, hq, hkv, d, page, fmt, causal, window=0):
    return {"name": name, "op": "attn", "n_seqs": n_seqs, "q_min": q[0], "q_max": q[1], "kv_min": kv[0],
            "kv_max": kv[1], "hq": hq, "hkv": hkv, "d": d, "page": page, "fmt": fmt, "causal": causal,
            "window": window, "lens": 1}


def listed():
    """kv is the range of tokens cached before the new ones, q that of a sequence's new tokens."""
    return [
        # one decode step of a small batch: pure latency
        _append("append_step", 8, (1, 1), (200, 4000), 32, 8, 128, 16, "bf16"),
        # three latent frames (24 x 42 tokens each) of a streamed video, the heads of the video workload
        _append("append_frames", 1, (3024, 3024), (12610, 12610), 56, 56, 128, 128, "bf16"),
        # a ragged batch of prompts into an 8-bit cache, 64-channel heads
        _append("append_ragged_e4m3", 48, (1, 500), (0, 3000), 24, 24, 64, 64, "e4m3"),
        # single tokens, few and short sequences: latency of one step
        _attn("decode_few", 4, (1, 1), (300, 1000), 32, 8, 128, 16, "bf16", True),
        # single tokens of a full serving batch with ragged contexts: the cache's bandwidth
        _attn("decode_batch", 64, (1, 1), (2000, 14000), 64, 8, 128, 64, "bf16", True),
        # one sequence with a very long context: the key axis has to be split
        _attn("decode_long", 1, (1, 1), (130001, 130001), 32, 8, 128, 256, "bf16", True),
        # single tokens over an 8-bit cache
        _attn("decode_e4m3", 32, (1, 1), (1000, 16000), 32, 4, 128, 32, "e4m3", True),
        # a few drafted tokens of each sequence, one K/V head per query head, 64-channel heads
        _attn("draft_tokens", 16, (4, 7), (1000, 6000), 24, 24, 64, 32, "bf16", True),
        # a short prompt behind a long shared context: few query rows, many keys
        _attn("short_chunk_long", 1, (65, 65), (32003, 32003), 32, 8, 128, 64, "bf16", True),
        # prompts of a ragged batch, some behind cached prefixes
        _attn("prompts_causal", 6, (300, 2500), (0, 6000), 32, 8, 128, 16, "bf16", True),
        # the same with a sliding window over an 8-bit cache, 64-channel heads
        _attn("window_e4m3", 3, (700, 1500), (4000, 12000), 24, 24, 64, 64, "e4m3", True, 4096),
        # three latent frames attending to the whole video so far and to each other
        _attn("chunk_frames", 1, (3024, 3024), (34786, 34786), 56, 56, 128, 128, "bf16", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 12, 24, 56])
    hq = hkv * rng.choice([g for g in (1, 1, 2, 4, 5, 7, 8) if hkv * g <= 64])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["bf16", "bf16", "e4m3"])
    kind = rng.choice(["append", "append", "decode", "decode", "draft", "chunk", "chunk"])
    if kind == "append":
        n = _log_int(rng, 1, 64)
        tokens = _log_int(rng, n, min(60000, 6000 * n))
        q = max(1, tokens // n)
        c = _append("", n, (max(1, q // 2), q), (0, _log_int(rng, 10, 2000)), hq, hkv, d, page, fmt,
                    rng.random() < 0.7)
        # the cache and the plain form's temporaries stay near a few GB
        while c["n_seqs"] * (c["q_max"] + c["kv_max"]) * hkv * d > 1 << 29 or c["n_seqs"] * c["q_max"] * hq * d > 1 << 28:
            c["n_seqs"] = max(1, c["n_seqs"] // 2)
            c["kv_max"] = max(8, c["kv_max"] // 2)
            c["q_max"] = max(1, c["q_max"] // 2)
            c["q_min"] = min(c["q_min"], c["q_max"])
    else:
        causal = kind != "chunk" or rng.random() < 0.6
        if kind == "chunk":
            n = _log_int(rng, 1, 8)
            q = _log_int(rng, 30, 3000)
        elif kind == "draft":
            n = _log_int(rng, 1, 48)
            q = rng.randint(2, 8)
        else:
            n = _log_int(rng, 1, 100)
            q = 1
        kv = _log_int(rng, 200, 40000)
        window = _log_int(rng, 100, 8000) if causal and rng.random() < 0.25 else 0
        c = _attn("", n, (max(1, q // 2), q), (kv // 3, kv), hq, hkv, d, page, fmt, causal, window)
        # keys and scores of the plain form (both in fp32) stay within those of the listed cases
        while (c["n_seqs"] * (c["kv_max"] + c["q_max"]) * hkv * d > 1 << 29
               or c["n_seqs"] * hq * c["q_max"] * (c["kv_max"] + c["q_max"]) > 3 << 30):
            if c["n_seqs"] > 1:
                c["n_seqs"] = c["n_seqs"] // 2
            else:
                c["kv_max"] = c["kv_max"] * 2 // 3
                c["kv_min"] = min(c["kv_min"], c["kv_max"])
    c["lens"] = rng.randint(2, 1 << 20)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens cached after them) of every sequence."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["n_seqs"])]
    return q, [n + r.randint(case["kv_min"], case["kv_max"]) for n in q]


# ------------------------------------------------------------------------------------- inputs
def _rope_table(rows, d, dev):
    pos = torch.arange(rows, dtype=torch.float64, device=dev)
    freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device=dev) / (d // 2))
    ang = pos[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
    q_len, kv_len = _lengths(case)
    n = sum(q_len)
    pages = [(k + ps - 1) // ps for k in kv_len]
    n_pages, width = sum(pages) + 3, max(pages)
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu().tolist()
    table, at = [], 0
    for p in pages:
        table.append(order[at:at + p] + [0] * (width - p))
        at += p
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    starts = [0]
    for x in q_len:
        starts.append(starts[-1] + x)
    s = {"case": case, "cu_q": i32(starts), "kv_len": i32(kv_len), "page_table": i32(table),
         "max_q": max(q_len), "max_kv": max(kv_len)}
    # K channels carry a common offset and Q rows have unit norm per channel, as behind a per-head norm
    bias = torch.randn((hkv, d), generator=g, device=dev)
    kv_shape = (n_pages, ps, hkv, d)
    s["k_scale"] = s["v_scale"] = None
    if case["op"] == "append":
        s["k_pages"] = torch.zeros(kv_shape, dtype=torch.bfloat16, device=dev)
        s["v_pages"] = torch.zeros(kv_shape, dtype=torch.bfloat16, device=dev)
    else:
        s["k_pages"] = (torch.randn(kv_shape, generator=g, device=dev) + bias).to(torch.bfloat16)
        s["v_pages"] = torch.randn(kv_shape, generator=g, device=dev).to(torch.bfloat16)
    if case["fmt"] == "e4m3":
        s["k_scale"] = 0.02 + 0.02 * torch.rand(hkv, generator=g, device=dev)
        s["v_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device=dev)
        for p, c in (("k_pages", "k_scale"), ("v_pages", "v_scale")):
            x = s[p].float() / s[c][:, None]
            s[p] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            del x
    if case["op"] == "append":
        proj = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=dev).to(torch.bfloat16)
        s["q"] = proj[:, :hq * d].view(n, hq, d)
        s["k"] = proj[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = proj[:, (hq + hkv) * d:].view(n, hkv, d)
        s["gamma_q"] = s["gamma_k"] = None
        if case["norm"]:
            s["gamma_q"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=dev)
            s["gamma_k"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=dev)
        s["cos"], s["sin"] = _rope_table(max(kv_len), d, dev)
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = torch.randn((n, hq, d), generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=dev)
    if own:   # the handles a serving loop keeps: the cache, the batch's tables, the workspace
        import video_diffusion_transformer_sage_gb300 as sage
        s["cache"] = sage.PagedKV(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        s["batch"] = sage.PagedBatch(s["cu_q"], s["kv_len"], s["page_table"])
        s["ws"] = sage.paged_workspace(d)
    return s


# ------------------------------------------------------------------------------------- the plain form
def _plain_norm_rope(x, gamma, cos, sin):
    x = x.float()
    if gamma is not None:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * gamma
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _token_places(s):
    """(sequence, position) of every new token."""
    n = s["q"].shape[0]
    t = torch.arange(n, device=s["q"].device)
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    return b, kv[b] - (cu[b + 1] - cu[b]) + (t - cu[b])


def _plain_append(s):
    ps = s["k_pages"].shape[1]
    b, pos = _token_places(s)
    page, slot = s["page_table"].long()[b, pos // ps], pos % ps
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["q_out"].copy_(_plain_norm_rope(s["q"], s["gamma_q"], cos, sin))
    k, v = _plain_norm_rope(s["k"], s["gamma_k"], cos, sin), s["v"].float()
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_pages"].view(torch.uint8)[page, slot] = k
        s["v_pages"].view(torch.uint8)[page, slot] = v
    else:
        s["k_pages"][page, slot] = k.to(torch.bfloat16)
        s["v_pages"][page, slot] = v.to(torch.bfloat16)
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _gather(pages, scale, page, slot, dt):
    if scale is None:
        return pages[page, slot].to(dt)
    return pages.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).to(dt) * scale.to(dt)[:, None]


def _places(s):
    """Indices of the padded batch: token rows [B, max_q], key pages and slots [B, max_kv], and the
    visible (row, key) pairs [B, max_q, max_kv]."""
    case, dev, ps = s["case"], s["q"].device, s["k_pages"].shape[1]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    q_len = cu[1:] - cu[:-1]
    j = torch.arange(s["max_q"], device=dev)
    live = j < q_len[:, None]
    rows = torch.where(live, cu[:-1, None] + j, 0)
    key = torch.arange(s["max_kv"], device=dev)
    stored = key < kv[:, None]
    page = torch.where(stored, s["page_table"].long().gather(1, (key // ps).expand(len(kv), -1)), 0)
    slot = (key % ps).expand(len(kv), -1)
    seen = stored[:, None].expand(-1, s["max_q"], -1)
    if case["causal"]:
        pos = (kv - q_len)[:, None] + j
        seen = seen & (key <= pos[..., None])
        if case["window"]:
            seen = seen & (key > pos[..., None] - case["window"])
    return live, rows, page, slot, seen


def _plain_attn(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    live, rows, page, slot, seen = _places(s)
    nb, mq = rows.shape
    k = _gather(s["k_pages"], s["k_scale"], page, slot, torch.float32).permute(0, 2, 3, 1)     # [B, Hkv, D, keys]
    v = _gather(s["v_pages"], s["v_scale"], page, slot, torch.float32).permute(0, 2, 1, 3)     # [B, Hkv, keys, D]
    q = s["q"][rows].float().view(nb, mq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(nb, hkv, -1, d)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(nb, hkv, hq // hkv, mq, -1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(nb, hkv, -1, x.shape[-1]), v).view(nb, hkv, hq // hkv, mq, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, mq, hq, d)
    s["out"].copy_(o[live])
    return s["out"]


def run(state):
    if own:
        import video_diffusion_transformer_sage_gb300 as sage
        s = state
        if s["case"]["op"] == "append":
            sage.sage_paged_append(s["k"], s["v"], s["cache"], s["batch"], q=s["q"], gamma_q=s["gamma_q"],
                                   gamma_k=s["gamma_k"], rope_cos=s["cos"], rope_sin=s["sin"], eps=EPS,
                                   q_out=s["q_out"], status=s["ws"])
            return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return sage.sage_paged_attn(s["q"], s["cache"], s["batch"], causal=s["case"]["causal"],
                                    window=s["case"]["window"], out=s["out"], ws=s["ws"])
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attn(state)


# ------------------------------------------------------------------------------------- what it costs
def work(case):
    """New tokens' rows read and written once, every visible key and value read once."""
    q_len, kv_len = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n, e = sum(q_len), 1 if case["fmt"] == "e4m3" else 2
    if case["op"] == "append":
        return {"bytes": n * d * (2 * hq * 2 + 2 * hkv * (2 + e)) + n * d * 4 + 4 * n, "flops": n * (hq + hkv) * d * 8}
    keys = pairs = 0
    for q, kv in zip(q_len, kv_len):
        w = case["window"] or kv
        keys += min(kv, w + q - 1) if case["causal"] else kv
        pairs += sum(min(p + 1, w) for p in range(kv - q, kv)) if case["causal"] else q * kv
    return {"bytes": 2 * n * hq * d * 2 + keys * 2 * hkv * d * e + 4 * (keys // case["page"]), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """From the definitions, sequence by sequence and head by head, in 64 bits.  Values that the
    cache holds in 8 bits have none: a rounding border falls to either side."""
    s = prepare(case, seed)
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
    q_len, kv_len = _lengths(case)
    starts, table = s["cu_q"].tolist(), s["page_table"].long()
    if case["op"] == "append":
        def turned(x, gamma, pos):
            x = x.double()
            if gamma is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * gamma.double()
            c, w = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
            z = torch.empty_like(x)
            z[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * w
            z[..., 1::2] = x[..., 0::2] * w + x[..., 1::2] * c
            return z
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        store = case["fmt"] == "bf16"
        kp = s["k_pages"].double() if store else None
        vp = s["v_pages"].double() if store else None
        for b, (n, kv) in enumerate(zip(q_len, kv_len)):
            r = slice(starts[b], starts[b] + n)
            pos = torch.arange(kv - n, kv, device="cuda")
            out[r] = turned(s["q"][r], s["gamma_q"], pos)
            if store:
                kp[table[b, pos // ps], pos % ps] = turned(s["k"][r], s["gamma_k"], pos)
                vp[table[b, pos // ps], pos % ps] = s["v"][r].double()
        return {"q": out, "k_pages": kp, "v_pages": vp}
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, kv) in enumerate(zip(q_len, kv_len)):
        key = torch.arange(kv, device="cuda")
        page, slot = table[b, key // ps], key % ps
        hidden = None
        if case["causal"]:
            pos = torch.arange(kv - n, kv, device="cuda")[:, None]
            hidden = key > pos
            if case["window"]:
                hidden = hidden | (key <= pos - case["window"])
        for h in range(hkv):
            def column(pages, scale):
                if scale is None:
                    return pages[page, slot, h].double()
                return pages.view(torch.uint8)[page, slot, h].view(torch.float8_e4m3fn).double() * scale[h].double()
            k, v = column(s["k_pages"], s["k_scale"]), column(s["v_pages"], s["v_scale"])
            for u in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][starts[b]:starts[b] + n, u].double() @ k.T / math.sqrt(d)
                if hidden is not None:
                    x.masked_fill_(hidden, -math.inf)
                out[starts[b]:starts[b] + n, u] = torch.softmax(x, -1) @ v
    return out
