"""Cases of the operators that drafted trees and beams need beside the paged K/V cache: the ancestor bits of a tree of
drafted tokens, attention of a tree over the cache, tokens kept and moved together in the cache, pages copied, and
the pages' accounting (given out, shared by a fork, given back).

`own` false: the plain form, elementary torch operations.  `own` true: the library.
Sequence lengths follow from the case alone; values, trees, page order and weights from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
KEEP_ALL = 2 ** 31 - 1


# ------------------------------------------------------------------------------------- the cases
def _tree(name, n_seqs, q, kv=(100, 4000), window=0):
    return {"name": name, "op": "tree", "n_seqs": n_seqs, "q_min": q[0], "q_max": q[1], "kv_min": kv[0], "kv_max": kv[1],
            "window": window, "lens": 1}


def _attn(name, n_seqs, q, kv, hq, hkv, d, page, fmt, window=0):
    return {"name": name, "op": "attn", "n_seqs": n_seqs, "q_min": q[0], "q_max": q[1], "kv_min": kv[0], "kv_max": kv[1],
            "hq": hq, "hkv": hkv, "d": d, "page": page, "fmt": fmt, "window": window, "lens": 1}


def _compact(name, n_seqs, kv, block, blocks, gone, hkv, d, page, fmt):
    """`blocks` blocks of `block` tokens behind the kept ones, of which `gone` are dropped."""
    return {"name": name, "op": "compact", "n_seqs": n_seqs, "kv_min": kv[0], "kv_max": kv[1], "block": block,
            "blocks": blocks, "gone": gone, "hkv": hkv, "d": d, "page": page, "fmt": fmt, "lens": 1}


def _copy(name, n, tokens, hkv, d, page, fmt, n_pages):
    return {"name": name, "op": "copy", "n": n, "t_min": tokens[0], "t_max": tokens[1], "hkv": hkv, "d": d, "page": page,
            "fmt": fmt, "n_pages": n_pages, "lens": 1}


def _pool(name, kind, rows, kv, more, page, n_pages, used):
    """`used`: how many of 1000 pages other requests hold."""
    return {"name": name, "op": "pool", "kind": kind, "rows": rows, "kv_min": kv[0], "kv_max": kv[1], "more": more,
            "page": page, "n_pages": n_pages, "used": used, "lens": 1}


def listed():
    """kv is the range of tokens cached before the new ones, q that of a sequence's drafted tokens."""
    return [
        # the drafts of a small batch: pure latency
        _tree("tree_small", 8, (8, 16)),
        # a full batch with wide trees
        _tree("tree_large", 256, (100, 250)),
        # a few drafted tokens of few and short sequences: latency of one step
        _attn("verify_few", 4, (6, 8), (300, 1000), 32, 8, 128, 16, "bf16"),
        # trees of a serving batch with ragged contexts: the cache's bandwidth
        _attn("verify_batch", 32, (24, 60), (1000, 9000), 32, 8, 128, 64, "bf16"),
        # the same over an 8-bit cache, 64-channel heads of their own
        _attn("verify_e4m3", 16, (20, 64), (2000, 10000), 24, 24, 64, 32, "e4m3"),
        # wide trees behind long contexts: arithmetic
        _attn("verify_wide", 2, (230, 256), (20000, 32000), 32, 8, 128, 128, "bf16"),
        # the accepted paths of a batch of drafted trees: a few tokens of each sequence
        _compact("compact_accepted", 64, (500, 4000), 1, 32, 27, 8, 128, 16, "bf16"),
        # latent frames (24 x 42 tokens each) dropped from a streamed video, the heads of the video workload
        _compact("compact_frames", 1, (4032, 4032), 1008, 30, 6, 56, 128, 128, "bf16"),
        # the begun pages of forked sequences
        _copy("copy_begun", 16, (1, 15), 8, 128, 16, "bf16", 600),
        # pages moved in bulk
        _copy("copy_pages", 1500, (64, 64), 8, 128, 64, "bf16", 3300),
        # beams chosen anew: the last ones' pages given back, the chosen ones forked
        _pool("pool_beams", "beams", 32, (500, 4000), 0, 16, 20000, 600),
        # room for the drafts of a full batch, after the last ones' was given back
        _pool("pool_drafts", "drafts", 512, (500, 8000), 64, 16, 400000, 700),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "attn", "attn", "attn", "attn", "compact", "compact", "copy", "pool"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 12, 24, 56])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "tree":
        q = _log_int(rng, 1, 250)
        c = _tree("", _log_int(rng, 1, 256), (max(1, q // 2), q), (0, 4000), rng.choice([0, 0, _log_int(rng, 2, 40)]))
    elif op == "attn":
        hq = hkv * rng.choice([g for g in (1, 1, 2, 4, 5, 7, 8) if hkv * g <= 64])
        n, q, kv = _log_int(rng, 1, 64), _log_int(rng, 2, 256), _log_int(rng, 200, 32000)
        window = _log_int(rng, 100, 8000) if rng.random() < 0.25 else 0
        c = _attn("", n, (max(1, q // 2), q), (kv // 3, kv), hq, hkv, d, page, fmt, window)
        # keys and scores of the plain form (both in fp32) stay within those of the listed cases
        while (c["n_seqs"] * (c["kv_max"] + c["q_max"]) * hkv * d > 290 << 20
               or c["n_seqs"] * hq * c["q_max"] * (c["kv_max"] + c["q_max"]) > 520 << 20):
            if c["n_seqs"] > 1:
                c["n_seqs"] = c["n_seqs"] // 2
            else:
                c["kv_max"] = c["kv_max"] * 2 // 3
                c["kv_min"] = min(c["kv_min"], c["kv_max"])
    elif op == "compact":
        n, block = _log_int(rng, 1, 64), rng.choice([1, 1, 1, _log_int(rng, 2, 1008)])
        blocks = _log_int(rng, 2, 64) if block > 1 else _log_int(rng, 4, 4000)
        while n * block * blocks * hkv * d > 200 << 20:
            n, blocks = max(1, n // 2), max(2, blocks // 2)
        c = _compact("", n, (0, _log_int(rng, 10, 2000)), block, blocks, rng.randint(1, blocks - 1), hkv, d, page, fmt)
        while c["n_seqs"] * (c["kv_max"] + block * blocks) * hkv * d > 280 << 20:
            c["kv_max"] //= 2
    elif op == "copy":
        most = max(2, (48 << 20) // (page * hkv * d))
        n = min(most, _log_int(rng, 1, 1500))
        whole = rng.random() < 0.5
        c = _copy("", n, (page if whole else 1, page), hkv, d, page, fmt, 2 * n + rng.randint(3, 50))
    else:
        rows, kv = _log_int(rng, 1, 512), _log_int(rng, 20, 8000)
        kind = rng.choice(["beams", "drafts"])
        need = (kv // page + 2 + 64 // page) * rows
        c = _pool("", kind, rows, (kv // 3, kv), rng.randint(1, 64) if kind == "drafts" else 0, page,
                  min(400000, max(1000, need + _log_int(rng, rows, 40 * rows + 1000)) * 2), rng.randint(0, 450))
    c["lens"] = rng.randint(2, 1 << 20)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens cached after them) of every sequence."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["n_seqs"])]
    return q, [n + r.randint(case["kv_min"], case["kv_max"]) for n in q]


def _kept(case):
    """(first position that may change, kept positions from there on, length) of every sequence."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["n_seqs"]):
        first = r.randint(case["kv_min"], case["kv_max"])
        stay = sorted(r.sample(range(case["blocks"]), case["blocks"] - case["gone"]))
        out.append((first, [first + x * case["block"] + i for x in stay for i in range(case["block"])],
                    first + case["blocks"] * case["block"]))
    return out


def _pool_lengths(case):
    r = random.Random(case["lens"])
    return [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["rows"])]


# ------------------------------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(case, g, kv_len):
    """The pages of every sequence in random order, and how many pages there are."""
    ps = case["page"]
    pages = [(k + ps - 1) // ps for k in kv_len]
    n_pages, width = sum(pages) + 3, max(pages)
    order = torch.randperm(n_pages - 1, generator=g, device="cuda").to(torch.int32).cpu().tolist()   # the last one is nobody's
    table, at = [], 0
    for p in pages:
        table.append(order[at:at + p] + [-1] * (width - p))
        at += p
    return _i32(table), n_pages


def _pages(case, g, n_pages, s):
    """K channels carry a common offset, as behind a per-head norm."""
    hkv, d = case["hkv"], case["d"]
    shape = (n_pages, case["page"], hkv, d)
    bias = torch.randn((hkv, d), generator=g, device="cuda")
    s["k_pages"] = torch.randn(shape, generator=g, device="cuda").add_(bias).to(torch.bfloat16)
    s["v_pages"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    s["k_scale"] = s["v_scale"] = None
    if case["fmt"] == "e4m3":
        s["k_scale"] = 0.02 + 0.02 * torch.rand(hkv, generator=g, device="cuda")
        s["v_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device="cuda")
        for p, c in (("k_pages", "k_scale"), ("v_pages", "v_scale")):
            s[p] = (s[p].float() / s[c][:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _starts(q_len):
    out = [0]
    for x in q_len:
        out.append(out[-1] + x)
    return out


def _parents(q_len, seed):
    """Of every drafted token, -1 for one that hangs off the cached text: chains, binary and bushier trees."""
    r, out = random.Random(seed), []
    for n in q_len:
        b = r.choice([1, 2, 2, 3])
        out += [min(j - 1, r.randint(max(-1, j // b - 3), max(0, j // b))) for j in range(n)]
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("tree", "attn"):
        q_len, kv_len = _lengths(case)
        n = sum(q_len)
        s.update(cu_q=_i32(_starts(q_len)), kv_len=_i32(kv_len), max_q=max(q_len), max_kv=max(kv_len), words=(max(q_len) + 31) // 32,
                 parents=_i32(_parents(q_len, seed)))
        s["mask"] = torch.empty((n, s["words"]), dtype=torch.int32, device=dev)
        s["depth"], s["positions"] = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2))
        if case["op"] == "attn":
            _plain_tree(s)
            s["page_table"], n_pages = _tables(case, g, kv_len)
            _pages(case, g, n_pages, s)
            s["q"] = torch.randn((n, case["hq"], case["d"]), generator=g, device=dev).to(torch.bfloat16)
            s["out"] = torch.empty_like(s["q"])
        else:
            s["page_table"] = torch.zeros((len(q_len), 1), dtype=torch.int32, device=dev)
    elif case["op"] == "compact":
        kept = _kept(case)
        s["page_table"], n_pages = _tables(case, g, [x[2] for x in kept])
        _pages(case, g, n_pages, s)
        s["first"], s["kv_len"] = _i32([x[0] for x in kept]), _i32([x[2] for x in kept])
        s["n_keep"], s["keep"] = _i32([len(x[1]) for x in kept]), _i32([x[1] for x in kept])
        s["cu_q"] = torch.zeros(len(kept) + 1, dtype=torch.int32, device=dev)
    elif case["op"] == "copy":
        _pages(case, g, case["n_pages"], s)
        order = torch.randperm(case["n_pages"], generator=g, device=dev).to(torch.int32)
        r = random.Random(case["lens"])
        s["src"], s["dst"] = order[:case["n"]].contiguous(), order[case["n"]:2 * case["n"]].contiguous()
        s["tokens"] = _i32([r.randint(case["t_min"], case["t_max"]) for _ in range(case["n"])])
    else:
        _prepare_pool(case, g, s)
    if own:   # the handles a serving loop keeps: the cache, the batch's tables, the tree, the pool, the workspace
        import video_diffusion_transformer_sage_gb300 as sage
        if "k_pages" in s:
            s["cache"] = sage.PagedKV(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        if "cu_q" in s:
            s["batch"] = sage.PagedBatch(s["cu_q"], s["kv_len"], s["page_table"])
            s["ws"] = sage.paged_workspace(case.get("d", 64))
        if "mask" in s:
            s["tree"] = sage.PagedTree(s["mask"], s["depth"], s["positions"])
        if case["op"] == "pool":
            s["pool"] = sage.PagedPool(s["refs"], s["table"], case["page"])
    return s


def _prepare_pool(case, g, s):
    """Pages in random order; some are held by requests that are not in this table."""
    n, ps, kv = case["n_pages"], case["page"], _pool_lengths(case)
    held = [(x + ps - 1) // ps for x in kv]
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    mine = order[:sum(held)].cpu().tolist()
    width, at, table = max((x + case["more"] + ps - 1) // ps for x in kv), 0, []
    for h in held:
        table.append(mine[at:at + h] + [-1] * (width - h))
        at += h
    s["refs"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["refs"][order[:at].long()] = 1
    other = order[at:at + min(n - at, n * case["used"] // 1000)].long()
    s["refs"][other] = 1
    if case["kind"] == "beams":   # rows of the chosen beams' successors behind those of the beams
        rows = case["rows"]
        s["table"] = _i32(table + [[-1] * width] * rows)
        s["src"] = torch.randint(0, rows, (rows,), generator=g, device="cuda").to(torch.int32)
        s["dst"] = torch.arange(rows, 2 * rows, dtype=torch.int32, device="cuda")
        s["hi"] = _i32([KEEP_ALL] * rows + [0] * rows)
        s["len"] = _i32(kv)[s["src"].long()]
    else:
        s["table"], s["hi"] = _i32(table), _i32(kv)
        s["want"] = _i32([x + case["more"] for x in kv])


# ------------------------------------------------------------------------------------- the plain form
def _rows_of(cu, max_q):
    """Token rows of the padded batch [B, max_q] and which of them exist."""
    j = torch.arange(max_q, device=cu.device)
    live = j < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + j, 0), live


def _plain_tree(s):
    """Ancestors by squaring (own edge or parent's): after k steps those up to 2^k further up."""
    cu, kv, m, window = s["cu_q"].long(), s["kv_len"].long(), s["max_q"], s["case"]["window"]
    rows, live = _rows_of(cu, m)
    parent = torch.where(live, s["parents"].long()[rows], -1)
    i = torch.arange(m, device=cu.device)
    up = ((parent[..., None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (m - 1).bit_length())):
        up = torch.matmul(up, up).clamp_(max=1.0)
    seen = up > 0.5
    depth = seen.sum(-1) - 1
    if window:
        seen = seen & (depth[..., None] - depth[:, None] < window)
    bits = torch.zeros((*seen.shape[:2], s["words"] * 32), dtype=torch.int64, device=cu.device)
    bits[..., :m] = seen
    bits = (bits.view(*seen.shape[:2], s["words"], 32) << torch.arange(32, device=cu.device)).sum(-1)
    prefix = (kv - (cu[1:] - cu[:-1])).clamp(min=0)[:, None]
    # rows that do not exist go behind the last one, which is left out
    at, n = torch.where(live, rows, s["mask"].shape[0]), s["mask"].shape[0]
    for name, x in (("mask", bits), ("depth", depth), ("positions", prefix + depth)):
        wide = torch.empty((n + 1, *s[name].shape[1:]), dtype=torch.int32, device=cu.device)
        wide[at] = torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)
        s[name].copy_(wide[:n])
    return {"mask": s["mask"], "depth": s["depth"], "positions": s["positions"]}


def _gather(pages, scale, page, slot):
    if scale is None:
        return pages[page, slot].float()
    return pages.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float() * scale[:, None]


def _plain_attn(s):
    case, dev, ps = s["case"], s["q"].device, s["k_pages"].shape[1]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    rows, live = _rows_of(cu, s["max_q"])
    nb, mq = rows.shape
    key = torch.arange(s["max_kv"], device=dev)
    stored = key < kv[:, None]
    page = torch.where(stored, s["page_table"].long().gather(1, (key // ps).expand(nb, -1)), 0)
    slot = (key % ps).expand(nb, -1)
    prefix = (kv - (cu[1:] - cu[:-1]))[:, None, None]
    seen = (key < prefix).expand(-1, mq, -1)
    if case["window"]:
        seen = seen & (key > prefix + s["depth"].long()[rows][..., None] - case["window"])
    i = (key - prefix).expand(-1, mq, -1)
    word = s["mask"].long()[rows].gather(-1, (i // 32).clamp(0, s["words"] - 1))
    seen = seen | ((i >= 0) & stored[:, None] & ((word >> (i % 32)) & 1).bool())
    k = _gather(s["k_pages"], s["k_scale"], page, slot).permute(0, 2, 3, 1)     # [B, Hkv, D, keys]
    v = _gather(s["v_pages"], s["v_scale"], page, slot).permute(0, 2, 1, 3)     # [B, Hkv, keys, D]
    q = s["q"][rows].float().view(nb, mq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(nb, hkv, -1, d)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(nb, hkv, hq // hkv, mq, -1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(nb, hkv, -1, x.shape[-1]), v).view(nb, hkv, hq // hkv, mq, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, mq, hq, d)
    # rows that do not exist go behind the last one, which is left out
    wide = torch.empty((s["out"].shape[0] + 1, hq, d), dtype=torch.bfloat16, device=dev)
    wide[torch.where(live, rows, s["out"].shape[0])] = o.to(torch.bfloat16)
    s["out"].copy_(wide[:-1])
    return s["out"]


def _bytes(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _plain_compact(s):
    ps, nobody = s["case"]["page"], s["k_pages"].shape[0] - 1
    i = torch.arange(s["keep"].shape[1], device="cuda")
    live = i < s["n_keep"][:, None]
    src, dst = torch.where(live, s["keep"].long(), 0), torch.where(live, s["first"].long()[:, None] + i, 0)
    table = s["page_table"].long()
    sp = torch.where(live, table.gather(1, src // ps), nobody).flatten()
    dp = torch.where(live, table.gather(1, dst // ps), nobody).flatten()
    ss, ds = (src % ps).flatten(), (dst % ps).flatten()
    _bytes(s["k_pages"])[dp, ds] = _bytes(s["k_pages"])[sp, ss]
    _bytes(s["v_pages"])[dp, ds] = _bytes(s["v_pages"])[sp, ss]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    take = (torch.arange(s["case"]["page"], device="cuda") < s["tokens"][:, None])[..., None, None]
    k, v = _bytes(s["k_pages"]), _bytes(s["v_pages"])
    k[dst] = torch.where(take, k[src], k[dst])
    v[dst] = torch.where(take, v[src], v[dst])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_release(s):
    table, ps = s["table"], s["case"]["page"]
    at = torch.arange(table.shape[1], device="cuda") * ps
    gone = (table >= 0) & (at >= s["hi"][:, None])
    s["refs"].scatter_add_(0, table.clamp(min=0).long().flatten(), -gone.int().flatten())
    table.masked_fill_(gone, -1)


def _free_pages(refs, k):
    """The k-th (from 1) page that nobody holds, in ascending order."""
    return torch.searchsorted(torch.cumsum(refs == 0, 0), k).clamp(max=refs.numel() - 1)


def _plain_reserve(s):
    table, refs, ps = s["table"], s["refs"], s["case"]["page"]
    need = (table < 0) & (torch.arange(table.shape[1], device="cuda") * ps < s["want"][:, None])
    per_row = need.sum(1)
    ok = (torch.cumsum(per_row, 0) <= (refs == 0).sum()) | (per_row == 0)
    need &= ok[:, None]
    page = _free_pages(refs, torch.cumsum(need.flatten(), 0).view(need.shape))
    table.copy_(torch.where(need, page, table))
    refs.scatter_add_(0, page.flatten(), need.int().flatten())
    return ok.int()


def _plain_fork(s):
    table, refs, ps = s["table"], s["refs"], s["case"]["page"]
    full, part = (s["len"] // ps).long(), s["len"] % ps
    begun = part > 0
    ok = (torch.cumsum(begun, 0) <= (refs == 0).sum()) | ~begun
    give = begun & ok
    page = _free_pages(refs, torch.cumsum(give, 0))
    i = torch.arange(table.shape[1], device="cuda")
    of_src = table[s["src"].long()]
    share = (i < full[:, None]) & ok[:, None]
    new = torch.where(share, of_src, -1)
    new = torch.where((i == full[:, None]) & give[:, None], page[:, None], new)
    last = of_src.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    table[s["dst"].long()] = torch.where(ok[:, None], new, table[s["dst"].long()]).int()
    refs.scatter_add_(0, of_src.clamp(min=0).long().flatten(), share.int().flatten())
    refs.scatter_add_(0, page, give.int())
    none = torch.full_like(last, -1)
    return torch.where(give, last, none), torch.where(give, page.int(), none), torch.where(give, part, 0), ok.int()


def _plain_pool(s):
    _plain_release(s)
    if s["case"]["kind"] == "drafts":
        return {"ok": _plain_reserve(s), "table": s["table"], "refs": s["refs"]}
    src, dst, tokens, ok = _plain_fork(s)
    return {"ok": ok, "src": src, "dst": dst, "tokens": tokens, "table": s["table"], "refs": s["refs"]}


def _own_run(s):
    import video_diffusion_transformer_sage_gb300 as sage
    op = s["case"]["op"]
    if op == "tree":
        sage.sage_paged_tree(s["parents"], s["batch"], s["tree"], status=s["ws"], window=s["case"]["window"])
        return {"mask": s["mask"], "depth": s["depth"], "positions": s["positions"]}
    if op == "attn":
        return sage.sage_paged_attn_tree(s["q"], s["cache"], s["batch"], s["tree"], window=s["case"]["window"], out=s["out"],
                                         ws=s["ws"])
    if op == "compact":
        sage.sage_paged_compact(s["cache"], s["batch"], s["first"], s["keep"], s["n_keep"], ws=s["ws"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "copy":
        sage.sage_paged_copy(s["cache"], s["src"], s["dst"], s["tokens"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    sage.sage_paged_release(s["pool"], hi=s["hi"])
    if s["case"]["kind"] == "drafts":
        return {"ok": sage.sage_paged_reserve(s["pool"], hi=s["want"]), "table": s["table"], "refs": s["refs"]}
    src, dst, tokens, ok = sage.sage_paged_fork(s["pool"], s["src"], s["dst"], s["len"])
    return {"ok": ok, "src": src, "dst": dst, "tokens": tokens, "table": s["table"], "refs": s["refs"]}


def run(state):
    if own:
        return _own_run(state)
    return {"tree": _plain_tree, "attn": _plain_attn, "compact": _plain_compact, "copy": _plain_copy,
            "pool": _plain_pool}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- what it costs
def work(case):
    """Every input read once, every output written once: visible keys and values, moved tokens, table entries, counts."""
    op, e = case["op"], 1 if case.get("fmt") == "e4m3" else 2
    if op in ("tree", "attn"):
        q_len, kv_len = _lengths(case)
        n, words = sum(q_len), (max(q_len) + 31) // 32
    if op == "tree":
        return {"bytes": n * (4 + 4 * words + 8) + 8 * len(q_len), "flops": n * words}
    if op == "attn":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        keys = pairs = 0
        for q, kv in zip(q_len, kv_len):
            w = min(case["window"] or kv, kv - q)
            keys += w + q
            pairs += q * (w + (q + 1) // 2)
        return {"bytes": 2 * n * hq * d * 2 + keys * 2 * hkv * d * e + 4 * (keys // case["page"]) + 4 * words * n,
                "flops": 4 * pairs * hq * d}
    if op == "compact":
        kept = _kept(case)
        moved = sum(sum(x != first + i for i, x in enumerate(keep)) for first, keep, _ in kept)
        return {"bytes": moved * case["hkv"] * case["d"] * e * 4 + sum(len(x[1]) for x in kept) * 4, "flops": 0}
    if op == "copy":
        r = random.Random(case["lens"])
        tokens = sum(r.randint(case["t_min"], case["t_max"]) for _ in range(case["n"]))
        return {"bytes": tokens * case["hkv"] * case["d"] * e * 4 + 12 * case["n"], "flops": 0}
    kv, ps = _pool_lengths(case), case["page"]
    pages = sum((x + ps - 1) // ps for x in kv)
    if case["kind"] == "beams":   # the children's entries and counts go back and are written anew
        return {"bytes": 4 * case["n_pages"] + pages * 4 * 8, "flops": 0}
    new = sum((x + case["more"] + ps - 1) // ps for x in kv) - pages
    return {"bytes": 4 * case["n_pages"] + 4 * pages + new * 4 * 6 + 12 * len(kv), "flops": 0}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """From the definitions, sequence by sequence and head by head, in 64 bits.  What is copied comes out as it is, and
    whole numbers have no such values."""
    if case["op"] in ("tree", "pool"):
        return None
    s = prepare(case, seed)
    if case["op"] == "copy":
        out = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
        for x, y, n in zip(s["src"].tolist(), s["dst"].tolist(), s["tokens"].tolist()):
            for p in out.values():
                p[y, :n] = p[x, :n]
        return out
    ps, table = case["page"], s["page_table"].long()
    if case["op"] == "compact":
        out = {}
        for name in ("k_pages", "v_pages"):
            x = s[name].double()
            for b, (first, keep, length) in enumerate(_kept(case)):
                pos = torch.arange(length, device="cuda")
                seq = x[table[b, pos // ps], pos % ps]
                new = seq[torch.tensor(keep, device="cuda")]
                pos = pos[first:first + len(keep)]
                x[table[b, pos // ps], pos % ps] = new
                del seq, new
            out[name] = x
        return out
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q_len, kv_len = _lengths(case)
    starts, parents = _starts(q_len), _parents(q_len, seed)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, kv) in enumerate(zip(q_len, kv_len)):
        hidden = torch.ones((n, n), dtype=torch.bool)
        depth, above = [], []
        for t in range(n):
            up = parents[starts[b] + t]
            above.append([t] if up < 0 else above[up] + [t])
            depth.append(len(above[t]) - 1)
            hidden[t, above[t][-case["window"]:] if case["window"] else above[t]] = False
        key = torch.arange(kv, device="cuda")
        page, slot = table[b, key // ps], key % ps
        hidden = torch.cat((torch.zeros((n, kv - n), dtype=torch.bool), hidden), 1).cuda()
        if case["window"]:
            first = kv - n + torch.tensor(depth, device="cuda") - case["window"]
            hidden |= (key <= first[:, None]) & (key < kv - n)
        for h in range(hkv):
            def column(pages, scale):
                if scale is None:
                    return pages[page, slot, h].double()
                return pages.view(torch.uint8)[page, slot, h].view(torch.float8_e4m3fn).double() * scale[h].double()
            k, v = column(s["k_pages"], s["k_scale"]), column(s["v_pages"], s["v_scale"])
            for u in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = (s["q"][starts[b]:starts[b] + n, u].double() @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                out[starts[b]:starts[b] + n, u] = torch.softmax(x, -1) @ v
    return out
