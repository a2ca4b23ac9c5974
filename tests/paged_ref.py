"""Problems for the paged K/V cache and their answers in 64 bits, on any device, from the definitions alone."""
import math
import random

import torch

E4M3_MAX = 448.0


class Problem:
    """A batch of sequences with a paged cache: q_lens new tokens each, kv_lens tokens in the cache with
    them (fewer than the new ones: left padding).  Slots that hold no token are filled with NaN."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, page, fmt="bf16", layout="nhd", seed=0, device="cuda",
                 pad_rows=0, extra_width=1, share_first_page=False):
        g = torch.Generator("cpu").manual_seed(seed)
        r = random.Random(seed)
        self.q_lens, self.kv_lens, self.hq, self.hkv, self.d, self.page, self.fmt = q_lens, kv_lens, hq, hkv, d, page, fmt
        self.dev = torch.device(device)
        n = sum(q_lens)
        self.n, self.rows = n, n + pad_rows
        need = [max(0, -(-k // page)) for k in kv_lens]
        self.n_pages = sum(need) + 3
        order = list(range(self.n_pages))
        r.shuffle(order)
        width = max(need + [0]) + extra_width
        table, at = [], 0
        for p in need:
            table.append(order[at:at + p] + [-7] * (width - p))   # entries behind the end: never read
            at += p
        if share_first_page:
            for row, p in zip(table[1:], need[1:]):
                if p > 1:
                    row[0] = table[0][0]
        cu = [0]
        for x in q_lens:
            cu.append(cu[-1] + x)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.dev)  # noqa: E731
        self.cu_q, self.kv_len = i32(cu), i32(kv_lens)
        self.table = i32(table).reshape(len(q_lens), width)
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        proj = rnd(self.rows, (hq + 2 * hkv) * d).to(torch.bfloat16).to(self.dev)
        self.q = proj[:, :hq * d].view(self.rows, hq, d)
        self.k = proj[:, hq * d:(hq + hkv) * d].view(self.rows, hkv, d)
        self.v = proj[:, (hq + hkv) * d:].view(self.rows, hkv, d)
        shape = (self.n_pages, page, hkv, d)
        self.k_scale = self.v_scale = None
        kf, vf = rnd(*shape) + rnd(hkv, d), rnd(*shape)
        used = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for b, k in enumerate(kv_lens):
            for pos in range(max(k, 0)):
                used[table[b][pos // page], pos % page] = True
        self.used = used.to(self.dev)
        if fmt == "e4m3":
            self.k_scale = (0.01 + 0.02 * torch.rand(hkv, generator=g)).to(self.dev)
            self.v_scale = (0.01 + 0.02 * torch.rand(hkv, generator=g)).to(self.dev)
            kf = (kf / self.k_scale.cpu()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            vf = (vf / self.v_scale.cpu()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        kf[~used], vf[~used] = float("nan"), float("nan")
        dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
        self.k_pages, self.v_pages = (self._lay(x.to(dt), layout) for x in (kf, vf))
        if layout == "kv":   # K and V side by side in one buffer, heads before slots
            both = torch.empty((self.n_pages, 2, hkv, page, d), dtype=dt, device=self.dev)
            both[:, 0].view(torch.uint8).copy_(self.k_pages.permute(0, 2, 1, 3).contiguous().view(torch.uint8))
            both[:, 1].view(torch.uint8).copy_(self.v_pages.permute(0, 2, 1, 3).contiguous().view(torch.uint8))
            self.k_pages, self.v_pages = both[:, 0].permute(0, 2, 1, 3), both[:, 1].permute(0, 2, 1, 3)
        self.gamma_q, self.gamma_k = ((1 + 0.2 * rnd(d)).to(self.dev) for _ in range(2))
        pos = torch.arange(max([1] + kv_lens), dtype=torch.float64)
        ang = pos[:, None] * 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))
        self.cos, self.sin = ang.cos().float().to(self.dev), ang.sin().float().to(self.dev)

    def _lay(self, x, layout):
        x = x.to(self.dev)
        if layout == "hnd":
            return x.view(torch.uint8).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(x.dtype) \
                if x.dtype == torch.float8_e4m3fn else x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        return x

    def token_positions(self):
        """[(row, sequence, position)] of the new tokens."""
        out, t = [], 0
        for b, (n, k) in enumerate(zip(self.q_lens, self.kv_lens)):
            for j in range(n):
                out.append((t, b, k - n + j))
                t += 1
        return out

    def values(self, pages, scale):
        """The page values in 64 bits, [n_pages, page, hkv, d]."""
        x = pages.double()
        return x if scale is None else x * scale.double()[:, None]


def transform(x, gamma, cos, sin, eps):
    """RMSNorm and rotation of rows [n, h, d] in 64 bits (gamma, cos: None leaves the step out)."""
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    if cos is not None:
        c, s = cos.double()[:, None], sin.double()[:, None]
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    return x


def attention(p: Problem, q, causal, window=0, sm_scale=None, hide_pages=()):
    """(out, lse, weight of |v|, largest score error unit) of the new tokens in 64 bits, [n, hq, ...]:
    the third is sum_j w_j |v_j|, the fourth max_j sum_c |q_c k_jc| over the visible keys."""
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
        k, v = kp[page, key % p.page], vp[page, key % p.page]            # [kv, hkv, d]
        pos = torch.arange(kv - n, kv, device=dev)[:, None]
        seen = torch.ones((n, kv), dtype=torch.bool, device=dev)
        if causal:
            seen = key <= pos
            if window:
                seen = seen & (key > pos - window)
        for bad in hide_pages:
            seen = seen & (key // p.page != bad[1] if bad[0] == b else torch.ones_like(key, dtype=torch.bool))
        for h in range(p.hq):
            kh, vh, qh = k[:, h // group], v[:, h // group], q[t:t + n, h].double()
            s = (qh @ kh.T * sm).masked_fill(~seen, -math.inf)
            some = seen.any(-1)
            w = torch.softmax(s[some], -1)
            w = torch.where(seen[some], w, torch.zeros_like(w))
            rows = torch.nonzero(some).squeeze(-1) + t
            # a value that no row sees plays no part
            vz = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
            out[rows, h] = w @ vz
            wv[rows, h] = w @ vz.abs()
            lse[rows, h] = torch.logsumexp(s[some], -1)
            unit[rows, h] = (qh[some].abs() @ torch.nan_to_num(kh.abs()).T).masked_fill(~seen[some], 0).amax(-1)
        t += n
    return out, lse, wv, unit


def attention_bound(p: Problem, ref, sm_scale=None):
    """How far a kernel may be off, element by element, from the arithmetic it states.

    - p_j rounded to bf16: a factor 1 + e_j, |e_j| <= 2^-8; where the sum takes the rounded p too, the
      weights are off by at most |e_j - mean e| <= 2^-7, else by 2^-8: 1.01 * 2^-7 sum_j w_j |v_j|.
    - scores from fp32 accumulation of d products: |ds| <= d 2^-23 sum_c |q_c k_c| sm; a weight is a ratio of
      two such exponentials, so off by at most 2 |ds| relative.  The scale's own rounding, ex2, the
      rescales and the fp32 sums add a few 2^-22 each on scores up to some tens: 1e-5 relative.
    - the output rounded to bf16: 2^-8 |out|."""
    out, _, wv, unit = ref
    sm = 1 / math.sqrt(p.d) if sm_scale is None else sm_scale
    ds = p.d * 2.0 ** -23 * unit * sm
    return (1.01 * 2.0 ** -7 + 2 * ds[..., None] + 1e-5) * wv + 2.0 ** -8 * out.abs() + 1e-30


def check_attention(p, got, ref, sm_scale=None):
    off = (got[:p.n].double() - ref[0]).abs() - attention_bound(p, ref, sm_scale)
    assert torch.isfinite(got[:p.n].float()).all()
    assert float(off.max()) <= 0.0, (float(off.max()), [int(i) for i in torch.nonzero(off == off.max())[0]])
