"""The cache's operators together, as a serving loop runs them: drafted trees verified and kept, beams forked and grown, each
step against lists of the tokens that every sequence should hold."""
import random

import pytest
import torch

import paged_ref
import tree_ref
import video_diffusion_transformer_sage_gb300 as sage
from paged_ref import Problem

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _World:
    """A cache of one layer, its pool, and for every row the K and V (as stored) of the tokens that it should hold."""

    def __init__(self, rows, n_pages, page, hq, hkv, d, fmt, width, seed):
        self.r, self.page, self.hq, self.hkv, self.d, self.fmt = random.Random(seed), page, hq, hkv, d, fmt
        self.g = torch.Generator("cuda").manual_seed(seed)
        dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
        self.k_pages, self.v_pages = (torch.full((n_pages, page, hkv, d), float("nan"), device="cuda").to(dt) for _ in range(2))
        self.k_scale = self.v_scale = None
        if fmt == "e4m3":
            self.k_scale, self.v_scale = (0.01 + 0.01 * torch.rand(hkv, generator=self.g, device="cuda") for _ in range(2))
        self.cache = sage.PagedKV(self.k_pages, self.v_pages, self.k_scale, self.v_scale)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.pool = sage.PagedPool(torch.zeros(n_pages, dtype=torch.int32, device="cuda"), self.table, page)
        self.kv_len = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.ws = sage.paged_workspace(d)
        self.tokens = [[] for _ in range(rows)]      # (k, v) of each token, as the cache holds it
        ang = torch.arange(2000, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        self.gamma = 1 + 0.1 * torch.randn(d, generator=self.g, device="cuda")

    def rows_of(self, n, h):
        return torch.randn((n, h, self.d), generator=self.g, device="cuda").to(torch.bfloat16)

    def batch(self, q_lens):
        cu = [0]
        for n in q_lens:
            cu.append(cu[-1] + n)
        return sage.PagedBatch(_i32(cu), self.kv_len, self.table)

    def append(self, q_lens, batch, positions=None):
        """New tokens into the cache; (their treated queries, their K and V as stored)."""
        n = sum(q_lens)
        q, k, v = self.rows_of(n, self.hq), self.rows_of(n, self.hkv), self.rows_of(n, self.hkv)
        q = sage.sage_paged_append(k, v, self.cache, batch, q=q, gamma_q=self.gamma, gamma_k=self.gamma, rope_cos=self.cos,
                                   rope_sin=self.sin, positions=positions)
        stored, t = [], 0
        for b, m in enumerate(q_lens):
            kv = int(self.kv_len[b])
            at = [(int(self.table[b, p // self.page]), p % self.page) for p in range(kv - m, kv)]
            stored.append([(self.k_pages[x].clone(), self.v_pages[x].clone()) for x in at])
            t += m
        return q, stored

    def check(self):
        """Every row's tokens stand in its pages, and the counts are those of the table."""
        for b, want in enumerate(self.tokens):
            for pos, (k, v) in enumerate(want):
                x = int(self.table[b, pos // self.page]), pos % self.page
                assert torch.equal(self.k_pages[x].view(torch.uint8), k.view(torch.uint8)), (b, pos)
                assert torch.equal(self.v_pages[x].view(torch.uint8), v.view(torch.uint8)), (b, pos)
        held = torch.bincount(self.table[self.table >= 0].long(), minlength=self.pool.n_pages)
        assert torch.equal(held.int(), self.pool.refs)
        need = [-(-len(t) // self.page) for t in self.tokens]
        assert (self.table >= 0).sum(1).tolist() == need
        for block in (self.ws, self.cache.status, self.pool.status):
            assert sage.sage_check_device_status(block) == (0, 0)

    def problem(self, q_lens):
        """What paged_ref and tree_ref ask of a batch."""
        p = Problem.__new__(Problem)
        p.q_lens, p.kv_lens, p.hq, p.hkv, p.d, p.page, p.fmt = q_lens, self.kv_len.tolist(), self.hq, self.hkv, self.d, self.page, self.fmt
        p.n = p.rows = sum(q_lens)
        p.dev, p.table, p.k_pages, p.v_pages = self.table.device, self.table, self.k_pages, self.v_pages
        p.k_scale, p.v_scale = self.k_scale, self.v_scale
        return p


@pytest.mark.parametrize("fmt,d,hq,page,most", [("bf16", 128, 8, 16, 7), ("e4m3", 64, 4, 8, 40), ("bf16", 64, 12, 32, 24)])
def test_speculative_decoding(fmt, d, hq, page, most):
    """A prompt, then drafted trees: pages for them, their tokens stored, attention, a path accepted and moved together, the
    pages behind it given back."""
    rows = 3
    w = _World(rows, 80, page, hq, 2, d, fmt, 40, seed=most)
    prompt = [30, 1, 75]
    w.kv_len.copy_(_i32(prompt))
    assert sage.sage_paged_reserve(w.pool, w.kv_len).tolist() == [1] * rows
    _, stored = w.append(prompt, w.batch(prompt))
    w.tokens = [list(s) for s in stored]
    w.check()
    for step in range(6):
        q_lens = [w.r.randint(1, most) for _ in range(rows)]
        prefix = [len(t) for t in w.tokens]
        parents = tree_ref.parents_of(q_lens, step + most)
        w.kv_len += _i32(q_lens)
        assert sage.sage_paged_reserve(w.pool, w.kv_len).tolist() == [1] * rows
        batch = w.batch(q_lens)
        tree = sage.sage_paged_tree(_i32(parents), batch, status=w.ws, words=(most + 31) // 32)
        q, stored = w.append(q_lens, batch, tree.positions)
        out = sage.sage_paged_attn_tree(q, w.cache, batch, tree, ws=w.ws)
        p, seen = w.problem(q_lens), tree_ref.closure(q_lens, parents)[0]
        tree_ref.check_attention(p, out, tree_ref.attention(p, q, seen), q)
        # one path from a root to some node, or nothing, is accepted
        keep, at = [], 0
        for b, n in enumerate(q_lens):
            i, path = w.r.randint(-1, n - 1), []
            while i >= 0:
                path.insert(0, i)
                i = parents[at + i]
            keep.append([prefix[b] + i for i in path])
            w.tokens[b] += [stored[b][i] for i in path]
            at += n
        wide = max(len(k) for k in keep) + 1
        sage.sage_paged_compact(w.cache, batch, _i32(prefix), _i32([k + [0] * (wide - len(k)) for k in keep]),
                                _i32([len(k) for k in keep]), ws=w.ws)
        w.kv_len.copy_(_i32([len(t) for t in w.tokens]))
        sage.sage_paged_release(w.pool, w.kv_len)
        w.check()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_beams(fmt):
    """Beams chosen anew at each step: children share their parents' full pages, the begun ones are copied, each grows on its
    own; attention over the shared pages; at the end all pages are free."""
    beams, page, d = 4, 8, 64
    w = _World(2 * beams, 60, page, 4, 2, d, fmt, 12, seed=5)
    now, then = list(range(beams)), list(range(beams, 2 * beams))
    lens = [21] * beams + [0] * beams
    w.kv_len.copy_(_i32(lens))
    sage.sage_paged_reserve(w.pool, w.kv_len)
    _, stored = w.append(lens, w.batch(lens))
    w.tokens = [list(s) for s in stored]
    w.check()
    for step in range(9):
        chosen = [w.r.choice(now) for _ in range(beams)]
        lens = [len(w.tokens[c]) for c in chosen]
        src, dst, tokens, ok = sage.sage_paged_fork(w.pool, _i32(chosen), _i32(then), _i32(lens))
        assert ok.tolist() == [1] * beams and tokens.tolist() == [n % page for n in lens]
        sage.sage_paged_copy(w.cache, src, dst, tokens)
        for c, t in zip(chosen, then):
            w.tokens[t] = list(w.tokens[c])
        gone = [0 if b in now else 2 ** 31 - 1 for b in range(2 * beams)]
        sage.sage_paged_release(w.pool, _i32(gone))
        for b in now:
            w.tokens[b] = []
        w.check()
        grow = [0 if b in now else w.r.randint(1, 3) for b in range(2 * beams)]
        w.kv_len.copy_(_i32([len(t) + g for t, g in zip(w.tokens, grow)]))
        assert sage.sage_paged_reserve(w.pool, w.kv_len).tolist() == [1] * (2 * beams)
        batch = w.batch(grow)
        q, stored = w.append(grow, batch)
        out = sage.sage_paged_attn(q, w.cache, batch, ws=w.ws)
        p = w.problem(grow)
        paged_ref.check_attention(p, out, paged_ref.attention(p, q, True))
        for t, s in zip(w.tokens, stored):
            t += s
        w.check()
        now, then = then, now
    sage.sage_paged_release(w.pool, torch.zeros_like(w.kv_len))
    assert not w.pool.refs.any() and bool((w.table == -1).all())
