"""Drafted trees on the GPU: mxsa_tree_fwd and mxsa_tree_mask against the
definition (attention in 64 bits, masks exactly), mxsa_tree_commit byte by
byte, and a speculative step's calls in a row.

Tolerances of tree_fwd's rows: those of tests/test_gpu_shared.py (the same
roundings: weights and result to 16 bits, FP32 sums).
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
I32, I64 = torch.int32, torch.int64


def dev(x, dt):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dt, device="cuda")


def random_parents(r, n, chain=False):
    if chain:
        return list(range(-1, n - 1))
    return [-1 if r.rand() < 0.2 else int(r.randint(-1, i)) for i in range(n)]


def ancestors(parents):
    rows = np.zeros((len(parents), len(parents)), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            rows[i] = rows[p]
        rows[i, i] = True
    return rows


def words_of(rows, words):
    """bool [n, tokens] -> int32 [n, words]"""
    b = np.zeros((rows.shape[0], 32 * words), bool)
    b[:, :min(rows.shape[1], 32 * words)] = rows[:, :32 * words]
    return np.packbits(b, axis=1, bitorder="little").view(np.int32)


class Trees:
    """seqs: (new tokens, committed keys); groups: (first, end, prefix)."""

    def __init__(self, seqs, hq=16, hkv=2, q="bf16", ps=64, seed=0, lead=0, tail=0, words=None, groups=None,
                 masks="tree", scale=0.0, wide=False):
        r = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        t = TDT[q]
        self.qn, self.seqs, self.hq, self.hkv = q, seqs, hq, hkv
        self.scale = scale or 128 ** -0.5
        B = len(seqs)
        self.cu = [lead]
        for n, _ in seqs:
            self.cu.append(self.cu[-1] + n)
        self.total = self.cu[-1] + tail
        lens = [n + c for n, c in seqs]
        width = max(1, max(-(-L // ps) for L in lens))
        if wide:  # a table of long rows: the general path also where one launch would do
            width = max(width, 130 * 128 // ps)
        table, pages = np.full((B, width), -3, np.int32), 0
        first_of, common = list(range(B)), [0] * B
        for a, b, P in groups or []:
            P = min([P] + [seqs[i][1] for i in range(a, b) if seqs[i][0] > 0]) if b - a > 1 else 0
            for i in range(a, b):
                first_of[i], common[i] = a, P
        for i, L in enumerate(lens):
            whole = 0 if i == first_of[i] else common[i] // ps
            n = max(-(-L // ps), whole)
            table[i, whole:n] = np.arange(pages, pages + n - whole)
            pages += n - whole
        pages = max(pages, 1) + 2
        perm = r.permutation(pages).astype(np.int32)
        table = np.where(table >= 0, perm[np.maximum(table, 0)], table)
        k, v = (torch.randn(pages, hkv, ps, 128, generator=g) for _ in range(2))
        read, self.slots = torch.zeros(pages, ps, dtype=torch.bool), []
        for i, L in enumerate(lens):
            p = np.arange(L)
            page = table[np.where(p < common[i], first_of[i], i), p // ps] if L else p
            assert (page >= 0).all()
            self.slots.append((torch.from_numpy(page.astype(np.int64)), torch.from_numpy(p % ps)))
            read[self.slots[-1]] = True
        k.transpose(1, 2)[~read] = float("nan")  # what nobody reads
        v.transpose(1, 2)[~read] = float("nan")
        self.k, self.v = k.to(t).cuda(), v.to(t).cuda()
        self.q = (torch.randn(self.total, hq, 128, generator=g) * 2).to(t).cuda()
        self.words = words or max(1, max(-(-n // 32) for n, _ in seqs))
        self.seen, mask = [], np.full((self.total, self.words), -1, np.int32)
        for i, (n, _) in enumerate(seqs):
            if masks == "random":  # any set, also the empty one
                rows = r.rand(n, n) < 0.3
                rows[::3] = False
            else:
                rows = ancestors(random_parents(r, n, masks == "chain"))
            rows[:, 32 * self.words:] = False
            self.seen.append(rows)
            mask[self.cu[i]:self.cu[i + 1]] = words_of(rows, self.words)
        self.mask = dev(mask, I32)
        self.dt, self.dcu, self.dl = dev(table, I32), dev(self.cu, I64), dev(lens, I32)
        self.lens = lens
        self.gp = dev([a for a, _, _ in groups] + [groups[-1][1]], I32) if groups else None
        self.pl = dev([P for _, _, P in groups], I32) if groups else None
        # (causal is not used: set where the case's number is odd)
        self.prob = mx.make_problem(B, self.total, hq, hkv, 0, ps, pages, width, bool(seed & 1), scale, q_dtype=t)
        self.ws = torch.full((mx.dense_shared_workspace_size(self.prob),), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.total, hq, 128), 9.0, dtype=t, device="cuda")
        self.lse = torch.full((hq, self.total), 9.0, device="cuda")
        self.flags = torch.zeros(1, dtype=I32, device="cuda")

    def run(self, **kw):
        a = dict(group_ptr=self.gp, prefix_lens=self.pl, ws=self.ws, out=self.out, lse=self.lse, flags=self.flags)
        a.update(kw)
        mx.tree_fwd(self.prob, self.q, self.k, self.v, self.dt, self.dcu, self.dl, self.mask, **a)
        return self

    def check(self, flags=0):
        torch.cuda.synchronize()
        assert self.flags.item() == flags
        u = U[self.qn]
        for s, (n, base) in enumerate(self.seqs):
            if n == 0:
                continue
            a, b, L = self.cu[s], self.cu[s + 1], self.lens[s]
            page, off = (x.cuda() for x in self.slots[s])
            q = self.q[a:b].double().view(n, self.hkv, -1, 128)
            k, v = self.k[page, :, off].double(), self.v[page, :, off].double()
            x = torch.einsum("tgrd,pgd->tgrp", q, k) * self.scale
            seen = torch.ones(n, L, dtype=torch.bool)
            seen[:, base:] = torch.from_numpy(self.seen[s])
            x.masked_fill_(~seen.cuda()[:, None, None], -math.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.where(lse[..., None] == -math.inf, torch.zeros_like(x), torch.exp(x - lse[..., None]))
            o = torch.einsum("tgrp,pgd->tgrd", p, v).reshape(n, self.hq, 128)
            A = torch.einsum("tgrp,pgd->tgrd", p, v.abs()).reshape(n, self.hq, 128)
            lse = lse.reshape(n, self.hq)
            got, gl = self.out[a:b].double(), self.lse[:, a:b].T.double()
            small = L * 2.0 ** -25 * 5 if self.qn == "fp16" else 0.0
            bad = ~((got - o).abs() <= u * (o.abs() + A) * 1.01 + 6.2e-4 * A + small)
            assert not bad.any(), f"seq {s}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"
            fin = lse.isfinite()
            assert torch.equal(fin, gl.isfinite()) and (gl[~fin] == lse[~fin]).all()
            assert ((gl - lse)[fin].abs() <= 1e-3).all()
        for a, b in ((0, self.cu[0]), (self.cu[-1], self.total)):  # tokens of no sequence
            assert (self.out[a:b] == 9).all() and (self.lse[:, a:b] == 9).all()
        return self


def rand(n, lo, hi, seed):
    return [int(x) for x in np.random.RandomState(seed).randint(lo, hi + 1, n)]


CASES = {
    "one_token": dict(seqs=[(1, 0)]),
    "one_token_long": dict(seqs=[(1, 5000)], ps=128),
    "small": dict(seqs=[(8, 1000)]),
    "no_committed": dict(seqs=[(40, 0), (7, 0)], q="fp16"),
    "edges": dict(seqs=[(16, 112), (16, 113), (16, 111), (32, 96), (33, 95), (31, 97), (5, 128), (64, 64), (64, 65)]),
    "page_edges": dict(seqs=[(3, 61), (3, 62), (9, 120), (9, 125)], hq=12, hkv=4, q="fp16"),
    "empty_between": dict(seqs=[(0, 100), (9, 300), (0, 0), (12, 1), (0, 5)], lead=3, tail=4),
    "verify": dict(seqs=[(16, n) for n in rand(12, 100, 3000, 1)], hq=64, hkv=8, ps=128),
    "wide": dict(seqs=[(61, n) for n in rand(6, 0, 900, 2)], hq=16, hkv=2),
    "wide_g3": dict(seqs=[(125, 700), (100, 33)], hq=12, hkv=4, q="fp16"),
    "g1": dict(seqs=[(150, 90), (128, 128), (129, 1)], hq=4, hkv=4),
    "g128": dict(seqs=[(5, 300), (2, 0)], hq=128, hkv=1),
    "deep_chain": dict(seqs=[(300, 50)], masks="chain", hq=8, hkv=2),
    "random_masks": dict(seqs=[(37, 200), (64, 0), (1, 0), (130, 100)], masks="random"),
    "random_masks_few_rows": dict(seqs=[(3, 0), (2, 30), (4, 0), (8, 125)], masks="random", hq=8, hkv=2, q="fp16"),
    "2048_tokens": dict(seqs=[(2048, 100)], hq=2, hkv=1),
    "spare_words": dict(seqs=[(8, 100), (40, 33)], words=5),
    "groups": dict(seqs=[(9, 1000 + n) for n in rand(8, 0, 60, 3)] + [(7, 400), (20, 10)], groups=[(0, 8, 1000)]),
    "groups_capped": dict(seqs=[(16, 500), (16, 300), (0, 900), (16, 350)], groups=[(0, 4, 5000)], ps=128, hq=64,
                          hkv=8),
    "two_groups": dict(seqs=[(5, 700)] * 6 + [(33, 260)] * 5, groups=[(0, 6, 650), (6, 11, 129)], q="fp16", hq=12,
                       hkv=4),
    # a cluster of 8, 4, 2 and 1 CTAs, sequences of very different lengths
    "cluster_8": dict(seqs=[(9, 8183)], ps=128),
    "cluster_4": dict(seqs=[(5, 4000), (12, 3), (0, 9), (16, 1100)], hq=64, hkv=8),
    "cluster_2": dict(seqs=[(16, n) for n in rand(7, 0, 2000, 6)], hq=64, hkv=8, q="fp16"),
    "cluster_1": dict(seqs=[(n, m) for n, m in zip(rand(14, 0, 16, 7), rand(14, 0, 1000, 8))], hq=64, hkv=8, lead=1,
                      tail=2),
    "many": dict(seqs=[(n, m) for n, m in zip(rand(200, 0, 12, 4), rand(200, 0, 600, 5))], hq=8, hkv=1, tail=3),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_against_the_definition(name, wide):
    Trees(seed=len(name), wide=wide, **CASES[name]).run().check()


def test_a_causal_chain_is_the_dense_causal_call():
    t = Trees([(20, 300), (7, 0)], masks="chain", seed=4).run().check()
    prob = mx.make_problem(*[getattr(t.prob, n) for n in ("num_seqs", "total_q", "num_q_heads", "num_kv_heads", "topk",
                                                         "page_size", "num_pages", "max_pages_per_seq")], True)
    out, lse = torch.empty_like(t.out), torch.empty_like(t.lse)
    mx.dense_shared_fwd(prob, t.q, t.k, t.v, t.dt, t.dcu, t.dl, None, None, t.ws, out, lse)
    torch.cuda.synchronize()
    # (both within u (|o| + A) of the definition, A <= 4.5 sigma of V here)
    assert ((out.double() - t.out.double()).abs() <= 2 * 2.0 ** -8 * (out.double().abs() + 4.5)).all()
    assert ((lse - t.lse).abs() <= 1e-3).all()


@pytest.mark.parametrize("wide", [False, True])
def test_nan_and_infinite_keys_that_a_row_does_not_see(wide):
    """K of drafted tokens outside a row's ancestors does not matter, whatever it holds."""
    t = Trees([(40, 100)], masks="chain", seed=2, wide=wide).run().check()
    want = t.out[:20].clone()
    page, off = (x.cuda() for x in t.slots[0])
    t.k[page[130:], :, off[130:]] = float("nan")
    t.k[page[135:], :, off[135:]] = float("inf")
    t.run()
    torch.cuda.synchronize()
    assert torch.equal(t.out[:20], want)


@pytest.mark.parametrize("wide", [False, True])
def test_too_many_tokens_for_the_mask(wide):
    t = Trees([(40, 100), (9, 3)], words=1, seed=6, wide=wide)
    t.run().check(flags=1024)  # (the further tokens' keys are seen by nobody)


@pytest.mark.parametrize("wide", [False, True])
def test_shorter_than_its_new_tokens(wide):
    t = Trees([(10, 0), (4, 50)], masks="chain", seed=8, wide=wide)
    t.dl.copy_(torch.tensor([6, 54]))
    t.run()
    torch.cuda.synchronize()
    assert t.flags.item() == 8
    # tokens 0 .. 3 have no key; key p is token p + 4's
    assert (t.out[:4] == 0).all() and t.lse[:, :4].isneginf().all()
    page, off = (x.cuda() for x in t.slots[0])
    v = t.v[page[0], :, off[0]].repeat_interleave(8, 0)
    assert torch.equal(t.out[4], v)  # token 4 sees key 0 alone


def test_repeated_captured_and_two_at_once():
    t = Trees([(16, n) for n in rand(9, 100, 2000, 21)], seed=3).run()
    torch.cuda.synchronize()
    out, lse = t.out.clone(), t.lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.run()
    for _ in range(3):
        t.out.fill_(9)
        t.ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.out, out) and torch.equal(t.lse, lse)
    b = Trees([(33, n) for n in rand(7, 0, 900, 22)], hq=12, hkv=4, seed=5)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        t.run(stream=s[0])
        b.run(stream=s[1])
    t.check()
    b.check()
    assert torch.equal(t.out, out)


@pytest.mark.parametrize("wide", [False, True])
def test_lengths_pages_and_starts_that_do_not_fit(wide):
    t = Trees([(9, 100), (4, 700), (16, 30)], hq=64, hkv=8, seed=9, wide=wide).run().check()
    good = t.out.clone()
    t.dcu.copy_(torch.tensor([0, 9, 8, 29]))
    t.out.fill_(9)
    t.run()
    torch.cuda.synchronize()
    assert t.flags.item() == 128 and (t.out == 9).all()
    t.dcu.copy_(torch.tensor(t.cu))
    t.flags.zero_()
    t.dl[0] = t.prob.max_pages_per_seq * 64 + 1
    t.dl[2] = -1
    t.run()
    torch.cuda.synchronize()
    # (the first one's further pages are no pages of the cache; the other length
    # may split the second one's keys otherwise: both within u (|o| + A) of the
    # definition, A <= 4.5 sigma of V here)
    assert t.flags.item() == 16 + 8 + 4
    mine, want = t.out[9:13].double(), good[9:13].double()
    assert ((mine - want).abs() <= 2 * 2.0 ** -8 * (want.abs() + 4.5)).all()
    assert (t.out[13:] == 0).all() and t.lse[:, 13:].isneginf().all()
    t.dl.copy_(torch.tensor(t.lens))
    t.flags.zero_()
    page = t.dt[1, 3].clone()
    t.dt[1, 3] = 10 ** 6
    t.run()
    torch.cuda.synchronize()
    assert t.flags.item() == 4
    t.dt[1, 3] = page
    t.flags.zero_()
    t.run().check()
    assert torch.equal(t.out, good)


@pytest.mark.parametrize("wide", [False, True])
def test_scores_that_grow_along_the_keys(wide):
    """The running maximum is passed again and again, also within a block's second half."""
    t = Trees([(16, 3000), (7, 500)], hq=16, hkv=2, seed=10, wide=wide, q="fp16")
    t.q.abs_()
    for page, off in t.slots:
        at = torch.arange(len(page), device="cuda")[:, None, None]
        rows = t.k[page.cuda(), :, off.cuda()].float()
        t.k[page.cuda(), :, off.cuda()] = ((rows * 0.1 + 1) * (at * 0.004 - 2) + 10 * (at % 300 == 290)).half()
    t.run()
    torch.cuda.synchronize()
    u = U["fp16"]
    for s, (n, base) in enumerate(t.seqs):
        a, b, L = t.cu[s], t.cu[s + 1], t.lens[s]
        page, off = (x.cuda() for x in t.slots[s])
        q = t.q[a:b].double().view(n, t.hkv, -1, 128)
        k, v = t.k[page, :, off].double(), t.v[page, :, off].double()
        x = torch.einsum("tgrd,pgd->tgrp", q, k) * t.scale
        mag = (torch.einsum("tgrd,pgd->tgrp", q.abs(), k.abs()) * t.scale).max().item()
        seen = torch.ones(n, L, dtype=torch.bool)
        seen[:, base:] = torch.from_numpy(t.seen[s])
        x.masked_fill_(~seen.cuda()[:, None, None], -math.inf)
        p = torch.softmax(x, -1)
        o, A = (torch.einsum("tgrp,pgd->tgrd", p, y).reshape(n, t.hq, 128) for y in (v, v.abs()))
        # FP32 sums of 128 products: a score is off by 128 * 2^-24 of its magnitudes' sum, p / l by twice that
        tol = u * (o.abs() + A) * 1.01 + (2 * 128 * 2.0 ** -24 * mag + 1e-5) * A + L * 2.0 ** -25 * 5
        assert ((t.out[a:b].double() - o).abs() <= tol).all()


def test_rows_that_are_no_tokens_change_no_bits():
    """Three heads to a kv head leave rows of a tile without a query: whatever stands there."""
    t = Trees([(16, 700), (7, 500), (42, 130)], hq=12, hkv=4, seed=11)
    t.run().check()
    want, lse = t.out.clone(), t.lse.clone()
    for size in (1e-3, 300.0, float("inf")):
        other = Trees([(16, 900)] * 3, hq=16, hkv=4, seed=12)
        other.q.fill_(size)
        other.run()
        t.out.fill_(9)
        t.run()
        torch.cuda.synchronize()
        assert torch.equal(t.out, want) and torch.equal(t.lse, lse)


# ------------------------------------------------------------------ the masks
@pytest.mark.parametrize("sizes,words", [([1], 1), ([8, 16, 3], 1), ([0, 33, 0, 64, 65], 3), ([2048], 64),
                                         ([125] * 30, 4), ([5, 7], 64), (rand(1024, 0, 6, 7), 1)])
def test_masks_and_positions(sizes, words):
    r = np.random.RandomState(len(sizes) + words)
    cu = np.cumsum([2] + sizes)
    total = int(cu[-1]) + 5
    parents, mask = np.full(total, -9, np.int32), np.full((total, words), 9, np.int32)
    pos = np.full(total, -5, np.int64)
    lens = [n + int(r.randint(0, 3000)) for n in sizes]
    want, wpos = mask.copy(), pos.copy()
    for i, n in enumerate(sizes):
        p = random_parents(r, n, chain=i % 3 == 2)
        parents[cu[i]:cu[i + 1]] = p
        rows = ancestors(p)
        want[cu[i]:cu[i + 1]] = words_of(rows, words) if n else 0
        wpos[cu[i]:cu[i + 1]] = lens[i] - n + rows.sum(1) - 1
    prob = mx.make_problem(len(sizes), total, 8, 8, 0, 64, 1, 100)
    m, p, f = dev(mask, I32), dev(pos, I64), dev([0], I32)
    a = (prob, dev(parents, I32), dev(cu, I64), dev(lens, I32), m)
    mx.tree_mask(*a, p, flags=f)
    assert f.item() == 0 and torch.equal(m, dev(want, I32)) and torch.equal(p, dev(wpos, I64))
    m.copy_(dev(mask, I32))
    mx.tree_mask(*a)
    assert torch.equal(m, dev(want, I32))


def test_mask_data_errors():
    prob = mx.make_problem(2, 6, 8, 8, 0, 64, 1, 2)
    cu, m, p, f = dev([0, 3, 6], I64), dev(np.zeros((6, 1)), I32), dev([0] * 6, I64), dev([0], I32)

    def run(parents, lens, cu=cu, m=m):
        f.zero_()
        mx.tree_mask(prob, dev(parents, I32), cu, dev(lens, I32), m, p, flags=f)
        return f.item(), m[:, 0].tolist(), p.tolist()

    # a parent that is no earlier token stands for -1
    assert run([-1, 1, 0, -2, 3, 1], [9, 9]) == (1024, [1, 2, 5, 1, 2, 6], [6, 6, 7, 6, 6, 7])
    assert run([-1, 0, 1, -1, 0, 1], [2, 200])[0] == 8 + 16
    assert p.tolist() == [-1, 0, 1, 125, 126, 127]
    m.fill_(7)
    assert run([-1] * 6, [9, 9], dev([0, 4, 3], I64))[:2] == (128, [7] * 6)
    assert run([-1] * 6, [9, 9], dev([0, 4, 7], I64))[:2] == (128, [7] * 6)


# ---------------------------------------------------------- the accepted paths
KINDS = {"bf16": (torch.bfloat16, torch.bfloat16), "fp8": (torch.float16, torch.float8_e4m3fn),
         "nvfp4": (torch.bfloat16, "nvfp4")}


def random_path(r, tq, cap):
    n = int(r.randint(0, min(tq, cap) + 1))
    return sorted(r.choice(tq, n, replace=False).tolist())


@pytest.mark.parametrize("kind,hkv,ps,sizes,idx", [
    ("bf16", 2, 64, [(8, 100)], 64), ("bf16", 8, 128, [(64, 1000), (1, 0), (0, 70), (33, 95), (64, 64)], 0),
    ("bf16", 1, 64, [(300, 20)], 128), ("fp8", 4, 64, [(64, 61), (125, 700), (16, 0)], 64),
    ("fp8", 1, 128, [(200, 3)], 0), ("nvfp4", 3, 64, [(64, 61), (125, 700), (16, 0), (100, 1)], 0),
    ("nvfp4", 2, 128, [(90, 100)], 0), ("fp8", 2, 64, [(5, n) for n in range(0, 130, 13)], 8),
])
def test_commit_moves_the_rows(kind, hkv, ps, sizes, idx):
    r = np.random.RandomState(hkv * ps + len(sizes))
    qd, kd = KINDS[kind]
    B, cu = len(sizes), np.cumsum([0] + [n for n, _ in sizes])
    lens = [a + b for a, b in sizes]
    width = max(1, max(-(-L // ps) for L in lens))
    table, pages = np.full((B, width), -1, np.int32), 0
    for i, L in enumerate(lens):
        n = -(-L // ps)
        table[i, :n] = np.arange(pages, pages + n)
        pages += n
    perm = r.permutation(pages + 1).astype(np.int32)
    table = np.where(table >= 0, perm[np.maximum(table, 0)], -1)
    pages += 1
    row = {"bf16": 256, "fp8": 128, "nvfp4": 72}[kind]
    elem = 2 if kind == "bf16" else 1
    caches = [torch.from_numpy(r.randint(0, 256, (pages, hkv, ps * row)).astype(np.uint8)) for _ in range(2)]
    ix = torch.from_numpy(r.randint(0, 256, (pages, 3, ps, idx * elem)).astype(np.uint8)) if idx else None
    cap = max(n for n, _ in sizes) + 2
    paths = [random_path(r, n, cap) for n, _ in sizes]
    paths[0] = sorted(set(paths[0]) | {0, sizes[0][0] - 1})
    path = np.full((B, cap), -77, np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p

    def want(cache, heads, parts):
        """parts: (bytes before the slab's rows, bytes of a row): codes and scales stand apart."""
        c = cache.clone()
        src = cache.view(pages, heads, -1)
        dst = c.view(pages, heads, -1)
        for i, p in enumerate(paths):
            base = sizes[i][1]
            for k, j in enumerate(p):
                a, b = base + j, base + k
                for at, n in parts:
                    x, y = at + a % ps * n, at + b % ps * n
                    dst[table[i, b // ps], :, y:y + n] = src[table[i, a // ps], :, x:x + n]
        return c

    parts = [(0, 64), (ps * 64, 8)] if kind == "nvfp4" else [(0, row)]
    k, v = (c.cuda() for c in caches)
    view = lambda c, shape: c if kind == "nvfp4" else c.view(kd).view(*shape)
    shape = (pages, hkv, ps, 128)
    dix = ix.cuda() if idx else None
    prob = mx.make_problem(B, int(cu[-1]), hkv, hkv, 0, ps, pages, width, q_dtype=qd, kv_dtype=kd)
    out, f = dev([-1] * B, I32), dev([0], I32)
    mx.tree_commit(prob, dev(cu, I64), dev(lens, I32), dev(table, I32), dev(path, I32), dev([len(p) for p in paths], I32),
                   view(k, shape), view(v, shape), kv_lens_out=out,
                   idx_cache=dix.view(kd).view(pages, 3, ps, idx) if idx else None, flags=f)
    assert f.item() == 0
    assert out.tolist() == [b + len(p) for (_, b), p in zip(sizes, paths)]
    assert torch.equal(k.cpu(), want(caches[0], hkv, parts)) and torch.equal(v.cpu(), want(caches[1], hkv, parts))
    if idx:
        assert torch.equal(dix.cpu(), want(ix, 3, [(0, idx * elem)]))


def test_commit_data_errors():
    ps, pages = 64, 4
    k0 = torch.randn(pages, 2, ps, 128, device="cuda").to(torch.bfloat16)

    def run(cu=(0, 8, 16), lens=(20, 100), path=((1, 3, 5), (0, 2, 7)), n=(3, 3), table=((0, -1), (1, 2))):
        prob = mx.make_problem(2, 16, 2, 2, 0, ps, pages, 2)
        k, v = k0.clone(), k0.clone()
        out, f = dev([-1, -1], I32), dev([0], I32)
        mx.tree_commit(prob, dev(cu, I64), dev(lens, I32), dev(table, I32), dev(path, I32), dev(n, I32), k, v, out,
                       flags=f)
        assert torch.equal(k, v)
        moved = (k != k0).any(-1).any(1).nonzero().tolist()  # (page, offset)
        return f.item(), out.tolist(), moved

    first, second = [[0, 12], [0, 13], [0, 14]], [[2, 29], [2, 30]]
    assert run() == (0, [15, 95], first + second)
    # a path out of order, twice the same, out of range, too long: nothing of that sequence moves
    for p in ((3, 1, 5), (1, 1, 5), (-1, 3, 5), (1, 3, 8)):
        assert run(path=(p, (0, 2, 7))) == (1024, [12, 95], second)
    for n in (4, -1):
        assert run(n=(n, 3)) == (1024, [12, 95], second)
    assert run(n=(0, 1)) == (0, [12, 93], [])
    assert run(lens=(7, 100)) == (8, [0, 95], second)
    assert run(lens=(-3, 100)) == (8 + 16, [0, 95], second)
    assert run(lens=(20, 129)) == (16, [15, 120], first)
    assert run(cu=(0, 17, 16)) [0] == 128 and run(cu=(0, 17, 16))[2] == []
    assert run(table=((7, -1), (1, 2))) == (4, [15, 95], second)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
def test_caches_past_two_to_the_32_bytes(kind):
    """Drafted tokens in the last pages of a cache of more than 2^32 bytes: commit and, in 16 bits, attention."""
    row, hkv, ps = {"bf16": 256, "fp8": 128, "nvfp4": 72}[kind], 8, 128
    pages = 2 ** 32 // (hkv * ps * row) + 5
    qd, kd = KINDS[kind]
    k, v = (torch.zeros(pages, hkv, ps * row, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3, pages - 4]], dtype=I32, device="cuda")
    tq, base = 20, 250
    view = lambda c: c if kind == "nvfp4" else c.view(kd).view(pages, hkv, ps, 128)
    prob = mx.make_problem(1, tq, 16, hkv, 0, ps, pages, 3, q_dtype=qd, kv_dtype=kd)
    cu, lens, f = dev([0, tq], I64), dev([tq + base], I32), dev([0], I32)
    g = torch.Generator(device="cuda").manual_seed(3)
    if kind == "bf16":
        for page in table[0].tolist():
            for c in (k, v):
                view(c)[page].copy_(torch.randn(hkv, ps, 128, device="cuda", generator=g))
        q = torch.randn(tq, 16, 128, device="cuda", generator=g).to(qd)
        mask = dev(words_of(ancestors(list(range(-1, tq - 1))), 1), I32)
        out = torch.empty_like(q)
        ws = torch.empty(mx.dense_shared_workspace_size(prob), dtype=torch.uint8, device="cuda")
        mx.tree_fwd(prob, q, view(k), view(v), table, cu, lens, mask, None, None, ws, out, flags=f)
        pos = torch.arange(tq + base, device="cuda")
        kk, vv = (view(c)[table[0].long()[pos // ps], :, pos % ps].double() for c in (k, v))
        x = torch.einsum("tgrd,pgd->tgrp", q.double().view(tq, hkv, 2, 128), kk) / math.sqrt(128)
        late = pos[None] > base + torch.arange(tq, device="cuda")[:, None]
        x.masked_fill_(late[:, None, None], -math.inf)
        p = torch.softmax(x, -1)
        o, A = (torch.einsum("tgrp,pgd->tgrd", p, y).reshape(tq, 16, 128) for y in (vv, vv.abs()))
        assert ((out.double() - o).abs() <= 2.0 ** -8 * (o.abs() + A) * 1.01 + 6.2e-4 * A).all()
    else:
        for page in table[0].tolist():
            for c in (k, v):
                c[page].random_(0, 256, generator=g)
    before = [c[table[0].long()].clone() for c in (k, v)]
    path = [1, 7, 8, 19]
    mx.tree_commit(prob, cu, lens, table, dev([path], I32), dev([4], I32), view(k), view(v), flags=f)
    assert f.item() == 0
    parts = [(0, 64), (ps * 64, 8)] if kind == "nvfp4" else [(0, row)]
    for c, old in zip((k, v), before):
        new = old.clone()
        for i, j in enumerate(path):
            a, b = base + j, base + i
            for at, n in parts:
                new[b // ps, :, at + b % ps * n:at + b % ps * n + n] = old[a // ps, :, at + a % ps * n:at + a % ps * n + n]
        assert torch.equal(c[table[0].long()], new)


# ------------------------------------------------------------- all in a row
def test_speculative_steps_in_a_row():
    """Prompts into the cache, then two rounds of drafted trees: tables, masks, norm + rotation + store, attention
    and commit, each round's attention against the definition over the tokens that the trees say."""
    r = np.random.RandomState(3)
    B, hq, hkv, ps, cap, pages, width = 5, 16, 2, 64, 512, 40, 8
    t = torch.bfloat16
    prob = lambda n: mx.make_problem(B, n, hq, hkv, 0, ps, pages, width, True, q_dtype=t)
    e = lambda *s, dt=I32: torch.zeros(*s, dtype=dt, device="cuda")
    lens, held, table, free = e(B), e(B), e(B, width), dev(r.permutation(pages), I32)
    count, f = dev([pages], I32), e(1)
    kc, vc = (torch.full((pages, hkv, ps, 128), float("nan"), dtype=t, device="cuda") for _ in range(2))
    cu, used, positions, loc = e(B + 1, dt=I64), e(B), e(cap, dt=I64), e(cap, dt=I64)
    half = torch.arange(64, dtype=torch.float64, device="cuda") / 64
    angle = torch.arange(600, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** -half
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    w = (1 + 0.1 * torch.randn(128, device="cuda")).to(t)
    held_rows = [[] for _ in range(B)]  # per sequence: (rotated key, value) of its committed tokens, as cached

    def step(new, parents):
        """One step of the model: q rows and, per sequence, the cached rows of its new tokens."""
        mx.build_tables(prob(cap), lens, dev(new, I32), held, table, free, count, cu, used, positions, loc, flags=f)
        assert f.item() == 0 and cu.tolist() == np.cumsum([0] + new).tolist()
        mask = None
        if parents is not None:
            flat = dev(sum(parents, []) + [0] * (cap - sum(new)), I32)
            mask = e(cap, 2)
            mx.tree_mask(prob(cap), flat, cu, used, mask, positions, flags=f)
        qkv = torch.randn(cap, (hq + 2 * hkv) * 128, device="cuda").to(t)
        q, k, v = (qkv[:, a * 128:b * 128].unflatten(1, (b - a, 128)) for a, b in
                   ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        q_out = torch.zeros(cap, hq, 128, dtype=t, device="cuda")
        mx.norm_rope_store(prob(cap), positions, loc, cos_sin, q, k, v, q_out, kc, vc, q_weight=w, k_weight=w, flags=f)
        rows = [torch.empty(cap, hkv, 128, dtype=t, device="cuda") for _ in range(2)]
        mx.load_kv(prob(cap), loc, kc, vc, *rows, flags=f)
        assert f.item() == 0
        return q_out, rows, mask

    def reference(q, keys, vals, seen):
        x = torch.einsum("tgrd,pgd->tgrp", q.double().view(len(q), hkv, -1, 128), keys.double()) / math.sqrt(128)
        x.masked_fill_(~seen.cuda()[:, None, None], -math.inf)
        p = torch.softmax(x, -1)
        o, A = (torch.einsum("tgrp,pgd->tgrd", p, y).reshape(len(q), hq, 128) for y in (vals.double(), vals.double().abs()))
        return o, A

    def close(got, o, A):
        assert ((got.double() - o).abs() <= 2.0 ** -8 * (o.abs() + A) * 1.01 + 6.2e-4 * A).all()

    new = [100, 1, 64, 30, 129]
    q, (k, v), _ = step(new, None)
    p = prob(sum(new))
    out = torch.empty(sum(new), hq, 128, dtype=t, device="cuda")
    n = sum(new)
    mx.prompt_fwd(p, q[:n], k[:n], v[:n], cu, torch.empty(mx.prompt_workspace_size(p), dtype=torch.uint8, device="cuda"),
                  out, flags=f)
    at = 0
    for s, x in enumerate(new):
        o, A = reference(q[at:at + x], k[at:at + x], v[at:at + x], torch.ones(x, x, dtype=torch.bool).tril())
        close(out[at:at + x], o, A)
        held_rows[s] = [(k[i].clone(), v[i].clone()) for i in range(at, at + x)]
        at += x
    lens.copy_(used)
    for rnd in range(2):
        new = [int(x) for x in r.randint(1, 41, B)]
        parents = [random_parents(r, x) for x in new]
        q, (k, v), mask = step(new, parents)
        out = torch.full((cap, hq, 128), 9.0, dtype=t, device="cuda")
        ws = torch.empty(mx.dense_shared_workspace_size(prob(cap)), dtype=torch.uint8, device="cuda")
        mx.tree_fwd(prob(cap), q, kc, vc, table, cu, used, mask, None, None, ws, out, flags=f)
        at, paths = 0, []
        for s, x in enumerate(new):
            rows = ancestors(parents[s])
            keys, vals = (torch.stack([h[i] for h in held_rows[s]] + list(y[at:at + x])) for i, y in ((0, k), (1, v)))
            seen = torch.cat([torch.ones(x, len(held_rows[s]), dtype=torch.bool), torch.from_numpy(rows)], 1)
            close(out[at:at + x], *reference(q[at:at + x], keys, vals, seen))
            node = int(r.randint(x))
            paths.append(np.flatnonzero(rows[node]).tolist() if s else [])  # the first sequence accepts nothing
            held_rows[s] += [(k[at + i].clone(), v[at + i].clone()) for i in paths[-1]]
            at += x
        assert (out[at:] == 9).all()
        path = np.full((B, 41), -1, np.int32)
        for s, x in enumerate(paths):
            path[s, :len(x)] = x
        mx.tree_commit(prob(cap), cu, used, table, dev(path, I32), dev([len(x) for x in paths], I32), kc, vc, lens,
                       flags=f)
        assert f.item() == 0 and lens.tolist() == [len(h) for h in held_rows]
        for s in range(B):  # the cache holds the accepted tokens in their places
            pos = np.arange(len(held_rows[s]))
            page, off = table[s].long()[dev(pos // ps, I64)], dev(pos % ps, I64)
            for cache, i in ((kc, 0), (vc, 1)):
                assert torch.equal(cache[page, :, off], torch.stack([h[i] for h in held_rows[s]]))


@pytest.mark.parametrize("width", [6, 400])  # tables that the one launch takes, and ones that the three do
def test_captured_steps_give_what_eager_ones_do(width):
    """Tables, masks, store, attention and commit of a step as one graph on a stream of its own, replayed with other
    trees and paths: the same bits as the same calls one by one."""
    B, n, hq, hkv, ps, pages, t = 6, 12, 16, 2, 64, 60, torch.float16
    cap = B * n + 3
    prob = mx.make_problem(B, cap, hq, hkv, 0, ps, pages, width, q_dtype=t)
    half = torch.arange(64, dtype=torch.float64, device="cuda") / 64
    angle = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** -half
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    def play(captured):
        r, g = np.random.RandomState(8), torch.Generator(device="cuda").manual_seed(4)
        e = lambda *s, dt=I32: torch.zeros(*s, dtype=dt, device="cuda")
        lens, held, table, free, count = e(B), e(B), e(B, width), dev(np.arange(pages), I32), dev([pages], I32)
        new, parents, path, plens, f = e(B), e(cap), e(B, n), e(B), e(1)
        kc, vc = (e(pages, hkv, ps, 128, dt=t) for _ in range(2))
        cu, used, positions, loc, mask = e(B + 1, dt=I64), e(B), e(cap, dt=I64), e(cap, dt=I64), e(cap, 1)
        qkv, q, out = e(cap, (hq + 2 * hkv) * 128, dt=t), e(cap, hq, 128, dt=t), e(cap, hq, 128, dt=t)
        lse = e(hq, cap, dt=torch.float32)
        ws = torch.empty(mx.dense_shared_workspace_size(prob), dtype=torch.uint8, device="cuda")
        rows = [qkv[:, a * 128:b * 128].unflatten(1, (b - a, 128)) for a, b in
                ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]

        def step():
            mx.build_tables(prob, lens, new, held, table, free, count, cu, used, positions, loc, flags=f)
            mx.tree_mask(prob, parents, cu, used, mask, positions, flags=f)
            mx.norm_rope_store(prob, positions, loc, cos_sin, *rows, q, kc, vc, flags=f)
            mx.tree_fwd(prob, q, kc, vc, table, cu, used, mask, None, None, ws, out, lse, flags=f)
            mx.tree_commit(prob, cu, used, table, path, plens, kc, vc, lens, flags=f)

        graph, side, got = torch.cuda.CUDAGraph(), torch.cuda.Stream(), []
        if captured:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                step()
        for i in range(6):
            sizes = [int(x) for x in r.randint(0, n + 1, B)]
            trees = [random_parents(r, x) for x in sizes]
            ends = [np.flatnonzero(ancestors(p)[r.randint(len(p))]).tolist() if len(p) else [] for p in trees]
            new.copy_(dev(sizes, I32))
            parents[:sum(sizes)].copy_(dev(sum((list(p) for p in trees), []), I32))
            path.copy_(dev([x + [-1] * (n - len(x)) for x in ends], I32))
            plens.copy_(dev([len(x) for x in ends], I32))
            qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=g))
            torch.cuda.synchronize()
            if captured:
                with torch.cuda.stream(side):
                    graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            assert f.item() == 0
            got.append([x.clone() for x in (out, lse, kc, vc, lens, table, mask, positions, loc)])
        return got

    for a, b in zip(play(False), play(True)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_commits_at_once_and_captured(kind):
    """Two layers' caches committed on two streams at once, then both in replayed graphs with other paths."""
    qd, kd = KINDS[kind]
    r = np.random.RandomState(6)
    B, hkv, ps, pages, width, n = 40, 4, 64, 400, 6, 50
    prob = mx.make_problem(B, B * n, 16, hkv, 0, ps, pages, width, q_dtype=qd, kv_dtype=kd)
    table = dev(r.permutation(pages)[:B * width].reshape(B, width), I32)
    cu, lens = dev(np.arange(B + 1) * n, I64), dev(r.randint(n, width * ps + 1, B), I32)
    g = torch.Generator(device="cuda").manual_seed(1)
    layers = [[torch.randint(0, 256, (pages, hkv, ps, 256 if kind == "bf16" else 128), dtype=torch.uint8, device="cuda",
                             generator=g) for _ in range(2)] for _ in range(2)]
    path, plens, f = torch.zeros(B, n, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda"), dev([0], I32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    # raw bytes of a cache as its rows' type
    views = [[c.view(kd).view(pages, hkv, ps, 128) for c in x] for x in layers]
    commit = lambda i: mx.tree_commit(prob, cu, lens, table, path, plens, *views[i], flags=f)

    def draw_paths():
        paths = [random_path(r, n, n) for _ in range(B)]
        path.copy_(dev([x + [0] * (n - len(x)) for x in paths], I32))
        plens.copy_(dev([len(x) for x in paths], I32))
        return paths

    def check(run):
        paths, old = draw_paths(), [[c.clone() for c in x] for x in layers]
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                run(i)
        torch.cuda.synchronize()
        tab, ln = table.cpu().numpy(), lens.tolist()
        for x, was in zip(layers, old):
            for c, o in zip(x, was):
                want = o.clone()
                for s, p in enumerate(paths):
                    src, dst = (np.asarray(p, int) + ln[s] - n, np.arange(len(p)) + ln[s] - n)
                    a, b = (dev(tab[s][y // ps], I64) for y in (src, dst))
                    want[b, :, dev(dst % ps, I64)] = o[a, :, dev(src % ps, I64)]
                assert torch.equal(c, want)
        assert f.item() == 0

    check(commit)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            commit(i)
    for _ in range(3):
        check(lambda i: graphs[i].replay())
