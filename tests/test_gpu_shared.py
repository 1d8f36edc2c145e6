"""mxsa_dense_shared_fwd on the GPU against the definition in 64 bits, and the
serving step's calls in a row.

Tolerance of an output element, with u half a step of the 16-bit type
(bf16 2^-8, fp16 2^-11) and A = sum p |v| of the row and column: the softmax
weights are rounded (u A), the result is rounded (u |ref|), FP32 sums of 128
products change a score by at most 128 * 2^-24 of its magnitudes' sum (below
40 here, so 3.1e-4 relative in p, at most twice that in p / l), and fp16
weights below 2^-14 lose up to 2^-25 each (n keys, l >= 1).  lse: the scores'
error and a few FP32 steps, 1e-3 at most.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


class Case:
    """groups: list of (prefix, [(tokens, own keys), ...]); a prefix of None: the sequences are in no group."""

    def __init__(self, groups, hq=16, hkv=2, q="bf16", ps=64, causal=False, seed=0, lead=0, tail=0, scale=0.0,
                 poison=True):
        r = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        t = TDT[q]
        self.qn, self.ps, self.hq, self.hkv, self.causal = q, ps, hq, hkv, causal
        self.scale = scale or 128 ** -0.5
        seqs, gp, prefix = [], [], []
        order = [x for x in groups if x[0] is not None] + [x for x in groups if x[0] is None]
        for P, members in order:
            if P is not None:
                gp.append(len(seqs))
                prefix.append(P)
            first = len(seqs)
            for tq, own in members:
                seqs.append((tq, (P or 0) + own, first, P or 0))
        ng = len(prefix)
        self.gp = gp + [gp[-1] + len([x for x in groups if x[0] is not None][-1][1])] if ng else None
        self.prefix = prefix if ng else None
        self.B = len(seqs)
        self.lens = [s[1] for s in seqs]
        cu = [lead]
        for s in seqs:
            cu.append(cu[-1] + s[0])
        self.cu, self.total = cu, cu[-1] + tail
        width = max(1, max(-(-L // ps) for L in self.lens))
        pages, table = 0, np.full((self.B, width), -7, np.int32)  # entries nothing needs: no page at all
        for i, (tq, L, first, P) in enumerate(seqs):
            a = 0 if i == first else P // ps  # whole prefix pages come from the first sequence
            n = -(-L // ps)
            if n > a:
                table[i, a:n] = np.arange(pages, pages + n - a)
                pages += n - a
        pages = max(pages, 1) + 2
        perm = r.permutation(pages).astype(np.int32)
        table = np.where(table >= 0, perm[np.maximum(table, 0)], table)
        k = torch.randn(pages, hkv, ps, 128, generator=g)
        v = torch.randn(pages, hkv, ps, 128, generator=g)
        # what each sequence reads, and NaN everywhere else
        read = torch.zeros(pages, ps, dtype=torch.bool)
        self.slots = []
        for i, (tq, L, first, P) in enumerate(seqs):
            P = min([P] + [s[1] for s in seqs if s[2] == first and s[0] > 0]) if P else 0
            if sum(s[2] == first for s in seqs) < 2:
                P = 0
            p = np.arange(L)
            row = np.where(p < P, first, i)
            page = table[row, p // ps] if L else p
            assert (page >= 0).all()
            self.slots.append((torch.from_numpy(page.astype(np.int64)), torch.from_numpy(p % ps)))
            read[self.slots[-1]] = True
        if poison:
            k.transpose(1, 2)[~read] = float("nan")
            v.transpose(1, 2)[~read] = float("nan")
        self.k, self.v = k.to(t).cuda(), v.to(t).cuda()
        self.q = (torch.randn(self.total, hq, 128, generator=g) * 2).to(t).cuda()
        dev = lambda x, dt: None if x is None else torch.tensor(x, dtype=dt, device="cuda")
        self.dt, self.dcu, self.dl = dev(table, torch.int32), dev(cu, torch.int64), dev(self.lens, torch.int32)
        self.dgp, self.dp = dev(self.gp, torch.int32), dev(self.prefix, torch.int32)
        self.prob = mx.make_problem(self.B, self.total, hq, hkv, 1, ps, pages, width, causal, scale, q_dtype=t)
        self.ws = torch.full((mx.dense_shared_workspace_size(self.prob),), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.total, hq, 128), 9.0, dtype=t, device="cuda")
        self.lse = torch.full((hq, self.total), 9.0, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, groups=True, **kw):
        a = dict(group_ptr=self.dgp if groups else None, prefix_lens=self.dp if groups else None, ws=self.ws,
                 out=self.out, lse=self.lse, flags=self.flags)
        a.update(kw)
        mx.dense_shared_fwd(self.prob, self.q, self.k, self.v, self.dt, self.dcu, self.dl, **a)
        return self

    def ref(self, s):
        """(out, A, lse) of sequence s in float64: [tq, hq, 128] twice, [tq, hq]."""
        page, off = (x.cuda() for x in self.slots[s])
        a, b = self.cu[s], self.cu[s + 1]
        tq, L, G = b - a, self.lens[s], self.hq // self.hkv
        q = self.q[a:b].double().view(tq, self.hkv, G, 128)
        k, v = self.k[page, :, off].double(), self.v[page, :, off].double()  # [L, hkv, 128]
        x = torch.einsum("tgrd,pgd->tgrp", q, k) * self.scale
        if self.causal:
            late = torch.arange(L, device="cuda")[None] > L - tq + torch.arange(tq, device="cuda")[:, None]
            x.masked_fill_(late[:, None, None], -math.inf)
        lse = torch.logsumexp(x, -1) if L else torch.full((tq, self.hkv, G), -math.inf, device="cuda",
                                                          dtype=torch.float64)
        p = torch.exp(x - lse[..., None])
        p = torch.where(lse[..., None] == -math.inf, torch.zeros_like(p), p)
        o = torch.einsum("tgrp,pgd->tgrd", p, v).reshape(tq, self.hq, 128)
        return o, torch.einsum("tgrp,pgd->tgrd", p, v.abs()).reshape(tq, self.hq, 128), lse.reshape(tq, self.hq)

    def check(self, flags=0):
        torch.cuda.synchronize()
        assert self.flags.item() == flags
        u = U[self.qn]
        for s in range(self.B):
            a, b = self.cu[s], self.cu[s + 1]
            if a == b:
                continue
            o, A, lse = self.ref(s)
            got, gl = self.out[a:b].double(), self.lse[:, a:b].T.double()
            small = self.lens[s] * 2.0 ** -25 * 5 if self.qn == "fp16" else 0.0
            tol = u * (o.abs() + A) * 1.01 + 6.2e-4 * A + small
            bad = ~((got - o).abs() <= tol)
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
    "one_key": dict(groups=[(None, [(1, 1)])]),
    "decode": dict(groups=[(1000, [(1, n) for n in rand(8, 1, 64, 1)])]),
    "decode_aligned": dict(groups=[(1024, [(1, n) for n in rand(9, 1, 300, 2)])], ps=128, q="fp16"),
    # 40 x 8 rows: a row tile of two halves and one of one half, over several chunks
    "two_row_tiles": dict(groups=[(3001, [(1, n) for n in rand(40, 1, 400, 3)])], hq=16, hkv=2),
    "three_row_tiles_g1": dict(groups=[(700, [(1, n) for n in rand(600, 1, 40, 4)])], hq=2, hkv=2, ps=128),
    "verify_g3": dict(groups=[(901, [(5, n) for n in rand(8, 5, 300, 5)]), (64, [(5, 77), (5, 5)]),
                              (1, [(5, 9), (5, 500)])], hq=12, hkv=4, q="fp16", causal=True),
    "g128": dict(groups=[(513, [(2, 3), (1, 130)])], hq=128, hkv=1, causal=True, ps=128),
    "g96": dict(groups=[(130, [(1, 3), (3, 130), (1, 1)])], hq=96, hkv=1, q="fp16"),
    "g5": dict(groups=[(300, [(30, 200), (11, 64)])], hq=10, hkv=2, causal=True),
    "no_groups_long": dict(groups=[(None, [(1, 20011), (1, 3)])], hq=8, hkv=1),
    "prefill": dict(groups=[(None, [(700, 900), (33, 33)])], hq=8, hkv=2, causal=True),
    "prefill_not_causal": dict(groups=[(200, [(100, 150), (77, 300)])], hq=4, hkv=2),
    # tokens that do not see all of the prefix, prefixes longer than a sequence, empty sequences
    "inside_prefix": dict(groups=[(256, [(90, 10), (3, 300), (0, 0), (40, 0)])], hq=16, hkv=2, causal=True),
    "empty_and_alone": dict(groups=[(0, [(1, 50), (2, 0)]), (300, [(4, 20)]), (None, [(0, 0), (3, 0), (1, 129)])]),
    "more_tokens_than_keys": dict(groups=[(None, [(40, 17), (5, 2)])], causal=True),
    "padded": dict(groups=[(100, [(1, 7), (1, 90)]), (None, [(2, 3)])], lead=3, tail=5),
    "scale": dict(groups=[(190, [(1, 40), (1, 60)])], scale=0.21),
    "mixed": dict(groups=[(5000, [(1, n) for n in rand(20, 1, 900, 6)]), (130, [(7, 40), (1, 4)]),
                          (None, [(1, 3000), (64, 700)])], hq=32, hkv=4, causal=True, ps=128),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    Case(**CASES[name], seed=len(name)).run().check()


def test_1024_sequences():
    n = rand(1024, 1, 200, 7)
    Case([(256, [(1, x) for x in n[:600]]), (None, [(i % 3, x) for i, x in enumerate(n[600:])])], hq=8, hkv=1,
         causal=True, seed=8).run().check()


def test_prefix_length_is_clamped_and_groups_are_optional():
    c = Case([(256, [(1, 40), (2, 90), (1, 0)])], poison=False, seed=3)
    c.dt[1:, :4] = c.dt[0, :4]  # (every row lists the whole prefix, so that no group is needed)
    c.run().check()
    with_groups = c.out.clone()
    c.dp.fill_(10 ** 6)  # longer than any: the shortest sequence's 256
    c.run().check()
    assert torch.equal(c.out, with_groups)
    c.dp.fill_(-5)
    c.run().check()
    c.run(groups=False).check()


def test_equals_dense_fwd_without_groups():
    c = Case([(None, [(3, 500), (1, 64), (20, 700)])], causal=True, hq=16, hkv=2, seed=4).run().check()
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    mx.dense_fwd(c.prob, c.q, c.k, c.v, c.dt, c.dcu, c.dl, out, lse)
    torch.cuda.synchronize()
    assert ((out.float() - c.out.float()).abs() <= 2.0 ** -6 * out.float().abs() + 2e-2).all()
    assert ((lse - c.lse).abs() <= 2e-3).all()


def test_same_bits_every_time_and_in_a_graph():
    c = Case(**CASES["mixed"], seed=5).run().check()
    first, lse = c.out.clone(), c.lse.clone()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run()
    for _ in range(3):
        c.out.zero_()
        c.ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)
    # the captured call follows new lengths, tables and prefixes
    d = Case(**CASES["mixed"], seed=6)
    for x in ("q", "k", "v", "dt", "dcu", "dl", "dgp", "dp"):
        getattr(c, x).copy_(getattr(d, x))
    graph.replay()
    d.run().check()
    assert torch.equal(c.out, d.out)


def test_two_calls_at_once_on_two_streams():
    a, b = Case(**CASES["two_row_tiles"], seed=1), Case(**CASES["mixed"], seed=2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(stream=sa)
        b.run(stream=sb)
    a.check()
    b.check()


def test_no_lse_no_flags():
    c = Case(**CASES["decode"], seed=1)
    c.run(lse=None, flags=None)
    torch.cuda.synchronize()
    assert (c.lse == 9).all()
    c.run().check()


def test_bad_page_is_flagged_and_only_its_rows_suffer():
    c = Case([(None, [(1, 300), (1, 300), (1, 300)])], seed=2, poison=False)
    c.run().check()
    good = c.out.clone()
    c.dt[1, 2] = c.prob.num_pages
    c.run()
    torch.cuda.synchronize()
    assert c.flags.item() == 4
    assert torch.equal(c.out[0], good[0]) and torch.equal(c.out[2], good[2])


def test_bad_cu_writes_nothing():
    c = Case([(None, [(1, 30), (2, 30), (1, 30)])], seed=2)
    c.dcu.copy_(torch.tensor([0, 3, 1, 4]))
    c.run()
    torch.cuda.synchronize()
    assert c.flags.item() == 128 and (c.out == 9).all() and (c.lse == 9).all()
    c.dcu.copy_(torch.tensor([0, 1, 3, 5]))  # past total_q
    c.flags.zero_()
    c.run()
    assert c.flags.item() == 128 and (c.out == 9).all()


@pytest.mark.parametrize("gp", [[1, 0, 2], [0, 2, 4], [-1, 1, 2]])
def test_bad_groups_are_ignored(gp):
    c = Case([(128, [(1, 30), (1, 3)]), (64, [(2, 30)])], seed=2, poison=False)
    c.dt[1, :2] = c.dt[0, :2]
    c.run(groups=False).check()
    want = c.out.clone()
    c.dgp.copy_(torch.tensor(gp))
    c.run()
    torch.cuda.synchronize()
    assert c.flags.item() == 512 and torch.equal(c.out, want)


def test_bad_lengths_are_clamped_and_flagged():
    c = Case([(None, [(1, 64), (1, 64)])], seed=2, poison=False)
    c.dl.copy_(torch.tensor([10 ** 9, -3]))
    c.run()
    torch.cuda.synchronize()
    assert c.flags.item() == 16
    assert c.out[0].isfinite().all() and (c.out[1] == 0).all() and (c.lse[:, 1] == -math.inf).all()


def test_nan_of_a_key_reaches_the_rows_that_see_it():
    c = Case([(200, [(1, 90), (1, 70), (1, 60)])], seed=2)
    c.run().check()
    good = c.out.clone()
    page, off = (x[250] for x in c.slots[1])  # a key of the second sequence's own
    c.k[page, 1, off, 3] = float("nan")
    c.run()
    torch.cuda.synchronize()
    assert c.out[1, 8:].isnan().all() and c.lse[8:, 1].isnan().all()
    assert torch.equal(c.out[1, :8], good[1, :8])
    assert torch.equal(c.out[0], good[0]) and torch.equal(c.out[2], good[2])


def test_large_scores_raise_the_running_maximum():
    """Scores that grow along the keys by far more than 2^8: O is rescaled block by block."""
    c = Case([(2000, [(1, 500), (1, 300), (1, 1)])], seed=9, poison=False)
    for s in range(c.B):
        page, off = (x.cuda() for x in c.slots[s])
        ramp = (torch.arange(len(page), device="cuda") / 150.0).to(c.k.dtype)
        c.k[page, :, off, 0] = ramp[:, None].expand(-1, c.hkv)
    c.q[:, :, 0] = 60.0  # score += 60 / sqrt(128) * p / 150
    c.run().check()


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    r = np.random.RandomState(seed)
    hq, hkv = [(8, 1), (16, 2), (12, 4), (4, 4), (128, 1), (10, 2), (64, 8), (96, 1)][r.randint(8)]
    causal = bool(r.randint(2))

    def members(n, lo):
        return [(int(r.choice([0, 1, 1, 1, 2, r.randint(1, 70)])), int(r.choice([lo, lo + r.randint(0, 900)])))
                for _ in range(n)]

    groups = [(int(r.choice([0, 1, 127, 128, 129, r.randint(1, 5000)])), members(r.randint(1, 30), 0))
              for _ in range(r.randint(0, 4))]
    groups += [(None, members(r.randint(1, 9), 1))]
    Case(groups, hq=hq, hkv=hkv, q=["bf16", "fp16"][r.randint(2)], ps=[64, 128][r.randint(2)], causal=causal, seed=seed,
         lead=int(r.randint(3)), tail=int(r.randint(3))).run().check()


@pytest.mark.parametrize("ps", [64, 128])
def test_long_columns(ps):
    """Tiles of more blocks than a page window holds, columns that end in small tiles, both queues."""
    Case([(100000, [(40, 37 + 300 * i) for i in range(7)]), (None, [(1, 9000), (3, 50)])], hq=16, ps=ps, seed=5).run().check()
    Case([(None, [(1, 200000), (0, 10), (2, 513)])], hq=32, hkv=4, ps=ps, seed=6, tail=2).run().check()


def test_pages_past_two_to_the_31_elements():
    """A cache of 2^31 elements and more: the sequences' pages are its last ones."""
    c = Case([(300, [(1, 90), (2, 70)])], seed=3, poison=False, hkv=2)
    used, per = c.k.shape[0], c.k[0].numel()
    pages = (1 << 31) // per + used + 5
    big = [torch.empty(pages, *c.k.shape[1:], dtype=c.k.dtype, device="cuda") for _ in range(2)]
    for b, x in zip(big, (c.k, c.v)):
        b[pages - used:] = x
    c.k, c.v = big
    shift = pages - used
    c.dt = torch.where(c.dt >= 0, c.dt + shift, c.dt)
    c.slots = [(p + shift, o) for p, o in c.slots]
    c.prob.num_pages = pages
    c.run().check()


# --------------------------------------------------- the calls of a serving step
@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_a_step_of_all_three(kv):
    """One document prefilled, eight continuations decoded for three steps: norm_rope_store writes the cache
    (16-bit; or a quantised one, read back with load_kv into 16-bit pages), dense_shared_fwd attends."""
    t, hq, hkv, ps, P, n = torch.bfloat16, 16, 2, 64, 333, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)
    width = -(-(P + 3) // ps) + 1
    table = torch.arange(n * width, device="cuda", dtype=torch.int32).view(n, width)
    table[:, :P // ps] = table[0, :P // ps]
    # the page where the prefix ends is each sequence's own for its new keys, the first one's for the prefix
    pages = n * width
    shape = (pages, hkv, ps, 128)
    kvt = {"bf16": t, "fp8": torch.float8_e4m3fn, "nvfp4": "nvfp4"}[kv]
    if kv == "nvfp4":
        kc, vc = (torch.zeros(pages, hkv, ps * 72, dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.zeros(shape, device="cuda").to(kvt) for _ in range(2))
    k16, v16 = (kc, vc) if kv == "bf16" else (torch.zeros(shape, dtype=t, device="cuda") for _ in range(2))
    ang = torch.rand(P + 8, 32, generator=g, device="cuda") * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    qw, kw = 1 + 0.1 * rnd(128), 1 + 0.1 * rnd(128)
    sprob = mx.make_problem(1, 1, hq, hkv, 1, ps, pages, width, True, q_dtype=t, kv_dtype=kvt)
    aprob16 = mx.make_problem(1, 1, hq, hkv, 1, ps, pages, width, True, q_dtype=t)
    keys, vals = [], []  # per sequence, what its cache stands for, in float64

    def step(pos, loc, count):
        x = rnd(count, (hq + 2 * hkv) * 128)
        q = x[:, :hq * 128].unflatten(1, (hq, 128))
        k = x[:, hq * 128:(hq + hkv) * 128].unflatten(1, (hkv, 128))
        v = x[:, (hq + hkv) * 128:].unflatten(1, (hkv, 128))
        q_out = torch.empty(count, hq, 128, dtype=t, device="cuda")
        mx.norm_rope_store(sprob, pos, loc, cs, q, k, v, q_out, kc, vc, q_weight=qw, k_weight=kw)
        rows = [torch.empty(count, hkv, 128, dtype=t, device="cuda") for _ in range(2)]
        mx.load_kv(sprob, loc, kc, vc, *rows)
        if kv != "bf16":
            mx.store_kv(aprob16, loc, rows[0], rows[1], k16, v16)
        return q_out, rows[0].double(), rows[1].double()

    at = torch.arange(P, device="cuda")
    _, pk, pv = step(at, table[0, at // ps].long() * ps + at % ps, P)
    own = [[], []]
    for i in range(3):
        pos = torch.full((n,), P + i, device="cuda", dtype=torch.int64)
        q, k, v = step(pos, table[:, (P + i) // ps].long() * ps + (P + i) % ps, n)
        own[0].append(k)
        own[1].append(v)
        prob = mx.make_problem(n, n, hq, hkv, 1, ps, pages, width, True, q_dtype=t)
        out, lse = torch.empty_like(q), torch.empty(hq, n, device="cuda")
        ws = torch.empty(mx.dense_shared_workspace_size(prob), dtype=torch.uint8, device="cuda")
        dev = lambda x, dt: torch.tensor(x, dtype=dt, device="cuda")
        mx.dense_shared_fwd(prob, q, k16, v16, table, dev(list(range(n + 1)), torch.int64),
                            dev([P + i + 1] * n, torch.int32), dev([0, n], torch.int32), dev([P], torch.int32), ws, out,
                            lse)
        for s in range(n):
            K = torch.cat([pk] + [x[s:s + 1] for x in own[0]])
            V = torch.cat([pv] + [x[s:s + 1] for x in own[1]])
            x = torch.einsum("grd,pgd->grp", q[s].double().view(hkv, -1, 128), K) * 128 ** -0.5
            p = torch.softmax(x, -1)
            o, A = (torch.einsum("grp,pgd->grd", p, y).reshape(hq, 128) for y in (V, V.abs()))
            tol = U["bf16"] * (o.abs() + A) * 1.01 + 6.2e-4 * A
            assert ((out[s].double() - o).abs() <= tol).all()
            assert ((lse[:, s].double() - torch.logsumexp(x, -1).reshape(hq)).abs() <= 1e-3).all()
