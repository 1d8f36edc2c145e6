"""mxsa_prompt_fwd on the GPU against the definition in 64 bits.

Tolerance of an output element, with u half a step of the 16-bit type
(bf16 2^-8, fp16 2^-11) and A = sum p |v| of the row and column: the softmax
weights are rounded (u A), the result is rounded (u |ref|), FP32 sums of 128
products change a score by at most 128 * 2^-24 of its magnitudes' sum M (the
largest of the case), which is twice that in p / l, and fp16 weights below
2^-14 lose up to 2^-25 each, n keys of weights whose sum is at least 1 in the
same units.  lse: the scores' error and a few FP32 steps of its size.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


class Prompts:
    def __init__(self, lens, hq=16, hkv=2, q="bf16", causal=True, seed=0, lead=0, tail=0, packed=True, scale=0.0,
                 grow=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = TDT[q]
        self.qn, self.lens, self.hq, self.hkv, self.causal = q, lens, hq, hkv, causal
        self.scale = scale or 128 ** -0.5
        self.cu = [lead]
        for n in lens:
            self.cu.append(self.cu[-1] + n)
        self.total = self.cu[-1] + tail
        rows = torch.randn(self.total, hq + 2 * hkv, 128, device="cuda", generator=g)
        rows[:, :hq] *= 2
        if grow:  # scores that grow along the keys: the running maximum is passed again and again
            at = torch.arange(self.total, device="cuda")[:, None, None]
            rows[:, :hq] = rows[:, :hq].abs()
            rows[:, hq:hq + hkv] = (rows[:, hq:hq + hkv] * 0.1 + 1) * (at * grow)
        for a, b in ((0, lead), (self.cu[-1], self.total)):  # tokens of no sequence
            rows[a:b] = float("nan")
        if packed:
            flat = rows.to(t).reshape(self.total, -1)
            cut = lambda a, n: flat[:, a * 128:(a + n) * 128].unflatten(1, (n, 128))
        else:
            cut = lambda a, n: rows[:, a:a + n].to(t).contiguous()
        self.q, self.k, self.v = cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)
        self.prob = mx.make_problem(len(lens), self.total, hq, hkv, 0, 64, 0, 0, causal, scale, q_dtype=t)
        self.ws = torch.full((mx.prompt_workspace_size(self.prob),), 0xFF, dtype=torch.uint8, device="cuda")
        self.dcu = torch.tensor(self.cu, dtype=torch.int64, device="cuda")
        self.out = torch.full((self.total, hq, 128), 9.0, dtype=t, device="cuda")
        self.lse = torch.full((hq, self.total), 9.0, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        a = dict(ws=self.ws, out=self.out, lse=self.lse, flags=self.flags)
        a.update(kw)
        mx.prompt_fwd(self.prob, self.q, self.k, self.v, self.dcu, **a)
        return self

    def check(self, flags=0, seqs=None):
        torch.cuda.synchronize()
        assert self.flags.item() == flags
        u = U[self.qn]
        for s in range(len(self.lens)) if seqs is None else seqs:
            lo, hi = self.cu[s], self.cu[s + 1]
            for a in range(lo, hi, 512):
                b = min(hi, a + 512)
                end = b if self.causal else hi
                q = self.q[a:b].double().view(b - a, self.hkv, -1, 128)
                k, v = self.k[lo:end].double(), self.v[lo:end].double()
                x = torch.einsum("tgrd,pgd->tgrp", q, k) * self.scale
                mag = (torch.einsum("tgrd,pgd->tgrp", q.abs(), k.abs()) * self.scale).max().item()
                if self.causal:
                    late = torch.arange(lo, end, device="cuda")[None] > torch.arange(a, b, device="cuda")[:, None]
                    x.masked_fill_(late[:, None, None], -math.inf)
                lse = torch.logsumexp(x, -1)
                p = torch.exp(x - lse[..., None])
                o = torch.einsum("tgrp,pgd->tgrd", p, v).reshape(b - a, self.hq, 128)
                A = torch.einsum("tgrp,pgd->tgrd", p, v.abs()).reshape(b - a, self.hq, 128)
                got, gl = self.out[a:b].double(), self.lse[:, a:b].T.double()
                score = 128 * 2.0 ** -24 * max(mag, 1.0)
                small = (end - lo) * 2.0 ** -25 * 5 if self.qn == "fp16" else 0.0
                bad = ~((got - o).abs() <= u * (o.abs() + A) * 1.01 + (2 * score + 1e-5) * A + small)
                assert not bad.any(), f"seq {s}, {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"
                lse = lse.reshape(b - a, self.hq)
                assert ((gl - lse).abs() <= 2 * score + 1e-5 + 4e-7 * lse.abs()).all()
        for a, b in ((0, self.cu[0]), (self.cu[-1], self.total)):  # tokens of no sequence
            assert (self.out[a:b] == 9).all() and (self.lse[:, a:b] == 9).all()
        return self


def rand(n, lo, hi, seed):
    return [int(x) for x in np.random.RandomState(seed).randint(lo, hi + 1, n)]


CASES = {
    "one_token": dict(lens=[1]),
    "two_tokens_mha": dict(lens=[2], hq=3, hkv=3, q="fp16"),
    "block": dict(lens=[128]),
    "past_a_block": dict(lens=[129], hq=12, hkv=4, q="fp16"),
    "half_tile_edges": dict(lens=[15, 16, 17, 31, 32, 33, 64]),
    "empty_between": dict(lens=[0, 5, 0, 0, 300, 0], lead=3, tail=70),
    "g1": dict(lens=[100, 127, 128, 129, 255, 256, 257, 600], hq=2, hkv=2),
    "g5": dict(lens=[37, 501, 1], hq=10, hkv=2, q="fp16"),
    "g128": dict(lens=[3, 130, 1], hq=128, hkv=1),
    "g48": dict(lens=[90, 300], hq=96, hkv=2, packed=False),
    "full": dict(lens=[1, 200, 129, 777], causal=False),
    "full_fp16": dict(lens=[1000, 3], causal=False, q="fp16", hq=12, hkv=4, packed=False),
    # more tiles than CTAs: the plan's order
    "many": dict(lens=rand(60, 1, 700, 1), hq=16, hkv=4, lead=2, tail=5),
    "many_full": dict(lens=rand(40, 1, 500, 2), hq=16, hkv=4, causal=False, q="fp16"),
    "seqs_1024": dict(lens=rand(1024, 0, 9, 3), hq=8, hkv=1, tail=1),
    # tiles of one half, which the groups take in turn
    "one_half_each": dict(lens=rand(300, 0, 128, 4), hq=4, hkv=4, lead=1),
    "one_half_now_and_then": dict(lens=rand(150, 1, 90, 5), hq=12, hkv=4, q="fp16", causal=False, tail=2),
    "long": dict(lens=[5000, 77], hq=16, hkv=2),
    "scaled": dict(lens=[400], scale=0.03),
    # the running maximum is raised in most blocks (P made twice)
    "growing": dict(lens=[900, 1500], grow=0.004),
    "growing_fp16": dict(lens=[2100], grow=0.003, q="fp16", causal=False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    Prompts(seed=len(name), **CASES[name]).run().check()


# how far the scores of each 64 keys lie above those of the first ones (log2 units): below what raises the reference,
# in the first half of a block, in its second half below and past what may stay, far down, far up, and a first key
# above all others
STEPS = [0, 3, 5, 5, 5, 11, 11, 17, 17, 40, 40, 12, 200, 200, 150, 206, 215, 215, 226, -300, 226, 231, 226]


@pytest.mark.parametrize("q,sink", [("bf16", 0), ("fp16", 0), ("fp16", 240), ("bf16", 240)])
@pytest.mark.parametrize("causal", [False, True])
def test_scores_in_steps(q, sink, causal):
    n = 64 * len(STEPS) - 10
    p = Prompts([n], hq=12, hkv=4, q=q, causal=causal, seed=15, packed=False)
    up = torch.tensor(STEPS, dtype=torch.float32, device="cuda").repeat_interleave(64)[:n]
    up[0] = sink
    p.q.mul_(0.25)
    p.q[..., 0] = 16
    p.k[..., 0] = (up * math.log(2) / (16 * p.scale))[:, None].to(p.k.dtype)
    p.run().check()


def test_rows_that_are_no_tokens_change_no_bits():
    """Three heads to a kv head leave two rows of a half without a query: whatever stands there."""
    p = Prompts([700, 41, 130], hq=12, hkv=4, seed=16)
    p.run().check()
    want, lse = p.out.clone(), p.lse.clone()
    for size in (1e-3, 300.0, float("inf")):
        other = Prompts([900] * 3, hq=16, hkv=4, seed=17, packed=False)
        other.q.copy_(torch.full_like(other.q, size))
        other.run()
        p.out.fill_(9)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.out, want) and torch.equal(p.lse, lse)


def test_without_lse_and_flags_and_on_a_given_stream():
    p = Prompts([300, 20], seed=5).run()
    torch.cuda.synchronize()
    want = p.out.clone()
    p.out.fill_(9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.run(lse=None, flags=None, stream=s)
    s.synchronize()
    assert torch.equal(p.out, want)


def test_the_same_call_gives_the_same_bits():
    p = Prompts(rand(50, 1, 600, 9), hq=32, hkv=4, seed=6).run()
    torch.cuda.synchronize()
    out, lse = p.out.clone(), p.lse.clone()
    for _ in range(5):
        p.out.fill_(9)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


def test_two_calls_at_once_with_a_workspace_each():
    a, b = Prompts(rand(40, 1, 500, 11), hkv=4, seed=7), Prompts(rand(30, 1, 900, 12), hkv=2, seed=8)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(stream=s[0])
        b.run(stream=s[1])
    a.check()
    b.check()


def test_captured_and_replayed_with_other_lengths():
    p = Prompts([500, 400, 300], hkv=4, seed=9)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for cu in ([0, 1, 700, 1200], [0, 0, 1150, 1200], [0, 400, 800, 1200]):
        p.cu, p.lens = cu, [y - x for x, y in zip(cu, cu[1:])]
        p.dcu.copy_(torch.tensor(cu))
        p.out.fill_(9)
        g.replay()
        p.check()


def test_nan_of_one_sequence_stays_there():
    p = Prompts([200, 130, 77, 300], hq=12, hkv=4, seed=10)
    a, b = p.cu[1], p.cu[2]
    for t in (p.q, p.k, p.v):
        t[a:b] = float("nan")
    p.run().check(seqs=[0, 2, 3])
    p.v[a:b] = float("inf")
    p.run().check(seqs=[0, 2, 3])


def test_nan_and_infinite_keys_behind_a_row_do_not_reach_it():
    p = Prompts([300], hq=8, hkv=2, seed=11)
    p.k[200:] = float("nan")
    p.k[250:] = float("inf")
    p.run()
    torch.cuda.synchronize()
    got = p.out[:200].clone()
    q = Prompts([300], hq=8, hkv=2, seed=11)
    q.run().check()
    assert torch.equal(got, q.out[:200])


def test_bad_starts_are_flagged_and_nothing_is_written():
    for cu in ([0, 200, 100, 300], [0, 100, 200, 301], [-1, 100, 200, 300]):
        for hkv in (2, 16):  # without and with a plan
            p = Prompts([100, 100, 100], hq=16, hkv=hkv)
            if hkv == 16:
                p = Prompts([700, 700, 700], hq=128, hkv=16)
                cu = [c * 7 for c in cu]
            p.dcu.copy_(torch.tensor(cu))
            p.run()
            torch.cuda.synchronize()
            assert p.flags.item() == 128
            assert (p.out == 9).all() and (p.lse == 9).all()


def test_no_tokens():
    p = mx.make_problem(2, 0, 8, 2, 1, 64, 1, 1, True)
    ws = torch.empty(mx.prompt_workspace_size(p), dtype=torch.uint8, device="cuda")
    e = lambda h: torch.empty(0, h, 128, dtype=torch.bfloat16, device="cuda")
    mx.prompt_fwd(p, e(8), e(2), e(2), torch.zeros(3, dtype=torch.int64, device="cuda"), ws, e(8))
    torch.cuda.synchronize()


def test_equals_the_paged_path():
    """The same prompts through a cache and dense_fwd: both within their roundings."""
    p = Prompts([300, 129, 64], hq=16, hkv=2, seed=12).run()
    ps, pages = 64, 5 + 3 + 1
    loc = torch.cat([torch.arange(n) + 64 * a for n, a in ((300, 0), (129, 5), (64, 8))]).cuda()
    prob = mx.make_problem(3, p.total, 16, 2, 1, ps, pages, 5, True)
    kc, vc = (torch.zeros(pages, 2, ps, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mx.store_kv(prob, loc, p.k.contiguous(), p.v.contiguous(), kc, vc)
    bt = torch.tensor([[0, 1, 2, 3, 4], [5, 6, 7, -1, -1], [8, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(p.out)
    mx.dense_fwd(prob, p.q.contiguous(), kc, vc, bt, p.dcu, torch.tensor(p.lens, dtype=torch.int32, device="cuda"), out)
    p.check()
    # (each within u (|o| + A) of the definition, A <= 4.5 sigma of V here)
    assert ((out.double() - p.out.double()).abs() <= 2 * 2.0 ** -8 * (p.out.double().abs() + 4.5)).all()


def test_strides_of_their_own_and_sixteen_byte_offsets():
    """q, k, v and out that begin at any 16 bytes, each with another distance between its tokens."""
    a = Prompts([150, 37, 300], hq=12, hkv=4, q="fp16", seed=13, packed=False)
    a.run().check()
    want = a.out.clone()
    for t, pad in (("q", 8), ("k", 24), ("v", 128)):
        x = getattr(a, t)
        n, h, _ = x.shape
        flat = torch.full((n * (h * 128 + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = flat[8:].view(n, h * 128 + pad)[:, :h * 128].unflatten(1, (h, 128))
        view.copy_(x)
        setattr(a, t, view)
    flat = torch.full((a.out.numel() + 16,), 9.0, dtype=a.out.dtype, device="cuda")
    out = flat[8:-8].view_as(a.out)
    a.run(out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (flat[:8] == 9).all() and (flat[-8:] == 9).all()


def test_rows_past_two_to_the_31_elements():
    """More than 2^31 elements of q and out: many short prompts, the last ones checked."""
    p = Prompts([270] * 1000, hq=64, hkv=4, seed=14)
    assert p.out.numel() > 2 ** 31 and p.q.numel() > 2 ** 31
    p.run().check(seqs=[0, 499, 998, 999])
