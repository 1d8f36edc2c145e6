"""The workspace of mxsa_dense_shared_fwd: its layout, restated, is what the
library asks for; every plan fits it; and it grows with the rows that can
exist, not with four of each.

Partial rows: a tile of two halves has one for each of its rows, a tile of one
half (the last row tile of a job, at most T tokens) two.  A token lies in at
most two jobs, its group's prefix and its sequence's own keys; without a second
sequence there is no prefix.
"""
import random

import pytest

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B
from tests.test_shared_models import MAXC, PER_CTA, cdiv, plan, random_problem


def layout(prob):
    """Byte offsets and bounds of the workspace."""
    G, hkv, seqs, tq = prob.num_q_heads // prob.num_kv_heads, prob.num_kv_heads, prob.num_seqs, prob.total_q
    T = 128 // G
    triples = hkv * (2 * (tq // (2 * T)) + 2 * seqs)
    blocks = cdiv(prob.max_pages_per_seq * prob.page_size, 128)
    by_cost = PER_CTA * 2 * MAXC
    extra = min(by_cost, triples * (blocks - 1))
    L = dict(tile_cap=triples + extra)
    ways = 2 if seqs > 1 else 1
    jobs = seqs + seqs // 2
    L["row_cap"] = hkv * (ways * tq * G + min(ways * tq * G, jobs * T * G)) + min(256, 2 * tq * G) * extra
    o = 0
    for name, n in (("hdr", 24), ("tok", 32 * tq), ("pieces", 16 * L["tile_cap"]), ("queue", 96 * L["tile_cap"]),
                    ("part_o", 512 * L["row_cap"]), ("part_lse", 4 * L["row_cap"])):
        L[name] = o
        o = cdiv(o + n, 256) * 256
    L["total"] = o
    return L


def problem_of(p, ps=64):
    """The problem of a batch as random_problem makes them."""
    width = max(1, cdiv(max(p["lens"]), ps))
    return mx.make_problem(len(p["lens"]), p["total_q"], p["hq"], p["hkv"], 1, ps, max(1, width), width, p["causal"])


def crowded(r):
    """Many jobs with a short last row tile: sequences of one token, of one half and one more, in groups of two."""
    hq, hkv = r.choice([(8, 1), (16, 2), (12, 4), (4, 4), (128, 1), (96, 1), (10, 2)])
    T = 128 // (hq // hkv)
    n = r.choice([2, 3, 16, 101])
    tq = [r.choice([1, 1, T, T + 1, 2 * T, 2 * T + 1, 3 * T]) for _ in range(n)]
    cu = [0]
    for x in tq:
        cu.append(cu[-1] + x)
    ng = n // 2
    return dict(hq=hq, hkv=hkv, cu=cu, lens=[r.choice([700, 129, 1, r.randint(100, 20000)]) for _ in range(n)],
                gp=[2 * j for j in range(ng + 1)], prefix=[r.choice([64, 100, 600, 3000]) for _ in range(ng)],
                causal=r.random() < 0.5, ctas=r.choice([1, 148, 152, 160]), total_q=cu[-1])


@pytest.mark.parametrize("seed", range(60))
def test_every_plan_fits(seed):
    B.build()
    r = random.Random(seed)
    for p in (random_problem(r), crowded(r), crowded(r)):
        prob = problem_of(p)
        L = layout(prob)
        assert L["total"] == mx.dense_shared_workspace_size(prob)
        tiles, part = plan(p)
        assert len(tiles) <= L["tile_cap"] and part <= L["row_cap"]


def test_size_of_a_prompt():
    """8192 new tokens of 64 heads: an output of 134 MB.  Two sequences: each row once per job and the chunks' bound."""
    B.build()
    size = lambda seqs: mx.dense_shared_workspace_size(mx.make_problem(seqs, 8192, 64, 8, 1, 64, 1024, 512))
    rows, chunks = 8192 * 64 * 516, 640 * 256 * 516
    assert size(1) < 1.01 * (rows + chunks)
    assert size(2) < 1.01 * (2 * rows + chunks)
    assert size(64) < 1.1 * (2 * rows + chunks)
