"""What mxsa_norm_rope_store promises at its edges (slots that occur twice,
NaN in an FP8 cache), and the sparse path behind it: its index queries and
index cache through the selection into the attention."""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from tests.test_gpu_norm_rope import TDT, call, case

pytestmark = pytest.mark.gpu


def raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu()


@pytest.mark.parametrize("kv,inter,idx", [("bf16", False, 64), ("fp8", True, 128), ("fp8", False, 64),
                                          ("nvfp4", False, 0)])
def test_slots_that_occur_twice(kv, inter, idx):
    """Tokens in pairs of one slot: every value (NVFP4: every byte) there is one of the pair's, the rest stays."""
    n = 300
    c = case(n, 16, 4, "bf16", kv, 64, 64, inter=inter, idx=idx, seed=3)
    c["loc"][1::2] = c["loc"][::2]
    caches = ["kc", "vc"] + (["ic"] if idx else [])
    before = {k: c[k].clone() for k in caches}
    pos, alone = c["pos"].clone(), []
    for parity in range(2):  # the pair's other token left out as padding
        for k in caches:
            c[k].copy_(before[k])
        c["pos"] = torch.where(torch.arange(n, device="cuda") % 2 == parity, pos, -1)
        call(c)
        alone.append({k: raw(c[k]) for k in caches})
    for k in caches:
        c[k].copy_(before[k])
    c["pos"] = pos
    call(c)
    torch.cuda.synchronize()
    for k in caches:
        got = raw(c[k])
        assert ((got == alone[0][k]) | (got == alone[1][k])).all(), k
        same = (alone[0][k] == raw(before[k])) & (alone[1][k] == raw(before[k]))
        assert torch.equal(got[same], raw(before[k])[same]), k


@pytest.mark.parametrize("q,inter", [("bf16", False), ("fp16", True)])
def test_nan_of_a_key_row_in_an_fp8_cache(q, inter):
    """NaN of either sign, normed and not, rotated and not: code 0x7F; V keeps the sign, as mxsa_store_kv does."""
    for weights in (True, False):
        c = case(8, 4, 2, q, "fp8", 64, 32, inter=inter, weights=weights, packed=False, idx=64, seed=7)
        bits = c["k"].view(torch.int16)
        for t, (col, word) in enumerate([(100, 0x7FFF), (100, -1), (3, 0x7FFF), (3, -1)]):
            bits[t, 1, col] = word
            c["v"].view(torch.int16)[t, 0, col] = word
            c["ik"].view(torch.int16)[t, 1, col % 64] = word
        call(c)
        torch.cuda.synchronize()
        page, off = c["loc"].cpu() // 64, c["loc"].cpu() % 64
        kc, vc, ic = (raw(c[k])[page, :, off] for k in ("kc", "vc", "ic"))
        for t, col in enumerate([100, 100, 3, 3]):
            assert kc[t, 1, col] == 0x7F and ic[t, 1, col % 64] == 0x7F
            assert vc[t, 0, col] == (0x7F if t % 2 == 0 else 0xFF)
        assert not (kc[4:] & 0x7F == 0x7F).any() and not (kc[:, 0] & 0x7F == 0x7F).any()


@pytest.mark.parametrize("kv,idx", [("bf16", 128), ("fp8", 64), ("fp8", 128)])
def test_prologue_selection_attention(kv, idx):
    """A prompt chunk of two sequences and a decode token of a third: norm_rope_store writes the caches and the index
    queries, select_blocks picks blocks from them, the sparse attention reads those.  The selection is compared with
    the oracle's on the rows as written, the attention with the definition in 64 bits over the selected blocks."""
    import oracle
    from block_sparse_attention_builder_gb300 import workloads as W

    dev, hq, hkv, ps, topk = "cuda", 16, 2, 64, 4
    tq, lens = [40, 300, 1], [700, 1300, 2111]
    n, B = sum(tq), len(tq)
    w = W.custom(f"prologue_{kv}_{idx}", tq, lens, hq, hkv, ps, topk, True, "uniform", 5, q_dtype="bf16", kv_dtype=kv)
    g = torch.Generator(device=dev).manual_seed(idx)
    t, kvt = torch.bfloat16, TDT[kv]
    pages, width = w.num_pages, w.max_pages_per_seq
    prob = mx.make_problem(B, n, hq, hkv, topk, ps, pages, width, True, q_dtype=t, kv_dtype=kvt)
    table = torch.from_numpy(w.block_tables).to(dev)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(tq)]), dtype=torch.int64, device=dev)
    used = torch.tensor(lens, dtype=torch.int32, device=dev)
    cache = lambda d: (torch.randn(pages, hkv, ps, d, generator=g, device=dev)).to(kvt)
    kc, vc, ic = cache(128), cache(128), cache(idx)
    x = torch.randn(n, (hq + 2 * hkv) * 128 + 2 * hkv * idx, generator=g, device=dev).to(t)
    cut = np.cumsum([0, hq * 128, hkv * 128, hkv * 128, hkv * idx, hkv * idx])
    q, k, v, iq, ik = (x[:, a:b].unflatten(1, (-1, d)) for a, b, d in zip(cut, cut[1:], (128, 128, 128, idx, idx)))
    seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(tq, device=dev))
    pos = used.long()[seq] - (cu[1:][seq] - torch.arange(n, device=dev))  # the last tq positions of each sequence
    loc = table[seq, pos // ps].long() * ps + pos % ps
    ang = torch.rand(max(lens), idx // 2, generator=g, device=dev) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    q_out, iq_out = torch.empty(n, hq, 128, dtype=t, device=dev), torch.empty(n, hkv, idx, dtype=kvt, device=dev)
    wt = lambda d: (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(t)
    qw, kw, iqw, ikw = wt(128), wt(128), wt(idx), wt(idx)
    flags = torch.zeros(1, dtype=torch.int32, device=dev)
    mx.norm_rope_store(prob, pos, loc, cs, q, k, v, q_out, kc, vc, q_weight=qw, k_weight=kw, idx_q=iq, idx_k=ik,
                       idx_q_weight=iqw, idx_k_weight=ikw, idx_q_out=iq_out, idx_cache=ic, flags=flags)
    sel, _ = mx.select_blocks(prob, iq_out, ic, table, cu, used, flags=flags)
    out, lse = mx.kvouter_attention(q_out, kc, vc, sel, table, cu, used, ps, causal=True, return_lse=True)
    torch.cuda.synchronize()
    assert flags.item() == 0
    # the selection: the oracle's, an integer decision on the rows that the store wrote
    want = oracle.select_blocks(oracle.problem_for(w), idx, iq_out.cpu(), ic.cpu(), w.block_tables, cu.cpu().numpy(),
                                used.cpu().numpy())
    assert np.array_equal(sel.cpu().numpy(), want)
    # the attention: 16-bit weights and rows (2^-8 each), FP32 sums far below that, partials in 16 bits (2^-8 of A)
    G = hq // hkv
    for s in range(B):
        L, a, b = lens[s], int(cu[s]), int(cu[s + 1])
        p = torch.arange(L, device=dev)
        rows = lambda c: c.float()[table[s, p // ps].long(), :, p % ps].double()  # [L, hkv, 128]
        K, V = rows(kc), rows(vc)
        x = torch.einsum("tgrd,pgd->tgrp", q_out[a:b].double().view(b - a, hkv, G, 128), K) / math.sqrt(128)
        block = (sel[a:b, :, :, None] == (p // 128)[None, None, None]).any(2)  # [t, hkv, L]
        see = block & (p[None, None] <= pos[a:b, None, None])
        x.masked_fill_(~see[:, :, None], -math.inf)
        P = torch.softmax(x, -1)
        o, A = (torch.einsum("tgrp,pgd->tgrd", P, y).reshape(b - a, hq, 128) for y in (V, V.abs()))
        tol = 2.0 ** -8 * (o.abs() + 2 * A) * 1.01 + 6.2e-4 * A
        assert ((out[a:b].double() - o).abs() <= tol).all()
        assert ((lse[:, a:b].T.double() - torch.logsumexp(x, -1).reshape(b - a, hq)).abs() <= 2e-3).all()
