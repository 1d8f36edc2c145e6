"""mxsa_norm_rope_store and mxsa_load_kv on the GPU against plain statements
in 64 bits, and the two with the attention calls they serve.

Tolerances: a row's FP32 arithmetic (a sum of 128 squares as a tree of fused
adds, a root, four products and one sum) is off by less than 16 * 2^-24 of
the row's largest normed value, far below the one rounding to the output
type, at most eps / 2 of the value (bf16 2^-8, fp16 2^-11, e4m3 2^-4, with
half the smallest subnormal step next to zero).
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def rope_ref(x, w, cs, inter, eps):
    """[n, heads, D] in float64 from the formula, on the CPU."""
    x = x.double().cpu()
    y = x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    half = cs.shape[1] // 2
    cs = cs.double().cpu()[:, None]
    c, s = cs[..., :half], cs[..., half:]
    y = y.clone()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    ya, yb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def check(got, ref, dt, what):
    got = got.float().double().cpu()
    half, tiny = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25),
                  "fp8": (2.0 ** -4, 2.0 ** -10)}[dt]
    if dt == "fp8":
        ref = ref.clamp(-448, 448)
    slack = 16 * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True)
    bad = (got - ref).abs() > (half * ref.abs()).clamp(min=tiny) + slack * (1 + half)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def fp4_values(cache, ps):
    """[pages, heads, ps, 128] float64 of an NVFP4 cache's bytes, and the scales' values."""
    cache = cache.cpu()
    pages, heads = cache.shape[:2]
    code = cache[:, :, :ps * 64].reshape(pages, heads, ps, 64).long()
    sc = cache[:, :, ps * 64:].contiguous().view(torch.float8_e4m3fn).float().double().reshape(pages, heads, ps, 8)
    nib = torch.stack([code & 15, code >> 4], -1).reshape(pages, heads, ps, 128)
    v = GRID[nib & 7] * torch.where(nib >= 8, -1.0, 1.0).double()
    return v * sc.repeat_interleave(16, -1), sc


def case(n, hq, hkv, q, kv, ps, rot, inter=False, per_head=False, idx=0, weights=True, positions=500, packed=True,
         seed=0, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    t = TDT[q]
    rnd = lambda *s, k=scale: (torch.randn(*s, generator=g) * k).to(t).cuda()
    c = dict(n=n, hq=hq, hkv=hkv, qn=q, kvn=kv, ps=ps, rot=rot, inter=inter, idx=idx, eps=1e-5)
    if packed:
        x = rnd(n, (hq + 2 * hkv) * 128 + 8)  # a token's row is longer than its heads
        c["q"] = x[:, :hq * 128].unflatten(1, (hq, 128))
        c["k"] = x[:, hq * 128:(hq + hkv) * 128].unflatten(1, (hkv, 128))
        c["v"] = x[:, (hq + hkv) * 128:(hq + 2 * hkv) * 128].unflatten(1, (hkv, 128))
    else:
        c["q"], c["k"], c["v"] = rnd(n, hq, 128), rnd(n, hkv, 128), rnd(n, hkv, 128)
    w = lambda h, d: (1 + rnd(*((h, d) if per_head else (d,)), k=0.2)) if weights else None
    c["qw"], c["kw"] = w(hq, 128), w(hkv, 128)
    pages = -(-n // ps) + 1
    c["pages"] = pages
    c["loc"] = torch.randperm(pages * ps, generator=g)[:n].cuda()
    c["pos"] = torch.randint(0, positions, (n,), generator=g).cuda()
    ang = torch.rand(positions, rot // 2, generator=g, dtype=torch.float64) * 6.3
    c["cs"] = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    c["kc"], c["vc"] = new_cache(c, hkv, 128, g), new_cache(c, hkv, 128, g)
    c["q_out"] = torch.full((n, hq, 128), 7.0, dtype=t, device="cuda")
    if idx:
        c["iq"], c["ik"] = rnd(n, hkv, idx), rnd(n, hkv, idx)
        c["iqw"], c["ikw"] = w(hkv, idx), w(hkv, idx)
        c["ic"] = new_cache(c, hkv, idx, g)
        c["iq_out"] = torch.zeros(n, hkv, idx, device="cuda").to(TDT[kv])
    c["prob"] = mx.make_problem(1, n, hq, hkv, 1, ps, pages, pages, False, q_dtype=t,
                                kv_dtype="nvfp4" if kv == "nvfp4" else TDT[kv])
    return c


def new_cache(c, heads, dim, g):
    pages, ps, kv = c["pages"], c["ps"], c["kvn"]
    if kv == "nvfp4":
        return torch.randint(0, 0x38, (pages, heads, ps * 72), generator=g, dtype=torch.uint8).cuda()
    return torch.randn(pages, heads, ps, dim, generator=g).to(TDT[kv]).cuda()


def call(c, **kw):
    idx = dict(idx_q=c["iq"], idx_k=c["ik"], idx_q_weight=c["iqw"], idx_k_weight=c["ikw"], idx_q_out=c["iq_out"],
               idx_cache=c["ic"]) if c["idx"] else {}
    mx.norm_rope_store(c["prob"], c["pos"], c["loc"], c["cs"], c["q"], c["k"], c["v"], c["q_out"], c["kc"], c["vc"],
                       q_weight=c["qw"], k_weight=c["kw"], eps=c["eps"], interleaved=c["inter"], **idx, **kw)


def by_slot(cache):
    """[slots, heads, dim] of a cache [pages, heads, ps, dim], as its bits."""
    b = cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16).cpu()
    return b.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])


CASES = {
    "one_token": dict(n=1, hq=16, hkv=2, q="bf16", kv="bf16", ps=64, rot=128),
    "bf16_partial": dict(n=37, hq=64, hkv=8, q="bf16", kv="bf16", ps=128, rot=64, idx=128),
    "fp16_fp8_inter": dict(n=133, hq=12, hkv=4, q="fp16", kv="fp8", ps=64, rot=96, inter=True, per_head=True),
    "bf16_fp8_idx64": dict(n=70, hq=10, hkv=5, q="bf16", kv="fp8", ps=128, rot=48, per_head=True, idx=64),
    "rot16_no_norm": dict(n=9, hq=3, hkv=1, q="fp16", kv="fp16", ps=64, rot=16, weights=False, idx=64),
    "rot112_dense": dict(n=65, hq=128, hkv=1, q="bf16", kv="fp8", ps=64, rot=112, packed=False),
    "inter_idx64": dict(n=40, hq=7, hkv=7, q="bf16", kv="bf16", ps=64, rot=64, inter=True, idx=64),
    "fp16_fp8_plain": dict(n=300, hq=16, hkv=2, q="fp16", kv="fp8", ps=128, rot=128, idx=128),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_formula(name):
    c = case(**CASES[name], seed=len(name))
    before = {k: by_slot(c[k]) for k in ("kc", "vc") + (("ic",) if c["idx"] else ())}
    call(c)
    torch.cuda.synchronize()
    cs = c["cs"][c["pos"]]
    check(c["q_out"], rope_ref(c["q"], c["qw"], cs, c["inter"], c["eps"]), c["qn"], "q_out")
    loc = c["loc"].cpu()
    rest = torch.ones(c["pages"] * c["ps"], dtype=torch.bool)
    rest[loc] = False

    def rows(cache):
        return cache.float().transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[c["loc"]]

    check(rows(c["kc"]), rope_ref(c["k"], c["kw"], cs, c["inter"], c["eps"]), c["kvn"], "k")
    # V is exactly the store's cast
    v = c["v"].float()
    v = (v.clamp(-448, 448) if c["kvn"] == "fp8" else v).to(c["vc"].dtype)
    bits = torch.uint8 if v.element_size() == 1 else torch.int16
    assert torch.equal(by_slot(c["vc"])[loc], v.view(bits).cpu())
    if c["idx"]:
        check(c["iq_out"], rope_ref(c["iq"], c["iqw"], cs, c["inter"], c["eps"]), c["kvn"], "idx_q")
        check(rows(c["ic"]), rope_ref(c["ik"], c["ikw"], cs, c["inter"], c["eps"]), c["kvn"], "idx_k")
    for k, b in before.items():  # the other slots are as they were
        assert torch.equal(by_slot(c[k])[rest], b[rest]), k


@pytest.mark.parametrize("q,inter", [("bf16", False), ("fp16", True)])
def test_nvfp4_cache(q, inter):
    c = case(90, 15, 3, q, "nvfp4", 64, 64, inter=inter, seed=5)
    call(c)
    torch.cuda.synchronize()
    page, off = c["loc"].cpu() // 64, c["loc"].cpu() % 64
    cs = c["cs"][c["pos"]]
    for cache, ref, exact in ((c["kc"], rope_ref(c["k"], c["kw"], cs, inter, c["eps"]), False),
                              (c["vc"], c["v"].double().cpu(), True)):
        got, sc = fp4_values(cache, 64)
        got, sc = got[page, :, off], sc[page, :, off].repeat_interleave(16, -1)
        amax = ref.reshape(90, 3, 8, 16).abs().amax(-1).repeat_interleave(16, -1)
        # the scale: e4m3 of amax / 6, half a step (2^-4) off at most
        assert ((sc - amax / 6).abs() <= 2.0 ** -4 * amax / 6 * (1 + 1e-5) + 2.0 ** -10).all()
        # each value: at most half the widest gap of the grid (4..6: 1) off in units of its scale, or cut off at 6
        # where amax / 6 was rounded down (6 * 2^-4 of the scale, less than half a gap too)
        assert ((got - ref).abs() <= sc * (1 + 1e-5) + 1e-6).all()
        y = (ref / sc.clamp(min=2.0 ** -9)).abs()
        # ties go to the even code; a tie times a scale has at most 7 significant bits, so bf16 rows hit them
        odd = torch.arange(8) % 2 * 1e-12
        near = (GRID[((y[..., None] - GRID).abs() + odd).argmin(-1)] * torch.sign(ref) * sc)
        flip = (near - got).abs() > 1e-9
        assert flip.double().mean() < (1e-9 if exact else 1e-3)
    # V's bytes are the store's
    kc, vc = torch.zeros_like(c["kc"]), torch.zeros_like(c["vc"])
    mx.store_kv(c["prob"], c["loc"], c["k"].contiguous(), c["v"].contiguous(), kc, vc)
    got, _ = fp4_values(c["vc"], 64)
    want, _ = fp4_values(vc, 64)
    assert torch.equal(got[page, :, off], want[page, :, off])


def test_padding_bad_positions_and_bad_slots():
    c = case(40, 8, 2, "bf16", "bf16", 64, 128, idx=64 * 2, seed=9)
    ref = case(40, 8, 2, "bf16", "bf16", 64, 128, idx=64 * 2, seed=9)
    call(ref)
    before = by_slot(c["kc"])
    c["pos"][3], c["pos"][5] = -1, 10 ** 12          # padding; past the table
    c["loc"][7], c["loc"][8] = -4, c["pages"] * 64   # not stored; past the cache
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 256 | 4
    keep = torch.ones(40, dtype=torch.bool)
    keep[[3, 5]] = False
    assert torch.equal(c["q_out"][keep.cuda()], ref["q_out"][keep.cuda()])  # 7 and 8 have their queries
    assert (c["q_out"][[3, 5]] == 7).all()
    assert torch.equal(c["iq_out"][keep.cuda()], ref["iq_out"][keep.cuda()])
    loc = ref["loc"].cpu()
    stored = keep.clone()
    stored[[7, 8]] = False
    assert torch.equal(by_slot(c["kc"])[loc[stored]], by_slot(ref["kc"])[loc[stored]])
    assert torch.equal(by_slot(c["kc"])[loc[~stored]], before[loc[~stored]])
    only = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["pos"][5], c["loc"][8] = -3, -1
    call(c, flags=only)
    assert only.item() == 0


def test_in_place_empty_and_special_values():
    c = case(33, 16, 2, "bf16", "fp8", 64, 64, packed=False, seed=11)
    want = case(33, 16, 2, "bf16", "fp8", 64, 64, packed=False, seed=11)
    call(want)
    c["q_out"] = c["q"]
    call(c)
    torch.cuda.synchronize()
    assert torch.equal(c["q"], want["q_out"])
    # rows of zeros, an infinity, a NaN: their own rows only
    c = case(4, 4, 2, "bf16", "fp8", 64, 64, packed=False, seed=12)
    want = case(4, 4, 2, "bf16", "fp8", 64, 64, packed=False, seed=12)
    call(want)
    c["q"][0, 0] = 0
    c["q"][1, 1, 5] = float("nan")
    c["k"][2, 0, 9] = float("inf")
    c["k"][3, 1] = 1e4  # e4m3 saturates nothing here: the norm brings it back
    call(c)
    torch.cuda.synchronize()
    assert (c["q_out"][0, 0] == 0).all() and c["q_out"][1, 1].isnan().all()
    same = torch.ones(4, 4, dtype=torch.bool, device="cuda")
    same[0, 0] = same[1, 1] = False
    assert torch.equal(c["q_out"][same], want["q_out"][same])
    page, off = c["loc"] // 64, c["loc"] % 64
    rows = c["kc"].float()[page, :, off]
    assert rows[2, 0].isnan().any() and not rows[2, 1].isnan().any() and not rows[3].isnan().any()
    e = case(1, 4, 2, "bf16", "bf16", 64, 64, seed=13)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    mx.norm_rope_store(e["prob"], none, none, e["cs"], e["q"][:0], e["k"][:0], e["v"][:0], e["q_out"], e["kc"],
                       e["vc"])
    assert (e["q_out"] == 7).all()


@pytest.mark.parametrize("kv,inter", [("bf16", False), ("fp8", True), ("nvfp4", False), ("nvfp4", True)])
def test_infinities_past_the_rotated_columns_stay_in_their_column(kv, inter):
    c = case(6, 4, 2, "bf16", kv, 64, 32, inter=inter, weights=False, packed=False, seed=31)
    want = case(6, 4, 2, "bf16", kv, 64, 32, inter=inter, weights=False, packed=False, seed=31)
    call(want)
    c["q"][0, 0, 40], c["q"][1, 2, 100] = float("inf"), float("nan")
    call(c)
    torch.cuda.synchronize()
    same = torch.ones(6, 4, 128, dtype=torch.bool, device="cuda")
    same[0, 0, 40] = same[1, 2, 100] = False
    assert torch.equal(c["q_out"][same], want["q_out"][same])
    assert c["q_out"][0, 0, 40] == float("inf") and c["q_out"][1, 2, 100].isnan()


def test_captured_and_replayed_on_another_stream():
    c = case(64, 16, 2, "bf16", "bf16", 64, 128, idx=128, seed=21)
    want = case(64, 16, 2, "bf16", "bf16", 64, 128, idx=128, seed=22)
    call(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(c)
    for k in ("q", "k", "v", "iq", "ik", "pos", "loc", "cs", "qw", "kw", "iqw", "ikw", "kc", "vc", "ic"):
        c[k].copy_(want[k])
    graph.replay()
    call(want)
    torch.cuda.synchronize()
    for k in ("q_out", "kc", "vc", "iq_out", "ic"):
        assert torch.equal(c[k], want[k]), k


# -------------------------------------------------------------------- load_kv
@pytest.mark.parametrize("q", ["bf16", "fp16"])
@pytest.mark.parametrize("kv", ["same", "fp8", "nvfp4"])
@pytest.mark.parametrize("n,hkv,ps,idx", [(1, 1, 64, 0), (77, 3, 64, 24), (300, 8, 128, 64)])
def test_load_is_exact(q, kv, n, hkv, ps, idx):
    kv = q if kv == "same" else kv
    g = torch.Generator().manual_seed(n)
    t, pages = TDT[q], -(-n // ps) + 2
    kvt = "nvfp4" if kv == "nvfp4" else TDT[kv]
    prob = mx.make_problem(1, n, hkv, hkv, 1, ps, pages, pages, False, q_dtype=t, kv_dtype=kvt)
    loc = torch.randint(0, pages * ps, (n,), generator=g)  # slots may repeat
    if n > 20:
        loc[4], loc[11], loc[19] = -1, pages * ps, -2 ** 40
    ok = (loc >= 0) & (loc < pages * ps)
    page, off = loc.clamp(0, pages * ps - 1) // ps, loc.clamp(0, pages * ps - 1) % ps

    def cache(heads, dim):
        if kv == "nvfp4":  # every byte: all codes, all scales, NaN scales among them
            return torch.randint(0, 256, (pages, heads, ps * 72), generator=g, dtype=torch.uint8)
        if kv == "fp8":    # every code
            return torch.randint(0, 256, (pages, heads, ps, dim), generator=g, dtype=torch.uint8)
        return torch.randint(-2 ** 15, 2 ** 15, (pages, heads, ps, dim), generator=g, dtype=torch.int16)

    def want(c):
        if kv == "nvfp4":
            return fp4_values(c, ps)[0][page, :, off]
        if kv == "fp8":
            return c[page, :, off].view(torch.float8_e4m3fn).float().double()
        return c[page, :, off]

    kc, vc = cache(hkv, 128), cache(hkv, 128)
    k, v = (torch.full((n, hkv, 128), 5.0, dtype=t, device="cuda") for _ in range(2))
    extra, ik, ic = {}, None, None
    if idx and kv != "nvfp4":
        ic, ik = cache(2, idx), torch.full((n, 2, idx), 5.0, dtype=t, device="cuda")
        extra = dict(idx_cache=ic.cuda(), idx_k=ik)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.load_kv(prob, loc.cuda(), kc.cuda(), vc.cuda(), k, v, flags=flags, **extra)
    torch.cuda.synchronize()
    assert flags.item() == (4 if n > 20 else 0)
    for got, c in ((k, kc), (v, vc)) + (((ik, ic),) if ik is not None else ()):
        got = got.cpu()
        assert (got[~ok] == 5).all()
        ref = want(c)[ok]
        if kv in ("bf16", "fp16"):
            assert torch.equal(got[ok].view(torch.int16), ref)
        else:
            got = got[ok].double()
            assert torch.equal(got.isnan(), ref.isnan())
            assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(ref, nan=0.0))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_slots_past_two_to_the_31_elements(kv):
    """Written by norm_rope_store into the last slots of a cache of more than 2^31 elements, and read back."""
    c = case(70, 8, 2, "bf16", kv, 64, 64, seed=41)
    per = 2 * 64 * (72 if kv == "nvfp4" else 128)
    pages = (1 << 31) // per + 3
    kvt = "nvfp4" if kv == "nvfp4" else TDT[kv]
    shape = (pages, 2, 64 * 72) if kv == "nvfp4" else (pages, 2, 64, 128)
    big = [torch.empty(shape, dtype=c["kc"].dtype, device="cuda") for _ in range(2)]
    prob = mx.make_problem(1, 70, 8, 2, 1, 64, pages, pages, False, q_dtype=torch.bfloat16, kv_dtype=kvt)
    want = [torch.zeros_like(c["kc"]) for _ in range(2)]
    call(dict(c, kc=want[0], vc=want[1]))
    shift = (pages - c["pages"]) * 64
    call(dict(c, prob=prob, kc=big[0], vc=big[1], loc=c["loc"] + shift))
    back = [[torch.empty(70, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    mx.load_kv(c["prob"], c["loc"], *want, *back[0])
    mx.load_kv(prob, c["loc"] + shift, *big, *back[1])
    torch.cuda.synchronize()
    for x, y in zip(*back):
        assert torch.equal(x, y) and x.abs().sum() > 0


@pytest.mark.parametrize("q", ["bf16", "fp16"])
def test_load_of_what_the_store_wrote(q):
    """A 16-bit row, stored in e4m3 and read back, is its cast."""
    n, hkv, ps = 200, 4, 64
    t = TDT[q]
    prob = mx.make_problem(1, n, hkv, hkv, 1, ps, 5, 5, False, q_dtype=t, kv_dtype=torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = ((torch.randn(n, hkv, 128, generator=g, device="cuda") * 200).to(t) for _ in range(2))
    kc, vc = (torch.zeros(5, hkv, ps, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    loc = torch.randperm(5 * ps, generator=g, device="cuda")[:n]
    mx.store_kv(prob, loc, k, v, kc, vc)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    mx.load_kv(prob, loc, kc, vc, k2, v2)
    cast = lambda x: x.float().clamp(-448, 448).to(torch.float8_e4m3fn).to(t)
    assert torch.equal(k2, cast(k)) and torch.equal(v2, cast(v))
