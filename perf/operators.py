"""The serving step's operators around the paged KV cache, as measured cases.

Three operators, each as elementary torch operations (``own`` false) and as the
calls a user makes of the framework (``own`` true):

``norm_rope_store``  the prologue of an attention layer: RMS norm of every query
    and key head, rotation by position, and the cast and write of K, V and the
    index keys into the paged caches.
``load_kv``          the way back: rows of the paged caches, widened, by slot.
``shared``           dense paged attention of a batch whose sequences share a
    long prefix in groups (one document or system prompt, many continuations).

``round_trip`` is the first two in a row on an NVFP4 cache, whose packed bytes
only the pair makes comparable.
"""
import math
import random

import numpy as np
import torch

own = False

DIM = 128
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
ROW_BYTES = {"bf16": 256, "fp16": 256, "fp8": 128, "nvfp4": 72}  # one cached head row
EPS = 1e-6


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one small sequence: the latency of the call
        dict(name="store_one_token", op="norm_rope_store", n=1, hq=16, hkv=2, q="bf16", kv="bf16", ps=64, rot=128,
             inter=False, per_head=False, idx=0, positions=4096),
        # a decode step of 64 sequences into an FP8 cache, index queries and keys with it
        dict(name="store_decode_fp8", op="norm_rope_store", n=64, hq=64, hkv=8, q="bf16", kv="fp8", ps=128, rot=64,
             inter=False, per_head=False, idx=128, positions=32768),
        # a ragged prefill chunk, three query heads to a kv head, pairs side by side, a weight row for each head
        dict(name="store_chunk_odd", op="norm_rope_store", n=5003, hq=12, hkv=4, q="fp16", kv="fp8", ps=64, rot=96,
             inter=True, per_head=True, idx=128, positions=36864),
        # a large prefill batch from the packed projection into a 16-bit cache
        dict(name="store_prefill", op="norm_rope_store", n=32768, hq=64, hkv=8, q="bf16", kv="bf16", ps=128, rot=128,
             inter=False, per_head=False, idx=0, positions=65536),
        # a decode step of 256 sequences into an NVFP4 cache, and those rows read back
        dict(name="round_trip_nvfp4", op="round_trip", n=256, hq=16, hkv=2, q="bf16", kv="nvfp4", ps=64, rot=128,
             inter=False, per_head=False, idx=0, positions=32768),
        # a few rows of a cache, as a debugger or a cache migration of one block takes them
        dict(name="load_block", op="load_kv", n=129, hkv=8, q="bf16", kv="bf16", ps=128, idx=64),
        # a long FP8 prefix widened for an attention that takes 16-bit keys
        dict(name="load_prefix_fp8", op="load_kv", n=36864, hkv=8, q="bf16", kv="fp8", ps=128, idx=0),
        # the same of an NVFP4 cache, a ragged length
        dict(name="load_prefix_nvfp4", op="load_kv", n=30011, hkv=4, q="fp16", kv="nvfp4", ps=64, idx=0),
        # eight continuations of a short prompt
        dict(name="shared_small", op="shared", groups=1, per=8, tq=1, hq=16, hkv=2, q="bf16", ps=64, prefix=1000,
             smin=1, smax=64, causal=False),
        # verification of five drafted tokens, three prompts of odd lengths
        dict(name="shared_verify", op="shared", groups=3, per=8, tq=5, hq=12, hkv=4, q="fp16", ps=64, prefix=9001,
             smin=5, smax=700, causal=True),
        # 64 decoding sequences over one long document
        dict(name="shared_decode", op="shared", groups=1, per=64, tq=1, hq=64, hkv=8, q="bf16", ps=128, prefix=32768,
             smin=128, smax=2048, causal=False),
        # 256 decoding sequences over a longer one
        dict(name="shared_decode_large", op="shared", groups=1, per=256, tq=1, hq=64, hkv=8, q="bf16", ps=128,
             prefix=65536, smin=64, smax=2048, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(8, 1), (16, 2), (12, 4), (16, 16), (32, 4), (64, 8), (48, 8), (128, 1), (10, 2)]


def draw(rng):
    op = rng.choice(["norm_rope_store", "load_kv", "shared", "shared", "round_trip"])
    hq, hkv = rng.choice(HEADS)
    q, ps = rng.choice(["bf16", "fp16"]), rng.choice([64, 128])
    if op == "load_kv":
        kv = rng.choice([q, "fp8", "nvfp4"])
        return dict(op=op, n=_log(rng, 1, 30000), hkv=hkv, q=q, kv=kv, ps=ps,
                    idx=0 if kv == "nvfp4" else rng.choice([0, 64, 128]))
    if op in ("norm_rope_store", "round_trip"):
        kv = "nvfp4" if op == "round_trip" else rng.choice([q, "fp8"])
        idx = 0 if kv == "nvfp4" else rng.choice([0, 64, 128])
        return dict(op=op, n=_log(rng, 1, 400 if kv == "nvfp4" else 20000), hq=hq, hkv=hkv, q=q, kv=kv, ps=ps,
                    rot=rng.choice([16, 32, 64] if idx == 64 else [16, 32, 64, 96, 128]), inter=rng.random() < 0.5,
                    per_head=rng.random() < 0.5, idx=idx, positions=_log(rng, 500, 60000))
    groups, tq = rng.choice([1, 1, 2, 5]), rng.choice([1, 1, 1, 3, 8])
    per = max(1, _log(rng, 1, 128) // (groups * tq))
    smax = _log(rng, tq, 2000)
    return dict(op=op, groups=groups, per=per, tq=tq, hq=hq, hkv=hkv, q=q, ps=ps, prefix=_log(rng, 1, 30000),
                smin=rng.randint(min(tq, smax), smax), smax=smax, causal=tq > 1 and rng.random() < 0.7)


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _slots(case, g, n):
    """n different slots of a cache of a few more pages than they fill, and its page count."""
    pages = -(-n // case["ps"]) + 2
    return torch.randperm(pages * case["ps"], generator=g, device="cuda")[:n].contiguous(), pages


def _cache(case, g, pages, heads, dim=DIM):
    """A cache that holds earlier tokens, in the case's cache type."""
    kv, ps = case["kv"], case["ps"]
    if kv == "nvfp4":
        c = torch.randint(0, 256, (pages, heads, ps * 72), generator=g, device="cuda", dtype=torch.uint8)
        # the scales' bytes: e4m3 codes of 2^-4 up to 15/32
        c[:, :, ps * 64:] = torch.randint(0x18, 0x38, (pages, heads, ps * 8), generator=g, device="cuda",
                                          dtype=torch.uint8)
        return c
    return _normal(g, pages, heads, ps, dim, dtype=torch.float32).to(TORCH[kv])


def _lens(case):
    """Prefix length of every group and suffix length of every sequence: the
    case's own, the same for every seed."""
    r = random.Random(case["prefix"] * 7919 + case["smax"] * 31 + case["per"])
    ng, n = case["groups"], case["groups"] * case["per"]
    prefix = [max(1, case["prefix"] - j * case["prefix"] // (2 * ng)) for j in range(ng)]
    suffix = [r.randint(case["smin"], case["smax"]) for _ in range(n)]
    suffix[0] = case["smax"]
    return prefix, suffix


def _prepare_store(case, seed):
    g, t = _gen(seed), TORCH[case["q"]]
    n, hq, hkv, d, idx = case["n"], case["hq"], case["hkv"], DIM, case["idx"]
    loc, pages = _slots(case, g, n)
    s = {"case": case, "loc": loc}
    # q, k and v are views of one packed projection
    qkv = _normal(g, n, (hq + 2 * hkv) * d, dtype=t, scale=1.5)
    s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    weight = lambda heads, dim: 1 + _normal(g, *((heads, dim) if case["per_head"] else (dim,)), dtype=torch.float32,
                                            scale=0.1)
    s["q_weight"], s["k_weight"] = weight(hq, d).to(t), weight(hkv, d).to(t)
    s["k_cache"], s["v_cache"] = _cache(case, g, pages, hkv), _cache(case, g, pages, hkv)
    s["q_out"] = torch.empty(n, hq, d, dtype=t, device="cuda")
    s["positions"] = torch.randint(0, case["positions"], (n,), generator=g, device="cuda")
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(case["positions"], dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if idx:
        s["idx_q"], s["idx_k"] = _normal(g, n, hkv, idx, dtype=t), _normal(g, n, hkv, idx, dtype=t)
        s["idx_q_weight"], s["idx_k_weight"] = weight(hkv, idx).to(t), weight(hkv, idx).to(t)
        s["idx_cache"] = _cache(case, g, pages, hkv, idx)
        s["idx_q_out"] = torch.empty(n, hkv, idx, dtype=TORCH[case["kv"]], device="cuda")
    if case["op"] == "round_trip":
        s["k_back"], s["v_back"] = (torch.empty(n, hkv, d, dtype=t, device="cuda") for _ in range(2))
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(1, n, hq, hkv, 1, case["ps"], pages, pages, False, q_dtype=t,
                                    kv_dtype="nvfp4" if case["kv"] == "nvfp4" else TORCH[case["kv"]])
    return s


def _prepare_load(case, seed):
    g, t = _gen(seed), TORCH[case["q"]]
    n, hkv, idx = case["n"], case["hkv"], case["idx"]
    loc, pages = _slots(case, g, n)
    # whole pages in a random order, as block tables give them
    page = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(n, device="cuda")
    loc = page[at // case["ps"]] * case["ps"] + at % case["ps"]
    s = {"case": case, "loc": loc, "k_cache": _cache(case, g, pages, hkv), "v_cache": _cache(case, g, pages, hkv)}
    s["k"], s["v"] = (torch.empty(n, hkv, DIM, dtype=t, device="cuda") for _ in range(2))
    if idx:
        s["idx_cache"] = _cache(case, g, pages, hkv, idx)
        s["idx_k"] = torch.empty(n, hkv, idx, dtype=t, device="cuda")
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(1, n, hkv, hkv, 1, case["ps"], pages, pages, False, q_dtype=t,
                                    kv_dtype="nvfp4" if case["kv"] == "nvfp4" else TORCH[case["kv"]])
    return s


def _prepare_shared(case, seed):
    g, t = _gen(seed), TORCH[case["q"]]
    ps, per, ng, tq, hq, hkv = case["ps"], case["per"], case["groups"], case["tq"], case["hq"], case["hkv"]
    prefix, suffix = _lens(case)
    n = ng * per
    lens = [prefix[i // per] + suffix[i] for i in range(n)]
    width = max(-(-l // ps) for l in lens)
    table, pages = np.full((n, width), -1, np.int32), 0
    for i in range(n):
        first = i // per * per
        whole = 0 if i == first else prefix[i // per] // ps  # pages that hold nothing but the prefix
        last = -(-lens[i] // ps)
        table[i, :whole] = table[first, :whole]
        table[i, whole:last] = np.arange(pages, pages + last - whole)
        pages += last - whole
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages).astype(np.int32)
    table = np.where(table >= 0, order[np.maximum(table, 0)], -1)
    dev = lambda a, dt: torch.tensor(np.asarray(a), dtype=dt, device="cuda")
    s = {"case": case, "pmax": max(prefix), "smax": max(suffix)}
    s["k_cache"] = torch.empty(pages, hkv, ps, DIM, dtype=t, device="cuda").normal_(generator=g)
    s["v_cache"] = torch.empty(pages, hkv, ps, DIM, dtype=t, device="cuda").normal_(generator=g)
    s["q"] = _normal(g, n * tq, hq, DIM, dtype=t, scale=2.0)
    s["block_tables"] = dev(table, torch.int32)
    s["cu"] = dev(np.arange(n + 1) * tq, torch.int64)
    s["lens"] = dev(lens, torch.int32)
    s["group_ptr"] = dev(np.arange(ng + 1) * per, torch.int32)
    s["prefix_lens"] = dev(prefix, torch.int32)
    s["out"] = torch.empty(n * tq, hq, DIM, dtype=t, device="cuda")
    s["lse"] = torch.empty(hq, n * tq, dtype=torch.float32, device="cuda")
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(n, n * tq, hq, hkv, 1, ps, pages, width, case["causal"], q_dtype=t)
        s["ws"] = torch.empty(mx.dense_shared_workspace_size(s["prob"]), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return {"norm_rope_store": _prepare_store, "round_trip": _prepare_store, "load_kv": _prepare_load,
            "shared": _prepare_shared}[case["op"]](case, seed)


# ------------------------------------------------------------- the plain forms
def _norm_rope(x, weight, cos_sin, inter):
    """[n, heads, dim] in 32 bits, normed over dim, the leading columns rotated."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[:, None, :half], cos_sin[:, None, half:]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _cast(x, dtype):
    """float32 to a cache's type, e4m3 saturating."""
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _nvfp4_values(x):
    """The values that E2M1 codes with one e4m3 scale to 16 elements stand for."""
    g = x.float().unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1, keepdim=True) / 6).clamp(max=448).to(torch.float8_e4m3fn).float()
    y = torch.where(scale > 0, g / scale.clamp(min=2.0 ** -10), torch.zeros_like(g))
    a = y.abs()
    half = ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float()) * 0.5
    m = half + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5).float()
    return (m * torch.sign(y) * scale).flatten(-2)


def _write(cache, page, off, x):
    """cache[page, :, off, :] = x, as bits (an 8-bit type has no indexed write of its own)."""
    bits = torch.uint8 if cache.element_size() == 1 else torch.int16
    cache.view(bits)[page, :, off] = x.view(bits)


def _plain_store(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"]]
    q = _norm_rope(s["q"], s["q_weight"], cs, c["inter"]).to(s["q"].dtype)
    k = _norm_rope(s["k"], s["k_weight"], cs, c["inter"])
    if c["op"] == "round_trip":
        return q, _nvfp4_values(k).to(q.dtype), _nvfp4_values(s["v"]).to(q.dtype)
    page, off = s["loc"] // c["ps"], s["loc"] % c["ps"]
    kv = s["k_cache"].dtype
    _write(s["k_cache"], page, off, _cast(k, kv))
    _write(s["v_cache"], page, off, _cast(s["v"].float(), kv))
    out = [q, s["k_cache"], s["v_cache"]]
    if c["idx"]:
        _write(s["idx_cache"], page, off, _cast(_norm_rope(s["idx_k"], s["idx_k_weight"], cs, c["inter"]), kv))
        out += [_cast(_norm_rope(s["idx_q"], s["idx_q_weight"], cs, c["inter"]), kv), s["idx_cache"]]
    return out


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _read(s, cache, page, off, dtype):
    c = s["case"]
    if c["kv"] != "nvfp4":
        bits = torch.uint8 if cache.element_size() == 1 else torch.int16
        return cache.view(bits)[page, :, off].view(cache.dtype).float().to(dtype)
    ps = c["ps"]
    codes = cache[:, :, :ps * 64].unflatten(2, (ps, 64))[page, :, off]
    scales = cache[:, :, ps * 64:].unflatten(2, (ps, 8))[page, :, off].view(torch.float8_e4m3fn).float()
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    mag = (codes & 7).float()  # 0 .5 1 1.5 2 3 4 6 by the code's number
    mag = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2, mag * 2 - 8))
    mag = torch.where((codes & 8) > 0, -mag, mag)
    return (mag.unflatten(-1, (8, 16)) * scales[..., None]).flatten(-2).to(dtype)


def _plain_load(s):
    c, t = s["case"], s["k"].dtype
    page, off = s["loc"] // c["ps"], s["loc"] % c["ps"]
    out = [_read(s, s["k_cache"], page, off, t), _read(s, s["v_cache"], page, off, t)]
    if c["idx"]:
        out.append(_read(s, s["idx_cache"], page, off, t))
    return out


def _plain_shared(s):
    c = s["case"]
    ng, per, tq, hkv, ps = c["groups"], c["per"], c["tq"], c["hkv"], c["ps"]
    n, G = ng * per, c["hq"] // c["hkv"]
    scale = DIM ** -0.5
    q = s["q"].float().view(n, tq, hkv, G, DIM) * scale
    lens, plen = s["lens"].long(), s["prefix_lens"].long()
    tables = s["block_tables"].long()
    pos = lens[:, None] - tq + torch.arange(tq, device="cuda")  # [n, tq]: each token's own position
    # the prefix, once for a group: rows [ng, hkv, per * tq * G]
    at = torch.arange(s["pmax"], device="cuda")
    page = tables[::per][:, at // ps].clamp(min=0)  # [ng, pmax]
    kp = s["k_cache"][page, :, at % ps].permute(0, 2, 1, 3).float()  # [ng, hkv, pmax, DIM]
    vp = s["v_cache"][page, :, at % ps].permute(0, 2, 1, 3).float()
    qp = q.view(ng, per * tq, hkv, G, DIM).permute(0, 2, 1, 3, 4).reshape(ng, hkv, per * tq * G, DIM)
    sp = qp @ kp.transpose(-1, -2)
    gone = (at >= plen[:, None])[:, None, :].expand(ng, per * tq, -1)
    if c["causal"]:
        gone = gone | (at > pos.view(ng, per * tq, 1))
    sp = sp.view(ng, hkv, per * tq, G, -1).masked_fill_(gone[:, None, :, None, :], -math.inf)
    mp = sp.amax(-1, keepdim=True)
    # each sequence's own keys
    rel = torch.arange(s["smax"], device="cuda")
    at = plen.repeat_interleave(per)[:, None] + rel  # [n, smax]
    page = tables.gather(1, (at // ps).clamp(max=tables.shape[1] - 1)).clamp(min=0)
    ks = s["k_cache"][page, :, at % ps].permute(0, 2, 1, 3).float()  # [n, hkv, smax, DIM]
    vs = s["v_cache"][page, :, at % ps].permute(0, 2, 1, 3).float()
    qs = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, tq * G, DIM)
    ss = (qs @ ks.transpose(-1, -2)).view(n, hkv, tq, G, -1)
    gone = (at >= lens[:, None])[:, None, :].expand(n, tq, -1)
    if c["causal"]:
        gone = gone | (at[:, None, :] > pos[:, :, None])
    ss = ss.masked_fill_(gone[:, None, :, None, :], -math.inf)
    # one softmax over both
    mp = mp.view(ng, hkv, per, tq, G, 1).transpose(1, 2).reshape(n, hkv, tq, G, 1)
    m = torch.maximum(mp, ss.amax(-1, keepdim=True))
    back = m.view(ng, per, hkv, tq, G, 1).transpose(1, 2).reshape(ng, hkv, per * tq, G, 1)
    ep, es = sp.sub_(back).exp_(), ss.sub_(m).exp_()
    op = (ep.view(ng, hkv, per * tq * G, -1) @ vp).view(ng, hkv, per, tq, G, DIM).transpose(1, 2)
    os = (es.view(n, hkv, tq * G, -1) @ vs).view(n, hkv, tq, G, DIM)
    lp = ep.sum(-1, keepdim=True).view(ng, hkv, per, tq, G, 1).transpose(1, 2).reshape(n, hkv, tq, G, 1)
    l = lp + es.sum(-1, keepdim=True)
    o = ((op.reshape(n, hkv, tq, G, DIM) + os) / l).permute(0, 2, 1, 3, 4).reshape(n * tq, c["hq"], DIM)
    lse = (m + l.log())[..., 0].permute(1, 3, 0, 2).reshape(c["hq"], n * tq)
    return o.to(s["q"].dtype), lse


# ------------------------------------------------------- the framework's calls
def _own_store(s):
    import block_sparse_attention_builder_gb300 as mx
    c = s["case"]
    idx = {k: s[k] for k in ("idx_q", "idx_k", "idx_q_weight", "idx_k_weight", "idx_q_out", "idx_cache")} \
        if c["idx"] else {}
    mx.norm_rope_store(s["prob"], s["positions"], s["loc"], s["cos_sin"], s["q"], s["k"], s["v"], s["q_out"],
                       s["k_cache"], s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                       interleaved=c["inter"], **idx)
    if c["op"] == "round_trip":
        mx.load_kv(s["prob"], s["loc"], s["k_cache"], s["v_cache"], s["k_back"], s["v_back"])
        return s["q_out"], s["k_back"], s["v_back"]
    out = [s["q_out"], s["k_cache"], s["v_cache"]]
    return out + [s["idx_q_out"], s["idx_cache"]] if c["idx"] else out


def _own_load(s):
    import block_sparse_attention_builder_gb300 as mx
    if s["case"]["idx"]:
        mx.load_kv(s["prob"], s["loc"], s["k_cache"], s["v_cache"], s["k"], s["v"], s["idx_cache"], s["idx_k"])
        return [s["k"], s["v"], s["idx_k"]]
    mx.load_kv(s["prob"], s["loc"], s["k_cache"], s["v_cache"], s["k"], s["v"])
    return [s["k"], s["v"]]


def _own_shared(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.dense_shared_fwd(s["prob"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["cu"], s["lens"],
                        s["group_ptr"], s["prefix_lens"], s["ws"], s["out"], s["lse"])
    return s["out"], s["lse"]


def run(state):
    op = state["case"]["op"]
    if op == "shared":
        return _own_shared(state) if own else _plain_shared(state)
    if op == "load_kv":
        return _own_load(state) if own else _plain_load(state)
    return _own_store(state) if own else _plain_store(state)


# ------------------------------------------------------------------- the floor
def work(case):
    q_row = DIM * 2
    if case["op"] == "shared":
        prefix, suffix = _lens(case)
        per, tq, rows = case["per"], case["tq"], len(suffix) * case["tq"]
        keys = sum(prefix) + sum(suffix)
        seen = 0  # (token, key) pairs
        for i, x in enumerate(suffix):
            L = prefix[i // per] + x
            seen += tq * L - (tq * (tq - 1) // 2 if case["causal"] else 0)
        return {"bytes": keys * case["hkv"] * 2 * q_row + rows * case["hq"] * (2 * q_row + 4),
                "flops": 4.0 * DIM * case["hq"] * seen}
    cached = ROW_BYTES[case["kv"]]
    n, hkv, idx = case["n"], case["hkv"], case["idx"]
    icached = idx * (1 if case["kv"] == "fp8" else 2)
    if case["op"] == "load_kv":
        return {"bytes": n * (8 + hkv * (2 * (cached + q_row) + icached + idx * 2)), "flops": n * hkv * 2.0 * DIM}
    b = n * (16 + case["hq"] * 2 * q_row + hkv * 2 * (q_row + cached) + hkv * 2 * (idx * 2 + icached) + case["rot"] * 4)
    if case["op"] == "round_trip":
        b += n * (8 + hkv * 2 * (cached + q_row))
    return {"bytes": b, "flops": n * (case["hq"] + hkv) * 7.0 * DIM}


# --------------------------------------------------- the definition in 64 bits
def _exact_rows(x, weight, s):
    """Norm and rotation as a complex product, in 64 bits."""
    c = s["case"]
    x = x.double()
    y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * weight.double()
    half = c["rot"] // 2
    turn = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())[s["positions"]][:, None]
    i = torch.arange(half, device=x.device)
    re, im = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
    z = torch.complex(y[..., re], y[..., im]) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_fp4(x):
    """The nearest E2M1 value under the group's scale, found by looking at all of them."""
    g = x.double().reshape(-1, 16)
    scale = (g.abs().max(1).values / 6).float().to(torch.float8_e4m3fn).double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    y = torch.where(scale[:, None] > 0, g / scale[:, None], torch.zeros((), dtype=torch.float64, device=x.device))
    far = (y.abs()[..., None] - grid).abs()
    # of two equally near, the one of the even code
    at = (far + torch.tensor([0, 1, 0, 1, 0, 1, 0, 1], device=x.device) * 1e-12).argmin(-1)
    return (grid[at] * y.sign() * scale[:, None]).reshape(x.shape)


def _exact_store(s):
    c = s["case"]
    q, k = _exact_rows(s["q"], s["q_weight"], s), _exact_rows(s["k"], s["k_weight"], s)
    if c["op"] == "round_trip":
        return q, _exact_fp4(k), _exact_fp4(s["v"])

    def cached(cache, x):
        flat = cache.to(torch.float32).double().transpose(1, 2).reshape(-1, *x.shape[1:]).clone()  # by slot
        flat[s["loc"]] = _cast(x.float(), cache.dtype).to(torch.float32).double() if c["kv"] == "fp8" else x.double()
        return flat.reshape(cache.shape[0], c["ps"], *x.shape[1:]).transpose(1, 2).contiguous()

    out = [q, cached(s["k_cache"], k), cached(s["v_cache"], s["v"])]
    if c["idx"]:
        iq = _exact_rows(s["idx_q"], s["idx_q_weight"], s)
        iq = _cast(iq.float(), torch.float8_e4m3fn).to(torch.float32).double() if c["kv"] == "fp8" else iq
        out += [iq, cached(s["idx_cache"], _exact_rows(s["idx_k"], s["idx_k_weight"], s))]
    return out


def _exact_load(s):
    c, n, ps = s["case"], s["case"]["n"], s["case"]["ps"]

    def rows(cache):
        if c["kv"] != "nvfp4":
            return cache.to(torch.float32).double().transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[s["loc"]]
        pages, heads = cache.shape[:2]
        b = cache.reshape(pages, heads, ps * 72)
        value = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=cache.device)
        code = b[..., :ps * 64].reshape(pages, heads, ps, 64).long()
        v = torch.empty(pages, heads, ps, DIM, dtype=torch.float64, device=cache.device)
        v[..., 0::2], v[..., 1::2] = value[code % 16], value[code // 16]
        sc = b[..., ps * 64:].contiguous().view(torch.float8_e4m3fn).float().double().reshape(pages, heads, ps, 8)
        v *= sc.repeat_interleave(16, -1)
        return v.transpose(1, 2).reshape(-1, heads, DIM)[s["loc"]]

    out = [rows(s["k_cache"]), rows(s["v_cache"])]
    assert out[0].shape[0] == n
    return out + [rows(s["idx_cache"])] if c["idx"] else out


def _exact_shared(s):
    """Sequence by sequence: its keys in order, then a softmax in 64 bits."""
    c = s["case"]
    per, tq, ps, hkv = c["per"], c["tq"], c["ps"], c["hkv"]
    prefix, suffix = _lens(c)
    out, lses, held = [], [], None
    for i, x in enumerate(suffix):
        first, P = i // per * per, prefix[i // per]
        L = P + x

        def keys(cache, lo, hi, row):
            p = torch.arange(lo, hi, device="cuda")
            return cache[s["block_tables"][row].long()[p // ps], :, p % ps].double()  # [hi - lo, hkv, DIM]

        if i == first:
            held = [keys(s[name], 0, P, first) for name in ("k_cache", "v_cache")]
        k, v = (torch.cat([h, keys(s[name], P, L, i)]) for h, name in zip(held, ("k_cache", "v_cache")))
        q = s["q"][i * tq:(i + 1) * tq].double().reshape(tq, hkv, -1, DIM)
        a = torch.einsum("tgrd,pgd->tgrp", q, k) / math.sqrt(DIM)
        if c["causal"]:
            late = torch.arange(L, device="cuda")[None] > (L - tq + torch.arange(tq, device="cuda"))[:, None]
            a.masked_fill_(late[:, None, None], -math.inf)
        out.append(torch.einsum("tgrp,pgd->tgrd", torch.softmax(a, -1), v).reshape(tq, -1, DIM))
        lses.append(torch.logsumexp(a, -1).reshape(tq, -1))
    return torch.cat(out), torch.cat(lses).T.contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope_store": _exact_store, "round_trip": _exact_store, "load_kv": _exact_load,
            "shared": _exact_shared}[case["op"]](s)
