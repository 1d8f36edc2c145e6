"""The steps around speculative decoding and whole prompts, as measured cases.

Five operators, each as elementary torch operations (``own`` false) and as the
calls a user makes of the framework (``own`` true):

``tables``  a serving step's bookkeeping on the GPU: pages for the new tokens
    taken from a free list (those of finished requests given back), block
    tables, lengths, positions and cache slots from the requests' lengths.
``mask``    the ancestor masks and positions of drafted token trees, from the
    tokens' parents.
``tree``    attention of drafted trees over the paged cache: every token sees
    its sequence's committed keys and its own ancestors.
``commit``  the accepted path of each tree moved to the positions it takes in
    the sequence, in the caches.
``prompt``  causal attention of whole prompts of different lengths, packed one
    behind the other, straight from the projection (no cache).
"""
import math
import random

import numpy as np
import torch

own = False

DIM = 128
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of 64 requests: one token each, a page now and then
        dict(name="tables_decode", op="tables", n=64, ps=64, new_min=1, new_max=1, old=32768, done=0),
        # a mixed step: ragged prompt chunks beside decoding, some requests finished
        dict(name="tables_prefill", op="tables", n=211, ps=128, new_min=1, new_max=4001, old=16384, done=9),
        # the trees of a small batch
        dict(name="mask_small", op="mask", n=8, tq=16, depth=5),
        # wide trees of a large batch, an odd size
        dict(name="mask_large", op="mask", n=256, tq=125, depth=10),
        # one sequence with a small tree: the latency of the call
        dict(name="tree_one", op="tree", n=1, per=1, tq=8, depth=3, hq=16, hkv=2, q="bf16", ps=64, lmin=1000,
             lmax=1000),
        # three query heads to a kv head, trees of an odd size, a prompt that eight continuations share
        dict(name="tree_shared_odd", op="tree", n=24, per=8, tq=37, depth=7, hq=12, hkv=4, q="fp16", ps=64, lmin=9001,
             lmax=9700),
        # a verification step: 64 sequences of different lengths, trees of 16 tokens
        dict(name="tree_verify", op="tree", n=64, per=1, tq=16, depth=5, hq=64, hkv=8, q="bf16", ps=128, lmin=4096,
             lmax=32768),
        # a handful of accepted tokens of one small sequence
        dict(name="commit_one", op="commit", n=1, tq=8, depth=3, hkv=2, kv="bf16", ps=64, lmax=1000),
        # a batch's accepted paths in an FP8 cache
        dict(name="commit_fp8", op="commit", n=128, tq=64, depth=8, hkv=8, kv="fp8", ps=128, lmax=1500),
        # one short prompt of an odd length, three query heads to a kv head: latency
        dict(name="prompt_short", op="prompt", n=1, lmin=77, lmax=77, hq=12, hkv=4, q="fp16"),
        # a prefill batch of prompts from a few words to some thousand
        dict(name="prompt_ragged", op="prompt", n=23, lmin=20, lmax=4096, hq=64, hkv=8, q="bf16"),
        # one long document
        dict(name="prompt_long", op="prompt", n=1, lmin=32768, lmax=32768, hq=64, hkv=8, q="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(8, 1), (16, 2), (12, 4), (16, 16), (32, 4), (64, 8), (48, 8), (128, 1), (10, 2)]


def draw(rng):
    op = rng.choice(["tables", "mask", "tree", "tree", "commit", "prompt", "prompt"])
    hq, hkv = rng.choice(HEADS)
    q, ps = rng.choice(["bf16", "fp16"]), rng.choice([64, 128])
    if op == "tables":
        n, new_max = _log(rng, 1, 250), rng.choice([1, 1, 5, _log(rng, 10, 4000)])
        return dict(op=op, n=n, ps=ps, new_min=rng.randint(0, new_max), new_max=new_max, old=_log(rng, 100, 16000),
                    done=rng.choice([0, n // 8]))
    tq = _log(rng, 1, 125)
    depth = rng.randint(1, 10)
    if op == "mask":
        return dict(op=op, n=_log(rng, 1, 250), tq=tq, depth=depth)
    if op == "commit":
        return dict(op=op, n=_log(rng, 1, 100), tq=tq, depth=depth, hkv=hkv, kv=rng.choice([q, "fp8"]), ps=ps,
                    lmax=tq + _log(rng, 1, 1200))
    if op == "tree":
        per = rng.choice([1, 1, 1, 2, 7])
        n = per * _log(rng, 1, max(1, 64 // per))
        lmax = min(tq + _log(rng, 1, 30000), 32768 * 32 // n, 32768 * 64 * 16 * 64 // (n * tq * hq))
        lmax = max(lmax, tq + 1)
        return dict(op=op, n=n, per=per, tq=tq, depth=depth, hq=hq, hkv=hkv, q=q, ps=ps,
                    lmin=rng.randint(max(tq, (lmax - 1) // 2), lmax), lmax=lmax)
    lmax = _log(rng, 1, 12000)
    return dict(op=op, n=min(_log(rng, 1, 64), max(1, 40000 // lmax)), lmin=rng.randint(1, lmax), lmax=lmax, hq=hq,
                hkv=hkv, q=q)


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _dev(a, dtype):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def _rng(*parts):
    """A generator of a case's own numbers, the same for every seed."""
    x = 17
    for p in parts:
        x = (x * 1000003 + int(p)) & 0x7FFFFFFF
    return random.Random(x)


def _pages(n, ps):
    return -(-n // ps)


def _tables_lens(case):
    """Cached and new tokens of every request (-1: finished)."""
    r = _rng(case["n"], case["new_max"], case["old"])
    old = [r.randint(0, case["old"]) for _ in range(case["n"])]
    new = [max(0, _log(r, 1, case["new_max"] + 1) - 1 if case["new_max"] > 8 else
               r.randint(case["new_min"], case["new_max"])) for _ in range(case["n"])]
    new[0] = case["new_max"]
    for i in range(case["done"]):
        new[(i * 7 + 3) % case["n"]] = -1
    return old, new


def _prepare_tables(case, seed):
    n, ps = case["n"], case["ps"]
    old, new = _tables_lens(case)
    # what a request holds: its cached tokens' pages, and one more where drafted tokens were rejected
    held = [_pages(o, ps) + (i % 5 == 4) for i, o in enumerate(old)]
    width = max(_pages(o + max(x, 0), ps) for o, x in zip(old, new)) + 2
    want = sum(max(0, _pages(o + max(x, 0), ps) - h) for o, x, h in zip(old, new, held))
    pages = sum(held) + want + 37
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages).astype(np.int32)
    table, at = np.full((n, width), -1, np.int32), 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    free = np.zeros(pages, np.int32)
    free[:pages - at] = order[at:]
    total = sum(max(x, 0) for x in new)
    cap = total + (-total) % 64  # a padded batch, as a captured step has it
    s = {"case": case, "total_q": cap, "width": width, "pages": pages, "new": new}
    s["kv_lens"], s["new_lens"], s["held"] = _dev(old, torch.int32), _dev(new, torch.int32), _dev(held, torch.int32)
    s["block_tables"], s["free_pages"] = _dev(table, torch.int32), _dev(free, torch.int32)
    s["free_count"] = _dev([pages - at], torch.int32)
    e = lambda k, dt: torch.empty(k, dtype=dt, device="cuda")
    s["cu"], s["used"] = e(n + 1, torch.int64), e(n, torch.int32)
    s["positions"], s["loc"] = e(cap, torch.int64), e(cap, torch.int64)
    s["held_out"], s["free_count_out"] = e(n, torch.int32), e(1, torch.int32)
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(n, cap, 8, 8, 1, ps, pages, width)
    return s


def _tree(r, tq, depth):
    """Parents of a tree's tokens, level by level; the first level is at least as wide as the tree is deep."""
    first = min(tq, max(depth + 1, -(-tq // depth)))
    parents, level, lo, d = [-1] * first, first, 0, 1
    while len(parents) < tq:
        width = tq - len(parents) if d >= depth - 1 else min(tq - len(parents), r.randint(1, max(1, tq // depth)))
        parents += sorted(r.randrange(lo, lo + level) for _ in range(width))
        lo, level, d = len(parents) - width, width, d + 1
    return parents


def _trees(case, seed):
    r = random.Random(seed * 31 + case["tq"])
    return [_tree(r, case["tq"], case["depth"]) for _ in range(case["n"])]


def _words(case):
    return -(-case["tq"] // 32)


def _tree_lens(case):
    r = _rng(case["n"], case["tq"], case["lmax"])
    lens = [r.randint(case["lmin"], case["lmax"]) for _ in range(case["n"])]
    lens[0] = case["lmax"]
    return lens


def _prepare_mask(case, seed):
    n, tq = case["n"], case["tq"]
    r = _rng(n, tq)
    s = {"case": case, "parents": _dev(np.array(_trees(case, seed)).reshape(-1), torch.int32)}
    s["cu"] = _dev(np.arange(n + 1) * tq, torch.int64)
    s["lens"] = _dev([tq + r.randint(0, 30000) for _ in range(n)], torch.int32)
    s["mask"] = torch.empty(n * tq, _words(case), dtype=torch.int32, device="cuda")
    s["positions"] = torch.empty(n * tq, dtype=torch.int64, device="cuda")
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(n, n * tq, 8, 8, 1, 64, 1, 1024)
    return s


def _shared_len(case):
    """Keys that a group's sequences have in common: nine tenths of the shortest's committed ones."""
    return 0 if case["per"] == 1 else (case["lmin"] - case["tq"]) * 9 // 10


def _prepare_tree(case, seed):
    g, t = _gen(seed), TORCH[case["q"]]
    n, per, tq, ps, hq, hkv = (case[k] for k in ("n", "per", "tq", "ps", "hq", "hkv"))
    lens, common = _tree_lens(case), _shared_len(case)
    width, pages = max(_pages(l, ps) for l in lens), 0
    table = np.full((n, width), -1, np.int32)
    for i, l in enumerate(lens):
        first, whole = i // per * per, 0 if i % per == 0 else common // ps
        table[i, :whole] = table[first, :whole]
        table[i, whole:_pages(l, ps)] = np.arange(pages, pages + _pages(l, ps) - whole)
        pages += _pages(l, ps) - whole
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages).astype(np.int32)
    s = {"case": case, "lens_host": lens}
    s["block_tables"] = _dev(np.where(table >= 0, order[np.maximum(table, 0)], -1), torch.int32)
    s["k_cache"] = torch.empty(pages, hkv, ps, DIM, dtype=t, device="cuda").normal_(generator=g)
    s["v_cache"] = torch.empty(pages, hkv, ps, DIM, dtype=t, device="cuda").normal_(generator=g)
    if common:  # the same keys through every row of a group, also in the page where the common part ends
        head, off = common // ps, common % ps
        for i in range(n):
            if off and i % per:
                a, b = (int(s["block_tables"][x, head]) for x in (i, i // per * per))
                s["k_cache"][a, :, :off] = s["k_cache"][b, :, :off]
                s["v_cache"][a, :, :off] = s["v_cache"][b, :, :off]
    s["q"] = _normal(g, n * tq, hq, DIM, dtype=t, scale=2.0)
    s["cu"], s["lens"] = _dev(np.arange(n + 1) * tq, torch.int64), _dev(lens, torch.int32)
    # every token's ancestors and itself, as bits
    bits = np.zeros((n * tq, 32 * _words(case)), bool)
    for i, parents in enumerate(_trees(case, seed)):
        for j, p in enumerate(parents):
            if p >= 0:
                bits[i * tq + j] = bits[i * tq + p]
            bits[i * tq + j, j] = True
    s["mask"] = _dev(np.packbits(bits, axis=1, bitorder="little").view(np.int32), torch.int32)
    s["out"] = torch.empty(n * tq, hq, DIM, dtype=t, device="cuda")
    s["lse"] = torch.empty(hq, n * tq, dtype=torch.float32, device="cuda")
    s["group_ptr"] = s["prefix_lens"] = None
    if common:
        s["group_ptr"] = _dev(np.arange(0, n + 1, per), torch.int32)
        s["prefix_lens"] = _dev([common] * (n // per), torch.int32)
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(n, n * tq, hq, hkv, 1, ps, pages, width, q_dtype=t)
        s["ws"] = torch.empty(mx.dense_shared_workspace_size(s["prob"]), dtype=torch.uint8, device="cuda")
    return s


def _paths(case, seed):
    """An accepted path of each tree: the first token, then children while there are any, sometimes cut short."""
    r, out = random.Random(seed * 17 + 5), []
    for parents in _trees(case, seed):
        path = [0]
        while r.random() < 0.85:
            kids = [j for j, p in enumerate(parents) if p == path[-1]]
            if not kids:
                break
            path.append(r.choice(kids))
        out.append(path if r.random() < 0.95 else [])
    return out


def _prepare_commit(case, seed):
    g = _gen(seed)
    n, tq, ps, hkv, t = case["n"], case["tq"], case["ps"], case["hkv"], TORCH[case["kv"]]
    r = _rng(n, tq, case["lmax"])
    lens = [r.randint(tq, case["lmax"]) for _ in range(n)]
    lens[0] = case["lmax"]
    width = max(_pages(l, ps) for l in lens)
    pages = sum(_pages(l, ps) for l in lens)
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages).astype(np.int32)
    table, at = np.full((n, width), -1, np.int32), 0
    for i, l in enumerate(lens):
        table[i, :_pages(l, ps)] = order[at:at + _pages(l, ps)]
        at += _pages(l, ps)
    paths = _paths(case, seed)
    path = np.full((n, case["depth"] + 1), -1, np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    s = {"case": case, "block_tables": _dev(table, torch.int32), "path": _dev(path, torch.int32)}
    s["path_lens"] = _dev([len(p) for p in paths], torch.int32)
    s["cu"], s["lens"] = _dev(np.arange(n + 1) * tq, torch.int64), _dev(lens, torch.int32)
    s["k_cache"], s["v_cache"] = (_normal(g, pages, hkv, ps, DIM, dtype=torch.float32).to(t) for _ in range(2))
    s["lens_out"] = torch.empty(n, dtype=torch.int32, device="cuda")
    if own:
        import block_sparse_attention_builder_gb300 as mx
        q = torch.bfloat16 if case["kv"] == "fp8" else t
        s["prob"] = mx.make_problem(n, n * tq, hkv, hkv, 1, ps, pages, width, q_dtype=q, kv_dtype=t)
    return s


def _prompt_lens(case):
    r = _rng(case["n"], case["lmin"], case["lmax"])
    lens = [_log(r, case["lmin"], case["lmax"]) for _ in range(case["n"])]
    lens[-1] = case["lmax"]
    return lens


def _prepare_prompt(case, seed):
    g, t, hq, hkv = _gen(seed), TORCH[case["q"]], case["hq"], case["hkv"]
    lens = _prompt_lens(case)
    total = sum(lens)
    # q, k and v are views of one packed projection
    qkv = _normal(g, total, (hq + 2 * hkv) * DIM, dtype=t)
    s = {"case": case, "lens_host": lens, "q": qkv[:, :hq * DIM].unflatten(1, (hq, DIM)).mul_(2),
         "k": qkv[:, hq * DIM:(hq + hkv) * DIM].unflatten(1, (hkv, DIM)),
         "v": qkv[:, (hq + hkv) * DIM:].unflatten(1, (hkv, DIM))}
    s["cu"] = _dev(np.cumsum([0] + lens), torch.int64)
    s["out"] = torch.empty(total, hq, DIM, dtype=t, device="cuda")
    s["lse"] = torch.empty(hq, total, dtype=torch.float32, device="cuda")
    if own:
        import block_sparse_attention_builder_gb300 as mx
        s["prob"] = mx.make_problem(len(lens), total, hq, hkv, 1, 64, 1, 1, True, q_dtype=t)
        s["ws"] = torch.empty(mx.prompt_workspace_size(s["prob"]), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return {"tables": _prepare_tables, "mask": _prepare_mask, "tree": _prepare_tree, "commit": _prepare_commit,
            "prompt": _prepare_prompt}[case["op"]](case, seed)


# ------------------------------------------------------------- the plain forms
def _plain_tables(s):
    c, cap, ps = s["case"], s["total_q"], s["case"]["ps"]
    old, new, held, table = s["kv_lens"].long(), s["new_lens"].long(), s["held"].long(), s["block_tables"].long()
    free, count = s["free_pages"].long(), s["free_count"].long()
    live = new >= 0
    n = new.clamp(min=0)
    used = torch.where(live, old + n, 0)
    col = torch.arange(s["width"], device="cuda")
    # finished requests give their pages back, behind the free ones
    back = (~live)[:, None] & (col < held[:, None])
    at = count + back.view(-1).long().cumsum(0).view_as(back) - 1
    spare = torch.cat([free, free.new_zeros(1)])
    spare[torch.where(back, at, len(free)).view(-1)] = table.view(-1)
    free = spare[:-1]
    top = count + back.sum()
    # pages for the new tokens, from the end of the list
    held = torch.where(live, held, 0)
    need = ((used + ps - 1) // ps - held).clamp(min=0)
    first = need.cumsum(0) - need
    k = first[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, free[(top - 1 - k).clamp(0, len(free) - 1)], table)
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    # every token's position and slot
    t = torch.arange(cap, device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["n"] - 1)
    there = t < cu[-1]
    pos = (used - n)[seq] + t - cu[seq]
    page = table[seq, (pos // ps).clamp(0, s["width"] - 1)]
    i32 = torch.int32
    return (cu, used.to(i32), torch.where(there, pos, -1), torch.where(there, page * ps + pos % ps, -1),
            table.to(i32), free.to(i32), (held + need).to(i32), (top - need.sum()).to(i32))


def _plain_mask(s):
    c = s["case"]
    n, tq, w = c["n"], c["tq"], _words(c)
    at = s["parents"].long().view(n, tq)
    seen = torch.eye(32 * w, dtype=torch.bool, device="cuda")[:tq].repeat(n, 1, 1)
    spare = torch.cat([seen, seen.new_zeros(n, tq, 1)], 2)  # the last column takes the roots' missing parents
    depth = torch.zeros_like(at)
    up = torch.cat([at, at.new_full((n, 1), -1)], 1)
    for _ in range(c["depth"]):
        spare.scatter_(2, torch.where(at >= 0, at, 32 * w)[..., None], True)
        depth += at >= 0
        at = up.gather(1, torch.where(at >= 0, at, tq))
    bits = spare[..., :32 * w].view(n * tq, w, 32).long() << torch.arange(32, device="cuda")
    word = bits.sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    return word, (s["lens"].long()[:, None] - tq + depth).view(-1)


def _plain_tree(s):
    c = s["case"]
    n, tq, ps, hkv, w = c["n"], c["tq"], c["ps"], c["hkv"], _words(c)
    scale = DIM ** -0.5
    j = torch.arange(tq, device="cuda")
    bit = (s["mask"].long()[:, j // 32] >> (j % 32)) & 1  # [n * tq, tq]
    out, lses = [], []
    for i, L in enumerate(s["lens_host"]):
        p = torch.arange(L, device="cuda")
        page = s["block_tables"][i].long()[p // ps]
        k = s["k_cache"][page, :, p % ps].float().transpose(0, 1)  # [hkv, L, DIM]
        v = s["v_cache"][page, :, p % ps].float().transpose(0, 1)
        q = s["q"][i * tq:(i + 1) * tq].float().view(tq, hkv, -1, DIM).permute(1, 0, 2, 3) * scale
        a = (q.reshape(hkv, -1, DIM) @ k.transpose(1, 2)).view(hkv, tq, -1, L)
        a[..., L - tq:].masked_fill_(bit[i * tq:(i + 1) * tq, None] == 0, -math.inf)
        m = a.amax(-1, keepdim=True)
        a = a.sub_(m).exp_()
        l = a.sum(-1, keepdim=True)
        o = (a.view(hkv, -1, L) @ v).view(hkv, tq, -1, DIM) / l
        out.append(o.permute(1, 0, 2, 3).reshape(tq, c["hq"], DIM))
        lses.append((m + l.log())[..., 0].permute(0, 2, 1).reshape(c["hq"], tq))
    return torch.cat(out).to(s["q"].dtype), torch.cat(lses, 1)


def _plain_commit(s):
    c = s["case"]
    ps, wide = c["ps"], s["path"].shape[1]
    base = (s["lens"].long() - c["tq"])[:, None]
    k = torch.arange(wide, device="cuda")
    there = k < s["path_lens"][:, None]
    src = base + torch.where(there, s["path"].long(), 0)
    dst = torch.where(there, base + k, src)  # (nothing to move: a row onto itself)
    last = s["block_tables"].shape[1] - 1
    page = lambda p: s["block_tables"].long().gather(1, (p // ps).clamp(max=last)).view(-1)
    sp, so, dp, do = page(src), (src % ps).view(-1), page(dst), (dst % ps).view(-1)
    there = there.view(-1)
    # (where nothing moves, the first slot of the sequence's path onto itself, with what it gets)
    home = torch.arange(len(there), device="cuda") // wide * wide
    pick = torch.where(there, torch.arange(len(there), device="cuda"), home)
    sp, so, dp, do = sp[pick], so[pick], dp[pick], do[pick]
    bits = torch.uint8 if s["k_cache"].element_size() == 1 else torch.int16
    for cache in (s["k_cache"].view(bits), s["v_cache"].view(bits)):
        cache[dp, :, do] = cache[sp, :, so]
    s["lens_out"].copy_(s["lens"] - c["tq"] + s["path_lens"])
    return s["k_cache"], s["v_cache"], s["lens_out"]


def _plain_prompt(s):
    c, hkv, hq = s["case"], s["case"]["hkv"], s["case"]["hq"]
    out, lses, at = [], [], 0
    for L in s["lens_host"]:
        k = s["k"][at:at + L].float().permute(1, 2, 0)  # [hkv, DIM, L]
        v = s["v"][at:at + L].float().transpose(0, 1)
        step = max(1, min(L, (1 << 30) // (hq * L)))  # rows whose scores fit in 4 GB
        for t0 in range(0, L, step):
            t1 = min(L, t0 + step)
            q = s["q"][at + t0:at + t1].float().view(t1 - t0, hkv, -1, DIM).permute(1, 0, 2, 3) * DIM ** -0.5
            a = (q.reshape(hkv, -1, DIM) @ k[..., :t1]).view(hkv, t1 - t0, -1, t1)
            late = torch.arange(t1, device="cuda") > torch.arange(t0, t1, device="cuda")[:, None]
            a.masked_fill_(late[:, None], -math.inf)
            m = a.amax(-1, keepdim=True)
            a = a.sub_(m).exp_()
            l = a.sum(-1, keepdim=True)
            o = (a.view(hkv, -1, t1) @ v[:, :t1]).view(hkv, t1 - t0, -1, DIM) / l
            out.append(o.permute(1, 0, 2, 3).reshape(t1 - t0, hq, DIM).to(s["q"].dtype))
            lses.append((m + l.log())[..., 0].permute(0, 2, 1).reshape(hq, t1 - t0))
        at += L
    return torch.cat(out), torch.cat(lses, 1)


# ------------------------------------------------------- the framework's calls
def _own_tables(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.build_tables(s["prob"], s["kv_lens"], s["new_lens"], s["held"], s["block_tables"], s["free_pages"],
                    s["free_count"], s["cu"], s["used"], s["positions"], s["loc"], pages_held_out=s["held_out"],
                    free_count_out=s["free_count_out"])
    return (s["cu"], s["used"], s["positions"], s["loc"], s["block_tables"], s["free_pages"], s["held_out"],
            s["free_count_out"])


def _own_mask(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.tree_mask(s["prob"], s["parents"], s["cu"], s["lens"], s["mask"], s["positions"])
    return s["mask"], s["positions"]


def _own_tree(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.tree_fwd(s["prob"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["cu"], s["lens"], s["mask"],
                s["group_ptr"], s["prefix_lens"], s["ws"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _own_commit(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.tree_commit(s["prob"], s["cu"], s["lens"], s["block_tables"], s["path"], s["path_lens"], s["k_cache"],
                   s["v_cache"], kv_lens_out=s["lens_out"])
    return s["k_cache"], s["v_cache"], s["lens_out"]


def _own_prompt(s):
    import block_sparse_attention_builder_gb300 as mx
    mx.prompt_fwd(s["prob"], s["q"], s["k"], s["v"], s["cu"], s["ws"], s["out"], s["lse"])
    return s["out"], s["lse"]


PLAIN = {"tables": _plain_tables, "mask": _plain_mask, "tree": _plain_tree, "commit": _plain_commit,
         "prompt": _plain_prompt}
OWN = {"tables": _own_tables, "mask": _own_mask, "tree": _own_tree, "commit": _own_commit, "prompt": _own_prompt}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- the floor
def work(case):
    op = case["op"]
    if op == "tables":
        old, new = _tables_lens(case)
        tokens = sum(max(x, 0) for x in new)
        fresh = sum(max(0, _pages(o + max(x, 0), case["ps"]) - _pages(o, case["ps"]) - (i % 5 == 4))
                    for i, (o, x) in enumerate(zip(old, new)))
        return {"bytes": case["n"] * 28 + fresh * 8 + tokens * 16, "flops": tokens * 4.0}
    if op == "mask":
        tokens = case["n"] * case["tq"]
        return {"bytes": tokens * (4 + 4 * _words(case) + 8), "flops": tokens * 4.0}
    if op == "commit":
        row = DIM * (1 if case["kv"] == "fp8" else 2)
        # (a path's expected length; its first token stays where it is)
        moved = case["n"] * max(1, min(case["depth"], case["tq"]) // 2)
        return {"bytes": moved * case["hkv"] * 4 * row + case["n"] * 20, "flops": moved * 4.0}
    row = DIM * 2
    if op == "tree":
        lens, common, tq = _tree_lens(case), _shared_len(case), case["tq"]
        keys = sum(lens) - common * (case["n"] - case["n"] // case["per"])
        rows = case["n"] * tq
        return {"bytes": keys * case["hkv"] * 2 * row + rows * case["hq"] * (2 * row + 4) + rows * 4 * _words(case),
                "flops": 4.0 * DIM * case["hq"] * tq * sum(l - tq + min(tq, case["depth"]) / 2 for l in lens)}
    lens = _prompt_lens(case)
    total = sum(lens)
    return {"bytes": total * (case["hq"] * (2 * row + 4) + case["hkv"] * 2 * row),
            "flops": 4.0 * DIM * case["hq"] * sum(l * (l + 1) / 2 for l in lens)}


# --------------------------------------------------- the definition in 64 bits
def _exact_tables(s):
    """Request by request, token by token, on the host."""
    c, ps = s["case"], s["case"]["ps"]
    old, new, held, free = (s[k].tolist() for k in ("kv_lens", "new_lens", "held", "free_pages"))
    table, top = s["block_tables"].cpu().numpy().copy(), int(s["free_count"][0])
    for i in range(c["n"]):
        if new[i] < 0:
            for p in table[i, :held[i]]:
                free[top] = int(p)
                top += 1
            old[i] = new[i] = held[i] = 0
    cu, used, pos, loc = [0], [], [], []
    for i in range(c["n"]):
        while held[i] * ps < old[i] + new[i]:
            top -= 1
            table[i, held[i]] = free[top]
            held[i] += 1
        for p in range(old[i], old[i] + new[i]):
            pos.append(p)
            loc.append(int(table[i, p // ps]) * ps + p % ps)
        cu.append(len(pos))
        used.append(old[i] + new[i])
    pad = [-1] * (s["total_q"] - len(pos))
    i32, i64 = torch.int32, torch.int64
    return (_dev(cu, i64), _dev(used, i32), _dev(pos + pad, i64), _dev(loc + pad, i64), _dev(table, i32),
            _dev(free, i32), _dev(held, i32), _dev([top], i32))


def _exact_mask(s):
    """Token by token: the parent's row and its own bit."""
    c = s["case"]
    tq, parents, lens = c["tq"], s["parents"].tolist(), s["lens"].tolist()
    rows, depth = [], []
    for t, p in enumerate(parents):
        up = t - t % tq + p
        rows.append((rows[up] if p >= 0 else 0) | 1 << (t % tq))
        depth.append(depth[up] + 1 if p >= 0 else 0)
    words = [[(r >> (32 * w) & 0xFFFFFFFF) for w in range(_words(c))] for r in rows]
    return (_dev(np.array(words, np.uint32).view(np.int32), torch.int32),
            _dev([lens[t // tq] - tq + d for t, d in enumerate(depth)], torch.int64))


def _softmax_rows(q, k, v, seen):
    """q [t, hkv, G, DIM], k and v [keys, hkv, DIM], seen [t, keys]: rows and log-sum-exps in 64 bits."""
    a = torch.einsum("tgrd,pgd->tgrp", q.double(), k.double()) / math.sqrt(DIM)
    a.masked_fill_(~seen[:, None, None], -math.inf)
    o = torch.einsum("tgrp,pgd->tgrd", torch.softmax(a, -1), v.double())
    return o.flatten(1, 2), torch.logsumexp(a, -1).flatten(1)


def _exact_tree(s):
    c = s["case"]
    tq, ps = c["tq"], c["ps"]
    out, lses = [], []
    words = s["mask"].cpu().numpy().view(np.uint32)
    for i, L in enumerate(s["lens_host"]):
        rows = s["block_tables"][i].long().repeat_interleave(ps)[:L] * ps + torch.arange(L, device="cuda") % ps
        flat = lambda cache: cache.transpose(1, 2).reshape(-1, c["hkv"], DIM)
        if i == 0:
            k_rows, v_rows = flat(s["k_cache"]), flat(s["v_cache"])  # by slot
        seen = np.ones((tq, L), bool)
        for t in range(tq):
            for j in range(tq):
                seen[t, L - tq + j] = words[i * tq + t, j // 32] >> (j % 32) & 1
        q = s["q"][i * tq:(i + 1) * tq].view(tq, c["hkv"], -1, DIM)
        o, l = _softmax_rows(q, k_rows[rows], v_rows[rows], torch.from_numpy(seen).cuda())
        out.append(o)
        lses.append(l)
    return torch.cat(out), torch.cat(lses).T.contiguous()


def _exact_commit(s):
    """Sequence by sequence, on copies of the rows."""
    c = s["case"]
    tq, ps = c["tq"], c["ps"]
    k, v = (x.to(torch.float32).double() for x in (s["k_cache"], s["v_cache"]))
    table, path, count, lens = (s[n].tolist() for n in ("block_tables", "path", "path_lens", "lens"))
    out, moves = [], []
    for i in range(c["n"]):
        base = lens[i] - tq
        for j in range(count[i]):
            a, b = base + path[i][j], base + j
            moves.append((table[i][a // ps], a % ps, table[i][b // ps], b % ps))
        out.append(base + count[i])
    if moves:
        sp, so, dp, do = (_dev(x, torch.int64) for x in zip(*moves))
        for cache in (k, v):
            rows = cache[sp, :, so].clone()
            cache[dp, :, do] = rows
    return k, v, _dev(out, torch.int32)


def _exact_prompt(s):
    c, out, lses, at = s["case"], [], [], 0
    for L in s["lens_host"]:
        for t0 in range(0, L, 256):
            t1 = min(L, t0 + 256)
            q = s["q"][at + t0:at + t1].reshape(t1 - t0, c["hkv"], -1, DIM)
            seen = torch.ones(t1 - t0, t1, dtype=torch.bool, device="cuda").tril(t0)
            o, l = _softmax_rows(q, s["k"][at:at + t1], s["v"][at:at + t1], seen)
            out.append(o)
            lses.append(l)
        at += L
    return torch.cat(out), torch.cat(lses).T.contiguous()


def exact(case, seed):
    if work(case)["flops"] > 4e12:  # (64-bit products of that size take over 20 seconds)
        return None
    s = prepare(case, seed)
    return {"tables": _exact_tables, "mask": _exact_mask, "tree": _exact_tree, "commit": _exact_commit,
            "prompt": _exact_prompt}[case["op"]](s)
