"""Refusals of the speculative step's and the whole-prompt calls before any
launch, in the C ABI and in the binding (no GPU)."""
import ctypes

import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B

P = ctypes.c_void_p
FAKE, FAKE2, FAKE8 = P(1 << 20), P((1 << 20) + 2), P((1 << 20) + 8)  # never dereferenced: validation fails first
BF, HALF, I32, I64 = torch.bfloat16, torch.float16, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mx.library()


def _prob(**kw):
    base = dict(num_seqs=2, total_q=4, num_q_heads=16, num_kv_heads=2, topk=0, page_size=64, num_pages=10,
                max_pages_per_seq=5, causal=True)
    base.update(kw)
    return mx.make_problem(**base)


BAD_SHAPES = [(dict(num_seqs=0), 1), (dict(num_q_heads=12, num_kv_heads=5), 1), (dict(total_q=-1), 1),
              (dict(softmax_scale=-1.0), 1), (dict(head_dim=64), 2), (dict(num_q_heads=256, num_kv_heads=1), 2),
              (dict(q_dtype=HALF, kv_dtype=BF), 2)]


def caller(fn, names, prob_at=0):
    """A call of fn by its arguments' names; None in `names`' values: the stream."""
    def call(prob=None, **kw):
        a = dict(names, **kw)
        pr = ctypes.byref(_prob() if prob is None else prob)
        return fn(pr, *a.values(), None)
    return call


def refuses(call, pointers, align, required, optional=()):
    for n in required:
        assert call(**{n: None}) == 1, n
    for n in tuple(required) + tuple(optional):
        bad = FAKE2 if align.get(n, 4) == 4 else (P((1 << 20) + 4) if align[n] == 8 else FAKE8)
        assert call(**{n: bad}) == 1, n


def test_tree_fwd(lib):
    p = _prob()
    nb = mx.dense_shared_workspace_size(p)
    names = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cu=FAKE, lens=FAKE, mask=FAKE, words=1, ng=0, gp=None, pl=None,
                 ws=FAKE, nb=nb, out=FAKE, lse=None, flags=None)
    call = caller(lib.mxsa_tree_fwd, names)
    refuses(call, None, dict(q=16, k=16, v=16, out=16, cu=8, ws=16), ["q", "k", "v", "bt", "cu", "lens", "mask", "ws", "out"],
            ["lse", "flags"])
    assert call(words=0) == 1 and call(words=-1) == 1 and call(words=65) == 2
    assert call(nb=nb - 256) == 3
    assert call(ng=3) == 1 and call(ng=-1) == 1 and call(ng=1) == 1 and call(ng=1, gp=FAKE) == 1
    for kw, status in BAD_SHAPES + [(dict(num_seqs=1025), 2), (dict(kv_dtype=torch.float8_e4m3fn), 2),
                                    (dict(page_size=32), 2)]:
        assert call(prob=_prob(**kw)) == status, kw
    assert lib.mxsa_tree_fwd(None, *names.values(), None) == 1


def test_tree_mask(lib):
    names = dict(parents=FAKE, cu=FAKE, lens=FAKE, words=1, mask=FAKE, pos=FAKE, flags=None)
    call = caller(lib.mxsa_tree_mask, names)
    refuses(call, None, dict(cu=8, pos=8), ["parents", "cu", "lens", "mask"], ["pos", "flags"])
    assert call(words=0) == 1 and call(words=65) == 2 and call(prob=_prob(num_seqs=1025)) == 2
    assert lib.mxsa_tree_mask(None, *names.values(), None) == 1


def test_tree_commit(lib):
    names = dict(cu=FAKE, lens=FAKE, bt=FAKE, path=FAKE, wide=4, n=FAKE, k=FAKE, v=FAKE, idx=None, ih=0, idim=0,
                 out=None, flags=None)
    call = caller(lib.mxsa_tree_commit, names)
    refuses(call, None, dict(cu=8, k=16, v=16, idx=16), ["cu", "lens", "bt", "path", "n", "k", "v"], ["out", "flags"])
    assert call(wide=0) == 1
    assert call(out=FAKE) == 1  # the lengths themselves: other heads still read them
    for off in (-4, 4):  # nor part of them
        assert call(out=P((1 << 20) + off)) == 1
    other = P(1 << 21)
    assert call(out=other, idx=FAKE, ih=0, idim=64) == 1 and call(idx=FAKE, ih=1, idim=60) == 1
    assert call(idx=FAKE8, ih=1, idim=64) == 1
    assert call(prob=_prob(kv_dtype="nvfp4"), idx=FAKE, ih=1, idim=64) == 2
    for kw, status in BAD_SHAPES + [(dict(page_size=32), 2)]:
        assert call(prob=_prob(**kw)) == status, kw
    assert lib.mxsa_tree_commit(None, *names.values(), None) == 1


def test_prompt_fwd(lib):
    p = _prob(page_size=0, num_pages=0, max_pages_per_seq=0)  # (no pages: not looked at)
    nb = mx.prompt_workspace_size(p)
    names = dict(q=FAKE, qs=2048, k=FAKE, ks=256, v=FAKE, vs=256, cu=FAKE, ws=FAKE, nb=nb, out=FAKE, lse=None, flags=None)
    call = caller(lib.mxsa_prompt_fwd, names)
    refuses(call, None, dict(q=16, k=16, v=16, out=16, cu=8, ws=16), ["q", "k", "v", "cu", "ws", "out"], ["lse", "flags"])
    assert call(nb=nb - 1) == 3
    for kw in (dict(qs=2040), dict(qs=2052), dict(ks=248), dict(vs=0), dict(vs=-256), dict(ks=1 << 37)):
        assert call(**kw) == 1, kw
    for kw, status in BAD_SHAPES + [(dict(num_seqs=1025), 2), (dict(kv_dtype=torch.float8_e4m3fn), 2)]:
        assert call(prob=_prob(**kw)) == status, kw
    assert call(prob=_prob(total_q=1 << 28)) == 2  # rows past 32 bits
    assert lib.mxsa_prompt_fwd(None, *names.values(), None) == 1
    assert lib.mxsa_prompt_workspace_size(ctypes.byref(p), None) == 1


def test_build_tables(lib):
    names = {n: FAKE for n in ("kv", "new", "held", "bt", "free", "count", "cu", "used", "pos", "loc", "held_out",
                               "count_out")}
    names["flags"] = None
    call = caller(lib.mxsa_build_tables, names)
    refuses(call, None, dict(cu=8, pos=16, loc=16), list(names)[:12], ["flags"])
    assert call(prob=_prob(num_seqs=1025)) == 2 and call(prob=_prob(page_size=32)) == 2
    assert call(prob=_prob(num_pages=0)) == 1
    assert lib.mxsa_build_tables(None, *names.values(), None) == 1


# ---------------------------------------------------------------- the binding
class Reached(Exception):
    pass


class NoCall:
    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(mx.library(), name)

        def call(*args):
            raise Reached(name)
        return call


def z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


@pytest.fixture
def check(lib, monkeypatch):
    monkeypatch.setattr(mx, "_lib", NoCall())
    monkeypatch.setattr(mx, "_stream", lambda s: 0)

    def run(fn, good, wrong, optional=(), raw=()):
        with pytest.raises(Reached):
            fn(**good)
        with pytest.raises(Reached):
            fn(**dict(good, **dict.fromkeys(optional)))
        for name, t in raw:
            with pytest.raises(Reached):
                fn(**dict(good, **{name: t}))
        for name, t in wrong:
            with pytest.raises(mx.MxsaError) as ei:
                fn(**dict(good, **{name: t}))
            assert ei.value.status == 1 and name in str(ei.value), (name, str(ei.value))
    return run


def ints(good, names):
    """Every integer tensor in the other width, and every tensor one element short."""
    for n in names:
        t = good[n]
        yield n, (t.long() if t.dtype is I32 else torch.zeros(2 * t.numel(), dtype=I32))
        yield n, t.flatten()[:-1].contiguous()
        yield n, t.double()


def test_binding_of_tree_fwd(check):
    p = _prob()
    cache = z(10, 2, 64, 128)
    good = dict(prob=p, q=z(4, 16, 128), k_cache=cache, v_cache=cache, block_tables=z(2, 5, dt=I32),
                cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32), tree_mask=z(4, 2, dt=I32),
                group_ptr=z(2, dt=I32), prefix_lens=z(1, dt=I32),
                ws=z(mx.dense_shared_workspace_size(p), dt=torch.uint8), out=z(4, 16, 128),
                lse=z(16, 4, dt=torch.float32), flags=z(1, dt=I32))
    wrong = list(ints(good, ["block_tables", "cu_seqlens_q", "used_kv_lens", "group_ptr"]))
    for n in ("q", "k_cache", "v_cache", "out"):
        wrong += [(n, good[n].to(HALF)), (n, good[n].float()), (n, good[n][:-1])]
    wrong += [("tree_mask", z(4, 2, dt=I64)), ("tree_mask", z(3, 2, dt=I32)), ("tree_mask", z(8, dt=I32)),
              ("tree_mask", z(4, 4, dt=I32)[:, ::2]), ("lse", z(16, 3, dt=torch.float32)), ("flags", z(1, dt=I64)),
              ("prefix_lens", None)]
    check(mx.tree_fwd, good, wrong, ("lse", "flags"), [("tree_mask", z(4, 2, dt=I32).view(torch.uint32)),
                                                       ("q", good["q"].view(torch.int16))])


def test_binding_of_tree_mask(check):
    good = dict(prob=_prob(), parents=z(4, dt=I32), cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32),
                mask=z(4, 1, dt=I32), positions=z(4, dt=I64), flags=z(1, dt=I32))
    wrong = list(ints(good, ["parents", "cu_seqlens_q", "used_kv_lens", "positions"])) + [("mask", z(4, 1, dt=I64))]
    check(mx.tree_mask, good, wrong, ("positions", "flags"))


@pytest.mark.parametrize("kv", [BF, torch.float8_e4m3fn, "nvfp4"])
def test_binding_of_tree_commit(check, kv):
    fp4 = kv == "nvfp4"
    cache = z(10, 2, 64 * 72, dt=torch.uint8) if fp4 else torch.zeros(10, 2, 64, 128).to(kv)
    good = dict(prob=_prob(kv_dtype=kv), cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32),
                block_tables=z(2, 5, dt=I32), path=z(2, 4, dt=I32), path_lens=z(2, dt=I32), k_cache=cache,
                v_cache=cache, kv_lens_out=z(2, dt=I32), flags=z(1, dt=I32))
    if not fp4:
        good["idx_cache"] = torch.zeros(10, 3, 64, 32).to(kv)
    wrong = list(ints(good, ["cu_seqlens_q", "used_kv_lens", "block_tables", "path_lens", "kv_lens_out"]))
    wrong += [("path", z(8, dt=I32)), ("path", z(2, 4, dt=I64)), ("path", z(1, 4, dt=I32)),
              ("k_cache", cache[:9]), ("v_cache", cache.view(torch.uint8).float())]
    if not fp4:
        wrong += [("idx_cache", good["idx_cache"][:9]), ("idx_cache", good["idx_cache"][:, :, :60]),
                  ("idx_cache", good["idx_cache"].float())]
    check(mx.tree_commit, good, wrong, ("kv_lens_out", "flags") + (() if fp4 else ("idx_cache",)))


def test_binding_of_prompt_fwd(check):
    p = _prob()
    flat = z(4, 20 * 128)
    good = dict(prob=p, q=flat[:, :2048].unflatten(1, (16, 128)), k=flat[:, 2048:2304].unflatten(1, (2, 128)),
                v=flat[:, 2304:].unflatten(1, (2, 128)), cu_seqlens=z(3, dt=I64),
                ws=z(mx.prompt_workspace_size(p), dt=torch.uint8), out=z(4, 16, 128), lse=z(16, 4, dt=torch.float32),
                flags=z(1, dt=I32))
    wrong = list(ints(good, ["cu_seqlens"]))
    for n, h in (("q", 16), ("k", 2), ("v", 2)):
        wrong += [(n, z(3, h, 128)), (n, z(4, h, 128, dt=HALF)), (n, z(4, h, 128, dt=torch.float32)), (n, z(4, h, 64)),
                  (n, z(4, 128, h).transpose(1, 2)), (n, z(h, 4, 128).transpose(0, 1))]
    wrong += [("out", z(3, 16, 128)), ("out", z(16, 4, 128).transpose(0, 1)), ("out", z(4, 16, 128, dt=HALF)),
              ("lse", z(16, 4, dt=torch.float64)), ("flags", z(1, dt=I64))]
    check(mx.prompt_fwd, good, wrong, ("lse", "flags"), [("q", z(4, 16, 128))])


def test_binding_of_build_tables(check):
    good = dict(prob=_prob(), kv_lens=z(2, dt=I32), new_lens=z(2, dt=I32), pages_held=z(2, dt=I32),
                block_tables=z(2, 5, dt=I32), free_pages=z(10, dt=I32), free_count=z(1, dt=I32),
                cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32), positions=z(4, dt=I64), loc=z(4, dt=I64),
                pages_held_out=z(2, dt=I32), free_count_out=z(1, dt=I32), flags=z(1, dt=I32))
    wrong = [x for n in list(good)[1:13] for x in ints(good, [n])] + [("block_tables", z(5, 2, dt=I32).T)]
    check(mx.build_tables, good, wrong, ("pages_held_out", "free_count_out", "flags"))
