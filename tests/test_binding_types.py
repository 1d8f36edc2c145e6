"""The binding refuses tensors of another type before the C call (no GPU).

A pointer carries no type: an int64 list of groups read as int32 would lose
its groups without a flag, and rows of the other 16-bit type would be read as
wrong numbers.  Integer tensors stand for raw bytes where rows are expected.
"""
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B

BF, HALF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
I32, I64 = torch.int32, torch.int64


class Reached(Exception):
    pass


class NoCall:
    """The library, of which only the size queries run: a call that comes through the checks raises Reached."""

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(mx.library(), name)

        def call(*args):
            raise Reached(name)
        return call


@pytest.fixture
def no_call(monkeypatch):
    B.build()
    monkeypatch.setattr(mx, "_lib", NoCall())
    monkeypatch.setattr(mx, "_stream", lambda s: 0)


def refused(fn, args, status=1, **kw):
    with pytest.raises(mx.MxsaError) as ei:
        fn(**dict(args, **kw))
    assert ei.value.status == status
    name, t = next(iter(kw.items()))
    assert name in str(ei.value) and str(t.dtype) in str(ei.value), str(ei.value)


def passes(fn, args, **kw):
    with pytest.raises(Reached):
        fn(**dict(args, **kw))


def z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=torch.uint8 if dt is F8 else dt).view(dt)


def test_dense_shared_fwd(no_call):
    p = mx.make_problem(3, 4, 16, 2, 1, 64, 10, 10)
    cache = z(10, 2, 64, 128)
    good = dict(prob=p, q=z(4, 16, 128), k_cache=cache, v_cache=cache, block_tables=z(3, 10, dt=I32),
                cu_seqlens_q=z(4, dt=I64), used_kv_lens=z(3, dt=I32), group_ptr=z(2, dt=I32), prefix_lens=z(1, dt=I32),
                ws=z(mx.dense_shared_workspace_size(p), dt=torch.uint8), out=z(4, 16, 128),
                lse=z(16, 4, dt=torch.float32), flags=z(1, dt=I32))
    passes(mx.dense_shared_fwd, good)
    passes(mx.dense_shared_fwd, good, group_ptr=None, prefix_lens=None, lse=None, flags=None)
    for name in ("block_tables", "used_kv_lens", "group_ptr", "prefix_lens", "flags"):
        refused(mx.dense_shared_fwd, good, **{name: good[name].long()})
    refused(mx.dense_shared_fwd, good, cu_seqlens_q=z(8, dt=I32))
    refused(mx.dense_shared_fwd, good, lse=z(16, 4, dt=torch.float64))
    for name in ("q", "k_cache", "v_cache", "out"):
        passes(mx.dense_shared_fwd, good, **{name: good[name].view(torch.int16)})
        refused(mx.dense_shared_fwd, good, **{name: good[name].to(HALF)})
        refused(mx.dense_shared_fwd, good, **{name: good[name].float()})


@pytest.mark.parametrize("q,kv", [(BF, BF), (HALF, F8), (BF, "nvfp4")])
def test_norm_rope_store_and_load_kv(no_call, q, kv):
    p = mx.make_problem(1, 4, 16, 2, 1, 64, 10, 10, q_dtype=q, kv_dtype=kv)
    other = HALF if q is BF else BF
    fp4 = kv == "nvfp4"
    cache = z(10, 2, 64 * 72, dt=torch.uint8) if fp4 else z(10, 2, 64, 128, dt=kv)
    row = lambda *s: z(4, *s, dt=q)
    good = dict(prob=p, positions=z(4, dt=I64), loc=z(4, dt=I64), cos_sin=torch.zeros(50, 64), q=row(16, 128),
                k=row(2, 128), v=row(2, 128), q_out=row(16, 128), k_cache=cache, v_cache=cache,
                q_weight=z(128, dt=q), k_weight=z(128, dt=q), flags=z(1, dt=I32))
    if not fp4:
        good.update(idx_q=row(2, 64), idx_k=row(2, 64), idx_q_weight=z(64, dt=q), idx_k_weight=z(64, dt=q),
                    idx_q_out=z(4, 2, 64, dt=kv), idx_cache=z(10, 2, 64, 64, dt=kv))
    fn = mx.norm_rope_store
    passes(fn, good)
    refused(fn, good, positions=z(8, dt=I32))
    refused(fn, good, loc=z(4, dt=torch.float64))
    refused(fn, good, flags=z(1, dt=I64))
    rows = ["q", "k", "v", "q_out", "q_weight", "k_weight"]
    if not fp4:
        rows += ["idx_q", "idx_k", "idx_q_weight", "idx_k_weight"]
    for name in rows:
        passes(fn, good, **{name: good[name].view(torch.int16)})
        refused(fn, good, **{name: good[name].view(other)})
    caches = ["k_cache", "v_cache"] + ([] if fp4 else ["idx_cache", "idx_q_out"])
    raw = torch.int16 if kv is q else torch.uint8
    wrong = other if kv is q else torch.float8_e5m2
    for name in caches:
        passes(fn, good, **{name: good[name].view(raw)})
        refused(fn, good, **{name: good[name].view(wrong)})
    load = dict(prob=p, loc=good["loc"], k_cache=cache, v_cache=cache, k=row(2, 128), v=row(2, 128), flags=good["flags"])
    if not fp4:
        load.update(idx_cache=good["idx_cache"], idx_k=row(2, 64))
    fn = mx.load_kv
    passes(fn, load)
    refused(fn, load, loc=z(4, dt=torch.float64))
    refused(fn, load, flags=z(1, dt=I64))
    for name in ("k", "v") + (() if fp4 else ("idx_k",)):
        passes(fn, load, **{name: load[name].view(torch.int16)})
        refused(fn, load, **{name: load[name].view(other)})
    for name in ("k_cache", "v_cache") + (() if fp4 else ("idx_cache",)):
        passes(fn, load, **{name: load[name].view(raw)})
        refused(fn, load, **{name: load[name].view(wrong)})


def test_none_is_left_to_the_library(no_call):
    """A missing tensor is the C entry's to refuse (or, with nothing to do, to take)."""
    p = mx.make_problem(1, 0, 16, 2, 1, 64, 10, 10)
    some = dict(block_tables=z(1, 10, dt=I32), cu_seqlens_q=z(2, dt=I64), used_kv_lens=z(1, dt=I32), group_ptr=None,
                prefix_lens=None, ws=z(mx.dense_shared_workspace_size(p), dt=torch.uint8))
    passes(mx.dense_shared_fwd, dict(prob=p, q=None, k_cache=None, v_cache=None, out=None, **some))
    passes(mx.dense_shared_fwd, dict(some, prob=p, q=None, k_cache=None, v_cache=None, out=None, block_tables=None))
    passes(mx.load_kv, dict(prob=p, loc=z(0, dt=I64), k_cache=None, v_cache=None, k=None, v=None))
    row = lambda *s: z(0, *s)
    passes(mx.norm_rope_store, dict(prob=p, positions=None, loc=z(0, dt=I64), cos_sin=torch.zeros(50, 64),
                                    q=row(16, 128), k=row(2, 128), v=row(2, 128), q_out=None, k_cache=None,
                                    v_cache=None))
    with pytest.raises(mx.MxsaError):  # a wrong type beside it is still refused
        mx.load_kv(p, z(0, dt=torch.float64), None, None, None, None)
