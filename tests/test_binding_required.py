"""A required tensor that is None is refused with MxsaError by the calls around
drafted trees and whole prompts, in the binding or in the library's own checks,
before any launch (no GPU)."""
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B

BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


def problem():
    return mx.make_problem(2, 4, 16, 2, 0, 64, 10, 5, True)


def tables():
    return mx.build_tables, (), dict(
        kv_lens=z(2, dt=I32), new_lens=z(2, dt=I32), pages_held=z(2, dt=I32), block_tables=z(2, 5, dt=I32),
        free_pages=z(10, dt=I32), free_count=z(1, dt=I32), cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32),
        positions=z(4, dt=I64), loc=z(4, dt=I64))


def mask():
    return mx.tree_mask, (), dict(parents=z(4, dt=I32), cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32),
                                  mask=z(4, 1, dt=I32))


def tree():
    cache = z(10, 2, 64, 128)
    return mx.tree_fwd, ("group_ptr", "prefix_lens"), dict(
        q=z(4, 16, 128), k_cache=cache, v_cache=cache, block_tables=z(2, 5, dt=I32), cu_seqlens_q=z(3, dt=I64),
        used_kv_lens=z(2, dt=I32), tree_mask=z(4, 1, dt=I32), group_ptr=None, prefix_lens=None,
        ws=z(mx.dense_shared_workspace_size(problem()), dt=torch.uint8), out=z(4, 16, 128))


def commit():
    cache = z(10, 2, 64, 128)
    return mx.tree_commit, (), dict(
        cu_seqlens_q=z(3, dt=I64), used_kv_lens=z(2, dt=I32), block_tables=z(2, 5, dt=I32), path=z(2, 4, dt=I32),
        path_lens=z(2, dt=I32), k_cache=cache, v_cache=cache)


def prompt():
    return mx.prompt_fwd, (), dict(q=z(4, 16, 128), k=z(4, 2, 128), v=z(4, 2, 128), cu_seqlens=z(3, dt=I64),
                                   ws=z(mx.prompt_workspace_size(problem()), dt=torch.uint8), out=z(4, 16, 128))


@pytest.mark.parametrize("call", [tables, mask, tree, commit, prompt], ids=lambda f: f.__name__)
def test_none(call, monkeypatch):
    B.build()
    monkeypatch.setattr(mx, "_stream", lambda s: 0)
    fn, optional, good = call()
    for name in good:
        if name in optional:
            continue
        with pytest.raises(mx.MxsaError) as e:
            fn(problem(), **dict(good, **{name: None}))
        assert e.value.status == 1, name
