"""A bounded wait of mxsa_tree_fwd's one-launch path that runs out, on the GPU.

The test-only library (50 ms limit) has a switch that makes one CTA's first warp
keep the tile to itself, so that its MMA issuers and its softmax groups wait for
what never comes; its copies are issued, and land.  The other CTAs of the cluster
meet it at the cluster's barriers all the same.  The launch must return with
MXSA_FLAG_TIMEOUT in the flags and the other clusters' rows right, and the next
calls, of this library and the regular one, must be right again.
"""
import time

import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B
from tests.test_gpu_tree import CASES, Trees

pytestmark = pytest.mark.gpu

FLAG_TIMEOUT = 32


@pytest.mark.parametrize("name", ["small", "cluster_2", "cluster_1"])
def test_a_wait_that_runs_out(name, monkeypatch):
    B.build()
    test_lib = mx._load_library(B.TEST_LIB)
    t = Trees(**CASES[name], seed=1).run().check()
    good = t.out.clone()
    monkeypatch.setattr(mx, "_lib_handle", test_lib)
    assert test_lib.mxsa_test_skip_found(0) == 0
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        t.run()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        assert test_lib.mxsa_test_skip_found(-1) == 0
    assert t.flags.item() & FLAG_TIMEOUT and dt < 5.0, (t.flags.item(), dt)
    rows = (t.out == good).all(-1)  # only the first cluster's: its tokens' rows of the first kv head
    G = t.hq // t.hkv
    first = torch.zeros_like(rows)
    first[t.cu[0]:t.cu[0] + 128 // G, :G] = True
    assert not rows.all() and rows[~first].all()
    t.flags.zero_()
    t.run().check()
    assert torch.equal(t.out, good)
    monkeypatch.setattr(mx, "_lib_handle", None)
    t.run().check()
    assert torch.equal(t.out, good)
