"""A bounded wait of mxsa_prompt_fwd that runs out, on the GPU.

The test-only library (50 ms limit) has a switch that makes one CTA's producer
keep its first tile's record to itself, so that its q warp, its MMA issuers and
its softmax groups wait for what never comes; the tile's first keys are copied,
and land.  The launch must return with MXSA_FLAG_TIMEOUT in the flags and every
other tile's rows right, and the next calls, of this library and the regular
one, must be right again.
"""
import time

import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B
from tests.test_gpu_prompt import CASES, Prompts

pytestmark = pytest.mark.gpu

FLAG_TIMEOUT = 32


@pytest.mark.parametrize("name", ["past_a_block", "many", "long"])  # one tile to a CTA, and the plan's order
def test_a_wait_that_runs_out(name, monkeypatch):
    B.build()
    test_lib = mx._load_library(B.TEST_LIB)
    p = Prompts(**CASES[name], seed=1).run().check()
    good = p.out.clone()
    monkeypatch.setattr(mx, "_lib_handle", test_lib)
    p.out.fill_(9)
    assert test_lib.mxsa_test_skip_record(0) == 0
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        p.run()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        assert test_lib.mxsa_test_skip_record(-1) == 0
    assert p.flags.item() & FLAG_TIMEOUT and dt < 5.0, (p.flags.item(), dt)
    lost, same = (p.out == 9).all(-1), (p.out == good).all(-1)
    assert lost.any() and (lost | same).all()  # CTA 0's first tile, and no other row
    p.flags.zero_()
    p.out.fill_(9)
    p.run().check()
    assert torch.equal(p.out, good)
    monkeypatch.setattr(mx, "_lib_handle", None)
    p.run().check()
    assert torch.equal(p.out, good)
