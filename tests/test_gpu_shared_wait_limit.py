"""A bounded wait of mxsa_dense_shared_fwd that runs out, on the GPU.

The test-only library (50 ms limit) has a switch that makes one CTA's
scheduler keep its first window of pages to itself, so that its producer, its
MMA issuers and its softmax groups wait for what never comes; only the tile's q
rows are copied, and land.  The launch must return with MXSA_FLAG_TIMEOUT in the
flags and every other CTA's rows right, and the next calls, of this library
and the regular one, must be right again.
"""
import time

import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B
from tests.test_gpu_shared import CASES, Case

pytestmark = pytest.mark.gpu

FLAG_TIMEOUT = 32


@pytest.mark.parametrize("name", ["decode", "two_row_tiles"])  # a first tile with copies, one of two halves
def test_a_wait_that_runs_out(name, monkeypatch):
    B.build()
    test_lib = mx._load_library(B.TEST_LIB)
    c = Case(**CASES[name], seed=1).run().check()
    good = c.out.clone()
    monkeypatch.setattr(mx, "_lib_handle", test_lib)
    c.ws.fill_(0xFF)  # partial rows that nobody writes are NaN
    assert test_lib.mxsa_test_skip_window(0) == 0
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        c.run()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        assert test_lib.mxsa_test_skip_window(-1) == 0
    assert c.flags.item() & FLAG_TIMEOUT and dt < 5.0, (c.flags.item(), dt)
    lost, same = c.out.isnan().any(-1), (c.out == good).all(-1)
    assert lost.any() and (lost | same).all()  # CTA 0's first tile, and no other row
    c.flags.zero_()
    c.run().check()
    assert torch.equal(c.out, good)
    monkeypatch.setattr(mx, "_lib_handle", None)
    c.run().check()
    assert torch.equal(c.out, good)
