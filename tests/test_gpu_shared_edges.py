"""mxsa_dense_shared_fwd at its edges: values that are not finite, and the plan
that its workspace holds after a call against the model of it."""
import numpy as np
import pytest
import torch

from tests.test_gpu_shared import CASES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["decode", "two_row_tiles", "decode_aligned"])
def test_an_infinity_in_v_stays_in_its_column(name):
    """A prefix key's V holds an infinity: that column of the kv head's rows is not finite, nothing else changes."""
    c = Case(**CASES[name], seed=1).run().check()
    good, lse = c.out.clone(), c.lse.clone()
    page, off = (x[50] for x in c.slots[0])
    c.v[page, 0, off, 7] = float("inf")
    c.run()
    torch.cuda.synchronize()
    G = c.hq // c.hkv
    assert not c.out[:, :G, 7].isfinite().any()
    same = torch.ones_like(c.out, dtype=torch.bool)
    same[:, :G, 7] = False
    assert torch.equal(c.out[same], good[same]) and torch.equal(c.lse, lse)
