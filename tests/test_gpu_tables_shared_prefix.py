"""mxsa_build_tables with requests that share a prefix's pages."""
import numpy as np
import pytest

import block_sparse_attention_builder_gb300 as mx
from tests.test_gpu_tables import I64, dev

pytestmark = pytest.mark.gpu


def test_requests_that_share_a_prefix():
    """Three requests on the same first two pages: one that finishes before the others has them moved out of the
    entries that it gives back; the last one gives them back.  Every page is then free once."""
    ps, pages, width, B = 64, 12, 6, 3
    prob = mx.make_problem(B, 64, 8, 8, 0, ps, pages, width)
    table = np.full((B, width), -1, np.int32)
    table[:, :2] = [4, 9]
    rest = [p for p in range(pages) if p not in (4, 9)]
    lens, held, table = dev([128] * B), dev([2] * B), dev(table)
    free, count = dev(rest + [0, 0]), dev([len(rest)])
    cu, pos, loc, f = dev([0] * (B + 1), I64), dev([0] * 64, I64), dev([0] * 64, I64), dev([0])
    step = lambda new: mx.build_tables(prob, lens, dev(new), held, table, free, count, cu, lens, pos, loc, flags=f)
    step([20, 10, 30])
    assert held.tolist() == [3, 3, 3] and count.item() == len(rest) - 3
    own = table[:, 2].tolist()
    assert len(set(own)) == 3 and not set(own) & {4, 9}
    # the second one finishes: its own page first, the prefix out of what it gives back
    table[1, 0], held[1] = own[1], 1
    step([1, -1, 1])
    assert held.tolist() == [3, 0, 3] and count.item() == len(rest) - 2
    assert own[1] in free[:count.item()].tolist() and not {4, 9} & set(free[:count.item()].tolist())
    assert loc[:2].tolist() == [own[0] * 64 + 20, own[2] * 64 + 30]  # the others still write behind the prefix
    # then the others: one gives the prefix back
    table[0, 0], held[0] = own[0], 1
    step([-1, -1, -1])
    assert f.item() == 0 and count.item() == pages and sorted(free.tolist()) == list(range(pages))
    assert lens.tolist() == held.tolist() == [0, 0, 0]
