"""mxsa_tree_fwd with tables of several widths around the same keys: on either
side of the width up to which one launch is taken, against the definition."""
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from tests.test_gpu_tree import I32, CASES, Trees

pytestmark = pytest.mark.gpu


def widen(t, blocks):
    """The same sequences in tables of so many blocks of 128 keys."""
    p = t.prob
    width = blocks * 128 // p.page_size
    assert width >= p.max_pages_per_seq
    table = torch.full((p.num_seqs, width), -3, dtype=I32, device="cuda")
    table[:, :p.max_pages_per_seq] = t.dt
    t.dt, t.prob = table, mx.make_problem(p.num_seqs, p.total_q, p.num_q_heads, p.num_kv_heads, 0, p.page_size,
                                          p.num_pages, width, bool(p.causal), p.softmax_scale,
                                          q_dtype=t.q.dtype)
    t.ws = torch.full((mx.dense_shared_workspace_size(t.prob),), 0xFF, dtype=torch.uint8, device="cuda")
    return t


@pytest.mark.parametrize("blocks", [33, 65, 127, 129, 191, 193, 2000])
@pytest.mark.parametrize("name", ["small", "empty_between", "cluster_2", "cluster_1", "wide_g3", "g128"])
def test_widths(name, blocks):
    widen(Trees(seed=len(name), **CASES[name]), blocks).run().check()


@pytest.mark.parametrize("case", [
    dict(seqs=[(5, 24000), (7, 100), (3, 9000), (1, 0), (6, 17000)], hq=16, hkv=2),  # a cluster of 8
    dict(seqs=[(n, 3000 * i % 16000) for i, n in enumerate([5, 1, 16, 0, 9, 3, 12] * 4)], hq=8, hkv=1, q="fp16"),  # 4
    dict(seqs=[(n, 1700 * i % 8000) for i, n in enumerate([9, 30, 1, 16] * 28)], hq=4, hkv=1, ps=128),  # 1
], ids=["8", "4", "1"])
def test_the_longest_keys_of_one_launch(case):
    """Lengths near the width where one launch ends."""
    t = Trees(seed=5, **case).run().check()
    widen(t, 300).run().check()
