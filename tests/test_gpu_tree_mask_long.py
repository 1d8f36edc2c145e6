"""mxsa_tree_mask on sequences of more tokens than its masks hold: flagged, with
a walk that ends after 2048 ancestors."""
import numpy as np
import pytest

import block_sparse_attention_builder_gb300 as mx
from tests.test_gpu_tree import I32, I64, dev

pytestmark = pytest.mark.gpu

LIMIT = 2048


def run(sizes, words, parents):
    cu, total = np.cumsum([0] + sizes), sum(sizes)
    prob = mx.make_problem(len(sizes), total, 8, 8, 0, 64, 1, 4096)
    m, p, f = dev(np.full((total, words), 9), I32), dev([-5] * total, I64), dev([0], I32)
    lens = [n + 100 for n in sizes]
    mx.tree_mask(prob, dev(parents, I32), dev(cu, I64), dev(lens, I32), m, p, flags=f)
    return f.item(), m.cpu().numpy().view(np.uint32), p.cpu().numpy()


def expected(sizes, words, parents):
    """Token by token: itself and up to LIMIT ancestors."""
    mask, pos, at = np.zeros((sum(sizes), words), np.uint32), [], 0
    for n in sizes:
        for i in range(n):
            j, depth = i, 0
            while True:
                if j < 32 * words:
                    mask[at + i, j // 32] |= np.uint32(1 << j % 32)
                if parents[at + j] < 0 or depth == LIMIT:
                    break
                j, depth = parents[at + j], depth + 1
            pos.append(100 + depth)
        at += n
    return mask, np.array(pos)


@pytest.mark.parametrize("words", [1, 64])
@pytest.mark.parametrize("chain", [2049, 2050, 4500])
def test_a_long_chain(chain, words):
    sizes = [7, chain, 3]
    parents = [-1, 0, 0, 1, 1, 2, -1] + list(range(-1, chain - 1)) + [-1, 0, 1]
    flags, mask, pos = run(sizes, words, parents)
    want, wpos = expected(sizes, words, parents)
    assert flags == 1024 and np.array_equal(mask, want) and np.array_equal(pos, wpos)


def test_a_wide_tree_past_the_mask():
    """Few ancestors: only the bits that the words do not reach are left out."""
    r = np.random.RandomState(1)
    parents = [-1] + [int(r.randint(-1, i)) for i in range(1, 3000)]
    flags, mask, pos = run([3000], 2, parents)
    want, wpos = expected([3000], 2, parents)
    assert flags == 1024 and np.array_equal(mask, want) and np.array_equal(pos, wpos)
