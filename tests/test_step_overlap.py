"""Outputs of the calls around drafted trees that overlap what other CTAs still
read: refused before any launch (no GPU)."""
import ctypes

import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B

P = ctypes.c_void_p
BASE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mx.library()


def problem():
    return mx.make_problem(3, 9, 16, 2, 0, 64, 10, 5)


# bytes that a call of `problem` reads
COMMIT = dict(cu=8 * 4, lens=4 * 3, bt=4 * 3 * 5, path=4 * 3 * 4, n=4 * 3)


@pytest.mark.parametrize("name", list(COMMIT))
def test_tree_commit(lib, name):
    at = {x: BASE * (i + 1) for i, x in enumerate(COMMIT)}

    def call(out):
        p = {x: P(v) for x, v in at.items()}
        # (index rows of 2^31 bytes: refused with another status after the overlaps, so that no call launches)
        return lib.mxsa_tree_commit(ctypes.byref(problem()), p["cu"], p["lens"], p["bt"], p["path"], 4, p["n"],
                                    P(64 * BASE), P(65 * BASE), P(66 * BASE), 1, 1 << 30, P(out), None, None)

    begin, end = at[name], at[name] + COMMIT[name]
    for out in (begin - 4 * 3 + 4, begin, end - 4):
        assert call(out) == 1, (name, out - begin)
    for out in (begin - 4 * 3, end):  # next to it
        assert call(out) == 2, (name, out - begin)


# the masks' call reads parents, starts and lengths and writes masks (one word a token) and positions
MASK = dict(parents=4 * 9, cu=8 * 4, lens=4 * 3)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would run on these pointers")
@pytest.mark.parametrize("out,size", [("mask", 4 * 9), ("pos", 8 * 9)])
@pytest.mark.parametrize("name", list(MASK) + ["the other output"])
def test_tree_mask(lib, name, out, size):
    at = {x: BASE * (i + 1) for i, x in enumerate(list(MASK) + ["mask", "pos"])}
    sizes = dict(MASK, mask=4 * 9, pos=8 * 9)
    name = {"mask": "pos", "pos": "mask"}[out] if name == "the other output" else name

    def call(where):
        p = {x: P(v) for x, v in dict(at, **{out: where}).items()}
        return lib.mxsa_tree_mask(ctypes.byref(problem()), p["parents"], p["cu"], p["lens"], 1, p["mask"], p["pos"],
                                  None, None)

    begin, end = at[name], at[name] + sizes[name]
    for where in (begin - size + 8, begin, end - 8 if end % 8 == 0 else end - 4):
        if out == "mask" or where % 8 == 0:
            assert call(where) == 1, where - begin
    for where in (begin - size, (end + 7) // 8 * 8):  # next to it: nothing to refuse (and no GPU here)
        assert call(where) == 4, where - begin
