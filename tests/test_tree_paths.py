"""Which of its two forms mxsa_tree_fwd takes, seen through a stand-in for the
CUDA runtime (tests/fake_launches.c; no GPU): the faster one of shapes where both
were timed and differ by more than the times' spread."""
import os
import subprocess

import pytest

from block_sparse_attention_builder_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))

# (sequences, tokens of one, query heads, kv heads, keys of the longest): the
# cluster of the one launch, or 0 for the three, and the two forms' times in us
# (one launch, three) for lengths from a third of the longest on
TIMED = {
    (1, 5, 16, 2, 1000): (8, 8, 16), (1, 5, 16, 2, 16000): (8, 23, 42), (4, 5, 16, 2, 16000): (8, 24, 32),
    (1, 60, 16, 2, 24000): (0, 35, 31), (1, 8, 12, 4, 32000): (0, 36, 33),
    (13, 5, 8, 1, 24000): (8, 32, 40), (7, 16, 16, 2, 24000): (8, 38, 43), (5, 3, 16, 2, 24000): (8, 31, 36),
    (2, 5, 128, 1, 24000): (8, 35, 38),
    (5, 20, 16, 4, 8000): (4, 27, 29), (5, 20, 16, 4, 24000): (0, 54, 45), (4, 40, 12, 4, 16000): (0, 42, 39),
    (30, 7, 8, 1, 16000): (4, 42, 47), (16, 5, 16, 2, 16000): (4, 42, 48), (4, 5, 64, 8, 16000): (4, 43, 50),
    (7, 33, 12, 4, 16000): (4, 46, 50), (28, 16, 8, 1, 16000): (4, 45, 48), (1, 200, 16, 2, 24000): (0, 57, 49),
    (2, 37, 64, 8, 4000): (2, 28, 36), (7, 16, 64, 8, 8000): (2, 47, 50), (16, 40, 12, 4, 8000): (2, 49, 60),
    (6, 16, 64, 8, 24000): (0, 101, 88), (70, 3, 8, 1, 8000): (2, 43, 52),
    (4, 40, 64, 8, 8000): (0, 69, 58), (80, 16, 8, 1, 8000): (0, 75, 70), (2, 100, 64, 8, 8000): (0, 72, 57),
    (16, 16, 64, 8, 4000): (1, 51, 63), (112, 5, 8, 1, 8000): (1, 72, 75), (16, 16, 64, 8, 8000): (1, 82, 91),
    (150, 8, 8, 1, 8000): (1, 84, 98), (4, 60, 64, 8, 8000): (1, 70, 84), (30, 20, 16, 4, 16000): (0, 135, 127),
    (110, 20, 8, 1, 8000): (0, 114, 97), (109, 8, 8, 1, 8000): (1, 74, 78), (9, 5, 8, 1, 24000): (8, 31, 37),
    (23, 8, 8, 1, 16000): (4, 39, 42), (12, 20, 8, 1, 16000): (0, 41, 36),
    (200, 5, 8, 1, 1000): (0, None, None),
}


@pytest.fixture(scope="module")
def taken(tmp_path_factory):
    B.build()
    exe = str(tmp_path_factory.mktemp("fake") / "fake_launches")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc())))
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-Wall", "-rdynamic", "-I", os.path.join(cuda, "include"), "-o", exe,
                    os.path.join(HERE, "fake_launches.c"), "-ldl"], check=True)
    r = subprocess.run([exe, B.LIB, *(",".join(map(str, c)) for c in TIMED)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return dict(zip(TIMED, (tuple(map(int, l.split())) for l in r.stdout.splitlines())))


@pytest.mark.parametrize("shape", list(TIMED), ids=lambda c: "-".join(map(str, c)))
def test_the_faster_form(taken, shape):
    cluster = TIMED[shape][0]
    assert taken[shape] == ((1, cluster) if cluster else (3, 0))
