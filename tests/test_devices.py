"""The launchers on more than one device, and after a failure of the runtime,
against a stand-in for the CUDA runtime (tests/fake_runtime.c; no GPU): the
shared-memory limit of a kernel belongs to a device, and a call that failed
once must not fail for the life of the process."""
import os
import subprocess

import pytest

from block_sparse_attention_builder_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    B.build()
    exe = str(tmp_path_factory.mktemp("fake") / "fake_runtime")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc())))
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-Wall", "-rdynamic", "-I", os.path.join(cuda, "include"), "-o", exe,
                    os.path.join(HERE, "fake_runtime.c"), "-ldl"], check=True)
    return exe


def run(program, *args):
    r = subprocess.run([program, B.LIB, *args], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_several_devices(program):
    run(program, "devices")


@pytest.mark.parametrize("call", range(4))
@pytest.mark.parametrize("kind", ["attributes", "entry points"])
def test_a_failure_is_not_kept(program, kind, call):
    run(program, kind, str(call))
