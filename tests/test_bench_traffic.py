"""The DRAM traffic that bench.py reports for the forward comes from committed
counter captures: they are of the current forward, and a change of the shared
headers that the forward does not use does not void them (no GPU)."""
import json
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "block_sparse_attention_builder_gb300", "csrc")


def headers():
    return [open(os.path.join(CSRC, f)).read() for f in ("ptx.cuh", "internal.h")]


def test_the_captures_are_of_the_current_forward():
    with open(os.path.join(bench.ROOT, "profiles", "k_fwd_traffic.json")) as f:
        names = [k for k in json.load(f) if not k.startswith("_")]
    assert {"skewed_decode", "gqa_decode", "shared_prefill", "fp8_varlen"} <= set(names)
    for w in names:
        assert bench.recorded_traffic(w) and bench.recorded_traffic(w) > 0, w


def test_only_what_the_forward_uses_counts():
    ptx, internal = headers()
    h = bench.fwd_source_hash()
    assert h == bench.fwd_source_hash([ptx, internal])
    new = ptx.replace("\n}  // namespace mxsa", """
// another kernel's helper
__device__ __forceinline__ float another_helper(float x) {
  return x;
}

struct AnotherArgs {
  int n;
};
}  // namespace mxsa""")
    assert new != ptx and bench.fwd_source_hash([new, internal]) == h
    declared = internal.replace("size_t shared_workspace_bytes", "size_t another_size(int n);\nsize_t shared_workspace_bytes")
    assert declared != internal and bench.fwd_source_hash([ptx, "// a comment\n" + declared]) == h
    # what it uses, directly or through another helper, does
    for name in ("tma_load_3d", "mbar_try_wait", "ex2_approx"):
        body = re.sub(r"(\b%s\([^)]*\)\s*\{)" % name, r"\1\n  int changed = 1;", ptx, count=1)
        assert body != ptx and bench.fwd_source_hash([body, internal]) != h, name
    moved = internal.replace("2000000000ull", "1000000000ull")
    assert moved != internal and bench.fwd_source_hash([ptx, moved]) != h
