"""Refusals of mxsa_norm_rope_store and mxsa_load_kv before any launch, in the
C ABI and in the binding (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx
from block_sparse_attention_builder_gb300 import build as B

P = ctypes.c_void_p
FAKE, FAKE8 = P(1 << 20), P((1 << 20) + 8)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mx.library()


def _prob(**kw):
    base = dict(num_seqs=1, total_q=4, num_q_heads=16, num_kv_heads=2, topk=1, page_size=64, num_pages=10,
                max_pages_per_seq=10, causal=False)
    base.update(kw)
    return mx.make_problem(**base)


def _cfg(**kw):
    c = mx.NormRope(q_stride=2048, k_stride=256, v_stride=256, idx_q_stride=0, idx_k_stride=0, num_positions=100,
                    rot_dim=64, interleaved=0, weight_per_head=0, idx_dim=0, eps=1e-6)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


NAMES = ["positions", "loc", "cos_sin", "q", "k", "v", "q_weight", "k_weight", "q_out", "k_cache", "v_cache",
         "idx_q", "idx_k", "idx_q_weight", "idx_k_weight", "idx_q_out", "idx_cache"]
BASE = dict.fromkeys(NAMES[:11], FAKE)
IDX = dict.fromkeys(NAMES[11:], FAKE)
IDX_CFG = dict(idx_dim=64, idx_q_stride=128, idx_k_stride=128)


def _call(lib, prob=None, cfg=None, n=4, flags=None, **kw):
    a = dict(BASE, **kw)
    prob, cfg = prob or _prob(), cfg or _cfg()
    return lib.mxsa_norm_rope_store(ctypes.byref(prob), ctypes.byref(cfg), n, *(a.get(x) for x in NAMES), flags, None)


@pytest.mark.parametrize("cfg,status", [
    (dict(rot_dim=0), 2), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(num_positions=0), 1), (dict(interleaved=2), 1),
    (dict(weight_per_head=-1), 1), (dict(q_stride=2040), 1), (dict(q_stride=2052), 1), (dict(k_stride=128), 1),
    (dict(v_stride=260), 1), (dict(idx_dim=32), 2),
])
def test_bad_configurations(lib, cfg, status):
    assert _call(lib, cfg=_cfg(**cfg)) == status


def test_null_misaligned_and_partial_arguments(lib):
    assert lib.mxsa_norm_rope_store(None, ctypes.byref(_cfg()), 4, *([FAKE] * 17), None, None) == 1
    assert lib.mxsa_norm_rope_store(ctypes.byref(_prob()), None, 4, *([FAKE] * 17), None, None) == 1
    assert _call(lib, n=-1) == 1
    for name in NAMES[:11]:
        if "weight" not in name:
            assert _call(lib, **{name: None}) == 1, name
        bad = P((1 << 20) + 4) if name in ("positions", "loc") else FAKE8
        assert _call(lib, **{name: bad}) == 1, name
    assert _call(lib, flags=P((1 << 20) + 2)) == 1
    # index rows: all or none, with a dimension, and not in NVFP4
    assert _call(lib, **IDX) == 1
    for name in ("idx_q", "idx_k", "idx_q_out", "idx_cache"):
        assert _call(lib, cfg=_cfg(**IDX_CFG), **dict(IDX, **{name: None})) == 1, name
        assert _call(lib, cfg=_cfg(**IDX_CFG), **dict(IDX, **{name: FAKE8})) == 1, name
    assert _call(lib, cfg=_cfg(**dict(IDX_CFG, rot_dim=96)), **IDX) == 1  # wider than the index rows
    assert _call(lib, cfg=_cfg(**dict(IDX_CFG, idx_k_stride=64)), **IDX) == 1
    assert _call(lib, prob=_prob(kv_dtype="nvfp4"), cfg=_cfg(**IDX_CFG), **IDX) == 2
    assert _call(lib, prob=_prob(page_size=32)) == 2
    assert _call(lib, prob=_prob(q_dtype=torch.float16, kv_dtype=torch.bfloat16)) == 2


def test_load_arguments(lib):
    p = _prob(kv_dtype=torch.float8_e4m3fn)

    def call(prob=p, n=4, loc=FAKE, kc=FAKE, vc=FAKE, k=FAKE, v=FAKE, ic=None, ik=None, ih=0, idim=0, flags=None):
        pr = ctypes.byref(prob) if prob is not None else None
        return lib.mxsa_load_kv(pr, n, loc, kc, vc, k, v, ic, ik, ih, idim, flags, None)

    assert call(prob=None) == 1 and call(n=-1) == 1
    for name in ("loc", "kc", "vc", "k", "v"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P((1 << 20) + 4)}) == 1, name
    assert call(ic=FAKE, ih=1, idim=64) == 1 and call(ik=FAKE, ih=1, idim=64) == 1
    assert call(ic=FAKE, ik=FAKE, ih=1, idim=60) == 1 and call(ic=FAKE, ik=FAKE, ih=0, idim=64) == 1
    assert call(prob=_prob(kv_dtype="nvfp4"), ic=FAKE, ik=FAKE, ih=1, idim=64) == 2
    assert call(prob=_prob(num_q_heads=12, num_kv_heads=5)) == 1
    assert call(flags=P((1 << 20) + 2)) == 1


def test_binding_refuses_what_the_shapes_rule_out(lib):
    p = _prob()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i64 = lambda n: torch.zeros(n, dtype=torch.int64)
    cs = torch.zeros(50, 64)
    cache = bf(10, 2, 64, 128)
    good = dict(positions=i64(4), loc=i64(4), cos_sin=cs, q=bf(4, 16, 128), k=bf(4, 2, 128), v=bf(4, 2, 128),
                q_out=bf(4, 16, 128), k_cache=cache, v_cache=cache)

    def refused(**kw):
        with pytest.raises(mx.MxsaError) as ei:
            mx.norm_rope_store(p, **dict(good, **kw))
        assert ei.value.status == 1

    refused(q=bf(4, 15, 128))
    refused(q=torch.zeros(4, 16, 128))                      # 32-bit rows
    refused(k=bf(2, 4, 128).transpose(0, 1))                # the heads of a token are apart
    refused(positions=i64(3))
    refused(cos_sin=cs.double())
    refused(cos_sin=torch.zeros(50, 128)[:, :64])           # rows of the table apart
    refused(q_out=bf(3, 16, 128))
    refused(k_cache=cache[:9])
    refused(q_weight=bf(64))
    refused(q_weight=bf(128), k_weight=bf(2, 128))          # one of each form
    refused(q_weight=torch.zeros(128))
    refused(idx_q=bf(4, 2, 64), idx_k=bf(4, 2, 64))         # without outputs
    refused(idx_q=bf(4, 2, 64), idx_k=bf(4, 2, 128), idx_q_out=bf(4, 2, 64), idx_cache=bf(10, 2, 64, 64))
    refused(idx_q=bf(4, 2, 64), idx_k=bf(4, 2, 64), idx_q_out=bf(4, 2, 64), idx_cache=bf(10, 2, 64, 63))
    for kw in (dict(k=bf(3, 2, 128)), dict(v_cache=cache[:9]), dict(loc=i64(8)[::2])):
        a = dict(loc=i64(4), k_cache=cache, v_cache=cache, k=bf(4, 2, 128), v=bf(4, 2, 128))
        with pytest.raises(mx.MxsaError) as ei:
            mx.load_kv(p, **dict(a, **kw))
        assert ei.value.status == 1


def test_dense_shared_arguments(lib):
    p = _prob(num_seqs=3)
    nbytes = mx.dense_shared_workspace_size(p)

    def call(prob=p, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cu=FAKE, lens=FAKE, ng=1, gp=FAKE, pl=FAKE, ws=FAKE, n=nbytes,
             out=FAKE, lse=None, flags=None):
        pr = ctypes.byref(prob) if prob is not None else None
        return lib.mxsa_dense_shared_fwd(pr, q, k, v, bt, cu, lens, ng, gp, pl, ws, n, out, lse, flags, None)

    assert call(prob=None) == 1
    for name in ("q", "k", "v", "bt", "cu", "lens", "gp", "pl", "ws", "out"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P((1 << 20) + 2)}) == 1, name
    assert call(ws=P((1 << 20) + 128)) == 1 and call(lse=P((1 << 20) + 2)) == 1 and call(flags=P((1 << 20) + 1)) == 1
    assert call(ng=-1) == 1 and call(ng=4) == 1
    assert call(n=nbytes - 1) == 3
    assert call(prob=_prob(num_seqs=1025)) == 2 and call(prob=_prob(kv_dtype=torch.float8_e4m3fn)) == 2
    assert call(prob=_prob(num_q_heads=256, num_kv_heads=1)) == 2 and call(prob=_prob(page_size=16)) == 2
    big = _prob(total_q=(1 << 31) - 1)
    assert call(prob=big) == 2
    assert lib.mxsa_shared_workspace_size(ctypes.byref(big), ctypes.byref(ctypes.c_size_t())) == 2
    assert lib.mxsa_shared_workspace_size(ctypes.byref(p), None) == 1
    # more tokens, more workspace; the index's limits do not apply
    assert mx.dense_shared_workspace_size(_prob(total_q=1 << 20, topk=256)) > nbytes
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cache, i32 = bf(10, 2, 64, 128), lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(q=bf(4, 16, 128), k_cache=cache, v_cache=cache, block_tables=i32(3, 10),
                cu_seqlens_q=torch.zeros(4, dtype=torch.int64), used_kv_lens=i32(3), group_ptr=i32(2),
                prefix_lens=i32(1), ws=torch.zeros(nbytes, dtype=torch.uint8), out=bf(4, 16, 128))
    for kw in (dict(group_ptr=i32(1)), dict(group_ptr=None), dict(prefix_lens=None), dict(q=bf(3, 16, 128)),
               dict(out=bf(4, 15, 128)), dict(block_tables=i32(3, 9)), dict(ws=good["ws"][::2])):
        with pytest.raises(mx.MxsaError) as ei:
            mx.dense_shared_fwd(p, **dict(good, **kw))
        assert ei.value.status == 1


def test_quotient_by_a_residual_step_is_the_division():
    """The NVFP4 casts' x / scale: q = x r, then q + (x - q s) r, r the rounded reciprocal; every E4M3 scale, values at
    and next to the ties of E2M1 and anywhere."""
    e = np.arange(1, 127)
    s = np.where(e < 8, e * 2.0 ** -9, (8 + e % 8) * 2.0 ** (e // 8 - 10.0)).astype(np.float32)[:, None]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6], np.float32)
    near = [s * ties]
    for _ in range(3):
        near.append(np.nextafter(near[-1], np.float32(np.inf)))
    low = s * ties
    for _ in range(3):
        low = np.nextafter(low, np.float32(0))
        near.append(low)
    rand = np.random.RandomState(0).rand(len(s), 20000).astype(np.float32) * s * 8
    x = np.concatenate(near + [rand, rand * np.float32(2.0 ** -100)], 1)
    L = np.longdouble
    r = np.float32(1) / s
    q = x * r
    rest = (L(x) - L(q) * L(s)).astype(np.float32)  # exact: one fused step
    y = (L(q) + L(rest) * L(r)).astype(np.float32)
    assert (y == x / s).all()
