"""Host-side checks of the drafted-token, rotation and eviction entry points:
every call here is refused before anything is launched, or needs no device."""
import ctypes
import math

import numpy as np
import pytest

import decode_attention_mla_gb300 as mla
from decode_attention_mla_gb300 import build as mla_build
import _tree_ref as ref

PTR = 0x100000                       # never dereferenced: the call is refused first


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()
    yield


def refused(fn, *args):
    return getattr(mla.lib(), fn)(*args)


# ---- rope ----------------------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(rot_dim=64, base=10000.0), dict(rot_dim=8, base=500.0), dict(rot_dim=64, base=1.0),
    dict(rot_dim=48, base=1e6, scaling="linear", factor=8.0),
    dict(rot_dim=64, base=10000.0, scaling="yarn", factor=40.0, original_ctx=4096, beta_fast=32.0, beta_slow=1.0),
    dict(rot_dim=32, base=5e5, scaling="yarn", factor=2.5, original_ctx=8192, beta_fast=16.0, beta_slow=0.5),
])
def test_table_is_the_formula(kw):
    turns = mla.rope_turns(**kw)
    want = ref.inv_freq(kw["rot_dim"], kw["base"], **{k: v for k, v in kw.items() if k not in ("rot_dim", "base")})
    assert len(turns) == kw["rot_dim"] // 2
    for t, f in zip(turns, want):
        # a few double roundings, and the last place of the 64-bit fraction
        assert abs(t / 2.0 ** 64 - f / (2 * math.pi)) <= 2.0 ** -50 * f + 2.0 ** -63


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=4), dict(rot_dim=12), dict(rot_dim=72), dict(rot_dim=-8), dict(base=0.5),
    dict(base=math.nan), dict(base=math.inf), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=math.nan), dict(scaling="yarn", factor=4.0, original_ctx=0),
    dict(scaling="yarn", factor=4.0, beta_fast=1.0, beta_slow=1.0), dict(scaling="yarn", factor=4.0, beta_slow=0.0),
    dict(scaling="yarn", factor=4.0, base=1.0), dict(scaling="yarn", factor=math.inf),
])
def test_table_refusals(kw):
    with pytest.raises(mla.MLADecodeError) as e:
        mla.rope_turns(**{**dict(rot_dim=64, base=10000.0), **kw})
    assert e.value.status == mla.EINVAL


def rope_args(**kw):
    a = dict(batch=2, tokens=3, heads=16, rot_dim=64, interleaved=1, amplitude=1.0, turns=PTR, positions=PTR,
             q_rope=PTR, q_rope_batch=576, q_rope_token=192, q_rope_head=64, q_out=PTR, q_out_batch=27648,
             q_out_token=9216, q_out_head=576, c=PTR, c_batch=1728, c_token=576, k_rope=PTR, k_rope_batch=1728,
             k_rope_token=576, kv=PTR, kv_rows=100, row_stride=576, kv_scale=1.0, d_pos=PTR, row_offset=PTR)
    a.update(kw)
    return mla.RopeArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), mla.EINVAL), (dict(batch=65536), mla.EINVAL), (dict(tokens=0), mla.EINVAL),
    (dict(heads=-1), mla.EUNSUPPORTED), (dict(heads=129), mla.EUNSUPPORTED), (dict(rot_dim=20), mla.EUNSUPPORTED),
    (dict(rot_dim=0), mla.EUNSUPPORTED), (dict(interleaved=2), mla.EINVAL), (dict(amplitude=0.0), mla.EINVAL),
    (dict(amplitude=math.nan), mla.EINVAL), (dict(turns=None), mla.EINVAL), (dict(positions=None), mla.EINVAL),
    (dict(q_rope=None), mla.EINVAL), (dict(q_out=None), mla.EINVAL), (dict(c=None), mla.EINVAL),
    (dict(k_rope=None), mla.EINVAL), (dict(kv=None), mla.EINVAL), (dict(d_pos=None), mla.EINVAL),
    (dict(row_offset=None), mla.EINVAL), (dict(kv_rows=0), mla.EINVAL), (dict(row_stride=575), mla.EINVAL),
    (dict(row_stride=580), mla.EALIGN), (dict(kv_fp8=2), mla.EINVAL), (dict(kv_fp8=1, kv_scale=0.0), mla.EINVAL),
    (dict(kv_fp8=1, row_stride=584), mla.EALIGN), (dict(q_rope=PTR + 8), mla.EALIGN), (dict(kv=PTR + 4), mla.EALIGN),
    (dict(q_rope_head=66), mla.EALIGN), (dict(q_out_token=9220), mla.EALIGN), (dict(c_token=577), mla.EALIGN),
    (dict(k_rope_batch=4), mla.EALIGN), (dict(d_pos=PTR + 2), mla.EALIGN), (dict(turns=PTR + 4), mla.EALIGN),
    (dict(heads=0, kv=None, c=None, k_rope=None), mla.EINVAL), (dict(row_weights=PTR + 1), mla.EALIGN),
    (dict(tokens=(1 << 28) + 1), mla.EINVAL),
])
def test_rope_refusals(kw, status):
    assert refused("mla_rope_append", ctypes.byref(rope_args(**kw)), None) == status


def test_rope_null():
    assert refused("mla_rope_append", None, None) == mla.EINVAL
    assert refused("mla_rope_table", None, None) == mla.EINVAL


# ---- tree ----------------------------------------------------------------------
def tree_plan(**kw):
    return mla.tree_plan(**{**dict(batch=2, tokens=8, heads=16, scale=0.04, num_sms=152), **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), mla.EINVAL), (dict(batch=4097), mla.EINVAL), (dict(tokens=0), mla.EINVAL),
    (dict(tokens=65), mla.EINVAL), (dict(heads=0), mla.EUNSUPPORTED), (dict(heads=129), mla.EUNSUPPORTED),
    (dict(scale=0.0), mla.EINVAL), (dict(scale=math.inf), mla.EINVAL), (dict(scale=math.nan), mla.EINVAL),
    (dict(num_sms=-1), mla.EINVAL), (dict(scale=3e38), mla.EINVAL),
])
def test_tree_plan_refusals(kw, status):
    with pytest.raises(mla.MLADecodeError) as e:
        tree_plan(**kw)
    assert e.value.status == status


def test_every_scale_that_a_plan_takes_is_a_number_in_base_2():
    """The kernels scale by float32(scale * log2 e): finite for the largest scale taken, infinite for the next."""
    def taken(bits):
        try:
            tree_plan(scale=float(np.int32(bits).view(np.float32)))
            return True
        except mla.MLADecodeError:
            return False
    lo, hi = int(np.float32(2e38).view(np.int32)), int(np.float32(3e38).view(np.int32))
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if taken(mid) else (lo, mid)
    with np.errstate(over="ignore"):
        in_base_2 = [np.float32(np.float64(np.int32(b).view(np.float32)) * math.log2(math.e)) for b in (lo, hi)]
    assert np.isfinite(in_base_2[0]) and np.isinf(in_base_2[1])


def test_tree_plan_layout():
    for sms in (2, 3, 152):
        p = tree_plan(num_sms=sms)
        assert p.scratch_bytes % 256 == 0 and p.part_offset % 256 == 0 and p.lse_part_offset % 256 == 0
        assert 0 == p.status_offset < p.part_offset <= p.lse_part_offset <= p.scratch_bytes
        assert 1 <= p.grid


def tree_args(**kw):
    a = dict(q=PTR, kv=PTR, kv_rows=100, row_stride=576, d_pos=PTR, row_offset=PTR, out=PTR, lse=PTR)
    a.update(kw)
    return mla.TreeArgs(**a)


TREE_BAD = [
    (dict(q=None), mla.EINVAL), (dict(kv=None), mla.EINVAL), (dict(d_pos=None), mla.EINVAL),
    (dict(lse=None), mla.EINVAL), (dict(row_offset=None), mla.EINVAL), (dict(kv_rows=0), mla.EINVAL),
    (dict(kv_rows=1 << 31), mla.EUNSUPPORTED), (dict(row_stride=568), mla.EINVAL), (dict(row_stride=580), mla.EALIGN),
    (dict(out_fp32=3), mla.EINVAL), (dict(q=PTR + 2), mla.EALIGN), (dict(kv=PTR + 8), mla.EALIGN),
    (dict(lse=PTR + 2), mla.EALIGN), (dict(mask=PTR + 4), mla.EALIGN), (dict(n_tokens=PTR + 1), mla.EALIGN),
    (dict(row_offset=PTR + 4), mla.EALIGN), (dict(d_pos=PTR + 1), mla.EALIGN),
]


@pytest.mark.parametrize("kw,status", TREE_BAD + [(dict(out=None), mla.EINVAL), (dict(out=PTR + 8), mla.EALIGN)])
def test_tree_forward_refusals(kw, status):
    p = tree_plan()
    assert refused("mla_tree_forward", ctypes.byref(p), ctypes.byref(tree_args(**kw)), PTR, p.scratch_bytes,
                   None) == status


@pytest.mark.parametrize("kw,status", TREE_BAD)
def test_tree_weights_refusals(kw, status):
    p = tree_plan()
    assert refused("mla_tree_weights", ctypes.byref(p), ctypes.byref(tree_args(out=None, **kw)), PTR, 1.0, PTR,
                   p.scratch_bytes, None) == status


@pytest.mark.parametrize("weights,decay,status", [
    (None, 1.0, mla.EINVAL), (PTR + 2, 1.0, mla.EALIGN), (PTR, -0.1, mla.EINVAL), (PTR, 1.5, mla.EINVAL),
    (PTR, math.nan, mla.EINVAL),
])
def test_tree_weights_own_arguments(weights, decay, status):
    p = tree_plan()
    assert refused("mla_tree_weights", ctypes.byref(p), ctypes.byref(tree_args()), weights, decay, PTR,
                   p.scratch_bytes, None) == status


def test_tree_scratch_and_plan_refusals():
    p, a = tree_plan(), tree_args()
    call = lambda pl, s, n: refused("mla_tree_forward", ctypes.byref(pl), ctypes.byref(a), s, n, None)  # noqa: E731
    assert call(p, None, p.scratch_bytes) == mla.ESCRATCH
    assert call(p, PTR + 16, p.scratch_bytes) == mla.ESCRATCH
    assert call(p, PTR, p.scratch_bytes - 1) == mla.ESCRATCH
    for field, value in (("magic", 0), ("grid", p.grid + 1), ("scratch_bytes", p.scratch_bytes + 256),
                         ("part_offset", p.part_offset + 256), ("lse_part_offset", p.lse_part_offset + 256),
                         ("status_offset", 4), ("num_sms", 0)):
        bad = mla.TreePlan.from_buffer_copy(p)
        setattr(bad, field, value)
        assert call(bad, PTR, p.scratch_bytes) == mla.EINVAL, field
    bad = mla.TreePlan.from_buffer_copy(p)
    bad.shape.tokens = 65
    assert call(bad, PTR, p.scratch_bytes) == mla.EINVAL
    assert refused("mla_tree_forward", None, ctypes.byref(a), PTR, 1 << 30, None) == mla.EINVAL
    assert refused("mla_tree_plan", None, None) == mla.EINVAL


# ---- commit and evict ---------------------------------------------------------
@pytest.mark.parametrize("kw,status", [
    (dict(kv=None), mla.EINVAL), (dict(accept=None), mla.EINVAL), (dict(n_accept=None), mla.EINVAL),
    (dict(d_pos=None), mla.EINVAL), (dict(batch=0), mla.EINVAL), (dict(batch=65536), mla.EINVAL),
    (dict(tokens=0), mla.EINVAL), (dict(tokens=65), mla.EINVAL), (dict(row_offset=None), mla.EINVAL),
    (dict(kv_rows=0), mla.EINVAL), (dict(row_stride=10), mla.EINVAL), (dict(kv_fp8=2), mla.EINVAL),
    (dict(row_stride=580), mla.EALIGN), (dict(kv_fp8=1, row_stride=584), mla.EALIGN), (dict(kv=PTR + 8), mla.EALIGN),
    (dict(d_pos_out=PTR + 2), mla.EALIGN), (dict(row_positions=PTR + 2), mla.EALIGN),
])
def test_commit_refusals(kw, status):
    a = dict(kv=PTR, kv_rows=100, row_stride=576, batch=2, tokens=8, accept=PTR, n_accept=PTR, d_pos=PTR,
             row_offset=PTR)
    a.update(kw)
    assert refused("mla_tree_commit", ctypes.byref(mla.TreeCommitArgs(**a)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kv=None), mla.EINVAL), (dict(weights=None), mla.EINVAL), (dict(positions=None), mla.EINVAL),
    (dict(next_pos=None), mla.EINVAL), (dict(weights_out=None), mla.EINVAL), (dict(d_pos_out=None), mla.EINVAL),
    (dict(positions_out=None), mla.EINVAL), (dict(batch=0), mla.EINVAL), (dict(keep=0), mla.EINVAL),
    (dict(sink=-1), mla.EINVAL), (dict(recent=-1), mla.EINVAL), (dict(max_rows=0), mla.EINVAL),
    (dict(kv_fp8=7), mla.EINVAL), (dict(row_offset=None), mla.EINVAL), (dict(row_stride=580), mla.EALIGN),
    (dict(weights=PTR + 2), mla.EALIGN), (dict(row_offset=PTR + 4), mla.EALIGN),
])
def test_evict_refusals(kw, status):
    a = dict(kv=PTR, kv_rows=100, row_stride=576, batch=2, keep=10, max_rows=50, weights=PTR, positions=PTR, d_pos=PTR,
             next_pos=PTR, row_offset=PTR, weights_out=PTR, positions_out=PTR, d_pos_out=PTR)
    a.update(kw)
    n = mla.lib().mla_evict_scratch_bytes(2, 10)
    assert refused("mla_evict", ctypes.byref(mla.EvictArgs(**a)), PTR, n, None) == status


def test_evict_scratch():
    L = mla.lib()
    assert L.mla_evict_scratch_bytes(0, 1) == 0 and L.mla_evict_scratch_bytes(1, 0) == 0
    n = L.mla_evict_scratch_bytes(3, 1000)
    assert n >= 3 * 4 + 2 * 3 * 1000 * 4 and n % 256 == 0
    assert L.mla_evict_scratch_bytes(65535, 1 << 20) >= 2 * 65535 * (1 << 20) * 4
    a = mla.EvictArgs(kv=PTR, kv_rows=100, row_stride=576, batch=1, keep=10, max_rows=50, weights=PTR, positions=PTR,
                      d_pos=PTR, next_pos=PTR, weights_out=PTR, positions_out=PTR, d_pos_out=PTR)
    need = L.mla_evict_scratch_bytes(1, 10)
    assert refused("mla_evict", ctypes.byref(a), PTR, need - 1, None) == mla.ESCRATCH
    assert refused("mla_evict", ctypes.byref(a), PTR + 64, need, None) == mla.ESCRATCH
    assert refused("mla_evict", ctypes.byref(a), None, need, None) == mla.ESCRATCH


def test_python_side_wants_cuda_tensors():
    import torch
    x = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mla.tree_make_args(x, torch.zeros(4, 576, dtype=torch.bfloat16), None, torch.zeros(1, 1, 16),
                           d_pos=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        mla.rope_turns(scaling="other")
    with pytest.raises(ValueError):
        mla.evict_alloc_scratch(batch=1, keep=0)


def test_packed_commit_arguments_have_the_structures_layout():
    v = list(range(1, 14))
    a = mla.TreeCommitArgs(*v)
    assert mla._COMMIT_ARGS.size == ctypes.sizeof(a) and mla._COMMIT_ARGS.pack(*v) == bytes(a)


@pytest.mark.parametrize("call", [
    lambda big: tree_plan(batch=big), lambda big: tree_plan(tokens=big), lambda big: tree_plan(heads=big),
    lambda big: tree_plan(num_sms=big), lambda big: mla.rope_turns(big), lambda big: mla._int(-big, "x"),
    lambda big: mla.evict_alloc_scratch(batch=big, keep=4), lambda big: mla.evict_alloc_scratch(batch=1, keep=big),
])
def test_integers_past_32_bits_are_refused(call):
    """A C int would take them modulo 2^32: 2^32 + 8 rows to keep would be 8."""
    with pytest.raises(ValueError, match="32-bit"):
        call(2 ** 32 + 8)
