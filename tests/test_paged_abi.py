"""Host-side checks of the paged cache's entry points: every call here is refused
before anything is launched, or needs no device."""
import ctypes
import math

import pytest
import torch

import decode_attention_mla_gb300 as mla
from decode_attention_mla_gb300 import build as mla_build
import _paged_ref as ref

PTR = 0x100000                       # never dereferenced: the call is refused first


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()
    yield


def cache(**kw):
    return mla.PagedCache(**{**dict(pages=PTR, page_stride=64 * 416, n_pages=10, page_rows=64, page_table=PTR,
                                    columns=4, kv_scale=1.0), **kw})


BAD_CACHE = [
    (dict(page_table=None), mla.EINVAL), (dict(n_pages=0), mla.EINVAL), (dict(n_pages=-1), mla.EINVAL),
    (dict(page_rows=0), mla.EINVAL), (dict(page_rows=4), mla.EINVAL), (dict(page_rows=48), mla.EINVAL),
    (dict(page_rows=2048, page_stride=2048 * 416), mla.EINVAL), (dict(page_stride=64 * 416 - 16), mla.EINVAL),
    (dict(page_stride=64 * 416 + 8), mla.EALIGN), (dict(columns=0), mla.EINVAL), (dict(columns=1 << 25), mla.EINVAL),
    (dict(kv_scale=0.0), mla.EINVAL), (dict(kv_scale=3.0), mla.EINVAL), (dict(kv_scale=-1.0), mla.EINVAL),
    (dict(kv_scale=math.nan), mla.EINVAL), (dict(kv_scale=math.inf), mla.EINVAL), (dict(kv_scale=2.0 ** 65), mla.EINVAL),
    (dict(kv_scale=2.0 ** -65), mla.EINVAL), (dict(pages=PTR + 8), mla.EALIGN), (dict(page_table=PTR + 2), mla.EALIGN),
]


def append_args(**kw):
    a = dict(cache=cache(), batch=2, tokens=3, heads=16, rot_dim=64, interleaved=1, amplitude=1.0, turns=PTR,
             positions=PTR, q_rope=PTR, q_rope_batch=576, q_rope_token=192, q_rope_head=64, q_out=PTR,
             q_out_batch=27648, q_out_token=9216, q_out_head=576, c=PTR, c_batch=1728, c_token=576, k_rope=PTR,
             k_rope_batch=1728, k_rope_token=576, eps=1e-6, d_pos=PTR)
    a.update(kw)
    return mla.PagedAppendArgs(**a)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**k)), s) for k, s in BAD_CACHE] + [
    (dict(batch=0), mla.EINVAL), (dict(batch=65536), mla.EINVAL), (dict(tokens=0), mla.EINVAL),
    (dict(tokens=(1 << 28) + 1), mla.EINVAL), (dict(heads=-1), mla.EUNSUPPORTED), (dict(heads=129), mla.EUNSUPPORTED),
    (dict(rot_dim=20), mla.EUNSUPPORTED), (dict(rot_dim=72), mla.EUNSUPPORTED), (dict(interleaved=2), mla.EINVAL),
    (dict(amplitude=0.0), mla.EINVAL), (dict(amplitude=math.inf), mla.EINVAL), (dict(eps=-1e-6), mla.EINVAL),
    (dict(eps=math.nan), mla.EINVAL), (dict(turns=None), mla.EINVAL), (dict(positions=None), mla.EINVAL),
    (dict(q_rope=None), mla.EINVAL), (dict(q_out=None), mla.EINVAL), (dict(c=None), mla.EINVAL),
    (dict(k_rope=None), mla.EINVAL), (dict(d_pos=None), mla.EINVAL), (dict(cache=cache(pages=None)), mla.EINVAL),
    (dict(heads=0, q_rope=None, q_out=None, q_norm=PTR), mla.EINVAL), (dict(heads=0), mla.EINVAL),
    (dict(cache=cache(pages=None), c=None, k_rope=None, d_pos=None, c_norm=PTR), mla.EINVAL),
    (dict(cache=cache(pages=None), c=None, k_rope=None, d_pos=None, heads=0, q_rope=None, q_out=None), mla.EINVAL),
    (dict(q_rope=PTR + 8), mla.EALIGN), (dict(q_rope_head=66), mla.EALIGN), (dict(q_out_token=9220), mla.EALIGN),
    (dict(c_token=577), mla.EALIGN), (dict(k_rope_batch=4), mla.EALIGN), (dict(d_pos=PTR + 2), mla.EALIGN),
    (dict(turns=PTR + 4), mla.EALIGN), (dict(c_norm=PTR + 8), mla.EALIGN), (dict(k_norm=PTR + 8), mla.EALIGN),
    (dict(q_norm=PTR + 8), mla.EALIGN), (dict(n_tokens=PTR + 1), mla.EALIGN),
])
def test_append_refusals(kw, status):
    assert mla.lib().mla_paged_append(ctypes.byref(append_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**k)), s) for k, s in BAD_CACHE] + [
    (dict(cache=cache(pages=None)), mla.EINVAL), (dict(batch=0), mla.EINVAL), (dict(batch=65536), mla.EINVAL),
    (dict(rows=0), mla.EINVAL), (dict(out=None), mla.EINVAL), (dict(out_row=568), mla.EINVAL),
    (dict(out_row=580), mla.EALIGN), (dict(out_batch=4), mla.EALIGN), (dict(out=PTR + 8), mla.EALIGN),
    (dict(first=PTR + 2), mla.EALIGN), (dict(n_rows=PTR + 1), mla.EALIGN),
])
def test_read_refusals(kw, status):
    a = mla.PagedReadArgs(**{**dict(cache=cache(), batch=2, rows=5, out=PTR, out_batch=2880, out_row=576), **kw})
    assert mla.lib().mla_paged_read(ctypes.byref(a), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), mla.EINVAL), (dict(batch=4097), mla.EINVAL), (dict(tokens=0), mla.EINVAL),
    (dict(tokens=65), mla.EINVAL), (dict(heads=0), mla.EUNSUPPORTED), (dict(heads=129), mla.EUNSUPPORTED),
    (dict(scale=0.0), mla.EINVAL), (dict(scale=-1.0), mla.EINVAL), (dict(scale=math.nan), mla.EINVAL),
    (dict(scale=2.0 ** 60), mla.EINVAL), (dict(num_sms=-1), mla.EINVAL),
])
def test_plan_refusals(kw, status):
    with pytest.raises(mla.MLADecodeError) as e:
        mla.paged_plan(**{**dict(batch=2, tokens=3, heads=16, scale=0.05, num_sms=152), **kw})
    assert e.value.status == status


def forward(plan, scratch=PTR, nbytes=None, **kw):
    a = mla.PagedArgs(**{**dict(cache=cache(), q=PTR, d_pos=PTR, out=PTR, lse=PTR), **kw})
    return mla.lib().mla_paged_forward(ctypes.byref(plan), ctypes.byref(a), scratch,
                                       plan.scratch_bytes if nbytes is None else nbytes, None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**k)), s) for k, s in BAD_CACHE] + [
    (dict(cache=cache(pages=None)), mla.EINVAL), (dict(q=None), mla.EINVAL), (dict(d_pos=None), mla.EINVAL),
    (dict(out=None), mla.EINVAL), (dict(lse=None), mla.EINVAL), (dict(window=-1), mla.EINVAL),
    (dict(sink=-1), mla.EINVAL), (dict(out_fp32=2), mla.EINVAL), (dict(q=PTR + 8), mla.EALIGN),
    (dict(out=PTR + 8), mla.EALIGN), (dict(lse=PTR + 2), mla.EALIGN), (dict(d_pos=PTR + 2), mla.EALIGN),
    (dict(n_tokens=PTR + 2), mla.EALIGN), (dict(scratch=None), mla.ESCRATCH), (dict(scratch=PTR + 16), mla.ESCRATCH),
    (dict(nbytes=1000), mla.ESCRATCH),
])
def test_forward_refusals(kw, status):
    assert forward(mla.paged_plan(batch=2, tokens=3, heads=16, scale=0.05, num_sms=152), **kw) == status


@pytest.mark.parametrize("field,value", [("magic", 1), ("num_sms", 0), ("grid", 7), ("scratch_bytes", 1 << 20),
                                         ("part_offset", 0), ("lse_part_offset", 256), ("status_offset", 4)])
def test_edited_plan_is_refused(field, value):
    plan = mla.paged_plan(batch=2, tokens=3, heads=16, scale=0.05, num_sms=152)
    setattr(plan, field, value)
    assert forward(plan, nbytes=1 << 40) == mla.EINVAL


POOL = dict(pages=PTR, page_stride=64 * 416, n_pages=10, page_rows=64, row_bytes=416, batch=3, columns=5,
            page_table=PTR, page_table_out=PTR)
BAD_POOL = [
    (dict(pages=None), mla.EINVAL), (dict(n_pages=0), mla.EINVAL), (dict(n_pages=(1 << 30) + 1), mla.EINVAL),
    (dict(page_rows=4), mla.EINVAL), (dict(page_rows=100), mla.EINVAL), (dict(row_bytes=0), mla.EINVAL),
    (dict(row_bytes=408), mla.EALIGN), (dict(row_bytes=65552), mla.EINVAL), (dict(page_stride=1024), mla.EINVAL),
    (dict(page_stride=64 * 416 + 4), mla.EALIGN), (dict(batch=0), mla.EINVAL), (dict(batch=4097), mla.EINVAL),
    (dict(columns=0), mla.EINVAL), (dict(columns=1 << 26), mla.EINVAL), (dict(batch=4096, columns=1 << 18), mla.EINVAL),
    (dict(page_table=None), mla.EINVAL), (dict(page_table_out=None), mla.EINVAL), (dict(pages=PTR + 8), mla.EALIGN),
    (dict(page_table=PTR + 1), mla.EALIGN), (dict(page_table_out=PTR + 2), mla.EALIGN),
]


@pytest.mark.parametrize("kw,status", BAD_POOL + [
    (dict(d_pos=None), mla.EINVAL), (dict(d_pos_out=None), mla.EINVAL), (dict(refs=None), mla.EINVAL),
    (dict(missing=None), mla.EINVAL), (dict(reserve=-1), mla.EINVAL), (dict(window=-1), mla.EINVAL),
    (dict(sink=-1), mla.EINVAL), (dict(parent=PTR + 2), mla.EALIGN), (dict(rows=PTR + 2), mla.EALIGN),
    (dict(refs=PTR + 2), mla.EALIGN), (dict(scratch=None), mla.ESCRATCH), (dict(scratch=PTR + 4), mla.ESCRATCH),
    (dict(nbytes=100), mla.ESCRATCH), (dict(page_table_out=PTR + 56), mla.EINVAL), (dict(d_pos_out=PTR - 8), mla.EINVAL),
])
def test_fork_refusals(kw, status):
    kw = dict(kw)
    scratch, nbytes = kw.pop("scratch", PTR), kw.pop("nbytes", 1 << 30)
    a = mla.PagesForkArgs(**{**POOL, **dict(d_pos=PTR, d_pos_out=PTR, refs=PTR, missing=PTR), **kw})
    assert mla.lib().mla_pages_fork(ctypes.byref(a), scratch, nbytes, None) == status


@pytest.mark.parametrize("kw,status", BAD_POOL + [
    (dict(refs=None), mla.EINVAL), (dict(refs_out=None), mla.EINVAL), (dict(used=None), mla.EINVAL),
    (dict(refs=PTR + 2), mla.EALIGN), (dict(used=PTR + 2), mla.EALIGN), (dict(scratch=None), mla.ESCRATCH),
    (dict(nbytes=100), mla.ESCRATCH), (dict(page_table_out=PTR - 56), mla.EINVAL), (dict(refs_out=PTR + 36), mla.EINVAL),
])
def test_compact_refusals(kw, status):
    kw = dict(kw)
    scratch, nbytes = kw.pop("scratch", PTR), kw.pop("nbytes", 1 << 30)
    a = mla.PagesCompactArgs(**{**POOL, **dict(refs=PTR, refs_out=PTR, used=PTR), **kw})
    assert mla.lib().mla_pages_compact(ctypes.byref(a), scratch, nbytes, None) == status


def test_null_arguments():
    L = mla.lib()
    assert L.mla_paged_append(None, None) == mla.EINVAL and L.mla_paged_read(None, None) == mla.EINVAL
    assert L.mla_pages_fork(None, PTR, 1 << 30, None) == mla.EINVAL
    assert L.mla_pages_compact(None, PTR, 1 << 30, None) == mla.EINVAL
    plan = mla.paged_plan(batch=1, tokens=1, heads=1, scale=1.0, num_sms=152)
    assert L.mla_paged_forward(None, None, PTR, 1 << 30, None) == mla.EINVAL
    assert L.mla_paged_forward(ctypes.byref(plan), None, PTR, 1 << 30, None) == mla.EINVAL
    assert L.mla_paged_plan(None, ctypes.byref(plan)) == mla.EINVAL


@pytest.mark.parametrize("batch,columns,n_pages", [(0, 1, 1), (4097, 1, 1), (1, 0, 1), (1, 1, 0), (4096, 1 << 18, 1),
                                                   (1, 1, (1 << 30) + 1)])
def test_scratch_of_sizes_out_of_range(batch, columns, n_pages):
    assert mla.lib().mla_pages_scratch_bytes(batch, columns, n_pages) == 0


def test_binding_refuses_cpu_tensors_and_wide_integers():
    q, pages = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 16, 416, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mla.paged_make_args(q, pages, torch.zeros(1, 4, dtype=torch.int32), q, q, d_pos=q)
    with pytest.raises(ValueError, match="CUDA"):
        mla.pages_fork_make_args(pages, torch.zeros(1, 4, dtype=torch.int32), q, q, missing=q)
    with pytest.raises(ValueError, match="32-bit"):
        mla.paged_plan(batch=2 ** 32 + 1, tokens=1, heads=16, scale=1.0, num_sms=152)


# ---- the references against small cases worked by hand ---------------------------
def test_values_of_a_row():
    raw = torch.zeros(1, 416, dtype=torch.uint8)
    raw[0, 0], raw[0, 8], raw[0, 255] = 0x72, 0xf1, 0x0b            # features 0, 1; 16, 17; 510, 511
    raw[0, 256:288] = 0x38                                          # 1.0
    raw[0, 257] = 0x40                                              # 2.0
    raw[0, 288:290] = torch.tensor([0x80, 0x3f], dtype=torch.uint8)  # 1.0 in bf16
    v = ref.row_values(raw, 0.5)[0]
    assert v[:2].tolist() == [0.5, 3.0] and v[16:18].tolist() == [0.5, -6.0] and v[510:512].tolist() == [-0.75, 0.0]
    assert v[512] == 1.0


def test_quantised_values_are_the_nearest():
    c = torch.zeros(1, 512, dtype=torch.float64)
    c[0, :16] = torch.tensor([6, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5.0, -3.5, -2.5, -1.75, -1.25, -0.75, -0.2])
    code, scale = ref.quantise(c, 1.0)
    assert scale[0, 0] == 1 and scale[0, 1] == 0
    assert ref.E2M1[code[0, :16]].tolist() == [6, 4, 4, 2, 2, 1, 1, 0, -6, -4, -4, -2, -2, -1, -1, 0]


def test_fork_by_hand():
    p = ref.Pages([[3, 5, -1], [3, 6, -1], [0, -1, -1]], [12, 16, 4], 8, 8)
    refs, missing, copies = p.fork(parent=[0, 0, -1], reserve=6)
    # request 0 keeps page 5, request 1 gets a copy in page 0; both need rows 12 .. 17
    assert p.table == [[3, 5, 0], [3, 1, 2], [-1, -1, -1]] and p.d_pos == [12, 12, 0]
    assert copies == [(5, 1, 4)] and missing == 0 and refs == [1, 1, 1, 2, 0, 1, 0, 0]
    out, live, moves = p.compact(refs)
    assert live == 5 and moves == [(5, 4)] and p.table[0] == [3, 4, 0] and out == [1, 1, 1, 2, 1, 0, 0, 0]
