"""Host-side checks of the paged cache at the ends of what its calls allow."""
import ctypes

import pytest
import torch

import decode_attention_mla_gb300 as mla
from decode_attention_mla_gb300 import build as mla_build
import _paged_ref as ref


def test_fork_of_rows_that_end_in_a_missing_page_by_hand():
    p = ref.Pages([[0, 1, -1, -1], [2, 3, 5, -1]], [20, 20], 8, 8)
    assert p.fork() == ([1, 1, 1, 1, 0, 1, 0, 0], 0, [])
    assert p.table == [[0, 1, -1, -1], [2, 3, 5, -1]] and p.d_pos == [16, 20]
    # a window gives back what no token from the rounded row on attends
    p = ref.Pages([[3, -1], [6, 4]], [12, 12], 8, 8)
    p.fork(window=4)
    assert p.table == [[3, -1], [-1, 4]] and p.d_pos == [8, 12]


# ---- outputs that lie in one place ------------------------------------------------
PTR = 0x100000                       # never dereferenced: the call is refused first


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()
    yield


@pytest.fixture
def on_host(monkeypatch):
    """The binding's layout of arguments, with CPU tensors for CUDA ones."""
    monkeypatch.setattr(mla, "_need", lambda t, name, dtypes, shape=None, contiguous=True: t.data_ptr())
    monkeypatch.setattr(mla, "_device", lambda: 0)


def read_args(out):
    pages, table = torch.zeros(4, 16, 416, dtype=torch.uint8), torch.zeros(out.shape[0], 4, dtype=torch.int32)
    return mla.paged_read_make_args(out, pages, table)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("out", [bf16(2, 1, 576).expand(2, 5, 576), bf16(1, 5, 576).expand(2, 5, 576),
                                 bf16(1, 1, 576).expand(3, 2, 576), bf16(1, 1, 576).expand(3, 1, 576)],
                         ids=lambda t: str((tuple(t.shape), t.stride())))
def test_reads_into_an_expanded_tensor_are_refused(out, on_host):
    """(The strides of an expanded dimension are 0: rows of 576 behind the first would lie behind the storage.)"""
    with pytest.raises(ValueError, match="expanded"):
        read_args(out)


@pytest.mark.parametrize("shape", [(2, 5, 576), (2, 1, 576), (1, 5, 576), (1, 1, 576)])
def test_reads_into_a_tensor_of_its_own(shape, on_host):
    out = bf16(*shape)
    a = read_args(out)
    last = (shape[0] - 1) * a.out_batch + (shape[1] - 1) * a.out_row + 576
    assert a.out_row >= 576 and last == out.numel()
    a = read_args(bf16(shape[1], shape[0], 600).transpose(0, 1)[..., :576])     # requests side by side
    assert a.out_row >= 576 and (shape[0] - 1) * a.out_batch + (shape[1] - 1) * a.out_row + 600 == 600 * shape[0] * shape[1]


@pytest.mark.parametrize("kw,status", [(dict(out_batch=0), mla.EINVAL), (dict(out_batch=568), mla.EINVAL),
                                       (dict(out_batch=-568), mla.EINVAL), (dict(out_row=0), mla.EINVAL)])
def test_library_refuses_reads_into_one_place(kw, status):
    c = mla.PagedCache(pages=PTR, page_stride=64 * 416, n_pages=10, page_rows=64, page_table=PTR, columns=4, kv_scale=1.0)
    a = mla.PagedReadArgs(**{**dict(cache=c, batch=2, rows=5, out=PTR, out_batch=2880, out_row=576), **kw})
    assert mla.lib().mla_paged_read(ctypes.byref(a), None) == status


def append_args(q):
    B, N = q.shape[:2]
    table = mla.RopeTable(torch.zeros(32, dtype=torch.int64), 64, True, 1.0)
    return mla.paged_append_make_args(table, torch.zeros(B, N, dtype=torch.int32), q_rope=bf16(*q.shape[:3], 64), q=q)


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_queries_written_to_an_expanded_tensor_are_refused(dim, on_host):
    shape = [2, 3, 4, 576]
    wide = list(shape)
    shape[dim] = 1
    append_args(bf16(*shape))
    append_args(bf16(*wide))
    with pytest.raises(ValueError, match="expanded"):
        append_args(bf16(*shape).expand(wide))


@pytest.mark.parametrize("kw", [dict(q_out_batch=0), dict(q_out_token=0), dict(q_out_head=0), dict(q_out_head=56),
                                dict(q_out_token=-56)])
def test_library_refuses_queries_in_one_place(kw):
    a = mla.PagedAppendArgs(**{**dict(batch=2, tokens=3, heads=16, rot_dim=64, interleaved=1, amplitude=1.0, turns=PTR,
                                      positions=PTR, q_rope=PTR, q_rope_batch=576, q_rope_token=192, q_rope_head=64,
                                      q_out=PTR, q_out_batch=27648, q_out_token=9216, q_out_head=576, eps=1e-6), **kw})
    assert mla.lib().mla_paged_append(ctypes.byref(a), None) == mla.EINVAL
