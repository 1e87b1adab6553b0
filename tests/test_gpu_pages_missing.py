"""Requests whose last page is missing: what goes on from them has no rows that
were never written."""
import pytest
import torch

import decode_attention_mla_gb300 as mla
from test_gpu_pages import I32, Pool

pytestmark = pytest.mark.gpu
# pools that one block forks, with its copies and without, and one that three launches fork
SIZES = pytest.mark.parametrize("n_pages,width", [(8, 416), (8, 16384), (70000, 16)])


@SIZES
def test_rows_end_before_a_last_page_that_is_missing(n_pages, width):
    p = Pool([[0, 1, -1, -1], [2, 3, 5, -1]], [20, 20], n_pages, 8, width=width)
    p.fork()
    assert p.table.tolist() == [[0, 1, -1, -1], [2, 3, 5, -1]] and p.d_pos.tolist() == [16, 20]
    assert int(p.count) == 0
    p = Pool([[0, 1, n_pages, -1], [2, 3, 5, -1]], [20, 20], n_pages, 8, width=width)
    p.fork(reserve=3)                                      # a page for rows 16 .. 18, and none for 20 .. 22 of the other
    assert p.table.tolist() == [[0, 1, 4, -1], [2, 3, 5, -1]] and p.d_pos.tolist() == [16, 20]
    p = Pool([[-7, 1, 6, -1]], [20], n_pages, 8, width=width)
    p.fork(None, [5], reserve=1)                           # back into a page that is missing
    assert p.table.tolist() == [[0, -1, -1, -1]] and p.d_pos.tolist() == [0]
    p = Pool([[0, 1, -1, -1]] * 3, [20, 20, 20], n_pages, 8, width=width)
    p.fork([0, 0, 2], [20, 13, 17], reserve=1)
    assert p.d_pos.tolist() == [16, 13, 16]


@SIZES
def test_a_window_keeps_what_the_rows_that_are_left_need(n_pages, width):
    p = Pool([[3, -1], [6, 4]], [12, 12], n_pages, 8, width=width)
    p.fork(None, window=4)                                 # from row 8 on rows 5 .. 7 are seen, from row 12 on 9 ..
    assert p.table.tolist() == [[3, -1], [-1, 4]] and p.d_pos.tolist() == [8, 12]


def test_attention_after_a_shortage():
    """Pages run out, a step's rows are dropped, pages come free: the request goes on from the rows it has."""
    H, R = 16, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    rope = mla.rope_table(64, base=10000.0)
    pages, table = mla.paged_alloc(4, R), torch.full((2, 6), -1, **I32)
    d_pos, refs, missing = torch.zeros(2, **I32), torch.zeros(4, **I32), torch.zeros(1, **I32)
    scratch = mla.pages_alloc_scratch(pages, table)

    def step(n, parent):
        mla.pages_fork(pages, table, d_pos, refs, scratch, parent=torch.tensor(parent, **I32), reserve=n, missing=missing)
        c, k = randn(2, n, 512), randn(2, n, 64)
        c[1] *= 50
        mla.paged_append(rope, d_pos[:, None] + torch.arange(n, **I32), c=c, k_rope=k, pages=pages, page_table=table,
                         d_pos=d_pos)
        return c, k

    c, k = step(16, [0, 1])
    d_pos += 16
    step(4, [0, 1])
    assert int(missing) == 2                               # rows 16 .. 19 have no page and were not written
    d_pos += 4
    c1, k1 = step(1, [0, -1])
    assert d_pos.tolist() == [16, 0] and int(missing) == 0
    plan = mla.paged_plan(batch=2, tokens=1, heads=H, scale=576 ** -0.5)
    attend = mla.paged_alloc_scratch(plan)
    q = randn(2, 1, H, 576)
    out, lse = torch.zeros(2, 1, H, 512, device="cuda"), torch.zeros(2, 1, H, device="cuda")
    mla.paged_forward(plan, q, pages, table, out, lse, attend, d_pos=d_pos)
    # the same 17 rows in pages of their own
    flat, ft = mla.paged_alloc(12, R), torch.arange(12, **I32).view(2, 6)
    mla.paged_append(rope, torch.arange(17, **I32).repeat(2, 1), c=torch.cat([c, c1], 1), k_rope=torch.cat([k, k1], 1),
                     pages=flat, page_table=ft, d_pos=torch.zeros(2, **I32))
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    mla.paged_forward(plan, q, flat, ft, out2, lse2, attend, d_pos=torch.tensor([16, 16], **I32))
    assert torch.equal(out[0], out2[0]) and torch.equal(lse[0], lse2[0])
