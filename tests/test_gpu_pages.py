"""Pages forked, copied, reserved, freed and compacted on the GPU, against the
definition worked out with lists; and a serving loop over the paged cache."""
import random

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _paged_ref as ref

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def start(rnd, lens, n_pages, page_rows, columns):
    """Tables in which requests share first pages, at random places of the pool."""
    order = list(range(n_pages))
    rnd.shuffle(order)
    table = []
    for b, n in enumerate(lens):
        have = -(-n // page_rows)
        shared = table[b - 1][:rnd.randint(0, min(lens[b - 1], n) // page_rows)] if b and rnd.random() < 0.6 else []
        table.append(shared + [order.pop() for _ in range(have - len(shared))] + [-1] * (columns - have))
    return table


class Pool:
    def __init__(self, table, d_pos, n_pages, page_rows, dtype=torch.uint8, width=416, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.model = ref.Pages(table, d_pos, n_pages, page_rows)
        raw = torch.randint(0, 256, (n_pages, page_rows, width * torch.empty(0, dtype=dtype).element_size()), generator=g,
                            dtype=torch.uint8)
        self.want = raw
        self.pages = raw.view(dtype).cuda()
        self.table, self.d_pos = torch.tensor(table, **I32), torch.tensor(d_pos, **I32)
        self.refs, self.count = torch.full((n_pages,), -7, **I32), torch.full((1,), -7, **I32)
        self.scratch = mla.pages_alloc_scratch(self.pages, self.table)
        self.scratch.fill_(0xa5)                          # it needs no initial value

    def same(self, refs, count):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.model.table
        assert self.d_pos.tolist() == self.model.d_pos
        assert self.refs.tolist() == refs and self.count.tolist() == [count]
        assert torch.equal(self.pages.cpu().view(torch.uint8).flatten(), self.want.flatten())

    def fork(self, parent=None, rows=None, separate=False, **kw):
        refs, missing, copies = self.model.fork(parent, rows, **kw)
        before = self.want.clone()
        for src, dst, n in copies:
            self.want[dst, :n] = before[src, :n]
        t = lambda v: None if v is None else torch.tensor(v, **I32)  # noqa: E731
        to = dict(page_table_out=torch.full_like(self.table, 9), d_pos_out=torch.full_like(self.d_pos, 9)) if separate else {}
        mla.pages_fork(self.pages, self.table, self.d_pos, self.refs, self.scratch, parent=t(parent), rows=t(rows),
                       missing=self.count, **kw, **to)
        if separate:
            self.table, self.d_pos = to["page_table_out"], to["d_pos_out"]
        self.same(refs, missing)
        return refs

    def compact(self, refs, separate=False):
        self.refs = torch.tensor(refs, **I32)
        out, live, moves = self.model.compact(refs)
        for src, dst in moves:
            self.want[dst] = self.want[src]
        to = dict(page_table_out=torch.full_like(self.table, 9), refs_out=torch.full_like(self.refs, 9)) if separate else {}
        mla.pages_compact(self.pages, self.table, self.refs, self.scratch, used=self.count, **to)
        if separate:
            self.table, self.refs = to["page_table_out"], to["refs_out"]
        self.same(out, live)
        return out


@pytest.mark.parametrize("seed", range(12))
def test_random_steps(seed):
    rnd = random.Random(seed)
    page_rows = rnd.choice([8, 16, 32])
    B = rnd.choice([1, 2, 3, 7, 20])
    lens = [rnd.randint(0, 150) for _ in range(B)]
    columns = 200 // page_rows + rnd.randint(0, 3)
    n_pages = B * (200 // page_rows + 1) + rnd.randint(0, 20)
    kind = rnd.choice([dict(), dict(dtype=torch.bfloat16, width=576), dict(width=576), dict(width=16)])
    p = Pool(start(rnd, lens, n_pages, page_rows, columns), lens, n_pages, page_rows, seed=seed, **kind)
    for _ in range(6):
        parent = rnd.choice([None, [rnd.randint(-2, B) for _ in range(B)], [rnd.randrange(B) for _ in range(B)]])
        rows = rnd.choice([None, [rnd.randint(-1, 160) for _ in range(B)]])
        window = rnd.choice([0, 0, rnd.randint(1, 60)])
        refs = p.fork(parent, rows, separate=rnd.random() < 0.5, reserve=rnd.choice([0, 1, 5, 40]), window=window,
                      sink=rnd.randint(0, 20) if window else 0)
        if rnd.random() < 0.5:
            p.compact(refs, separate=rnd.random() < 0.5)


def test_all_go_on_from_one():
    p = Pool([[4, 2, 7, -1]] + [[-1] * 4] * 5, [20, 0, 0, 0, 0, 0], 16, 8)
    refs = p.fork([0] * 6, reserve=1)
    assert refs[4] == 6 and refs[2] == 6 and refs[7] == 1
    p.fork([5, 5, 5, -1, -1, 9])
    p.fork([-1] * 6)
    assert p.refs.tolist() == [0] * 16


def test_a_page_that_another_has_whole_is_copied():
    """Request 1 goes back into a page that request 0 has read to its end."""
    p = Pool([[3, 1, -1], [3, 2, -1]], [16, 12], 6, 8)
    p.fork(None, [16, 5])
    assert p.table.tolist() == [[3, 1, -1], [0, -1, -1]]


def test_too_few_pages():
    p = Pool([[0, 1, -1, -1], [2, 3, -1, -1]], [12, 15], 5, 8)
    p.fork([0, 0], reserve=20)
    assert int(p.count) > 0
    q = Pool([[0, 1], [2, 3]], [12, 12], 4, 8)
    q.fork([0, 0])
    q = Pool([[0, 1]], [12], 2, 8)
    q.fork(None)                                           # nothing to take
    q = Pool([[0, 1, 2], [0, 1, 2]], [20, 20], 3, 8)
    q.fork(None)                                           # the copy has no page: n falls to 16
    assert q.d_pos.tolist() == [20, 16] and int(q.count) == 1


def test_tables_with_entries_that_are_no_pages():
    p = Pool([[-1, 3, 99, -9], [2, -1, 1, 0]], [28, 30], 8, 8)
    p.fork(None, reserve=3)
    p.compact(p.refs.tolist())
    p = Pool([[5, 6, 7, 2 ** 31 - 1]], [30], 8, 8)
    p.compact([0, 0, 0, 0, 0, 1, 0, 2])                    # an entry whose page is not in use
    p = Pool([[-1] * 3], [-4], 8, 8)
    p.fork(None, reserve=9)


@pytest.mark.parametrize("n_pages,batch,columns,page_rows", [(5000, 40, 130, 8), (9000, 3, 1500, 8), (4096, 64, 33, 16),
                                                             (20000, 600, 20, 8), (8193, 2, 2, 64), (65536, 30, 400, 8),
                                                             (65537, 300, 40, 8), (80000, 2, 9000, 8), (8192, 4, 2048, 8),
                                                             (33, 1, 32, 8), (65535, 65, 300, 16),
                                                             (9000, 2500, 3, 8), (12000, 3000, 8, 8)])
def test_larger_pools(n_pages, batch, columns, page_rows):
    rnd = random.Random(n_pages)
    most = min(columns * page_rows - 1, (n_pages * page_rows) // (2 * batch))
    lens = [rnd.randint(0, most) for _ in range(batch)]
    p = Pool(start(rnd, lens, n_pages, page_rows, columns), lens, n_pages, page_rows, width=32)
    for step in range(3):
        refs = p.fork([rnd.randint(-1, batch - 1) if rnd.random() < 0.4 else b for b in range(batch)], None, step > 1,
                      reserve=rnd.choice([0, 1, 30]))
        p.compact(refs, step > 1)


def test_pool_with_a_stride():
    rnd = random.Random(3)
    lens = [50, 21, 33]
    table = start(rnd, lens, 30, 16, 6)
    p = Pool(table, lens, 30, 16)
    wide = torch.zeros(30, 2, 16, 416, dtype=torch.uint8, device="cuda")
    wide[:, 1] = p.pages
    p.pages = wide[:, 1]
    refs = p.fork([1, 1, 0], reserve=4)
    p.compact(refs)
    assert bool((wide[:, 0] == 0).all())
    with pytest.raises(ValueError, match="contiguous"):
        mla.pages_fork_make_args(wide[:, :, 0], p.table, p.d_pos, p.refs, missing=p.count)


def test_captured_fork_and_compact_go_on():
    """A graph that forks in place and compacts, replayed: each replay goes on from the one before."""
    rnd = random.Random(9)
    lens = [40, 61, 17, 8]
    p = Pool(start(rnd, lens, 64, 8, 12), lens, 64, 8)
    parent, rows = [1, 1, 0, 3], [60, 37, 100, 7]
    tp, tr = torch.tensor(parent, **I32), torch.tensor(rows, **I32)
    used = torch.zeros(1, **I32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.pages_fork(p.pages, p.table, p.d_pos, p.refs, p.scratch, parent=tp, rows=tr, reserve=2, missing=p.count)
        mla.pages_compact(p.pages, p.table, p.refs, p.scratch, used=used)
    for _ in range(4):
        refs, missing, copies = p.model.fork(parent, rows, reserve=2)
        before = p.want.clone()
        for src, dst, n in copies:
            p.want[dst, :n] = before[src, :n]
        refs, live, moves = p.model.compact(refs)
        for src, dst in moves:
            p.want[dst] = p.want[src]
        graph.replay()
        p.same(refs, missing)
        assert used.tolist() == [live]


def test_a_serving_loop():
    """Requests that fork, grow, end and are compacted give what the same rows give without any of it."""
    B, H, ps, columns, n_pages = 4, 16, 16, 12, 60
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = random.Random(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    rope = mla.rope_table(64, base=10000.0)
    pages = mla.paged_alloc(n_pages, ps)
    table, d_pos = torch.full((B, columns), -1, **I32), torch.zeros(B, **I32)
    refs, count = torch.zeros(n_pages, **I32), torch.zeros(1, **I32)
    scratch = mla.pages_alloc_scratch(pages, table)
    norms = dict(c_norm=randn(512) * 0.1 + 1, k_norm=randn(64) * 0.1 + 1, q_norm=randn(64) * 0.1 + 1)
    plan = mla.paged_plan(batch=B, tokens=20, heads=H, scale=576 ** -0.5, pdl=True)
    attend = mla.paged_alloc_scratch(plan)
    history = [[] for _ in range(B)]                       # (c, k_rope) of every row, per request
    for step in range(9):
        n = 20 if step == 0 else rnd.choice([1, 2, 5])
        parent = [b if rnd.random() < 0.6 else rnd.randrange(B) for b in range(B)]
        keep = [max(0, len(history[p]) - rnd.choice([0, 0, 1, 17])) for p in parent]
        history = [history[p][:k] for p, k in zip(parent, keep)]
        mla.pages_fork(pages, table, d_pos, refs, scratch, parent=torch.tensor(parent, **I32),
                       rows=torch.tensor(keep, **I32), reserve=n, missing=count)
        assert int(count) == 0 and d_pos.tolist() == keep
        if step % 3 == 2:
            mla.pages_compact(pages, table, refs, scratch, used=count)
            assert sorted(set(table.flatten().tolist()) - {-1}) == list(range(int(count)))
        q, q_proj, c, k = torch.zeros(B, 20, H, 576, device="cuda", dtype=torch.bfloat16), randn(B, 20, H, 64), randn(B, 20, 512), randn(B, 20, 64)
        q[..., :512] = randn(B, 20, H, 512)
        pos = d_pos[:, None] + torch.arange(20, **I32)
        n_tok = torch.full((B,), n, **I32)
        mla.paged_append(rope, pos, q_rope=q_proj, q=q, c=c, k_rope=k, pages=pages, page_table=table, d_pos=d_pos,
                         n_tokens=n_tok, **norms)
        out, lse = torch.zeros(B, 20, H, 512, device="cuda"), torch.zeros(B, 20, H, device="cuda")
        window, sink = (0, 0) if step % 2 else (24, 3)
        mla.paged_forward(plan, q, pages, table, out, lse, attend, d_pos=d_pos, n_tokens=n_tok, window=window, sink=sink)
        for b in range(B):
            history[b] = history[b] + [(c[b, i], k[b, i]) for i in range(n)]
        # the same rows in pages of their own, written in one go
        longest = max(map(len, history))
        flat = mla.paged_alloc(B * columns, ps)
        ft = torch.arange(B * columns, **I32).view(B, columns)
        fc, fk = (torch.zeros(B, longest, w, device="cuda", dtype=torch.bfloat16) for w in (512, 64))
        for b in range(B):
            for t, (x, y) in enumerate(history[b]):
                fc[b, t], fk[b, t] = x, y
        zero, lens = torch.zeros(B, **I32), torch.tensor([len(h) for h in history], **I32)
        mla.paged_append(rope, torch.arange(longest, **I32).expand(B, longest).contiguous(), c=fc, k_rope=fk, pages=flat,
                         page_table=ft, d_pos=zero, n_tokens=lens, c_norm=norms["c_norm"], k_norm=norms["k_norm"])
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        mla.paged_forward(plan, q, flat, ft, out2, lse2, attend, d_pos=d_pos, n_tokens=n_tok, window=window, sink=sink)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        rows, rows2 = (torch.zeros(B, longest, 576, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        mla.paged_read(rows, pages, table, n_rows=lens)
        mla.paged_read(rows2, flat, ft, n_rows=lens)
        assert torch.equal(rows, rows2)
        d_pos = d_pos + n
