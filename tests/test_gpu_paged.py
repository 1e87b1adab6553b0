"""The paged 4-bit cache on the GPU: its rows written and read back, and the
attention over them, against plain 64-bit forms."""
import math
import random

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _paged_ref as ref

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
NAN_ROW = 0xff                        # as a scale and in the key values: NaN


def random_pages(n_pages, page_rows, g, kv_scale=1.0, spread=1.0):
    """Pages of normal values, quantised by the reference."""
    raw = torch.zeros(n_pages * page_rows, 416, dtype=torch.uint8)
    c = torch.randn(n_pages * page_rows, 512, generator=g, dtype=torch.float64) * spread
    code, scale = ref.quantise(c, kv_scale)
    raw[:, :256] = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    raw[:, 256:288] = scale.float().to(torch.float8_e4m3fn).view(torch.uint8)
    raw[:, 288:] = torch.randn(n_pages * page_rows, 64, generator=g).bfloat16().view(torch.uint8)
    return raw.view(n_pages, page_rows, 416)


# heads, and SMs to plan for (0: all): few query rows and little work are one kernel's, 48 heads on two SMs the other's
BOTH = pytest.mark.parametrize("H,sms", [(16, 0), (48, 0), (48, 2)])
SMS = pytest.mark.parametrize("sms", [0, 2, 8])


class Case:
    """Requests over pages in random order; everything that no token attends is NaN."""

    def __init__(self, d_pos, Q=1, H=16, page_rows=16, n_tokens=None, window=0, sink=0, kv_scale=1.0, seed=0, gone=(),
                 fp32=False, spare=2, scale=576 ** -0.5, gain=1.0, sms=0):
        g = torch.Generator().manual_seed(seed)
        rnd = random.Random(seed)
        B = len(d_pos)
        self.d_pos, self.n_tokens, self.window, self.sink = d_pos, n_tokens or [Q] * B, window, sink
        self.kv_scale, self.scale, self.fp32, self.sms = kv_scale, scale, fp32, sms
        need = [-(-(max(d, -1) + Q) // page_rows) for d in d_pos]
        n_pages = sum(need) + spare
        order = list(range(n_pages))
        rnd.shuffle(order)
        columns = max(max(need), 1) + 1
        self.table = [[order.pop() for _ in range(k)] + [rnd.choice([-1, 0, n_pages, 1 << 30])] * (columns - k) for k in need]
        for b, c in gone:
            self.table[b][c] = rnd.choice([-1, -5, n_pages, 2 ** 31 - 1])
        self.pages = torch.full((n_pages, page_rows, 416), NAN_ROW, dtype=torch.uint8)
        good = random_pages(n_pages, page_rows, g, kv_scale)
        for b, d in enumerate(d_pos):
            for i in range(self.n_tokens[b]):
                at, _ = ref.rows_of(self.table, b, page_rows, ref.seen(d + i, window, sink) if d >= 0 else [], n_pages)
                if at:
                    x = torch.tensor(at)
                    self.pages[x[:, 0], x[:, 1]] = good[x[:, 0], x[:, 1]]
        self.q = (torch.randn(B, Q, H, 576, generator=g) * gain).bfloat16()

    def expected(self, device="cpu"):
        return ref.attention(self.q.to(device), self.pages.to(device), self.table, d_pos=self.d_pos,
                             n_tokens=self.n_tokens, scale=self.scale, window=self.window, sink=self.sink,
                             kv_scale=self.kv_scale, out_half=ref.F32 if self.fp32 else ref.BF16)

    def on_gpu(self):
        B, Q, H, _ = self.q.shape
        self.t_pages, self.t_table = self.pages.cuda(), torch.tensor(self.table, **I32)
        self.t_q, self.t_d, self.t_n = self.q.cuda(), torch.tensor(self.d_pos, **I32), torch.tensor(self.n_tokens, **I32)
        self.out = torch.full((B, Q, H, 512), 7.0, device="cuda", dtype=torch.float32 if self.fp32 else torch.bfloat16)
        self.lse = torch.full((B, Q, H), 7.0, device="cuda")
        return self

    def forward(self, pdl=False, plan=None, scratch=None, **kw):
        B, Q, H, _ = self.q.shape
        plan = plan or mla.paged_plan(batch=B, tokens=Q, heads=H, scale=self.scale, num_sms=self.sms, pdl=pdl)
        scratch = mla.paged_alloc_scratch(plan) if scratch is None else scratch
        mla.paged_forward(plan, self.t_q, self.t_pages, self.t_table, self.out, self.lse, scratch, d_pos=self.t_d,
                          n_tokens=self.t_n, window=self.window, sink=self.sink, kv_scale=self.kv_scale, **kw)
        return plan, scratch

    def check(self, expected=None, device="cpu"):
        torch.cuda.synchronize()
        out, lse = self.out.to(device).double(), self.lse.to(device).double()
        B, Q = out.shape[:2]
        expected = expected or self.expected(device)
        for b in range(B):
            for i in range(Q):
                if (b, i) not in expected:
                    assert bool((out[b, i] == 7).all()) and bool((lse[b, i] == 7).all()), f"{b, i}: written"
                    continue
                o, l, tol_o, tol_l = expected[b, i]
                none = l == -math.inf
                assert torch.equal(lse[b, i] == -math.inf, none), f"{b, i}: rows attended"
                assert bool((out[b, i][none] == 0).all())
                err_o, err_l = (out[b, i] - o).abs(), (lse[b, i] - l).abs()
                assert bool((err_o <= tol_o).all()), f"{b, i}: out off by {float((err_o / tol_o.clamp(min=1e-30)).max()):.3g} bounds"
                assert bool((err_l[~none] <= tol_l[~none]).all()), f"{b, i}: lse off by {float(err_l[~none].max()):.3g}"


@pytest.mark.parametrize("kw", [
    dict(d_pos=[0]), dict(d_pos=[1], H=1), dict(d_pos=[6], page_rows=8, H=128), dict(d_pos=[126]), dict(d_pos=[127]),
    dict(d_pos=[128], H=7), dict(d_pos=[255], page_rows=128), dict(d_pos=[256], page_rows=1024), dict(d_pos=[700], H=128),
    dict(d_pos=[1500, 3, 640], H=16, page_rows=64), dict(d_pos=[0], Q=64, H=3), dict(d_pos=[90], Q=64, H=128, page_rows=32),
    dict(d_pos=[200, 31, 0, 77], Q=5, H=40, n_tokens=[5, 0, 1, 3]), dict(d_pos=[-1, 30, -7], Q=2),
    dict(d_pos=[300, 301], Q=3, H=128, n_tokens=[1, 3], page_rows=128, kv_scale=0.25),
    dict(d_pos=[500], Q=4, kv_scale=8.0, page_rows=8), dict(d_pos=[1023, 1024, 1025], Q=1, H=64, page_rows=1024),
    dict(d_pos=[10, 20, 30, 40, 50, 60, 70], Q=7, H=20, n_tokens=[1, 2, 3, 4, 5, 6, 7], page_rows=8),
    dict(d_pos=[2500], Q=2, H=32), dict(d_pos=[64, 63], Q=1, H=17, page_rows=64),
], ids=str)
@pytest.mark.parametrize("fp32", [False, True])
@SMS
def test_attention(kw, fp32, sms):
    c = Case(**kw, fp32=fp32, sms=sms).on_gpu()
    plan, scratch = c.forward()
    c.check()
    assert mla.status_word(plan, scratch) == 0


@pytest.mark.parametrize("kw", [
    dict(d_pos=[300], window=1), dict(d_pos=[300], window=1, sink=1), dict(d_pos=[300], window=128, sink=4, H=128),
    dict(d_pos=[1000, 5, 129], Q=3, window=100, sink=130, page_rows=64), dict(d_pos=[1000], window=5000, sink=3),
    dict(d_pos=[1000], window=1000, sink=999), dict(d_pos=[1000], Q=4, window=2, sink=0, H=5),
    dict(d_pos=[2000, 700, 0, -1, 257], Q=9, H=24, window=257, sink=70, n_tokens=[9, 4, 2, 9, 0]),
    dict(d_pos=[640], Q=64, H=16, window=30, sink=1, page_rows=128), dict(d_pos=[1279], window=256, sink=128, page_rows=128),
    dict(d_pos=[3000], window=2 ** 31 - 1, sink=2 ** 31 - 1), dict(d_pos=[500], window=3, sink=2 ** 31 - 1),
], ids=str)
@BOTH
def test_window(kw, H, sms):
    c = Case(**{"H": H, **kw}, sms=sms).on_gpu()
    c.forward()
    c.check()


@pytest.mark.parametrize("kw", [
    dict(d_pos=[300], gone=[(0, 3)]), dict(d_pos=[300], gone=[(0, k) for k in range(19)]),
    dict(d_pos=[500, 260], Q=2, H=128, gone=[(0, 0), (0, 31), (1, 8), (1, 9)]),
    dict(d_pos=[400], window=50, sink=20, gone=[(0, 1), (0, 24)]),
    dict(d_pos=[256 + 127], page_rows=128, gone=[(0, 1)]),
], ids=str)
@BOTH
def test_rows_without_pages(kw, H, sms):
    c = Case(**{"H": H, **kw}, sms=sms).on_gpu()
    c.forward()
    c.check()


@BOTH
def test_rows_behind_the_table(H, sms):
    c = Case([47], H=H, page_rows=16, sms=sms)
    c.table[0][3] = -1                # rows 48 .. 63 have no page, and the table ends there
    want = c.expected()
    c.d_pos = [1000]
    c.on_gpu()
    c.forward()
    c.check(want)


@pytest.mark.parametrize("what", ["scale", "key"])
@BOTH
def test_nan_in_an_attended_row(what, H, sms):
    c = Case([300, 200], Q=2, H=H, sms=sms)
    page, slot = c.table[0][300 // 16], 300 % 16      # the first token's own row
    if what == "scale":
        c.pages[page, slot, 256 + 5] = 0x7f
    else:
        c.pages[page, slot, 288:290] = 0xff
    c.on_gpu()
    c.forward()
    torch.cuda.synchronize()
    assert bool(c.lse[0].isnan().all()) and bool(c.out[0].isnan().all())
    assert bool(c.lse[1].isfinite().all()) and bool(c.out[1].isfinite().all())


@BOTH
def test_nan_queries_stay_in_their_rows(H, sms):
    c = Case([300], Q=2, H=H, sms=sms)
    c.q[0, 0, 3, 17] = math.nan
    c.q[0, 1, 5, 570] = math.inf
    want = c.expected()
    c.on_gpu()
    c.forward()
    torch.cuda.synchronize()
    for i, h in ((0, 3), (1, 5)):
        assert bool(c.lse[0, i, h].isnan()) or bool(c.lse[0, i, h] == math.inf)
    for (_, i), (o, l, tol_o, tol_l) in want.items():
        ok = torch.tensor([(i, h) not in ((0, 3), (1, 5)) for h in range(H)])
        assert bool(((c.out[0, i].cpu().double() - o).abs() <= tol_o)[ok].all())


@pytest.mark.parametrize("gain", [1e-30, 1e-4, 300.0, 1e30])
@BOTH
def test_queries_of_any_size(gain, H, sms):
    """A query's size times the scale is what counts: far from f16's range, the same result."""
    c = Case([400], Q=2, H=H, sms=sms, gain=gain, scale=576 ** -0.5 / gain * 1.0)
    if not c.scale < 2.0 ** 60:
        c.scale = 2.0 ** 59
    c.on_gpu()
    c.forward()
    c.check()


@BOTH
def test_small_query_values_beside_large_ones(H, sms):
    c = Case([200], Q=1, H=H, sms=sms)
    c.q[..., 0] *= 2.0 ** 20          # the others still count, exactly
    c.scale = 2.0 ** -22
    c.on_gpu()
    c.forward()
    c.check()


@BOTH
def test_zero_queries_average_the_rows(H, sms):
    c = Case([999], H=H - 13, fp32=True, sms=sms)
    c.q.zero_()
    c.on_gpu()
    c.forward()
    c.check()
    assert float((c.lse - math.log(1000)).abs().max()) <= 4 * ref.F32 * math.log(1000) + 2.0 ** -21


@BOTH
def test_layers_of_one_pool(H, sms):
    """Pages with a stride: one layer of a pool that holds several."""
    c = Case([300, 77], Q=2, H=H, sms=sms, page_rows=32)
    c.on_gpu()
    pool = torch.full((c.pages.shape[0], 3, 32, 416), NAN_ROW, dtype=torch.uint8, device="cuda")
    pool[:, 1] = c.t_pages
    c.t_pages = pool[:, 1]
    c.forward()
    c.check()


@BOTH
def test_shared_pages(H, sms):
    """Two requests over the same pages, and one that goes on alone behind them."""
    c = Case([95, 95, 40], Q=2, H=H, sms=sms, page_rows=16)
    for k in range(4):
        c.table[1][k] = c.table[0][k]
    c.pages = torch.where((c.pages == NAN_ROW).all(-1, keepdim=True), torch.zeros(1, dtype=torch.uint8), c.pages)
    c.on_gpu()
    c.forward()
    c.check()


@pytest.mark.parametrize("kw", [
    dict(d_pos=[20000], H=16, page_rows=64), dict(d_pos=[9000, 12000], Q=2, H=128, page_rows=128),
    dict(d_pos=[16000], Q=16, H=128, page_rows=64, fp32=True), dict(d_pos=[30000, 100], Q=3, H=16, window=8000, sink=500),
    dict(d_pos=[13 * (b % 41) for b in range(300)], Q=1, H=16, page_rows=32),
    dict(d_pos=[1000 + 7 * b for b in range(40)], Q=2, H=128, page_rows=64),
    dict(d_pos=[4095] * 8, Q=5, H=128, page_rows=64),
], ids=lambda kw: str({k: v if k != "d_pos" else (len(v), max(v)) for k, v in kw.items()}))
def test_long_and_many(kw):
    c = Case(**kw).on_gpu()
    plan, scratch = c.forward(pdl=True)
    c.check(device="cuda")
    assert mla.status_word(plan, scratch) == 0
    out, lse = c.out.clone(), c.lse.clone()
    c.forward(plan=plan, scratch=scratch)
    c.forward(pdl=False)
    torch.cuda.synchronize()
    assert torch.equal(c.lse, lse) and torch.equal(c.out, out)


@BOTH
def test_pages_past_four_gigabytes(H, sms):
    page_rows, n_pages = 1024, 11000  # 4.7 GB
    c = Case([2500], Q=2, H=H, sms=sms, page_rows=page_rows, spare=0)
    pages = torch.zeros(n_pages, page_rows, 416, dtype=torch.uint8, device="cuda")
    to = {p: n_pages - 1 - 40 * k for k, p in enumerate(c.table[0][:3])}
    for p, far in to.items():
        pages[far] = c.pages[p].cuda()
    want = c.expected()
    c.table = [[to.get(p, -1) for p in c.table[0]]]
    c.on_gpu()
    c.t_pages = pages
    c.forward()
    c.check(want)


@BOTH
def test_replayed_graph_follows_lengths_and_tables(H, sms):
    a, b = Case([300, 40], Q=2, H=H, seed=1), Case([123, 290], Q=2, H=H, seed=2)
    a.on_gpu()
    b.on_gpu()
    n = max(a.pages.shape[0], b.pages.shape[0])
    columns = max(a.t_table.shape[1], b.t_table.shape[1])
    pages = torch.zeros(n, 16, 416, dtype=torch.uint8, device="cuda")
    table, d, q = torch.full((2, columns), -1, **I32), torch.zeros(2, **I32), torch.zeros_like(a.t_q)
    out, lse = torch.zeros_like(a.out), torch.zeros_like(a.lse)
    plan = mla.paged_plan(batch=2, tokens=2, heads=H, scale=a.scale, num_sms=sms, pdl=True)
    scratch = mla.paged_alloc_scratch(plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.paged_forward(plan, q, pages, table, out, lse, scratch, d_pos=d)
    for c in (a, b, a):
        pages[:c.pages.shape[0]].copy_(c.t_pages)
        table.fill_(-1)
        table[:, :c.t_table.shape[1]].copy_(c.t_table)
        d.copy_(c.t_d)
        q.copy_(c.t_q)
        graph.replay()
        torch.cuda.synchronize()
        c.out.copy_(out)
        c.lse.copy_(lse)
        c.check()


def test_two_streams_with_scratch_of_their_own():
    a, b = Case([3000], Q=2, H=128, seed=1).on_gpu(), Case([2000, 100], Q=1, H=16, seed=2).on_gpu()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    held = []
    for _ in range(3):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                held.append(c.forward())
    a.check()
    b.check()


@BOTH
def test_a_wait_that_runs_out_is_reported(H, sms):
    c = Case([300], H=H, sms=sms).on_gpu()
    plan = mla.paged_plan(batch=1, tokens=1, heads=H, scale=c.scale, num_sms=sms, stall_test=True)
    _, scratch = c.forward(plan=plan)
    torch.cuda.synchronize()
    assert mla.status_word(plan, scratch) == mla.EDEVICE
    c.forward()
    c.check()


def test_arguments_of_another_shape_are_refused():
    c = Case([30], H=16).on_gpu()
    plan = mla.paged_plan(batch=1, tokens=1, heads=32, scale=1.0)
    scratch = mla.paged_alloc_scratch(plan)
    with pytest.raises(ValueError, match="plan"):
        mla.paged_forward(plan, c.t_q, c.t_pages, c.t_table, c.out, c.lse, scratch, d_pos=c.t_d)
    with pytest.raises(ValueError, match="contiguous"):
        mla.paged_make_args(c.t_q, c.t_pages.permute(1, 0, 2), c.t_table, c.out, c.lse, d_pos=c.t_d)
    with pytest.raises(ValueError, match="416"):
        mla.paged_make_args(c.t_q, c.t_pages[..., :400].contiguous(), c.t_table, c.out, c.lse, d_pos=c.t_d)
    with pytest.raises(mla.MLADecodeError):
        a = mla.paged_make_args(c.t_q, c.t_pages, c.t_table, c.out, c.lse, d_pos=c.t_d, kv_scale=0.3)
        mla.paged_forward_args(mla.paged_plan(batch=1, tokens=1, heads=16, scale=1.0), a, scratch)


# ---- rows written and read back ---------------------------------------------------
def inv_freq(rot):
    return [10000.0 ** (-2 * j / rot) for j in range(rot // 2)]


class Append:
    def __init__(self, d_pos, N=3, H=4, page_rows=16, n_tokens=None, norms=True, kv_scale=1.0, interleaved=True, rot=64,
                 seed=0, amplitude=1.0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        rnd = random.Random(seed)
        B = len(d_pos)
        self.__dict__.update(d_pos=d_pos, N=N, H=H, n_tokens=n_tokens or [N] * B, kv_scale=kv_scale, rot=rot, eps=1e-5,
                             interleaved=interleaved, page_rows=page_rows, amplitude=amplitude)
        need = [-(-(max(d, -1) + N) // page_rows) for d in d_pos]
        self.n_pages = sum(need) + 2
        order = list(range(self.n_pages))
        rnd.shuffle(order)
        columns = max(max(need), 1)
        self.table = [[order.pop() for _ in range(k)] + [-1] * (columns - k) for k in need]
        self.q_proj = torch.randn(B, N, H, 192, generator=g).bfloat16()
        self.kv_proj = (torch.randn(B, N, 576, generator=g) * spread).bfloat16()
        self.w = [(1 + 0.3 * torch.randn(n, generator=g)).bfloat16() if norms else None for n in (512, 64, 64)]
        self.positions = torch.tensor([[max(d, 0) + i for i in range(N)] for d in d_pos], dtype=torch.int32)
        self.pages = torch.randint(0, 255, (self.n_pages, page_rows, 416), generator=g, dtype=torch.uint8)

    def run(self):
        B, N, H = len(self.d_pos), self.N, self.H
        table = mla.rope_table(self.rot, base=10000.0, interleaved=self.interleaved, amplitude=self.amplitude)
        qp, kp = self.q_proj.cuda(), self.kv_proj.cuda()
        w = [x if x is None else x.cuda() for x in self.w]
        self.t_q = torch.full((B, N, H, 576), 3.0, device="cuda", dtype=torch.bfloat16)
        self.t_pages, self.t_table = self.pages.cuda(), torch.tensor(self.table, **I32)
        mla.paged_append(table, self.positions.cuda(), q_rope=qp[..., 128:], q=self.t_q, c=kp[..., :512],
                         k_rope=kp[..., 512:], pages=self.t_pages, page_table=self.t_table,
                         d_pos=torch.tensor(self.d_pos, **I32), n_tokens=torch.tensor(self.n_tokens, **I32), c_norm=w[0],
                         k_norm=w[1], q_norm=w[2], eps=self.eps, kv_scale=self.kv_scale)
        return self

    def check(self):
        q, pages = self.t_q.cpu(), self.t_pages.cpu()
        assert bool((q[..., :512] == 3).all())
        want_pages, written = self.pages.clone(), torch.zeros(self.n_pages, self.page_rows, dtype=torch.bool)
        f = inv_freq(self.rot)
        x = ref.rotate(ref.norm(self.q_proj[..., 128:], self.w[2], self.eps), self.positions[..., None], f,
                       self.interleaved, self.rot, self.amplitude)
        k = ref.rotate(ref.norm(self.kv_proj[..., 512:], self.w[1], self.eps), self.positions, f, self.interleaved,
                       self.rot, self.amplitude)
        c = ref.norm(self.kv_proj[..., :512], self.w[0], self.eps)
        for b, d in enumerate(self.d_pos):
            for i in range(self.N):
                if i >= self.n_tokens[b]:
                    assert bool((q[b, i, :, 512:] == 3).all())
                    continue
                # one rounding to bf16; products and the norm in fp32 (80 steps: a sum of 64 squares, and the rest)
                err = (q[b, i, :, 512:].double() - x[b, i]).abs()
                assert bool((err <= ref.BF16 * x[b, i].abs() + 80 * ref.F32 * x[b, i].abs().amax(-1, keepdim=True)).all())
                at, _ = ref.rows_of(self.table, b, self.page_rows, [d + i] if d >= 0 else [], self.n_pages)
                if not at:
                    continue
                page, slot = at[0]
                written[page, slot] = True
                row = pages[page, slot]
                err = (row[288:].view(torch.bfloat16).double() - k[b, i]).abs()
                assert bool((err <= ref.BF16 * k[b, i].abs() + 80 * ref.F32 * k[b, i].abs().amax()).all())
                code, scale = ref.quantise(c[b, i][None], self.kv_scale)
                got_scale = row[256:288].view(torch.float8_e4m3fn).double()
                got_code = torch.stack([row[:256] & 15, row[:256] >> 4], -1).flatten().long()
                # the same codes, but where the exact value lies within four fp32 steps of a border
                top = c[b, i].view(32, 16).abs().amax(-1) / 6 / self.kv_scale
                near = lambda v, border: (v / border - 1).abs() <= 5 * ref.F32  # noqa: E731
                low, high = torch.minimum(got_scale, scale[0]), torch.maximum(got_scale, scale[0])
                assert bool(((got_scale == scale[0]) | near(top, (low + high) / 2)).all())
                unit = torch.where(got_scale > 0, c[b, i].view(32, 16).T / (got_scale * self.kv_scale), 0).T.flatten()
                want = (unit.abs()[:, None] - ref.E2M1[:8]).abs().amin(-1)
                gap = (unit - ref.E2M1[got_code]).abs()
                assert bool((gap <= want + 5 * ref.F32 * unit.abs()).all())
        assert torch.equal(pages[~written], want_pages[~written])


@pytest.mark.parametrize("kw", [
    dict(d_pos=[0], N=1, H=1), dict(d_pos=[15, 16, 17]), dict(d_pos=[100, 3, -1], N=5, n_tokens=[5, 0, 3]),
    dict(d_pos=[7, 1000], N=40, H=128, page_rows=64, n_tokens=[33, 40]), dict(d_pos=[5], N=9, norms=False, interleaved=False),
    dict(d_pos=[63], N=2, H=33, kv_scale=0.125, interleaved=False, rot=48, page_rows=8),
    dict(d_pos=[0], N=300, H=2, kv_scale=4.0, rot=16, amplitude=1.25), dict(d_pos=[12], N=4, spread=1e-6, norms=False),
    dict(d_pos=[12], N=4, spread=1e5, norms=False), dict(d_pos=[3], N=130, spread=1e12, page_rows=1024),
    dict(d_pos=[3], N=20, spread=1e-12), dict(d_pos=[250000], N=2, page_rows=1024),
], ids=str)
def test_append(kw):
    Append(**kw).run().check()


def test_append_gives_the_same_bits_as_the_formula_in_its_own_roundings():
    """Beside a border every rounding counts: scales and codes are those of the documented fp32 steps."""
    a = Append([0], N=2000, H=1, page_rows=64, seed=5)
    a.run()
    x = a.kv_proj[0, :, :512].float()
    rstd = (1 / (x.double().square().mean(-1, keepdim=True) + torch.tensor(a.eps, dtype=torch.float32).double()).sqrt()).float()
    y = (x * rstd * a.w[0].float()).view(-1, 32, 16)
    scale = (y.abs().amax(-1) * torch.tensor(1 / 6)).clamp(max=448).to(torch.float8_e4m3fn)
    unit = y * (1.0 / scale.float())[..., None]
    dist = (unit.abs().double()[..., None] - ref.E2M1[:8]).abs()
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7])
    code = torch.where(dist == dist.amin(-1, keepdim=True), order, 99).argmin(-1) + 8 * torch.signbit(unit).long()
    code = code.flatten(-2)
    at = torch.tensor([[a.table[0][t // 64], t % 64] for t in range(2000)])
    rows = a.t_pages.cpu()[at[:, 0], at[:, 1]]
    same = (rows[:, :256] == (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)) & (
        (rows[:, 256:288] == scale.view(torch.uint8)).repeat_interleave(8, 1))
    # (rstd is the nearest fp32 number but for about one row in 2^20)
    assert bool(same.all())


def test_append_of_blocks_that_are_zero_nan_or_infinite():
    a = Append([0], N=4, H=1, norms=False)
    a.kv_proj[0, 0, 32:48] = 0
    a.kv_proj[0, 1, 5] = math.nan
    a.kv_proj[0, 2, 5] = math.inf
    a.kv_proj[0, 3, :16] = 1e-30
    a.run()
    rows = a.t_pages.cpu()[[a.table[0][0]] * 4, range(4)]
    v = ref.row_values(rows, 1.0)
    assert bool((v[0, 32:48] == 0).all()) and bool(v[1, :16].isnan().all()) and bool(v[1, 16:512].isfinite().all())
    assert v[2, 5] == 6 * 448 and bool((v[3, :16] == 0).all())
    b = Append([0], N=2, H=1)
    b.kv_proj[0, 0, 5] = math.nan
    b.kv_proj[0, 1, 512 + 3] = math.nan
    b.run()
    v = ref.row_values(b.t_pages.cpu()[[b.table[0][0]] * 2, range(2)], 1.0)
    assert bool(v[0, :512].isnan().all()) and bool(v[0, 512:].isfinite().all())
    assert bool(v[1, :512].isfinite().all()) and bool(v[1, 512:].isnan().all())


def test_append_without_pages_writes_nothing():
    a = Append([16, 5], N=3, H=2)
    a.table[0] = [-1, a.n_pages] + a.table[0][2:]
    a.run()
    a.check()
    a = Append([10], N=3, H=2, page_rows=8)
    a.d_pos = [2 ** 31 - 2]           # past the table, and past 32 bits
    a.run()
    assert torch.equal(a.t_pages.cpu(), a.pages)


def test_parts_alone():
    a = Append([20, 7], N=3, H=5)
    a.run()
    table = mla.rope_table(64, base=10000.0)
    q = torch.full_like(a.t_q, 3.0)
    w = [x.cuda() for x in a.w]
    pos, n, d = a.positions.cuda(), torch.tensor(a.n_tokens, **I32), torch.tensor(a.d_pos, **I32)
    mla.paged_append(table, pos, q_rope=a.q_proj.cuda()[..., 128:], q=q, q_norm=w[2], eps=a.eps, n_tokens=n)
    pages, kp = a.pages.cuda(), a.kv_proj.cuda()
    mla.paged_append(table, pos, c=kp[..., :512], k_rope=kp[..., 512:], pages=pages, page_table=a.t_table, d_pos=d,
                     c_norm=w[0], k_norm=w[1], eps=a.eps, n_tokens=n)
    assert torch.equal(q, a.t_q) and torch.equal(pages, a.t_pages)
    in_place = a.q_proj.cuda()[..., 128:].contiguous()
    wide = torch.zeros(2, 3, 5, 576, device="cuda", dtype=torch.bfloat16)
    wide[..., 512:] = in_place
    mla.paged_append(table, pos, q_rope=wide[..., 512:], q=wide, q_norm=w[2], eps=a.eps)
    assert torch.equal(wide[..., 512:], a.t_q[..., 512:])
    for bad in (dict(c=kp[..., :512]), dict(c_norm=w[0]), dict(q_rope=in_place), dict(q_norm=w[2])):
        with pytest.raises(ValueError):
            mla.paged_append(table, pos, **bad)


@pytest.mark.parametrize("page_rows,kv_scale", [(8, 1.0), (64, 0.25), (1024, 2.0 ** 20)])
def test_read(page_rows, kv_scale):
    g = torch.Generator().manual_seed(page_rows)
    n_pages = 30 if page_rows < 1024 else 5
    pages = random_pages(n_pages, page_rows, g, kv_scale, spread=kv_scale)
    pages[0, 0, 256] = 0x7f                            # a NaN scale
    table = [[3, 0, -1, 2], [1, n_pages, 4, 4]]
    first, n_rows = [page_rows - 3, 2 * page_rows + 1], [2 * page_rows + 7, 9]
    N = 2 * page_rows + 8
    buf = torch.full((2, N, 600), 5.0, device="cuda", dtype=torch.bfloat16)
    out = buf[..., :576]
    mla.paged_read(out, pages.cuda(), torch.tensor(table, **I32), first=torch.tensor(first, **I32),
                   n_rows=torch.tensor(n_rows, **I32), kv_scale=kv_scale)
    got = buf.cpu()
    assert bool((got[..., 576:] == 5).all())
    for b in range(2):
        assert bool((got[b, n_rows[b]:] == 5).all())
        for i in range(n_rows[b]):
            at, _ = ref.rows_of(table, b, page_rows, [first[b] + i], n_pages)
            want = ref.row_values(pages[at[0][0], at[0][1]][None], kv_scale)[0] if at else torch.zeros(576).double()
            assert torch.equal(got[b, i, :576].double().nan_to_num(nan=99.0), want.nan_to_num(nan=99.0))
    whole = torch.zeros(2, 4, 576, device="cuda", dtype=torch.bfloat16)
    mla.paged_read(whole, pages.cuda(), torch.tensor(table, **I32), kv_scale=kv_scale)
    assert torch.equal(whole[0, 1].cpu().double(), ref.row_values(pages[3, 1][None], kv_scale)[0])
