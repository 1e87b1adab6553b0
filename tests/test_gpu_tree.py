"""Attention of drafted tokens (mla_tree_forward) and the weights that cache
rows get from it (mla_tree_weights), against the 64-bit forms."""
import math
import random

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(576)
NAN = float("nan")


class Case:
    """Inputs of one call; stale rows around and behind every request hold NaN."""

    def __init__(self, seed, lens, Q, H, n_tokens=None, mask="tree", stride=576, kv_rows=None, gain=1.5, offsets=None):
        g = torch.Generator().manual_seed(seed)
        rnd = random.Random(seed)
        B = len(lens)
        self.B, self.Q, self.H, self.lens = B, Q, H, lens
        self.n = list(n_tokens) if n_tokens is not None else [Q] * B
        self.offs, at = [], 3
        for b in range(B):
            self.offs.append(at)
            at += max(lens[b], 0) + Q + rnd.randint(0, 5)
        if offsets is not None:
            self.offs, at = list(offsets), max(at, max(offsets) + max(lens) + Q)
        rows = at
        kv = torch.full((rows, 576), NAN)
        for b in range(B):
            live = max(lens[b], -1) + self.n[b] if lens[b] >= 0 else 0
            lo, hi = max(self.offs[b], 0), min(self.offs[b] + live, rows)
            if hi > lo:
                kv[lo:hi] = torch.randn(hi - lo, 576, generator=g)
        self.kv = kv.bfloat16()
        self.q = (torch.randn(B, Q, H, 576, generator=g) * gain).bfloat16()
        if mask == "tree":
            self.bits = [ref.masks_of_tree(rnd, Q) for _ in range(B)]
        elif mask == "chain":
            self.bits = [[(2 << i) - 1 for i in range(Q)] for _ in range(B)]
        elif mask == "random":
            self.bits = [[rnd.getrandbits(64) for _ in range(Q)] for _ in range(B)]
        elif mask == "none":
            self.bits = [[0] * Q for _ in range(B)]
        self.mask_given = mask != "chain"
        self.stride, self.kv_rows = stride, kv_rows or rows
        d = "cuda"
        self.d = dict(
            q=self.q.to(d), d_pos=torch.tensor(lens, dtype=torch.int32, device=d),
            row_offset=torch.tensor(self.offs, dtype=torch.int64, device=d),
            n_tokens=torch.tensor(self.n, dtype=torch.int32, device=d),
            mask=torch.tensor([[ref.signed(w) for w in r] for r in self.bits], dtype=torch.int64, device=d)
            if self.mask_given else None)
        wide = torch.full((rows, stride), NAN, dtype=torch.bfloat16, device=d)
        wide[:, :576] = self.kv.to(d)
        self.d["kv"] = wide[:, :576]

    def kw(self):
        return dict(d_pos=self.d["d_pos"], row_offset=self.d["row_offset"], mask=self.d["mask"],
                    n_tokens=self.d["n_tokens"], kv_rows=self.kv_rows)

    def plan(self, **kw):
        return mla.tree_plan(batch=self.B, tokens=self.Q, heads=self.H, scale=SCALE, **kw)

    def outputs(self, dtype=torch.bfloat16):
        return (torch.full((self.B, self.Q, self.H, 512), 7.0, dtype=dtype, device="cuda"),
                torch.full((self.B, self.Q, self.H), 7.0, device="cuda"))

    def run(self, dtype=torch.bfloat16, **plan_kw):
        p = self.plan(**plan_kw)
        scratch = mla.tree_alloc_scratch(p)
        out, lse = self.outputs(dtype)
        mla.tree_forward(p, self.d["q"], self.d["kv"], out, lse, scratch, **self.kw())
        torch.cuda.synchronize()
        assert mla.status_word(p, scratch) == 0
        return out, lse

    def reference(self):
        return ref.tree(self.q, self.kv, d_pos=self.lens, row_offset=self.offs, n_tokens=self.n, bits=self.bits,
                        scale=SCALE, kv_rows=self.kv_rows)

    def check(self, out, lse, want=None):
        o, l = out.double().cpu(), lse.double().cpu()
        want = want or self.reference()
        for b in range(self.B):
            for i in range(self.Q):
                if (b, i) not in want:
                    assert (o[b, i] == 7).all() and (l[b, i] == 7).all(), f"token {(b, i)} is behind the drafts"
                    continue
                ro, rl, to, tl = want[b, i]
                empty = torch.isinf(rl)
                assert torch.equal(torch.isinf(l[b, i]), empty)
                assert ((l[b, i] - rl).abs()[~empty] <= tl[~empty]).all(), (b, i, (l[b, i] - rl).abs().max())
                if out.dtype == torch.bfloat16:
                    to = to + ref.BF16 * (ro.abs() + to)
                err = (o[b, i] - ro).abs()
                assert (err <= to + 1e-30).all(), (b, i, float((err - to).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Q,H", [
    ([0], 1, 1), ([1], 1, 16), ([0], 5, 16), ([63], 1, 16), ([64], 2, 16), ([127], 1, 128), ([128], 4, 32),
    ([120], 8, 16), ([121], 8, 16), ([255], 3, 5), ([300], 7, 48), ([1000], 64, 16), ([513], 64, 128),
    ([2000], 13, 17), ([700, 0, 129, 64, 3], 6, 16), ([200] * 9, 3, 64),
    # query rows that are not a whole number of boxes, in several requests
    ([3000], 1, 16), ([200] * 5, 1, 5), ([300] * 6, 3, 7), ([500, 300], 5, 70), ([90, 400, 7], 12, 33),
])
def test_trees_against_the_64_bit_form(lens, Q, H, dtype):
    c = Case(11 * len(lens) + Q + H, lens, Q, H)
    c.check(*c.run(dtype))


# Runs of 96 tiles and more, on few pairs: a request's row blocks are cut along the
# cache, and their pieces lie in several runs.
@pytest.mark.parametrize("num_sms", [0, 2, 10, 20, 24])
@pytest.mark.parametrize("lens,Q,H", [
    ([50000], 2, 65), ([24000, 0, 9000, 130, 20000], 3, 100), ([13000] * 4, 5, 64), ([49100, 30], 64, 6),
])
def test_long_caches_of_several_row_blocks(lens, Q, H, num_sms):
    c = Case(13 + Q, lens, Q, H, gain=0.5)
    out, lse = c.run(num_sms=num_sms)
    c.check(out, lse, long_reference(c))


def long_reference(c):
    """Case.reference, once per case."""
    key = (tuple(c.lens), c.Q, c.H)
    if key not in LONG:
        LONG[key] = c.reference()
    return LONG[key]


LONG = {}


# Queries of zero weigh all rows alike, and sums of latents of 0 and 1 are exact: a row
# left out or taken twice shows in the mean and in the log of the count.  Bound: the
# merge's weights are within 2^-22, each product and sum of a piece within 2^-24.
@pytest.mark.parametrize("num_sms,lens,Q,H", [
    (0, [1000], 1, 1), (1200, [50000], 1, 5), (1200, [60000], 2, 65), (400, [1300000], 2, 65),
    (2, [20000, 5000], 3, 128), (6, [20000, 5000, 0, 30000], 3, 128), (10, [9000] * 7, 4, 128),
    (14, [12288 + 64 * i for i in range(9)], 2, 128), (0, [30000 + 7777 * i for i in range(12)], 5, 128),
    (0, [300000, 250000], 5, 128), (38, [100, 150000, 37, 60000, 1], 9, 50), (24, [200000], 64, 8),
    # row blocks of one length, a whole number of them per run
    (0, [1000], 64, 128), (0, [4000] * 64, 1, 128), (6, [900] * 5, 2, 128), (0, [500] * 40, 1, 16),
    (0, [500] * 39 + [700], 1, 16), (0, [500, 0, 500, 500], 30, 128), (10, [600] * 12, 3, 128),
    # short ones of several lengths, whole as well
    (0, [357, 567], 45, 128), (0, [300 + 97 * (i % 11) for i in range(100)], 1, 128),
    (0, [20, 0, 900, 4, 130, 1, 400], 40, 64), (0, [(i * 37) % 140 for i in range(70)], 6, 128), (8, [700, 300], 20, 100),
    (0, [(i * 7) % 23 for i in range(4096)], 1, 1),
])
def test_every_row_counts_once(num_sms, lens, Q, H):
    g = torch.Generator(device="cuda").manual_seed(len(lens) + Q)
    offs = [sum(lens[:b]) + b * Q for b in range(len(lens))]
    rows = sum(lens) + len(lens) * Q
    kv = torch.randint(0, 2, (rows, 576), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    B, i32 = len(lens), dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(B, Q, H, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(B, Q, H, 512, device="cuda"), torch.empty(B, Q, H, device="cuda")
    p = mla.tree_plan(batch=B, tokens=Q, heads=H, scale=SCALE, num_sms=num_sms)
    scratch = mla.tree_alloc_scratch(p)
    mla.tree_forward(p, q, kv, out, lse, scratch, d_pos=torch.tensor(lens, **i32),
                     row_offset=torch.tensor(offs, dtype=torch.int64, device="cuda"))
    assert mla.status_word(p, scratch) == 0
    tol = 2.0 ** -21 + 2 * p.grid * 2.0 ** -23
    for b, (o, n) in enumerate(zip(offs, lens)):
        whole = kv[o:o + n, :512].sum(0, dtype=torch.float64)
        for i in range(Q):
            want = (whole + kv[o + n:o + n + i + 1, :512].double().sum(0)) / (n + i + 1)
            assert (out[b, i].double() - want).abs().max() <= tol, (b, i)
            assert (lse[b, i].double() - math.log(n + i + 1)).abs().max() <= 2.0 ** -20 * 8, (b, i)


@pytest.mark.parametrize("mask", ["chain", "random", "none"])
@pytest.mark.parametrize("lens,n", [([0, 40, 0], [4, 9, 0]), ([130, 257, 5], [9, 1, 6])])
def test_masks_chains_empty_rows_and_ragged_drafts(mask, lens, n):
    c = Case(5, lens, 9, 16, n_tokens=n, mask=mask)
    c.check(*c.run())


def test_mask_bit_63_and_bits_behind_the_drafts():
    c = Case(6, [100, 100], 64, 4, n_tokens=[64, 63], mask="random")
    c.check(*c.run())


def test_inactive_requests_attend_nothing():
    c = Case(7, [90, -1, 33], 4, 16)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("kv_rows", [1, 60, 100, 131, 400])
def test_rows_outside_the_cache_are_not_attended(kv_rows):
    c = Case(8, [110], 8, 16)
    c.kv_rows = min(kv_rows, c.kv.shape[0])
    c.check(*c.run())


def test_negative_row_offset_starts_inside_the_request():
    c = Case(9, [150, 20], 4, 16, offsets=[-40, 200])
    c.check(*c.run())


def test_requests_over_the_same_rows():
    # reading only, so requests may share cache rows: one prefix, two of their own lengths
    c = Case(20, [700, 700, 260], 5, 16, offsets=[3, 3, 3])
    c.kv = c.kv.nan_to_num(0.25)
    c.d["kv"].copy_(c.kv)
    c.check(*c.run())


def test_offsets_at_which_no_row_can_lie_inside():
    c = Case(12, [30, 30, 30, 100], 4, 16)
    c.d["d_pos"] = torch.tensor([2**31 - 1, 50, 2**31 - 1, 100], dtype=torch.int32, device="cuda")
    c.d["row_offset"] = torch.tensor([-2**31, 2**62, -2**63, c.offs[3]], dtype=torch.int64, device="cuda")
    out, lse = c.run()
    assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    c.check(out, lse, {**{(b, i): (torch.zeros(16, 512), torch.full((16,), -math.inf), torch.zeros(16, 512),
                                   torch.zeros(16)) for b in range(3) for i in range(4)},
                       **{k: v for k, v in c.reference().items() if k[0] == 3}})
    w = torch.full((c.kv.shape[0],), 5.0, device="cuda")
    p = c.plan()
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, mla.tree_alloc_scratch(p), w, decay=0.0, **c.kw())
    assert (w[:c.offs[3]] == 5).all() and abs(float(w[c.offs[3]:c.offs[3] + 104].sum()) - 64) < 0.1


@pytest.mark.parametrize("stride", [584, 640, 1152])
def test_row_strides(stride):
    c = Case(10, [200, 77], 5, 16, stride=stride)
    c.check(*c.run())


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_non_finite_drafts_reach_only_the_tokens_that_attend_them(bad):
    c = Case(12, [140], 8, 16, mask="none")
    # token i attends itself only, except token 2, which attends draft 5 too; draft 5 is broken
    c.bits = [[1 << i for i in range(8)]]
    c.bits[0][2] |= 1 << 5
    c.d["mask"] = torch.tensor(c.bits, dtype=torch.int64, device="cuda")
    want = c.reference()
    row = c.offs[0] + 140 + 5
    c.d["kv"][row, 100:140] = bad
    if math.isinf(bad):
        c.d["q"][:, :, :, 100:140] = abs(c.d["q"][:, :, :, 100:140])     # the score is +-infinity, not NaN
    c.q = c.d["q"].cpu()
    want = c.reference()
    out, lse = c.run()
    for i in (2, 5):
        if bad != -math.inf:
            assert torch.isnan(out[0, i]).all(), i
        del want[0, i]
    sel = [i for i in range(8) if i not in (2, 5)]
    assert torch.isfinite(out[0, sel]).all() and torch.isfinite(lse[0, sel]).all()
    o, l = out.clone(), lse.clone()
    o[0, [2, 5]], l[0, [2, 5]] = 7, 7
    c.check(o, l, want)


def test_large_scores_and_a_growing_maximum():
    c = Case(13, [900], 4, 16, gain=1.0)
    # scores rise along the cache, so the running maximum moves in every tile
    ramp = torch.linspace(0.05, 30.0, 904)[:, None]
    body = c.kv[3:3 + 904].float() * 0.05
    body[:, :8] = ramp
    c.kv[3:3 + 904] = body.bfloat16()
    c.q[..., :8] = 3.0
    c.d["kv"][3:3 + 904] = c.kv[3:3 + 904].cuda()
    c.d["q"].copy_(c.q)
    c.check(*c.run())


@pytest.mark.parametrize("num_sms", [2, 6, 40, 0])
def test_any_number_of_sms_and_bitwise_repeats(num_sms):
    c = Case(14, [1500, 333, 0, 64], 12, 32)
    out, lse = c.run(num_sms=num_sms)
    c.check(out, lse)
    out2, lse2 = c.run(num_sms=num_sms, pdl=True)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)


def test_one_token_is_the_dense_decode():
    """With one drafted token and mask 1 the result is mla_decode_forward's, within both kernels' bounds."""
    c = Case(15, [777, 40], 1, 16)
    out, lse = c.run(torch.float32)
    p = mla.plan(batch=2, heads=16, max_ctx=778, scale=SCALE)
    o, l = torch.empty(2, 16, 512, device="cuda"), torch.empty(2, 16, device="cuda")
    mla.forward(p, c.d["q"], c.d["kv"], o, l, mla.alloc_scratch(p), d_pos=c.d["d_pos"], row_offset=c.d["row_offset"])
    want = c.reference()
    for b in range(2):
        assert ((out[b, 0] - o[b]).abs().double().cpu() <= 2 * want[b, 0][2]).all()
        assert ((lse[b, 0] - l[b]).abs().double().cpu() <= 2 * want[b, 0][3]).all()


def test_captured_on_a_side_stream_and_replayed_on_new_positions():
    c = Case(16, [400, 90], 8, 16)
    p = c.plan(pdl=True)
    scratch = mla.tree_alloc_scratch(p)
    out, lse = c.outputs()
    args = mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw())
    w = torch.zeros(c.kv.shape[0], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.tree_forward_args(p, args, scratch)
        mla.tree_weights_args(p, args, scratch, w, decay=0.0)
    for lens in ([400, 90], [130, 0], [399, 1]):
        c.lens = lens
        c.d["d_pos"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7), lse.fill_(7)
        # rows that were committed before and are drafts now are finite; nothing else changes
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
        total = sum(float(w[c.offs[b]:c.offs[b] + lens[b] + 8].sum()) for b in range(2))
        assert abs(total - 2 * 8 * 16) <= 1e-3 * 2 * 8 * 16
    assert mla.status_word(p, scratch) == 0


def test_two_calls_at_once_with_their_own_scratch():
    a, b = Case(17, [3000], 16, 16), Case(18, [2500, 10], 8, 32)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for c, s in ((a, s1), (b, s2)):
        p = c.plan(pdl=True)
        out, lse = c.outputs()
        runs.append((p, mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw()), mla.tree_alloc_scratch(p), s,
                     out, lse))
    torch.cuda.synchronize()
    for _ in range(4):
        for p, args, scratch, s, _, _ in runs:
            mla.tree_forward_args(p, args, scratch, stream=s)
    torch.cuda.synchronize()
    a.check(*runs[0][4:])
    b.check(*runs[1][4:])


@pytest.mark.parametrize("decay", [0.0, 0.875, 1.0])
@pytest.mark.parametrize("lens,Q,H,n,mask", [
    ([0], 1, 1, None, "tree"), ([1], 1, 16, None, "tree"), ([127], 1, 16, None, "chain"), ([128], 2, 64, None, "tree"),
    ([129], 2, 128, None, "tree"), ([500], 8, 33, None, "tree"), ([260, 0, -1, 64, 1000], 5, 16, [5, 5, 5, 0, 3], "random"),
    ([100], 64, 16, None, "tree"), ([300], 6, 16, None, "none"), ([100], 64, 1, None, "random"),
    ([70, 9], 30, 7, None, "random"), ([40], 5, 127, None, "tree"), ([500, 300], 5, 70, None, "tree"),
    ([200] * 5, 1, 5, None, "tree"), ([300] * 6, 3, 7, None, "chain"), ([90, 400, 7], 12, 33, [12, 1, 7], "random"),
])
def test_weights_against_the_64_bit_form(lens, Q, H, n, mask, decay):
    c = Case(21 + Q + H, lens, Q, H, n_tokens=n, mask=mask)
    out, lse = c.run()
    g = torch.Generator().manual_seed(3)
    old = torch.rand(c.kv.shape[0], generator=g)
    if decay == 0.0:
        for b in range(c.B):                                # with decay 0 the old values are not read
            if lens[b] >= 0:
                old[c.offs[b]:c.offs[b] + lens[b] + c.n[b]] = NAN
    w = old.cuda()
    p = c.plan()
    scratch = mla.tree_alloc_scratch(p)
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, scratch, w, decay=decay, **c.kw())
    torch.cuda.synchronize()
    assert mla.status_word(p, scratch) == 0
    new, tol = ref.weights(c.q, c.kv, lse.cpu(), old, d_pos=c.lens, row_offset=c.offs, n_tokens=c.n, bits=c.bits,
                           scale=SCALE, decay=decay, kv_rows=c.kv_rows)
    err = (w.double().cpu() - new).abs()
    assert (err <= tol).all(), float((err - tol).max())
    untouched = tol <= 2.0 ** -39
    assert torch.equal(w.cpu()[untouched & (new == old)], old[untouched & (new == old)])
    w2 = old.cuda()
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, scratch, w2, decay=decay, **c.kw())
    assert torch.equal(w, w2)


@pytest.mark.parametrize("bad", [NAN, math.inf])
def test_weights_of_rows_that_nobody_attends(bad):
    """A broken draft that no token attends gets its decayed weight and nothing else changes."""
    c = Case(30, [140], 8, 16, mask="none")
    c.bits = [[1 << i if i != 5 else 1 for i in range(8)]]
    c.d["mask"] = torch.tensor(c.bits, dtype=torch.int64, device="cuda")
    row = c.offs[0] + 145
    c.kv[row, 30:40] = bad
    c.d["kv"][row, 30:40] = bad
    out, lse = c.run()
    c.check(out, lse)
    old = torch.rand(c.kv.shape[0])
    w = old.cuda()
    p = c.plan(num_sms=3)
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, mla.tree_alloc_scratch(p), w, decay=0.5, **c.kw())
    new, tol = ref.weights(c.q, c.kv, lse.cpu(), old, d_pos=c.lens, row_offset=c.offs, n_tokens=c.n, bits=c.bits,
                           scale=SCALE, decay=0.5)
    assert ((w.double().cpu() - new).abs() <= tol).all()
    assert float(w[row]) == 0.5 * float(old[row])


def test_long_cache_weights_sum_to_the_tokens_and_heads():
    c = Case(31, [20000], 3, 128)
    out, lse = c.run()
    p = c.plan()
    w = torch.zeros(c.kv.shape[0], device="cuda")
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, mla.tree_alloc_scratch(p), w, **c.kw())
    assert abs(float(w.double().sum()) - 3 * 128) <= 3 * 128 * 1e-4
    c.check(out, lse)


@pytest.mark.parametrize("num_sms", [0, 10])
def test_many_requests_of_all_lengths(num_sms):
    rnd = random.Random(4)
    lens = [rnd.choice([-1, 0, 1, 63, 127, 128, 129, 200, 300]) for _ in range(70)]
    n = [rnd.randint(0, 3) for _ in range(70)]
    c = Case(40, lens, 3, 16, n_tokens=n)
    out, lse = c.run(num_sms=num_sms)
    c.check(out, lse)
    old = torch.rand(c.kv.shape[0])
    w = old.cuda()
    p = c.plan(num_sms=num_sms)
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, mla.tree_alloc_scratch(p), w, decay=0.25, **c.kw())
    new, tol = ref.weights(c.q, c.kv, lse.cpu(), old, d_pos=c.lens, row_offset=c.offs, n_tokens=c.n, bits=c.bits,
                           scale=SCALE, decay=0.25)
    assert ((w.double().cpu() - new).abs() <= tol).all()


def test_a_batch_with_nothing_to_attend():
    c = Case(41, [-1, 0, -1], 2, 16, n_tokens=[2, 0, 1])
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("Q,H", [(1, 16), (2, 128), (3, 128), (9, 128)])
@pytest.mark.parametrize("num_sms", [2, 4, 0])
def test_weights_of_several_requests_in_one_run(Q, H, num_sms):
    """All forms of the staging (one and two resident query blocks, streamed ones) across requests."""
    c = Case(50 + Q, [600, 0, 257, 1000, 255, 1, 511], Q, H, n_tokens=[Q, Q, 1, Q, 0, Q, max(1, Q - 1)])
    out, lse = c.run(num_sms=num_sms)
    old = torch.rand(c.kv.shape[0])
    results = []
    for pdl in (False, True):
        w = old.cuda()
        p = c.plan(num_sms=num_sms, pdl=pdl)
        scratch = mla.tree_alloc_scratch(p)
        mla.tree_weights(p, c.d["q"], c.d["kv"], lse, scratch, w, decay=0.75, **c.kw())
        torch.cuda.synchronize()
        assert mla.status_word(p, scratch) == 0
        results.append(w)
    new, tol = ref.weights(c.q, c.kv, lse.cpu(), old, d_pos=c.lens, row_offset=c.offs, n_tokens=c.n, bits=c.bits,
                           scale=SCALE, decay=0.75)
    assert ((results[0].double().cpu() - new).abs() <= tol).all()
    assert torch.equal(results[0], results[1])


def test_rows_past_4_gigabytes():
    """The same requests at the front of a cache and behind its first 4 GiB give the same bits."""
    far = (1 << 32) // 1152 + 1000
    rows = far + 1200
    kv = torch.empty(rows, 576, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    kv[:1200] = torch.randn(1200, 576, generator=g, device="cuda").bfloat16()
    kv[far:] = kv[:1200]
    c = Case(60, [1000], 7, 16)
    d_pos = torch.tensor([1000], dtype=torch.int32, device="cuda")
    weights, positions = torch.zeros(rows, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    seen = []
    for at in (0, far):
        off = torch.tensor([at], dtype=torch.int64, device="cuda")
        p = c.plan()
        scratch = mla.tree_alloc_scratch(p)
        new = torch.randn(1, 7, 576, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        pos = torch.arange(1000, 1007, dtype=torch.int32, device="cuda")[None]
        mla.rope_append(mla.rope_table(64), pos, c=new[..., :512], k_rope=new[..., 512:], kv=kv, d_pos=d_pos,
                        row_offset=off, row_positions=positions, row_weights=weights)
        out, lse = c.outputs()
        kw = dict(d_pos=d_pos, row_offset=off, mask=c.d["mask"])
        mla.tree_forward(p, c.d["q"], kv, out, lse, scratch, **kw)
        mla.tree_weights(p, c.d["q"], kv, lse, scratch, weights, decay=0.0, **kw)
        mla.tree_commit(kv, torch.tensor([[3, 5, 6]], dtype=torch.int32, device="cuda"),
                        torch.tensor([3], dtype=torch.int32, device="cuda"), d_pos=d_pos, row_offset=off,
                        row_weights=weights)
        d = d_pos + 3
        mla.evict(kv, weights, positions, mla.evict_alloc_scratch(batch=1, keep=600), d_pos=d,
                  next_pos=torch.tensor([1007], dtype=torch.int32, device="cuda"), keep=600, row_offset=off)
        seen.append((out, lse, weights[at:at + 1200].clone(), kv[at:at + 1200].clone(), d.clone()))
    for x, y in zip(*seen):
        assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y)


def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable():
    c = Case(61, [3000, 50], 8, 16)
    want = c.reference()
    p = c.plan(stall_test=True)
    good = c.plan()
    scratch = mla.tree_alloc_scratch(p)
    out, lse = c.outputs()
    args = mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw())
    w = torch.zeros(c.kv.shape[0], device="cuda")
    for call in (lambda q: mla.tree_forward_args(q, args, scratch),
                 lambda q: mla.tree_weights_args(q, args, scratch, w, decay=0.0)):
        mla.scratch_init(scratch)
        call(p)
        torch.cuda.synchronize()
        assert mla.status_word(p, scratch) == mla.EDEVICE
    mla.scratch_init(scratch)
    mla.tree_forward_args(good, args, scratch)
    torch.cuda.synchronize()
    assert mla.status_word(good, scratch) == 0
    c.check(out, lse, want)


def test_two_host_threads():
    import threading
    cases = [Case(70 + i, [500 + 300 * i, 40], 6, 16) for i in range(2)]
    got, failed = [None, None], []

    def work(i):
        try:
            c, s = cases[i], torch.cuda.Stream()
            p = c.plan(pdl=True)
            scratch, (out, lse) = mla.tree_alloc_scratch(p), c.outputs()
            torch.cuda.synchronize()
            for _ in range(20):
                mla.tree_forward(p, c.d["q"], c.d["kv"], out, lse, scratch, stream=s, **c.kw())
            s.synchronize()
            got[i] = (out, lse)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed
    for c, r in zip(cases, got):
        c.check(*r)


def test_arguments_of_another_shape_than_the_plan_are_refused():
    c = Case(62, [30], 4, 16)
    p = mla.tree_plan(batch=1, tokens=5, heads=16, scale=SCALE)
    out, lse = c.outputs()
    with pytest.raises(ValueError, match="plan"):
        mla.tree_forward(p, c.d["q"], c.d["kv"], out, lse, mla.tree_alloc_scratch(p), **c.kw())
    with pytest.raises(ValueError):
        mla.tree_make_args(c.d["q"], c.d["kv"].to(torch.float16), out, lse, **c.kw())
    with pytest.raises(ValueError):
        mla.tree_make_args(c.d["q"].transpose(1, 2), c.d["kv"], out, lse, **c.kw())
    with pytest.raises(ValueError):
        mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **{**c.kw(), "d_pos": c.d["d_pos"].long()})
