"""Runs of calls of the drafted-token kernels: one behind the other on the same
SMs, and the forms of a call that the other tests take once."""
import math

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref
import test_gpu_tree
from test_gpu_tree import SCALE, Case

pytestmark = pytest.mark.gpu
NAN = float("nan")


# Runs that end with every buffer of a form in use or not: one tile and several, one item
# and several, the odd CTAs with live rows and without, all forms of the staging.
@pytest.mark.parametrize("lens,Q,H,num_sms", [
    ([200], 1, 16, 0), ([2000], 1, 16, 2), ([100, 300, 60], 2, 16, 2), ([700], 2, 128, 2), ([90, 600], 2, 128, 4),
    ([300], 5, 128, 2), ([1500, 40], 5, 128, 6), ([64] * 12, 3, 16, 4),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_one_behind_the_other(lens, Q, H, num_sms, dtype):
    """Programmatic launches: a kernel's CTAs take the SMs of the one before as they end."""
    c = Case(80 + Q + H, lens, Q, H)
    p = c.plan(num_sms=num_sms, pdl=True)
    scratch = mla.tree_alloc_scratch(p)
    out, lse = c.outputs(dtype)
    args = mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw())
    w = torch.zeros(c.kv.shape[0], device="cuda")

    def calls():
        mla.tree_weights_args(p, args, scratch, w, decay=0.0)
        mla.tree_forward_args(p, args, scratch)
        mla.tree_weights_args(p, args, scratch, w, decay=0.0)

    mla.tree_forward_args(p, args, scratch)
    calls()
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, lse, w)]
    c.check(out, lse)
    for t in (out, w):
        t.zero_()
    out.fill_(7)
    for _ in range(50):
        calls()
    torch.cuda.synchronize()
    assert mla.status_word(p, scratch) == 0
    for a, b in zip(first, (out, lse, w)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def touched_rows(c):
    """Entries of the weights that a call writes (its rows inside the cache), from the definition."""
    touched = torch.zeros(c.kv.shape[0], dtype=torch.bool)
    for b in range(c.B):
        if c.lens[b] >= 0:
            lo, hi = max(c.offs[b], 0), min(c.offs[b] + c.lens[b] + c.n[b], c.kv_rows)
            touched[lo:hi] = True
    return touched


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("lens,Q,H,n", [([600], 8, 33, [5]), ([260, 0, -1, 64, 1000], 5, 16, [5, 5, 5, 0, 3]),
                                        ([300, 128], 2, 128, [1, 2]), ([255, 400], 5, 128, [5, 4])])
def test_entries_of_other_rows_keep_their_bits(lens, Q, H, n, decay):
    c = Case(90 + Q + H, lens, Q, H, n_tokens=n, mask="random")
    c.kv_rows -= 2 if n[-1] == Q else 0                     # the last request's last rows lie outside
    touched = touched_rows(c)
    assert not touched.all() and (~touched).sum() >= 3
    old = torch.rand(c.kv.shape[0], generator=torch.Generator().manual_seed(1))
    old[~touched] = torch.tensor([NAN, -0.0, math.inf, -3.0]).repeat(old.numel())[:int((~touched).sum())]
    out, lse = c.run()
    w = old.cuda()
    p = c.plan()
    mla.tree_weights(p, c.d["q"], c.d["kv"], lse, mla.tree_alloc_scratch(p), w, decay=decay, **c.kw())
    w = w.cpu()
    assert torch.equal(w[~touched].view(torch.int32), old[~touched].view(torch.int32))
    new, tol = ref.weights(c.q, c.kv, lse.cpu(), old.nan_to_num(0, 0, 0), d_pos=c.lens, row_offset=c.offs, n_tokens=c.n,
                           bits=c.bits, scale=SCALE, decay=decay, kv_rows=c.kv_rows)
    assert ((w.double() - new).abs() <= tol)[touched].all()


def test_a_wait_that_runs_out_with_fp32_outputs():
    c = Case(61, [3000, 50], 8, 16)
    bad, good = c.plan(stall_test=True), c.plan()
    scratch = mla.tree_alloc_scratch(bad)
    out, lse = c.outputs(torch.float32)
    args = mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw())
    mla.tree_forward_args(bad, args, scratch)
    torch.cuda.synchronize()
    assert mla.status_word(bad, scratch) == mla.EDEVICE
    mla.scratch_init(scratch)
    mla.tree_forward_args(good, args, scratch)
    torch.cuda.synchronize()
    assert mla.status_word(good, scratch) == 0
    c.check(out, lse)


@pytest.mark.parametrize("bad", [NAN, math.inf])
def test_non_finite_drafts_with_fp32_outputs(bad):
    """Only token 3 attends the broken draft 3; committed rows fill part of the drafts' tile and all of it."""
    for rows in (140, 256, 0):
        c = Case(12, [rows], 8, 16, mask="none")
        c.bits = [[1 << i for i in range(8)]]
        c.d["mask"] = torch.tensor(c.bits, dtype=torch.int64, device="cuda")
        c.d["kv"][c.offs[0] + rows + 3, 100:140] = bad
        c.d["q"][:, :, :, 100:140] = abs(c.d["q"][:, :, :, 100:140])
        c.q = c.d["q"].cpu()
        want = c.reference()
        del want[0, 3]
        out, lse = c.run(torch.float32)
        assert torch.isnan(out[0, 3]).all()
        out[0, 3], lse[0, 3] = 7, 7
        c.check(out, lse, want)


class Elsewhere:
    """A tensor that says it is on another device."""

    def __init__(self, t):
        self.t, self.is_cuda, self.dtype, self.nbytes = t, True, t.dtype, t.nbytes

    def get_device(self):
        return self.t.get_device() + 1

    def is_contiguous(self):
        return True


def test_scratch_and_arguments_of_another_device_are_refused():
    """Refused before anything is launched: scratch elsewhere, or with fewer bytes behind it than it
    counts (a broadcast one); arguments laid out while another device was current."""
    c = Case(63, [30], 4, 16)
    p = c.plan()
    scratch = mla.tree_alloc_scratch(p)
    out, lse = c.outputs()
    a = mla.tree_make_args(c.d["q"], c.d["kv"], out, lse, **c.kw())
    n = c.kv.shape[0]
    w, pos = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    kv = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    e = mla.evict_make_args(kv, w, pos, d_pos=c.d["d_pos"].clone(), next_pos=c.d["d_pos"], keep=8,
                            row_offset=c.d["row_offset"])
    r = mla.rope_make_args(mla.rope_table(), torch.zeros(1, 4, dtype=torch.int32, device="cuda"),
                           q_rope=c.d["q"][..., 512:], q=c.d["q"])
    ev = mla.evict_alloc_scratch(batch=1, keep=8)
    wide = torch.zeros(1, 256, dtype=torch.uint8, device="cuda").expand(p.scratch_bytes // 256 + 1, 256)
    for bad in (Elsewhere(scratch), wide, scratch.cpu()):
        for call in (lambda: mla.tree_forward_args(p, a, bad), lambda: mla.tree_weights_args(p, a, bad, w),
                     lambda: mla.evict_args(e, bad)):
            with pytest.raises(ValueError):
                call()
    for args, call in ((a, lambda: mla.tree_forward_args(p, a, scratch)),
                       (a, lambda: mla.tree_weights_args(p, a, scratch, w)),
                       (e, lambda: mla.evict_args(e, ev)), (r, lambda: mla.rope_append_args(r))):
        assert args._device == 0
        args._device = 1
        with pytest.raises(ValueError, match="device"):
            call()
        args._device = 0
    mla.tree_forward_args(p, a, scratch)
    torch.cuda.synchronize()
    c.check(out, lse)


ROWS_ONCE = next(m.args[1] for m in test_gpu_tree.test_every_row_counts_once.pytestmark if m.name == "parametrize")


@pytest.mark.parametrize("num_sms,lens,Q,H", ROWS_ONCE)
def test_every_row_counts_once_with_bf16_outputs(num_sms, lens, Q, H):
    """All splits of the work, in the other form of the kernel: queries of zero, so the log-sum-exp is the
    log of the count, and the means of latents of 0 and 1 differ from the fp32 ones by their rounding."""
    B, i32 = len(lens), dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(B + Q)
    offs = [sum(lens[:b]) + b * Q for b in range(B)]
    kv = torch.randint(0, 2, (sum(lens) + B * Q, 576), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    q = torch.zeros(B, Q, H, 576, dtype=torch.bfloat16, device="cuda")
    p = mla.tree_plan(batch=B, tokens=Q, heads=H, scale=SCALE, num_sms=num_sms)
    scratch = mla.tree_alloc_scratch(p)
    got = []
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = torch.empty(B, Q, H, 512, dtype=dtype, device="cuda"), torch.empty(B, Q, H, device="cuda")
        mla.tree_forward(p, q, kv, out, lse, scratch, d_pos=torch.tensor(lens, **i32),
                         row_offset=torch.tensor(offs, dtype=torch.int64, device="cuda"))
        got.append((out, lse))
    assert mla.status_word(p, scratch) == 0
    count = torch.tensor(lens, dtype=torch.float64, device="cuda")[:, None] + torch.arange(1, Q + 1, device="cuda")
    assert (got[0][1].double() - torch.log(count)[:, :, None]).abs().max() <= 2.0 ** -20 * 8
    # probabilities of one are exact in bf16: half a step of the output, and the fp32 sums' 2^-18
    out, exact = got[0][0].float(), got[1][0]
    assert ((out - exact).abs() <= ref.BF16 * exact.abs() + 2.0 ** -18).all()
