"""How near the drafted-token attention and the weights come to the 64-bit
forms where the scores are exact, and over short contexts.

U is half a step of fp32 (2^-24 relative).  Scores of queries with one non-zero
element, a power of two, are exact in the tensor cores' sums; the scale is one
fp32 number, so s = q k scale is known exactly, and what is left are the
roundings that the comments beside each bound count."""
import math

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref
import workloads
from _gpu import assert_parity, oracle_dense

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device="cuda")


def one_row_each(Q, H, values, scale, num_sms=0):
    """Q drafts behind no committed row, each attending itself alone: one score per (token, head).
    `values`: bf16 [Q], element 0 of the drafts' rows; head h's query has element 0 alone, 2^(h mod 3).
    Returns plan, scratch, tensors and the exact scores [Q, H]."""
    kv = torch.zeros(Q, 576, dtype=torch.bfloat16, device="cuda")
    kv[:, 0] = values.cuda()
    kv[:, 1] = 1
    q = torch.zeros(1, Q, H, 576, dtype=torch.bfloat16, device="cuda")
    gain = torch.tensor([2.0 ** (h % 3) for h in range(H)])
    q[..., 0] = gain.cuda()
    s = values.double()[:, None] * gain.double() * f32(scale)
    mask = torch.tensor([[ref.signed(1 << i) for i in range(Q)]], dtype=torch.int64, device="cuda")
    p = mla.tree_plan(batch=1, tokens=Q, heads=H, scale=scale, num_sms=num_sms)
    return p, mla.tree_alloc_scratch(p), q, kv, dict(d_pos=ints([0]), mask=mask), s


# Of the log-sum-exp of one row, in base 2: scale * log2 e rounded (U), the maximum's
# product (U), the sum of reference and log (U), then ln 2 and its product (2 U, of which
# ln 2's own rounding is half a step at most); the exponential of the maximum's residual
# and the log of the sum: 2^-22 each, twice for safety.
def lse_bound(s):
    return 5 * U * s.abs() + 2.0 ** -20


@pytest.mark.parametrize("scale", [1 / 8, 1 / 24, 0.1])
def test_log_sum_exps_of_exact_scores(scale):
    values = torch.cat([torch.arange(96, 128), -torch.arange(96, 128)]).bfloat16()     # scores of up to 64
    p, scratch, q, kv, kw, s = one_row_each(64, 128, values, scale)
    out, lse = torch.empty(1, 64, 128, 512, device="cuda"), torch.empty(1, 64, 128, device="cuda")
    mla.tree_forward(p, q, kv, out, lse, scratch, **kw)
    err = lse[0].double().cpu() - s
    assert (err.abs() <= lse_bound(s)).all(), float((err.abs() - lse_bound(s)).max())
    # No part of the scores is lost or added on average: only the two constants' roundings
    # (2 U) and half a step of the product that has no pair are one-sided.
    rel = (err / s)[s.abs() >= 8]
    assert abs(float(rel.mean())) <= 4 * U, float(rel.mean())
    # One row of weight 1: its probability is the exponential of the maximum's residual, U |s|
    # (and 2^-22), rounded for the product and not for the sum; quotient and product 2 U.
    assert ((out[0, :, :, 1].double().cpu() - 1).abs() <= 1.01 * U * s.abs() + 2.0 ** -22 + 2 * U).all()


@pytest.mark.parametrize("scale", [1 / 8, 1 / 24, 0.1])
def test_weights_of_exact_scores(scale):
    """Each draft's weight is the sum over heads of exp(s - lse), here of lse = s rounded to fp32."""
    values = torch.cat([torch.arange(96, 128), -torch.arange(96, 128)]).bfloat16()
    p, scratch, q, kv, kw, s = one_row_each(64, 128, values, scale)
    lse = s.float().cuda()[None].contiguous()
    w = torch.full((64,), 7.0, device="cuda")
    mla.tree_weights(p, q, kv, lse, scratch, w, decay=0.0, **kw)
    want = torch.exp(s - lse[0].double().cpu()).sum(1)
    # exponent: scale * log2 e (U), log2 e (U) and its product (U), each of |s|, the fused
    # sum's own rounding, of a number below 1; exponential 2^-22; 128 terms added
    bound = ((3 * U * s.abs()) + 2.0 ** -21).sum(1) * 1.01 + 128 * 128 * U
    err = w.double().cpu() - want
    assert (err.abs() <= bound).all(), float((err.abs() - bound).max())
    # one-sided: scale * log2 e and log2 e alone
    assert abs(float((err / s.abs().sum(1)).mean())) <= 2 * U + 2.0 ** -21 / 8


def largest_scale():
    """The largest scale that a plan takes (host only: the SM count is given)."""
    def taken(x):
        try:
            mla.tree_plan(batch=1, tokens=1, heads=1, scale=x, num_sms=2)
            return True
        except mla.MLADecodeError:
            return False
    lo, hi = torch.tensor([2.0e38]), torch.tensor([3.0e38])
    lo, hi = int(lo.view(torch.int32)), int(hi.view(torch.int32))
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if taken(float(torch.tensor([mid], dtype=torch.int32).view(torch.float32))):
            lo = mid
        else:
            hi = mid
    return float(torch.tensor([lo], dtype=torch.int32).view(torch.float32))


def test_the_largest_scale_is_a_number():
    """Scores of zero stay zero at every scale that a plan takes."""
    p = mla.tree_plan(batch=1, tokens=3, heads=5, scale=largest_scale())
    scratch = mla.tree_alloc_scratch(p)
    kv = torch.ones(20, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 3, 5, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(1, 3, 5, 512, device="cuda"), torch.empty(1, 3, 5, device="cuda")
    w = torch.empty(20, device="cuda")
    mla.tree_forward(p, q, kv, out, lse, scratch, d_pos=ints([17]))
    mla.tree_weights(p, q, kv, lse, scratch, w, decay=0.0, d_pos=ints([17]))
    for i in range(3):
        assert (lse[0, i].double() - math.log(18 + i)).abs().max() <= 2.0 ** -20
    assert (out - 1).abs().max() <= 2.0 ** -20
    assert abs(float(w.double().sum()) - 15) <= 15 * 2.0 ** -18


# ---- fp32 outputs ---------------------------------------------------------------
@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 16, 64, 129, 256, 1000])
def test_one_token_meets_the_dense_decodes_bar(T, H):
    """One drafted token is the dense decode: the same inputs, oracle and bar."""
    for seed in range(3):
        x = workloads.dense(1, H, T, seed=100 * T + seed)
        p = mla.tree_plan(batch=1, tokens=1, heads=H, scale=x.scale)
        scratch = mla.tree_alloc_scratch(p)
        out, lse = torch.empty(1, 1, H, 512, device="cuda"), torch.empty(1, 1, H, device="cuda")
        mla.tree_forward(p, x.q.cuda()[:, None].contiguous(), x.kv.cuda(), out, lse, scratch, d_pos=x.d_pos.int().cuda())
        assert_parity(out[:, 0], lse[:, 0], *oracle_dense(x), what=f"T={T}, H={H}, seed {seed}")


@pytest.mark.parametrize("num_sms", [0, 2, 6])
@pytest.mark.parametrize("lens,Q,H", [([3], 2, 16), ([0, 40, 7], 9, 16), ([300, 1, 128], 5, 33), ([500], 64, 16),
                                      ([700, 90], 3, 128)])
def test_fp32_outputs_of_exact_scores(lens, Q, H, num_sms):
    """Probabilities enter the product with V in 16 bits and more."""
    g = torch.Generator().manual_seed(Q + H)
    B, offs = len(lens), [sum(lens[:b]) + b * Q for b in range(len(lens))]
    rows = sum(lens) + B * Q
    kv = torch.randn(rows, 576, generator=g).bfloat16()
    kv[:, 570] = torch.randint(-40, 41, (rows,), generator=g).bfloat16()
    q = torch.zeros(B, Q, H, 576, dtype=torch.bfloat16)
    q[..., 570] = torch.tensor([2.0 ** -(h % 3) for h in range(H)]).bfloat16()
    p = mla.tree_plan(batch=B, tokens=Q, heads=H, scale=0.1, num_sms=num_sms)
    scratch = mla.tree_alloc_scratch(p)
    out, lse = torch.empty(B, Q, H, 512, device="cuda"), torch.empty(B, Q, H, device="cuda")
    mla.tree_forward(p, q.cuda(), kv.cuda(), out, lse, scratch, d_pos=ints(lens), row_offset=ints(offs, torch.int64))
    assert mla.status_word(p, scratch) == 0
    for b in range(B):
        for i in range(Q):
            n = lens[b] + i + 1
            k = kv[offs[b]:offs[b] + n].double()
            s = q[b, i].double() @ k.T * f32(0.1)
            rl = torch.logsumexp(s, 1)
            prob = torch.exp(s - rl[:, None])
            want, spread = prob @ k[:, :512], prob @ k[:, :512].abs()
            # a probability: its exponent (5 U of the largest |s|), exponential and reference 2^-20, the
            # pair of bf16 numbers 2^-16; sums over 2 n products drop 2^-23 each; l likewise over n; pieces
            # are joined with weights within 2^-20
            rel = 2 * (5 * U * s.abs().amax(1) + 2.0 ** -20) + 2.0 ** -16 + 3 * n * 2.0 ** -23 + 2.0 ** -20
            err = (out[b, i].double().cpu() - want).abs()
            assert (err <= rel[:, None] * spread).all(), (b, i, float((err / spread).max()), float(rel.max()))
            assert ((lse[b, i].double().cpu() - rl).abs() <= 5 * U * s.abs().amax(1) + 2.0 ** -19 + n * U).all()


@pytest.mark.parametrize("Q,H,rows,num_sms", [(1, 16, 300, 0), (1, 128, 300, 2), (2, 128, 300, 2), (2, 100, 900, 2),
                                              (2, 128, 300, 0), (5, 64, 300, 2)])
def test_weights_keep_half_of_what_one_chain_of_sums_drops(Q, H, rows, num_sms):
    """A score of 64 and 35 addends of 2^-24 of it, one in each of the other 16-column products that
    an MMA sums: towards zero, each is dropped where it is added to the large one.  Half a chain's are not."""
    kv = torch.zeros(rows + Q, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, Q, H, 576, dtype=torch.bfloat16, device="cuda")
    for t in (kv, q):
        t[..., 0] = 8
        t[..., 24::16] = 2.0 ** -9
    s = 64 + 35 * 2.0 ** -18
    lse = torch.full((1, Q, H), 64.0, device="cuda")
    w = torch.empty(rows + Q, device="cuda")
    p = mla.tree_plan(batch=1, tokens=Q, heads=H, scale=1.0, num_sms=num_sms)
    mla.tree_weights(p, q, kv, lse, mla.tree_alloc_scratch(p), w, decay=0.0, d_pos=ints([rows]))
    # the first half, 20 MMAs, drops 19 of the addends at most; roundings as in test_weights_of_exact_scores
    rel = 19 * 2.0 ** -18 + 3 * U * 64 + 2.0 ** -21 + Q * H * U
    want = Q * H * math.exp(s - 64)
    assert ((w[:rows].double() - want).abs() <= rel * want).all(), float((w[:rows].double() / want - 1).abs().max())
