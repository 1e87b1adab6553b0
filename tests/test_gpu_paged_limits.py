"""The paged 4-bit cache at the ends of what its arguments may be."""
import math

import pytest
import torch

import decode_attention_mla_gb300 as mla
import perf.more_operators as measured
import _paged_ref as ref
from test_gpu_paged import BOTH, Append, Case

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")

# a last tile that the rows end in; a window; rows without a page
WHERE = [dict(d_pos=[999]), dict(d_pos=[999, 40], Q=2, window=300, sink=5), dict(d_pos=[999], gone=[(0, 3), (0, 62)])]


@pytest.mark.parametrize("kw", [dict(kv_scale=2.0 ** -20), dict(kv_scale=2.0 ** -64), dict(scale=2.0 ** -26),
                                dict(scale=1e-40), dict(scale=2.0 ** -59, kv_scale=2.0 ** -64)], ids=str)
@pytest.mark.parametrize("where", WHERE, ids=str)
@BOTH
def test_zero_queries_at_any_scale(kw, where, H, sms):
    """All scores are 0, however small the factor on them is: the average of the rows."""
    c = Case(**where, **kw, H=H, sms=sms, fp32=True)
    c.q.zero_()
    c.on_gpu()
    c.forward()
    c.check()


@pytest.mark.parametrize("kw", [dict(kv_scale=2.0 ** -30, scale=2.0 ** -50), dict(kv_scale=2.0 ** -64, scale=1.0)], ids=str)
@pytest.mark.parametrize("where", WHERE, ids=str)
@BOTH
def test_tiny_queries_at_any_scale(kw, where, H, sms):
    c = Case(**where, **kw, H=H, sms=sms, gain=2.0 ** -100)
    c.on_gpu()
    c.forward()
    c.check()


@BOTH
def test_large_queries_over_rows_of_zeros(H, sms):
    """A factor past fp32's range on scores that are 0."""
    c = Case([300], H=H, sms=sms, gain=2.0 ** 100, scale=2.0 ** 59)
    c.pages = torch.zeros_like(c.pages)
    c.on_gpu()
    c.forward()
    c.check()


@pytest.mark.parametrize("d", [300, 5000])
@BOTH
def test_nan_and_infinite_scores_make_their_rows_nan(d, H, sms):
    """A query's NaN or infinity (over keys of both signs) is the whole result of its (token, head), and nobody else's."""
    c = Case([d], Q=2, H=H, sms=sms)
    c.q[0, 0, 3, 17] = math.nan
    c.q[0, 1, 5, 570] = math.inf
    c.q[0, 1, 9, 100] = -math.inf
    bad = {(0, 3), (1, 5), (1, 9)}
    want = c.expected()
    c.on_gpu()
    c.forward()
    torch.cuda.synchronize()
    out, lse = c.out.cpu().double(), c.lse.cpu().double()
    for i, h in bad:
        assert bool(lse[0, i, h].isnan()) and bool(out[0, i, h].isnan().all()), f"{i, h}"
    for (_, i), (o, l, tol_o, tol_l) in want.items():
        ok = torch.tensor([(i, h) not in bad for h in range(H)])
        assert bool(((out[0, i] - o).abs() <= tol_o)[ok].all())
        assert bool(((lse[0, i] - l).abs() <= tol_l)[ok].all())


@pytest.mark.parametrize("on", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norms_one_by_one(on, interleaved):
    """Weights for some of latents, keys and queries; the others go without a norm."""
    a = Append([37, 5], N=6, H=33, n_tokens=[6, 4], interleaved=interleaved, kv_scale=0.5)
    a.w = [w if use else None for w, use in zip(a.w, on)]
    a.run().check()


def test_measured_append_follows_weights_that_are_replaced(monkeypatch):
    """A state whose norm weights are other tensors than at its last pass gives what a state made with them gives."""
    monkeypatch.setattr(measured, "own", True)
    case = dict(op="append", B=2, N=5, H=16, lo=100, hi=200, ragged=True, interleaved=True, page_rows=16, norms=True,
                kv_scale=0.5)
    a, b = measured.prepare(case, 1), measured.prepare(case, 1)
    first = [t.clone() for t in measured.run(a)]
    for name in ("c_norm", "k_norm", "q_norm"):
        a[name] = b[name] = (b[name].float() * 1.5).bfloat16()
        b.pop("handle", None)
        got, want = measured.run(a), measured.run(b)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert not any(torch.equal(x, y) for x, y in zip(got, first))


@BOTH
def test_probabilities_are_rounded_once_to_f16(H, sms):
    """Two rows, of which the second's latents are 1: the output is its probability, off by half a step of f16's eleven bits
    (2^-11), and where that is subnormal by half of 2^-31 of the largest."""
    Q = 64
    pages = torch.zeros(1, 8, 416, dtype=torch.uint8)
    pages[0, 1, :256], pages[0, 1, 256:288] = 0x22, 0x38          # 1.0 times 1.0
    pages[0, 1, 288:290] = torch.tensor([0x80, 0x3f], dtype=torch.uint8)
    q = torch.zeros(Q, 1, H, 576)
    q[..., 512] = torch.linspace(-24, 24, Q * H).view(Q, 1, H)
    q = q.bfloat16()
    s = q[..., 512].double()
    plan = mla.paged_plan(batch=Q, tokens=1, heads=H, scale=1.0, num_sms=sms)
    out, lse = torch.zeros(Q, 1, H, 512, device="cuda"), torch.zeros(Q, 1, H, device="cuda")
    mla.paged_forward(plan, q.cuda(), pages.cuda(), torch.zeros(Q, 1, **I32), out, lse, mla.paged_alloc_scratch(plan),
                      d_pos=torch.ones(Q, **I32))
    p = torch.sigmoid(s)
    # besides: the score in base 2 (its factor's rounding and its own), the reference and the difference to it (each of the
    # score and 7 more at most), both exponentials (2^-21), the sum and its reciprocal
    rest = (4 * 1.4427 * s.abs() + 28) * ref.F32 + 2 * 2.0 ** -21 + 4 * ref.F32
    tol = p * (ref.F16 + rest) + 2.0 ** -32
    err = (out.cpu().double() - p[..., None]).abs()
    assert bool((err <= tol[..., None]).all()), f"off by {float((err / tol[..., None]).max()):.4g} bounds"
    want = torch.logaddexp(s, torch.zeros_like(s))
    assert bool(((lse.cpu().double() - want).abs() <= rest + want.abs() * 4 * ref.F32).all())
    assert float((err / p[..., None]).where((p > 1e-4)[..., None], 0).max()) > 2.0 ** -12
