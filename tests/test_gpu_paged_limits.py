"""The paged 4-bit cache at the ends of what its arguments may be."""
import math

import pytest
import torch

import perf.more_operators as measured
from test_gpu_paged import BOTH, Append, Case

pytestmark = pytest.mark.gpu

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
