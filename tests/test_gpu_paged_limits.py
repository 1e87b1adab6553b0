"""The paged 4-bit cache at the ends of what its arguments may be."""
import pytest
import torch

from test_gpu_paged import BOTH, Case

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
