"""Runs of calls of the drafted-token kernels: one behind the other on the same
SMs, and the forms of a call that the other tests take once."""
import math

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref
from test_gpu_tree import Case

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
