"""Rotation of the new tokens' queries and keys and the append of their rows
(mla_rope_append), against the 64-bit form."""
import math
import random

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref

pytestmark = pytest.mark.gpu


def make(seed, B, N, H, far=4000):
    g = torch.Generator().manual_seed(seed)
    rnd = random.Random(seed)
    pos = torch.tensor([[rnd.randint(0, far) for _ in range(N)] for _ in range(B)], dtype=torch.int32)
    return (pos, torch.randn(B, N, H, 192, generator=g).bfloat16(), torch.randn(B, N, 576, generator=g).bfloat16())


def bound(x, want, pos, amplitude):
    """Rounding to bf16, plus fp32 products and the angle's fp32 fraction of a turn (2^-24 of pi)."""
    size = amplitude * x.double().abs().amax(-1, keepdim=True) * 2
    return ref.BF16 * want.abs() + size * 16 * ref.F32


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rot", [8, 16, 40, 48, 64])
@pytest.mark.parametrize("B,N,H", [(1, 1, 16), (3, 5, 128), (2, 7, 1), (1, 2, 33)])
def test_rotation_and_append(B, N, H, rot, interleaved):
    pos, qp, kp = make(B + N + H + rot, B, N, H)
    d_pos, n = [4 + 3 * b for b in range(B)], [max(0, N - b) for b in range(B)]
    offs = [b * (N + 40) for b in range(B)]
    rows = B * (N + 40)
    yarn = dict(scaling="yarn", factor=16.0, original_ctx=2048, beta_fast=24.0, beta_slow=2.0)
    table = mla.rope_table(rot, 50000.0, interleaved=interleaved, amplitude=1.25, **yarn)
    f = ref.inv_freq(rot, 50000.0, **yarn)
    qd, kd = qp.cuda(), kp.cuda()
    q = torch.full((B, N, H, 576), 3.0, device="cuda", dtype=torch.bfloat16)
    kv = torch.full((rows, 576), 5.0, device="cuda", dtype=torch.bfloat16)
    rp = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    rw = torch.full((rows,), 2.0, device="cuda")
    dev = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    mla.rope_append(table, pos.cuda(), q_rope=qd[..., 128:], q=q, c=kd[..., :512], k_rope=kd[..., 512:], kv=kv,
                    d_pos=dev(d_pos, torch.int32), row_offset=dev(offs, torch.int64), n_tokens=dev(n, torch.int32),
                    row_positions=rp, row_weights=rw)
    want_q = ref.rotate(qp[..., 128:], pos[..., None], f, rot, interleaved, 1.25)
    want_k = ref.rotate(kp[..., 512:], pos, f, rot, interleaved, 1.25)
    got, kvc = q.double().cpu(), kv.double().cpu()
    assert (got[..., :512] == 3).all()
    touched = torch.zeros(rows, dtype=torch.bool)
    for b in range(B):
        for t in range(N):
            if t >= n[b]:
                assert (got[b, t] == 3).all()
                continue
            w = want_q[b, t]
            assert ((got[b, t, :, 512:] - w).abs() <= bound(qp[b, t, :, 128:], w, pos, 1.25)).all()
            assert torch.equal(got[b, t, :, 512 + rot:], qp[b, t, :, 128 + rot:].double())
            r = offs[b] + d_pos[b] + t
            touched[r] = True
            assert torch.equal(kvc[r, :512], kp[b, t, :512].double())
            assert ((kvc[r, 512:] - want_k[b, t]).abs() <= bound(kp[b, t, 512:], want_k[b, t], pos, 1.25)).all()
            assert int(rp[r]) == int(pos[b, t]) and float(rw[r]) == 0
    assert (kvc[~touched] == 5).all() and (rp.cpu()[~touched] == -9).all() and (rw.cpu()[~touched] == 2).all()


def test_far_positions_keep_their_angle():
    """Position 2^30 + i: a fp32 product of position and frequency would be off by whole radians."""
    pos = torch.tensor([[2 ** 30 + 12345, 2 ** 31 - 1, 0]], dtype=torch.int32)
    x = torch.zeros(1, 3, 1, 64)
    x[..., 0::2] = 1.0
    x = x.bfloat16()
    q = torch.zeros(1, 3, 1, 576, device="cuda", dtype=torch.bfloat16)
    table = mla.rope_table(64, 10000.0)
    mla.rope_append(table, pos.cuda(), q_rope=x.cuda(), q=q)
    # the reference in integers: the table's turn fractions are exact by definition
    turns = mla.rope_turns(64, 10000.0)
    for t in range(3):
        for j in range(32):
            frac = (int(pos[0, t]) * turns[j]) % (1 << 64) / 2.0 ** 64
            c, s = math.cos(2 * math.pi * frac), math.sin(2 * math.pi * frac)
            got = q[0, t, 0, 512 + 2 * j:514 + 2 * j].double().cpu()
            assert abs(float(got[0]) - c) <= ref.BF16 * abs(c) + 2 ** -20
            assert abs(float(got[1]) - s) <= ref.BF16 * abs(s) + 2 ** -20


def test_in_place_rotation_and_queries_alone():
    pos, qp, _ = make(3, 2, 3, 16)
    for interleaved in (True, False):
        q = torch.zeros(2, 3, 16, 576, device="cuda", dtype=torch.bfloat16)
        q[..., 512:] = qp[..., 128:].cuda()
        table = mla.rope_table(64, interleaved=interleaved)
        mla.rope_append(table, pos.cuda(), q_rope=q[..., 512:], q=q)
        want = ref.rotate(qp[..., 128:], pos[..., None], ref.inv_freq(64, 10000.0), 64, interleaved, 1.0)
        err = (q[..., 512:].double().cpu() - want).abs()
        assert (err <= bound(qp[..., 128:], want, pos, 1.0)).all()


def test_e4m3_rows_clamp_and_rows_outside_are_left():
    pos, _, kp = make(4, 2, 4, 1)
    kp[0, 0, 0], kp[0, 0, 1], kp[0, 1, 2], kp[0, 1, 3] = 3e4, -3e4, float("inf"), float("nan")
    kv = torch.zeros(20, 592, dtype=torch.uint8, device="cuda")
    table = mla.rope_table(64, interleaved=False)
    mla.rope_append(table, pos.cuda(), c=kp[..., :512].cuda(), k_rope=kp[..., 512:].cuda(), kv=kv[:, :576],
                    d_pos=torch.tensor([5, 2], dtype=torch.int32, device="cuda"),
                    row_offset=torch.tensor([0, 16], dtype=torch.int64, device="cuda"), kv_scale=0.25)
    got = kv[:, :576].contiguous().view(torch.float8_e4m3fn).double().cpu() * 0.25
    want = kp.double().clone()
    want[..., 512:] = ref.rotate(kp[..., 512:], pos, ref.inv_freq(64, 10000.0), 64, False, 1.0)
    want = want.clamp(-112, 112)
    for b, t, r in [(0, 0, 5), (0, 1, 6), (0, 2, 7), (0, 3, 8), (1, 0, 18), (1, 1, 19)]:
        nan = torch.isnan(want[b, t])
        assert torch.equal(torch.isnan(got[r]), nan)
        # e4m3: half a step is 2^-4 of the value, 2^-10 (times the scale) among the subnormals
        err = (got[r] - want[b, t]).abs()[~nan]
        assert (err <= want[b, t].abs()[~nan] * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10 * 0.25 + 2.0 ** -18).all()
    untouched = [r for r in range(20) if r not in (5, 6, 7, 8, 18, 19)]       # rows 20, 21 lie outside
    assert (kv[untouched] == 0).all() and (kv[:, 576:] == 0).all()
    mla.rope_append(table, pos.cuda(), c=kp[..., :512].cuda(), k_rope=kp[..., 512:].cuda(), kv=kv[:, :576],
                    d_pos=torch.tensor([-1, -3], dtype=torch.int32, device="cuda"),
                    row_offset=torch.tensor([0, 16], dtype=torch.int64, device="cuda"), kv_scale=0.25)
    assert (kv[untouched] == 0).all()


def test_many_tokens_linear_scaling():
    pos, qp, kp = make(5, 2, 700, 64, far=120000)
    q = torch.zeros(2, 700, 64, 576, device="cuda", dtype=torch.bfloat16)
    table = mla.rope_table(64, 1e6, scaling="linear", factor=4.0)
    mla.rope_append(table, pos.cuda(), q_rope=qp.cuda()[..., 128:], q=q)
    want = ref.rotate(qp[..., 128:], pos[..., None], ref.inv_freq(64, 1e6, "linear", 4.0), 64, True, 1.0)
    # the 64-bit reference's own product p f is exact to 2^-52 of 120000 radians
    assert ((q[..., 512:].double().cpu() - want).abs() <= bound(qp[..., 128:], want, pos, 1.0)).all()


def test_side_arrays_without_rows_are_refused():
    x = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="belong"):
        mla.rope_append(mla.rope_table(), pos, q_rope=x, q=q, row_weights=torch.zeros(4, device="cuda"))
