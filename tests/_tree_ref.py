"""Plain 64-bit forms of the drafted-token operators, written from their
definitions, with the error bounds that the kernels' types allow.

Bounds count roundings at half a step each: bf16 2^-8, fp32 2^-24 (relative).
A score is a fp32 sum of 576 products of bf16 values (exact in fp32): its error
is at most 576 steps of 2^-24 of the sum of magnitudes, here 600 to cover the
scale.  A probability carries the score's error and the base-2 exponential's
(2^-22); it enters P . V rounded to bf16."""
from __future__ import annotations

import math

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def masks_of_tree(rnd, Q):
    bits = []
    for i in range(Q):
        parent = rnd.randint(max(-1, i - 6), i - 1)
        bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
    return bits


def signed(word):
    return word - (1 << 64) if word >> 63 else word


def attended(d_pos, n, bits, base, kv_rows):
    """Request rows that a token with mask `bits` attends."""
    if d_pos < 0:
        return []
    t = list(range(d_pos)) + [d_pos + j for j in range(n) if bits >> j & 1]
    return [x for x in t if 0 <= base + x < kv_rows]


def tree(q, kv, *, d_pos, row_offset, n_tokens, bits, scale, kv_rows=None):
    """Per (b, i): out [H, 512], lse [H] and their bounds; None where i >= n_tokens[b]."""
    B, Q, H, _ = q.shape
    kv_rows = kv_rows or kv.shape[0]
    res = {}
    for b in range(B):
        for i in range(n_tokens[b]):
            rows = attended(d_pos[b], n_tokens[b], bits[b][i], row_offset[b], kv_rows)
            if not rows:
                z = torch.zeros(H, 512, dtype=torch.float64)
                res[b, i] = (z, torch.full((H,), -math.inf, dtype=torch.float64), z, torch.zeros(H).double())
                continue
            k = kv[torch.tensor(rows) + row_offset[b]].double()
            x = q[b, i].double()
            s = x @ k.T * scale
            mag = (x.abs() @ k.abs().T * scale).amax(1)
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            out = p @ k[:, :512]
            spread = p @ k[:, :512].abs()
            d_s = 600 * F32 * mag + 4 * F32 * (lse.abs() + s.abs().amax(1))
            tol_l = d_s + 2.0 ** -21 + len(rows) * F32
            tol_o = spread * (BF16 + 2 * (d_s + 2.0 ** -21 + len(rows) * F32))[:, None]
            res[b, i] = (out, lse, tol_o, tol_l)
    return res


def weights(q, kv, lse, old, *, d_pos, row_offset, n_tokens, bits, scale, decay, kv_rows=None):
    """New weights and their bounds (entries that are not touched: old, and a bound all the same)."""
    B, Q, H, _ = q.shape
    kv_rows = kv_rows or kv.shape[0]
    new, tol = old.double().clone(), torch.zeros(old.shape, dtype=torch.float64)
    for b in range(B):
        if d_pos[b] < 0:
            continue
        for t in range(d_pos[b] + n_tokens[b]):
            r = row_offset[b] + t
            if 0 <= r < kv_rows:
                was = new[r].clone()
                new[r] = decay * was if decay else 0.0
                tol[r] = 2 * F32 * abs(float(new[r]))
        for i in range(n_tokens[b]):
            rows = torch.tensor(attended(d_pos[b], n_tokens[b], bits[b][i], row_offset[b], kv_rows),
                                dtype=torch.int64) + row_offset[b]
            live = torch.isfinite(lse[b, i])
            if not len(rows) or not live.any():
                continue
            k, x, l = kv[rows].double(), q[b, i][live].double(), lse[b, i][live].double()
            s = x @ k.T * scale
            p = torch.exp(s - l[:, None])
            d_s = 600 * F32 * (x.abs() @ k.abs().T * scale) + 4 * F32 * (s.abs() + l.abs()[:, None]) + 2.0 ** -21
            new[rows] += p.sum(0)
            tol[rows] += (p * d_s).sum(0) * 2
    H_sum = Q * H * F32
    return new, tol + new.abs() * H_sum + 2.0 ** -40


def rotate(x, positions, inv_freq, rot, interleaved, amplitude):
    """[..., 64] rotated in 64 bits; positions broadcast over the leading dimensions."""
    y = x.double().clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        t = positions.double() * inv_freq[j]
        c, s = amplitude * torch.cos(t), amplitude * torch.sin(t)
        y[..., a] = x[..., a].double() * c - x[..., b].double() * s
        y[..., b] = x[..., b].double() * c + x[..., a].double() * s
    return y


def inv_freq(rot, base, scaling="none", factor=1.0, original_ctx=4096.0, beta_fast=32.0, beta_slow=1.0):
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "yarn":
        def pair(beta):
            return rot * math.log(original_ctx / (beta * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
        out = []
        for j, x in enumerate(f):
            r = min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0)
            out.append(x * (1 - r) + x / factor * r)
        return out
    return f


def evict_rows(weights, positions, n, keep, sink, recent_from):
    """Source row of each of the min(n, keep) kept places."""
    if n <= keep:
        return list(range(n))

    def rank(r):
        if positions[r] < sink or positions[r] >= recent_from:
            return (0, 0.0, r)
        w = weights[r]
        return (1, math.inf if math.isnan(w) else -w, r)
    stay = sorted(sorted(range(n), key=rank)[:keep])
    here = {r for r in stay if r < keep}
    behind = iter([r for r in stay if r >= keep])
    return [r if r in here else next(behind) for r in range(keep)]
