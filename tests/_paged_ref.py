"""Plain 64-bit forms of the paged 4-bit cache's operators, written from their
definitions, with the error bounds that the kernels' types allow.

Bounds count roundings at half a step each: bf16 2^-8, f16 2^-11, fp32 2^-24
(relative).  A score is a fp32 sum of 576 products (exact in fp32) whose error is
at most 576 steps of 2^-24 of the sum of magnitudes, here 600 to cover the scale.
A probability carries the score's error and the base-2 exponential's (2^-21), and
enters the second product in f16."""
from __future__ import annotations

import math

import torch

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64)


def row_values(raw, kv_scale):
    """Rows of bytes [n, 416] as 64-bit values [n, 576]."""
    code = raw[:, :256].long()
    code = torch.stack([code & 15, code >> 4], -1).flatten(1)
    scale = raw[:, 256:288].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    rope = raw[:, 288:].contiguous().view(torch.bfloat16).double()
    return torch.cat([E2M1.to(raw.device)[code] * scale * kv_scale, rope], 1)


def rows_of(table, b, page_rows, ts, n_pages):
    """(page, slot) of the rows ts of request b that have a page, and those rows."""
    found, kept = [], []
    for t in ts:
        col = t // page_rows
        page = int(table[b][col]) if col < len(table[b]) else -1
        if 0 <= page < n_pages:
            found.append((page, t % page_rows))
            kept.append(t)
    return found, kept


def seen(r, window, sink):
    return [t for t in range(r + 1) if window == 0 or t > r - window or t < sink]


def attention(q, pages, table, *, d_pos, n_tokens, scale, window, sink, kv_scale, out_half):
    """Per (b, i): out [H, 512], lse [H] and their bounds.  table, d_pos, n_tokens: lists."""
    B, Q, H, _ = q.shape
    n_pages, ps, _ = pages.shape
    res = {}
    for b in range(B):
        for i in range(min(max(n_tokens[b], 0), Q)):
            at, _ = rows_of(table, b, ps, seen(d_pos[b] + i, window, sink) if d_pos[b] >= 0 else [], n_pages)
            if not at:
                z = torch.zeros(H, 512, dtype=torch.float64, device=q.device)
                res[b, i] = (z, z[:, 0] - math.inf, z, z[:, 0])
                continue
            idx = torch.tensor(at, device=q.device)
            k = row_values(pages[idx[:, 0], idx[:, 1]], kv_scale)
            x = q[b, i].double()
            s = x @ k.T * scale
            mag = (x.abs() @ k.abs().T * scale).amax(1)
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            out = p @ k[:, :512]
            spread = p @ k[:, :512].abs()
            n = len(at)
            d_s = 600 * F32 * mag + 4 * F32 * (lse.abs() + s.abs().amax(1))
            tol_l = d_s + 2.0 ** -21 + n * F32
            # (a probability below 2^-17 of the largest is a multiple of 2^-31 of it)
            tol_o = spread * (F16 + 2 * (d_s + 2.0 ** -21 + 2 * n * F32))[:, None] + out.abs() * out_half
            tol_o = tol_o + n * 2.0 ** -31 * k[:, :512].abs().amax()
            res[b, i] = (out, lse, tol_o, tol_l)
    return res


def norm(x, weight, eps):
    x = x.double()
    if weight is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def rotate(x, positions, inv_freq, interleaved, rot_dim, amplitude=1.0):
    """x [.., 64] in 64 bits at positions [..]."""
    ang = positions.double()[..., None] * torch.tensor(inv_freq, dtype=torch.float64)
    cos, sin = amplitude * ang.cos(), amplitude * ang.sin()
    y = x.clone()
    h = rot_dim // 2
    a, b = (slice(0, rot_dim, 2), slice(1, rot_dim, 2)) if interleaved else (slice(0, h), slice(h, rot_dim))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def quantise(c, kv_scale):
    """[n, 512] in 64 bits: codes [n, 512], scales as E4M3 values [n, 32] (before kv_scale)."""
    blocks = c.unflatten(-1, (32, 16))
    scale = (blocks.abs().amax(-1) / 6 / kv_scale).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    unit = torch.where(scale[..., None] > 0, blocks / (scale * kv_scale)[..., None], torch.zeros_like(blocks))
    dist = (unit.abs()[..., None] - E2M1[:8]).abs()
    # nearest value, halfway the even code
    best = dist.amin(-1, keepdim=True)
    near = dist == best
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7])          # even codes before odd ones
    code = torch.where(near, order, 99).argmin(-1)
    return (code + 8 * (unit < 0).long()).flatten(-2), scale


class Pages:
    """What mla_pages_fork and mla_pages_compact say, with lists."""

    def __init__(self, table, d_pos, n_pages, page_rows):
        self.table, self.d_pos, self.n_pages, self.ps = [list(r) for r in table], list(d_pos), n_pages, page_rows

    def fork(self, parent=None, rows=None, reserve=0, window=0, sink=0):
        B, columns, ps = len(self.table), len(self.table[0]), self.ps
        parent = list(range(B)) if parent is None else parent
        new = [[-1] * columns for _ in range(B)]
        n = [0] * B
        full_of, ends = {}, {}
        for b in range(B):
            if not 0 <= parent[b] < B:
                continue
            have = max(self.d_pos[parent[b]], 0)
            n[b] = min(have, max(rows[b], 0) if rows is not None else have, columns * ps)
            if n[b] % ps and not 0 <= self.table[parent[b]][n[b] // ps] < self.n_pages:
                n[b] = n[b] // ps * ps                    # the rows of a last page that is missing are not there
            for c in range(columns):
                page = self.table[parent[b]][c]
                if c * ps >= n[b] or not 0 <= page < self.n_pages:
                    continue
                if window and c * ps >= sink and (c + 1) * ps <= n[b] + 1 - window:
                    continue
                new[b][c] = page
                if (c + 1) * ps <= n[b]:
                    full_of.setdefault(page, []).append(b)
                else:
                    ends.setdefault(page, []).append(b)
        wants, copies = [], []
        for b in range(B):
            if not 0 <= parent[b] < B:
                continue
            last, part = n[b] // ps, n[b] % ps
            copied = False
            if part and new[b][last] >= 0:
                page = new[b][last]
                copied = page in full_of or ends[page][0] != b
            end = min(columns, -(-(n[b] + reserve) // ps))
            for c in range(last, end):
                if c == last and part and new[b][last] >= 0:
                    if copied:
                        wants.append((b, c, new[b][last]))
                        new[b][c] = -1
                else:
                    wants.append((b, c, None))
        refs = [0] * self.n_pages
        for row in new:
            for page in row:
                if page >= 0:
                    refs[page] += 1
        free = [i for i in range(self.n_pages) if refs[i] == 0]
        missing = 0
        for k, (b, c, src) in enumerate(wants):
            if k >= len(free):
                missing += 1
                if src is not None:
                    n[b] = n[b] // ps * ps
                continue
            new[b][c] = free[k]
            refs[free[k]] = 1
            if src is not None:
                copies.append((src, free[k], n[b] % ps))
        self.table, self.d_pos = new, n
        return refs, missing, copies

    def compact(self, refs):
        live = sum(r > 0 for r in refs)
        holes = [i for i in range(live) if refs[i] <= 0]
        movers = [i for i in range(live, self.n_pages) if refs[i] > 0]
        to = {i: i for i in range(live) if refs[i] > 0}
        to.update(zip(movers, holes))
        out = [0] * self.n_pages
        for i, j in to.items():
            out[j] = refs[i]
        self.table = [[to.get(page, -1) for page in row] for row in self.table]
        return out, live, list(zip(movers, holes))
