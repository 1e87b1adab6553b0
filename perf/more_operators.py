"""Measured cases of a paged cache in 4 bits: what writes its rows, the attention
that reads them, and what keeps its pages.

A cache row is 416 bytes: 512 latent values in 4 bits (E2M1, two per byte, the
even feature in the low half), 32 scales (E4M3, one per 16 features) and 64
rotated key values in bf16.  A latent value is code * scale * kv_scale, kv_scale
a power of two.  Row t of request b is row t % page_rows of page
page_table[b, t // page_rows]; d_pos[b] rows are committed, and new token i
stands in row d_pos[b] + i.

  append   new tokens' latents normalised (RMS, 512), quantised and written to
           their pages; keys and every head's queries normalised (RMS, 64) and
           rotated by their positions
  attend   attention of 1 .. 64 new tokens per request over the cache: all rows up
           to their own, or a sliding window of them and the first `sink` ones
  fork     every request goes on from a parent's first rows: full pages are shared,
           a shared last page is copied, pages that nobody has are free, and
           pages for the next rows are taken from the free ones
  compact  the pages in use moved to the front of the pool

`run` computes them in elementary torch operations, or with `own` through
decode_attention_mla_gb300.
"""
import math
import random
from operator import is_not, itemgetter

import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
BLOCK = 16                                  # features per scale
ROW_BYTES = LATENT // 2 + LATENT // BLOCK + 2 * ROPE
SCALE = 1.0 / math.sqrt(ROW)
EPS = 1e-6
GOLDEN = 0.6180339887498949
LARGEST_SCORES = 16 * 4 * 128 * 20000       # requests * tokens * heads * rows of the largest attention


def listed():
    return [
        # one decode step of a 16-head rank
        dict(name="append_step", op="append", B=1, N=1, H=16, lo=8191, hi=8191, ragged=False, interleaved=True,
             page_rows=64, norms=True, kv_scale=1.0),
        # a prefill chunk of four ragged requests on all heads
        dict(name="append_prefill", op="append", B=4, N=2048, H=128, lo=2048, hi=100000, ragged=True,
             interleaved=False, page_rows=64, norms=True, kv_scale=0.25),
        # one token after a short prompt: latency
        dict(name="attend_small", op="attend", B=1, Q=1, H=16, lo=255, hi=255, ragged=False, page_rows=64, window=0,
             sink=0, kv_scale=1.0),
        # one token over a long cache on a 16-head rank
        dict(name="attend_long", op="attend", B=1, Q=1, H=16, lo=131071, hi=131071, ragged=False, page_rows=64,
             window=0, sink=0, kv_scale=1.0),
        # a decode step of a ragged batch on a 16-head rank: the cache's bytes
        dict(name="attend_batch", op="attend", B=32, Q=1, H=16, lo=4096, hi=65536, ragged=False, page_rows=64,
             window=0, sink=0, kv_scale=0.5),
        # long ragged requests that see a window and the first rows, all heads, small pages
        dict(name="attend_window", op="attend", B=16, Q=2, H=128, lo=1000, hi=131072, ragged=True, page_rows=16,
             window=4096, sink=4, kv_scale=1.0),
        # four new tokens per request on all heads: the tensor cores
        dict(name="attend_heads", op="attend", B=16, Q=4, H=128, lo=4096, hi=32768, ragged=False, page_rows=128,
             window=0, sink=0, kv_scale=1.0),
        # a beam search step of one prompt
        dict(name="fork_beams", op="fork", B=4, lo=1800, hi=2100, page_rows=64, pages=512, kind="q4", reserve=1,
             window=0, sink=0),
        # a serving batch: requests end, others go on from shared prefixes, pages for eight drafted tokens
        dict(name="fork_batch", op="fork", B=256, lo=500, hi=32000, page_rows=64, pages=65536, kind="q4", reserve=8,
             window=0, sink=0),
        # a small pool of bf16 pages with a few holes
        dict(name="compact_small", op="compact", B=4, lo=500, hi=2000, page_rows=32, pages=1024, kind="bf16"),
        # half of a large pool in use
        dict(name="compact_large", op="compact", B=64, lo=2000, hi=30000, page_rows=64, pages=32768, kind="q4"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "fork", "compact"])
    page_rows = rng.choice([16, 32, 64, 64, 128])
    if op in ("fork", "compact"):
        B = _log_int(rng, 1, 200)
        hi = _log_int(rng, 10, max(11, 1500000 // B))
        hi = min(hi, 100000)
        lo = rng.randint(hi // 8, hi)
        least = B * (hi // page_rows + 2)
        pages = min(_log_int(rng, 2 * least + 16, 4 * least + 64), 65536 * 64 // page_rows)
        case = dict(op=op, B=B, lo=lo, hi=hi, page_rows=page_rows, pages=max(pages, least + B + 8), kind=rng.choice(["q4", "q4", "bf16"]))
        if case["pages"] * page_rows > 2500000:
            case["kind"] = "q4"
        if op == "fork":
            case["reserve"] = rng.choice([0, 1, 1, 4, 16, 100])
            case["window"] = rng.choice([0, 0, rng.randint(1, hi)])
            case["sink"] = rng.choice([0, 4, 64]) if case["window"] else 0
        return case
    H = rng.choice([16, 16, 32, 64, 128])
    B = _log_int(rng, 1, 32)
    if op == "append":
        N = min(_log_int(rng, 1, max(1, 8192 * 128 // (B * H * 2))), 4096)
        lo = rng.randint(0, 2000)
        return dict(op=op, B=B, N=N, H=H, lo=lo, hi=lo + _log_int(rng, 1, 30000), ragged=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, page_rows=page_rows, norms=rng.random() < 0.7,
                    kv_scale=rng.choice([0.125, 0.5, 1.0, 2.0]))
    Q = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
    top = int(min(131072, LARGEST_SCORES / (B * Q * H), 1000000 / B))
    hi = _log_int(rng, 16, max(17, top - 64))
    lo = rng.randint(0, hi)
    window = rng.choice([0, 0, 0, rng.randint(1, hi), min(hi, 1024)])
    return dict(op=op, B=B, Q=Q, H=H, lo=lo, hi=hi, ragged=rng.random() < 0.5, page_rows=page_rows, window=window,
                sink=rng.choice([0, 4, 100]) if window else 0, kv_scale=rng.choice([0.125, 0.5, 1.0, 2.0]))


def _lengths(case):
    """Committed rows per request: spread over [lo, hi], the first request at hi."""
    lo, hi = case["lo"], case["hi"]
    return [hi - int((hi - lo) * ((b * GOLDEN) % 1.0)) for b in range(case["B"])]


def _tokens(case, n):
    """New tokens per request: n, or ragged ones in 1..n."""
    if not case.get("ragged"):
        return [n] * case["B"]
    return [n - int((n - 1) * ((b * GOLDEN) % 1.0)) for b in range(case["B"])]


def _quantise(y, kv_scale):
    """Rows [.., 512] in fp32 as bytes: 256 of codes, 32 of scales."""
    y = y.unflatten(-1, (LATENT // BLOCK, BLOCK))
    scale = (y.abs().amax(-1) * (1.0 / 6.0 / kv_scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale.float() * kv_scale
    v = y * torch.where(step > 0, 1.0 / step, torch.zeros_like(step))[..., None]
    a = v.abs()
    # halfway between two values: the one whose last bit is 0
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code + 8 * torch.signbit(v).byte()).flatten(-2)
    return torch.cat([code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8)], -1)


VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _pairs(device, dtype):
    """The two values of each byte."""
    v = torch.tensor(VALUES, dtype=dtype, device=device)
    byte = torch.arange(256, device=device)
    return torch.stack([v[byte & 15], v[byte >> 4]], -1)


def _row_values(rows, kv_scale, dtype):
    """Rows of bytes [.., 416] as values [.., 576]."""
    c = _pairs(rows.device, dtype)[rows[..., :LATENT // 2].int()].flatten(-2).unflatten(-1, (LATENT // BLOCK, BLOCK))
    scale = rows[..., LATENT // 2:LATENT // 2 + LATENT // BLOCK].contiguous().view(torch.float8_e4m3fn).to(dtype)
    c = (c * (scale * kv_scale)[..., None]).flatten(-2)
    return torch.cat([c, rows[..., ROW_BYTES - 2 * ROPE:].contiguous().view(torch.bfloat16).to(dtype)], -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rnd = random.Random(int(seed))
    B, op, dev, ps = case["B"], case["op"], "cuda", case["page_rows"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    lens = _lengths(case)
    s = dict(case=case, d_pos=ints(lens))
    if op in ("fork", "compact"):
        # a page more than the pool has, which no table names
        n_pages = case["pages"]
        columns = (case["hi"] + case.get("reserve", 0)) // ps + 2
        if case["kind"] == "q4":
            s["buffer"] = torch.randint(0, 256, (n_pages + 1, ps, ROW_BYTES), generator=g, device=dev, dtype=torch.uint8)
        else:
            s["buffer"] = normal(n_pages + 1, ps, ROW)
        s["pages"] = s["buffer"][:n_pages]
        order = torch.randperm(n_pages, generator=g, device=dev).tolist()
        table, refs = [], [0] * n_pages
        for b, n in enumerate(lens):
            have = -(-n // ps)
            shared = []
            if b % 4:  # its first pages are those of the request before it
                prefix = min(lens[b - 1], n) // ps // 2
                shared = table[-1][:prefix]
            row = shared + [order.pop() for _ in range(have - len(shared))]
            for page in row:
                refs[page] += 1
            table.append(row + [-1] * (columns - have))
        s["table"], s["refs"] = ints(table), ints(refs)
        s["table_out"], s["refs_out"] = torch.zeros_like(s["table"]), torch.zeros_like(s["refs"])
        s["count"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if op == "fork":
            # most requests go on by themselves, some from another one, some end, some give drafts back
            parent = [b if rnd.random() < 0.5 else rnd.randrange(B) if rnd.random() < 0.9 else -1 for b in range(B)]
            s["parent"] = ints(parent)
            s["rows"] = ints([max(0, lens[p] - rnd.choice([0, 0, 0, 1, 3, ps])) if p >= 0 else 0 for p in parent])
            s["d_pos_out"] = torch.zeros_like(s["d_pos"])
        return s
    extra = case["N"] if op == "append" else case["Q"]
    need = [-(-(n + extra) // ps) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    table = [[order.pop() for _ in range(k)] + [-1] * (max(need) - k) for k in need]
    s["table"] = ints(table)
    s["n_tokens"] = ints(_tokens(case, extra))
    if op == "append":
        N, H = case["N"], case["H"]
        s["pages"] = torch.zeros(n_pages, ps, ROW_BYTES, device=dev, dtype=torch.uint8)
        s["positions"] = s["d_pos"][:, None] + torch.arange(N, device=dev, dtype=torch.int32)
        s["q_proj"] = normal(B, N, H, 192)              # [q_nope | q_rope] of the query projection
        channel = torch.exp(0.5 * normal(ROW, dtype=torch.float32))   # channels of unlike size, as projections have
        s["kv_proj"] = (normal(B, N, ROW, dtype=torch.float32) * channel).to(torch.bfloat16)
        s["q"] = torch.zeros(B, N, H, ROW, device=dev, dtype=torch.bfloat16)
        for name, n in (("c_norm", LATENT), ("k_norm", ROPE), ("q_norm", ROPE)):
            s[name] = (1 + 0.2 * normal(n, dtype=torch.float32)).to(torch.bfloat16) if case["norms"] else None
        s["inv_freq"] = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device=dev) * 2 / ROPE)
        s["values"] = torch.zeros(B, N, ROW, device=dev, dtype=torch.bfloat16)
        return s
    Q, H = case["Q"], case["H"]
    s["pages"] = torch.empty(n_pages, ps, ROW_BYTES, device=dev, dtype=torch.uint8)
    each = max(1, 131072 // ps)
    for p0 in range(0, n_pages, each):
        part = s["pages"][p0:p0 + each]
        part[..., :ROW_BYTES - 2 * ROPE] = _quantise(normal(*part.shape[:2], LATENT, dtype=torch.float32), case["kv_scale"])
        part[..., ROW_BYTES - 2 * ROPE:] = normal(*part.shape[:2], ROPE).view(torch.uint8)
    gain = 0.25 + 2.0 * torch.rand(1, 1, H, 1, generator=g, device=dev)     # flat heads and peaked ones
    s["q"] = (normal(B, Q, H, ROW).float() * gain).to(torch.bfloat16)
    s["out"] = torch.zeros(B, Q, H, LATENT, device=dev, dtype=torch.bfloat16)
    s["lse"] = torch.zeros(B, Q, H, device=dev)
    return s


def _run_append(s):
    case = s["case"]
    ps, kv_scale = case["page_rows"], case["kv_scale"]
    ang = s["positions"].double()[..., None] * s["inv_freq"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def norm(x, weight, dtype):
        x = x.float()
        if weight is None:
            return x
        rstd = torch.rsqrt(x.to(dtype).square().mean(-1, keepdim=True) + EPS).float()
        return x * rstd * weight.float()

    def rotate(x, cos, sin):
        if case["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    N = s["positions"].shape[1]
    i = torch.arange(N, device=ang.device)
    here = i < s["n_tokens"][:, None]                                       # [B, N]
    q = rotate(norm(s["q_proj"][..., 128:], s["q_norm"], torch.float32), cos[:, :, None], sin[:, :, None])
    s["q"][..., LATENT:] = torch.where(here[..., None, None], q.to(torch.bfloat16), s["q"][..., LATENT:])
    # (the mean of squares in 64 bits: a value next to a border falls to one side)
    c = norm(s["kv_proj"][..., :LATENT], s["c_norm"], torch.float64)
    k = rotate(norm(s["kv_proj"][..., LATENT:], s["k_norm"], torch.float32), cos, sin).to(torch.bfloat16)
    new = torch.cat([_quantise(c, kv_scale), k.view(torch.uint8)], -1)
    t = s["d_pos"][:, None] + i
    page, at = s["table"].gather(1, (t // ps).long()), t % ps
    s["pages"][page, at] = torch.where(here[..., None], new, s["pages"][page, at])
    values = _row_values(s["pages"][page, at], kv_scale, torch.float32).to(torch.bfloat16)
    s["values"].copy_(torch.where(here[..., None], values, s["values"]))


def _rows_seen(s):
    """[B, T]: rows that some token of the request attends, and others."""
    case, d = s["case"], s["d_pos"][:, None]
    Q, window, sink = case["Q"], case["window"], case["sink"]
    dev = d.device
    if not window:
        return torch.arange(case["hi"] + Q, device=dev).expand(case["B"], -1)
    near = torch.clamp(d - window + 1, min=sink) + torch.arange(min(window, case["hi"]) + Q, device=dev)
    return torch.cat([torch.arange(sink, device=dev).expand(case["B"], -1), near], 1)


def _run_attend(s):
    case = s["case"]
    B, Q, H, ps, window, sink = (case[k] for k in ("B", "Q", "H", "page_rows", "window", "sink"))
    t = _rows_seen(s)
    page = s["table"].gather(1, (t // ps).clamp(max=s["table"].shape[1] - 1).long()).clamp(min=0)
    kv = _row_values(s["pages"][page, t % ps], case["kv_scale"], torch.float32)
    last = s["d_pos"][:, None] + torch.arange(Q, device=t.device)           # [B, Q]: the token's own row
    see = t[:, None] <= last[..., None]
    if window:
        see &= (t[:, None] > last[..., None] - window) | (t[:, None] < sink)
    x = torch.matmul(s["q"].float().view(B, Q * H, ROW), kv.transpose(1, 2)).view(B, Q, H, -1)
    x *= SCALE
    x.masked_fill_(~see[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, Q * H, -1), kv[..., :LATENT]).view(B, Q, H, LATENT) / total
    lse = (m + torch.log(total))[..., 0]
    here = (torch.arange(Q, device=t.device) < s["n_tokens"][:, None])[..., None]
    return torch.where(here[..., None], out.to(torch.bfloat16), s["out"]), torch.where(here, lse, s["lse"])


def _run_fork(s):
    case = s["case"]
    ps, reserve, window, sink, n_pages = (case[k] for k in ("page_rows", "reserve", "window", "sink", "pages"))
    B, columns = s["table"].shape
    dev = s["table"].device
    parent = s["parent"].long()
    goes_on = parent >= 0
    old = s["table"][parent.clamp(min=0)]
    n = torch.where(goes_on, torch.minimum(s["rows"], s["d_pos"][parent.clamp(min=0)]), 0)[:, None]
    p = torch.arange(columns, device=dev)
    b = torch.arange(B, device=dev)[:, None].expand(B, columns)
    full, last = (p + 1) * ps <= n, (p * ps < n) & ((p + 1) * ps > n)
    dropped = torch.zeros_like(full)
    if window:
        dropped = (p * ps >= sink) & ((p + 1) * ps <= n + 1 - window)
    valid = (old >= 0) & (old < n_pages)
    held = (full | last) & valid & ~dropped
    at = torch.where(held, old, n_pages).long().flatten()                    # (a page more for what is not held)
    frozen = torch.zeros(n_pages + 1, device=dev, dtype=torch.int32).scatter_add_(0, at, full.int().flatten()) > 0
    keeper = torch.full((n_pages + 1,), B, device=dev, dtype=torch.int64)
    keeper.scatter_reduce_(0, at, torch.where(last, b, B).flatten(), "amin")
    at = at.view(B, columns)
    copied = held & last & (frozen[at] | (keeper[at] != b))
    kept = held & ~copied
    need = copied | ((p * ps < n + reserve) & ~full & ~held & ~dropped & goes_on[:, None])
    refs = torch.zeros(n_pages + 1, device=dev, dtype=torch.int32)
    refs.scatter_add_(0, at.flatten(), kept.int().flatten())
    used = (refs[:n_pages] > 0).int()
    free, n_free = torch.argsort(used, stable=True), n_pages - used.sum()    # the free pages first, in order
    k = need.flatten().cumsum(0).view(B, columns) - 1
    gets = need & (k < n_free)
    fresh = torch.where(gets, free[k.clamp(0, n_pages - 1)], n_pages)
    table = torch.where(kept, old, torch.where(gets, fresh, -1).int())
    refs.scatter_add_(0, fresh.flatten(), gets.int().flatten())
    short = copied & ~gets
    # the copied rows of each request's last page
    r = torch.arange(ps, device=dev)
    moves = copied & gets
    src = torch.where(moves, at, 0).sum(1)
    dst = torch.where(moves.any(1), torch.where(moves, fresh, 0).sum(1), n_pages)
    rows = s["buffer"][src[:, None], r]
    to = torch.where(r < n % ps, dst[:, None], n_pages)
    s["buffer"][to, r] = rows
    return (table, torch.where(short.any(1), n[:, 0] // ps * ps, n[:, 0]), refs[:n_pages],
            (need.sum() - gets.sum()).int().view(1), s["pages"])


def _run_compact(s):
    n_pages = s["case"]["pages"]
    dev = s["table"].device
    used = s["refs"] > 0
    live = used.sum()
    page = torch.arange(n_pages, device=dev)
    hole, mover = (page < live) & ~used, (page >= live) & used
    # the k-th page behind the front goes to the k-th hole
    at = torch.full((n_pages + 1,), n_pages, device=dev, dtype=torch.int64)
    at.scatter_(0, torch.where(hole, hole.cumsum(0) - 1, n_pages), page)
    to = torch.where(mover, at[(mover.cumsum(0) - 1).clamp(min=0)], page)    # new number of each page in use
    refs = torch.where(page < live, s["refs"], 0)
    refs = torch.cat([refs, refs.new_zeros(1)]).scatter_(0, torch.where(mover, to, n_pages), s["refs"])[:n_pages]
    table = torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), -1)
    src = torch.nonzero(mover)[:, 0]
    s["buffer"][to[src]] = s["buffer"][src]
    return table, refs, live.int().view(1), s["pages"]


# The state's tensors whose addresses are in a call's arguments.
LAID_OUT = dict(
    append=itemgetter("positions", "q_proj", "q", "kv_proj", "pages", "table", "n_tokens", "d_pos", "values", "c_norm",
                      "k_norm", "q_norm"),
    attend=itemgetter("q", "pages", "table", "out", "lse", "n_tokens", "d_pos"),
    fork=itemgetter("pages", "table", "table_out", "d_pos", "d_pos_out", "refs_out", "count", "parent", "rows"),
    compact=itemgetter("pages", "table", "table_out", "refs", "refs_out", "count"))


def _own(s):
    """The calls a serving loop makes: arguments that stay the same are laid out once, and
    again if one of the state's tensors has been replaced by another."""
    import decode_attention_mla_gb300 as mla
    case, op = s["case"], s["case"]["op"]
    tensors = LAID_OUT[op](s)
    laid_out, h = s.get("handle", (tensors, None))
    if any(map(is_not, laid_out, tensors)):
        h = None
    if op == "append":
        if h is None:
            # (the base of every state's inv_freq)
            table = mla.rope_table(rot_dim=ROPE, base=10000.0, interleaved=case["interleaved"])
            a = mla.paged_append_make_args(
                table, s["positions"], q_rope=s["q_proj"][..., 128:], q=s["q"], c=s["kv_proj"][..., :LATENT],
                k_rope=s["kv_proj"][..., LATENT:], pages=s["pages"], page_table=s["table"], d_pos=s["d_pos"],
                n_tokens=s["n_tokens"], c_norm=s["c_norm"], k_norm=s["k_norm"], q_norm=s["q_norm"], eps=EPS,
                kv_scale=case["kv_scale"])
            r = mla.paged_read_make_args(s["values"], s["pages"], s["table"], first=s["d_pos"],
                                         n_rows=s["n_tokens"], kv_scale=case["kv_scale"])
            h = a, r
            s["handle"] = tensors, h
        mla.paged_append_args(h[0])
        mla.paged_read_args(h[1])
        return None
    if op == "attend":
        if h is None:
            plan = mla.paged_plan(batch=case["B"], tokens=case["Q"], heads=case["H"], scale=SCALE, pdl=True)
            args = mla.paged_make_args(s["q"], s["pages"], s["table"], s["out"], s["lse"], d_pos=s["d_pos"],
                                       n_tokens=s["n_tokens"], window=case["window"], sink=case["sink"],
                                       kv_scale=case["kv_scale"])
            h = plan, args, mla.paged_alloc_scratch(plan)
            s["handle"] = tensors, h
        mla.paged_forward_args(*h)
        return s["out"], s["lse"]
    if op == "fork":
        if h is None:
            args = mla.pages_fork_make_args(
                s["pages"], s["table"], s["d_pos"], s["refs_out"], parent=s["parent"], rows=s["rows"],
                reserve=case["reserve"], window=case["window"], sink=case["sink"], page_table_out=s["table_out"],
                d_pos_out=s["d_pos_out"], missing=s["count"])
            h = args, mla.pages_alloc_scratch(s["pages"], s["table"])
            s["handle"] = tensors, h
        mla.pages_fork_args(*h)
        return s["table_out"], s["d_pos_out"], s["refs_out"], s["count"], s["pages"]
    if h is None:
        args = mla.pages_compact_make_args(s["pages"], s["table"], s["refs"], page_table_out=s["table_out"],
                                           refs_out=s["refs_out"], used=s["count"])
        h = args, mla.pages_alloc_scratch(s["pages"], s["table"])
        s["handle"] = tensors, h
    mla.pages_compact_args(*h)
    return s["table_out"], s["refs_out"], s["count"], s["pages"]


def run(s):
    op = s["case"]["op"]
    if own:
        r = _own(s)
    else:
        r = {"append": _run_append, "attend": _run_attend, "fork": _run_fork, "compact": _run_compact}[op](s)
    return (s["q"][..., LATENT:], s["values"]) if op == "append" else r


def _rows_attended(case, d, n):
    """Rows that the n tokens behind d rows attend, and (token, row) pairs."""
    window, sink = case["window"], case["sink"]
    pairs, first = 0, d + n
    for i in range(n):
        r = d + i
        from_row = max(0, r + 1 - window) if window else 0
        pairs += r + 1 - from_row + min(sink, from_row)
        first = min(first, from_row)
    return d + n - first + min(sink, first), pairs


def work(case):
    B, op, ps = case["B"], case["op"], case["page_rows"]
    lens = _lengths(case)
    if op == "append":
        n = sum(_tokens(case, case["N"]))
        return {"bytes": n * (case["H"] * 2 * 2 * ROPE + 2 * ROW + ROW_BYTES + 4 + ROW_BYTES + 2 * ROW) + B * 8,
                "flops": n * (9 * LATENT + 10 * ROPE * (case["H"] + 1))}
    if op == "attend":
        H, bytes_, pairs = case["H"], 0, 0
        for d, n in zip(lens, _tokens(case, case["Q"])):
            rows, seen = _rows_attended(case, d, n)
            bytes_ += rows * ROW_BYTES + 4 * (rows // ps + 1) + n * H * (2 * ROW + 2 * LATENT + 4)
            pairs += seen * H
        return {"bytes": bytes_, "flops": pairs * 2 * (ROW + LATENT)}
    row = ROW_BYTES if case["kind"] == "q4" else 2 * ROW
    columns = (case["hi"] + case.get("reserve", 0)) // ps + 2
    if op == "fork":
        # tables read and written, references written, about a third of the requests copies half a page
        return {"bytes": B * columns * 8 + case["pages"] * 4 + B // 3 * ps * row, "flops": 0}
    held = [-(-n // ps) for n in lens]
    live = sum(k - (min(lens[b - 1], lens[b]) // ps // 2 if b % 4 else 0) for b, k in enumerate(held))
    moved = live * (1 - live / case["pages"])
    return {"bytes": B * columns * 8 + case["pages"] * 8 + moved * 2 * ps * row, "flops": 0}


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None                                     # whole numbers and bytes that are moved
    s = prepare(case, seed)
    ps, kv_scale = case["page_rows"], case["kv_scale"]
    lens, table = s["d_pos"].tolist(), s["table"].long()
    step = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    if op == "append":
        n = s["n_tokens"].tolist()
        out, rows = s["q"][..., LATENT:].double(), s["values"].double()
        pair = torch.arange(ROPE // 2, device="cuda")
        first = 2 * pair if case["interleaved"] else pair
        second = first + (1 if case["interleaved"] else ROPE // 2)

        def normed(x, weight):
            return x if weight is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()

        for b in range(case["B"]):
            turn = s["positions"][b, :n[b], None, None].double() * s["inv_freq"]
            unit = torch.polar(torch.ones_like(turn), turn)
            for x, dst in ((normed(s["q_proj"][b, :n[b], :, 128:].double(), s["q_norm"]), out[b, :n[b]]),
                           (normed(s["kv_proj"][b, :n[b], None, LATENT:].double(), s["k_norm"]), rows[b, :n[b], None, LATENT:])):
                z = torch.complex(x[..., first], x[..., second]) * unit
                dst[..., first], dst[..., second] = z.real, z.imag
            c = normed(s["kv_proj"][b, :n[b], :LATENT].double(), s["c_norm"]).view(n[b], -1, BLOCK)
            # (64-bit values go to E4M3 through 32 bits)
            scale = (c.abs().max(-1).values / (6 * kv_scale)).clamp(max=448).float().to(torch.float8_e4m3fn).double()
            scale = scale[..., None] * kv_scale
            unit = torch.where(scale > 0, c / scale, 0)
            positive = step[:8]
            middle = (positive[1:] + positive[:-1]) / 2
            up = torch.bucketize(unit.abs(), middle)                        # halfway: down
            up += ((unit.abs() == middle[up.clamp(max=6)]) & (up % 2 == 1)).long()   # to the even one
            rows[b, :n[b], :LATENT] = (positive[up] * unit.sign() * scale).flatten(-2)
        return [out, rows]
    n, H = s["n_tokens"].tolist(), case["H"]
    window, sink = case["window"], case["sink"]
    if sum(d + k for d, k in zip(lens, n)) * max(n) * H * 2 * (ROW + LATENT) > 4e12:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(case["B"]):
        last = lens[b] + n[b] - 1
        t = torch.arange(last + 1, device="cuda")
        if window:
            t = t[(t < sink) | (t > lens[b] - window)]
        raw = s["pages"][table[b, t // ps], t % ps]
        code = raw[:, :LATENT // 2].long()
        code = torch.stack([code % 16, code // 16], 2).view(len(t), LATENT // BLOCK, BLOCK)
        scale = raw[:, LATENT // 2:LATENT // 2 + LATENT // BLOCK].contiguous().view(torch.float8_e4m3fn).double()
        c = (step[code] * (scale * kv_scale)[:, :, None]).view(len(t), LATENT)
        kv = torch.cat([c, raw[:, -2 * ROPE:].contiguous().view(torch.bfloat16).double()], 1)
        for i in range(n[b]):
            at = t[:, None].T
            x = s["q"][b, i].double() @ kv.T * SCALE
            hidden = at > lens[b] + i
            if window:
                hidden |= (at <= lens[b] + i - window) & (at >= sink)
            x = x.masked_fill(hidden, -math.inf)
            lse[b, i] = torch.logsumexp(x, -1)
            out[b, i] = torch.exp(x - lse[b, i, :, None]) @ c
    return [out, lse]
