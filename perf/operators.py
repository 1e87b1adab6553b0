"""Measured cases of the operators around a latent (MLA) cache: drafted tokens
verified as a tree, the rotation that writes their rows, the accepted path's
commit, and eviction by accumulated attention weight.

A cache row is [c (512) | k_rope (64)] in bf16 (or E4M3 bytes); a query is
[q_lat (512) | q_rope (64)] per head.  Request b's rows start at row_offset[b];
d_pos[b] rows of it are committed, and drafted token j stands in row d_pos[b] + j.

  rope     q_rope and k_rope rotated by their positions, the new rows written
           to the cache behind each request's committed rows
  tree     every drafted token attends the committed rows and the drafted rows
           that its mask names (its ancestors and itself)
  commit   the accepted path's rows moved together behind the committed rows
  weights  w[row] = decay * w[row] + the attention weight that the row got from
           every token and head of the call
  evict    the rows of largest weight kept (the first positions and the last
           ones always), the holes below `keep` filled from behind

`run` computes them in elementary torch operations, or with `own` through
decode_attention_mla_gb300.
"""
import math
import random
from operator import is_not, itemgetter

import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
SCALE = 1.0 / math.sqrt(ROW)
LARGEST_SCORES = 8192 * 65600       # tokens * heads * rows of the largest tree
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one decode step of a tensor-parallel rank: 16 heads, one new token
        dict(name="rope_step", op="rope", B=1, N=1, H=16, lo=8191, hi=8191, ragged=False, interleaved=True,
             rot=64, yarn=False, kv8=False),
        # prefill chunks of four requests on all heads, long-context scaling, E4M3 cache
        dict(name="rope_prefill", op="rope", B=4, N=2048, H=128, lo=2048, hi=100000, ragged=True,
             interleaved=False, rot=64, yarn=True, kv8=True),
        # eight drafted tokens after a short prompt: latency
        dict(name="tree_small", op="tree", B=1, Q=8, H=16, lo=248, hi=248, ragged=False),
        # sixteen drafted tokens over a long cache on a 16-head rank: the cache's bytes
        dict(name="tree_long", op="tree", B=1, Q=16, H=16, lo=131072, hi=131072, ragged=False),
        # a serving batch, ragged lengths and drafts, all heads
        dict(name="tree_batch", op="tree", B=16, Q=5, H=128, lo=4096, hi=32768, ragged=True),
        # the widest tree on all heads over a long cache: the tensor cores
        dict(name="tree_wide", op="tree", B=1, Q=64, H=128, lo=65536, hi=65536, ragged=False),
        # the accepted path of one request
        dict(name="commit_one", op="commit", B=1, Q=8, lo=8192, hi=8192),
        # the accepted paths of a batch of wide trees
        dict(name="commit_batch", op="commit", B=64, Q=64, lo=1000, hi=5000),
        # one decode step's weights on a 16-head rank
        dict(name="weights_step", op="weights", B=1, Q=1, H=16, lo=8191, hi=8191, ragged=False, decay=1.0),
        # two-token steps of a ragged batch over long caches, all heads
        dict(name="weights_batch", op="weights", B=8, Q=2, H=128, lo=8192, hi=131072, ragged=True, decay=0.96875),
        # half of one request's cache
        dict(name="evict_one", op="evict", B=1, lo=8192, hi=8192, keep=4096, sink=4, recent=256),
        # a ragged batch of long caches down to one budget; some requests are below it
        dict(name="evict_batch", op="evict", B=16, lo=16384, hi=131072, keep=32768, sink=4, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "commit", "weights", "evict"])
    H = rng.choice([16, 32, 64, 128])
    B = _log_int(rng, 1, 16)
    if op == "rope":
        N = _log_int(rng, 1, max(1, 8192 * 128 // (B * H * 2)))
        N = min(N, 4096)
        lo = rng.randint(0, 2000)
        return dict(op=op, B=B, N=N, H=H, lo=lo, hi=lo + _log_int(rng, 1, 30000), ragged=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, rot=rng.choice([16, 32, 48, 64, 64, 64]),
                    yarn=rng.random() < 0.5, kv8=rng.random() < 0.3)
    if op == "commit":
        lo = rng.randint(0, 3000)
        return dict(op=op, B=_log_int(rng, 1, 64), Q=rng.randint(1, 64), lo=lo, hi=lo + _log_int(rng, 1, 2000))
    if op == "evict":
        hi = _log_int(rng, 200, 131072)
        lo = rng.randint(hi // 8, hi)
        sink = rng.randint(0, 8)
        recent = rng.randint(0, hi // 16)
        return dict(op=op, B=B, lo=lo, hi=hi, keep=rng.randint(hi // 8 + 1, hi), sink=sink, recent=recent)
    Q = rng.randint(1, 64) if op == "tree" else rng.randint(1, 8)
    most = 131072 if op == "tree" else 65536
    top = int(min(most, LARGEST_SCORES / (B * Q * H), 600000 / B))
    if op == "weights":
        top = int(min(top, 4 * LARGEST_SCORES / (B * 256 * 16)))
    hi = _log_int(rng, 16, max(17, top - 64))
    lo = rng.randint(0, hi)
    case = dict(op=op, B=B, Q=Q, H=H, lo=lo, hi=hi, ragged=rng.random() < 0.5)
    if op == "weights":
        case["decay"] = rng.choice([0.0, 0.5, 0.9375, 1.0])
    return case


def _lengths(case):
    """Committed rows per request: spread over [lo, hi], the first request at hi."""
    lo, hi = case["lo"], case["hi"]
    return [hi - int((hi - lo) * ((b * GOLDEN) % 1.0)) for b in range(case["B"])]


def _tokens(case, n):
    """Tokens per request: n, or ragged ones in 1..n."""
    if not case.get("ragged"):
        return [n] * case["B"]
    return [n - int((n - 1) * ((b * GOLDEN) % 1.0)) for b in range(case["B"])]


def _tree_masks(rnd, B, Q):
    """Ancestor bits (itself included) of random trees, as signed 64-bit words."""
    words = []
    for _ in range(B):
        bits = []
        for i in range(Q):
            parent = rnd.randint(max(-1, i - 8), i - 1)
            bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
        words.append([w - (1 << 64) if w >> 63 else w for w in bits])
    return torch.tensor(words, dtype=torch.int64)


def _inv_freq(case):
    """Angle per position of each pair, in 64 bits, as the user's configuration gives it."""
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) * 2 / case["rot"])
    if not case["yarn"]:
        return f, 1.0
    edge = [case["rot"] * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(10000.0)) for r in (32.0, 1.0)]
    low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), case["rot"] - 1)
    ramp = ((torch.arange(half, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / 40.0 * ramp + f * (1 - ramp), 0.1 * math.log(40.0) + 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rnd = random.Random(int(seed))
    B, op, dev = case["B"], case["op"], "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    lens = _lengths(case)
    extra = case["N"] if op == "rope" else case.get("Q", 0)
    room = [n + extra for n in lens]
    offs = [0]
    for r in room[:-1]:
        offs.append(offs[-1] + r)
    s = dict(case=case, d_pos=ints(lens), row_offset=ints(offs, torch.int64), rows=offs[-1] + room[-1],
             longest=max(lens) + extra)
    if op == "rope":
        N, H = case["N"], case["H"]
        n = _tokens(case, N)
        s["n_tokens"] = ints(n)
        s["positions"] = s["d_pos"][:, None] + torch.arange(N, device=dev, dtype=torch.int32)
        s["q_proj"] = normal(B, N, H, 192)             # [q_nope | q_rope] of the query projection
        s["kv_proj"] = normal(B, N, ROW)               # [c | k_rope] of the latent projection
        s["q"] = torch.zeros(B, N, H, ROW, device=dev, dtype=torch.bfloat16)
        s["kv"] = torch.zeros(s["rows"], ROW, device=dev, dtype=torch.uint8 if case["kv8"] else torch.bfloat16)
        f, s["amplitude"] = _inv_freq(case)
        s["inv_freq"] = f.to(dev)
        s["kv_scale"] = 0.03125 if case["kv8"] else 1.0
    elif op in ("tree", "weights"):
        Q, H = case["Q"], case["H"]
        gain = 0.25 + 2.0 * torch.rand(1, 1, H, 1, generator=g, device=dev)     # flat heads and peaked ones
        s["q"] = (normal(B, Q, H, ROW).float() * gain).to(torch.bfloat16)
        s["kv"] = normal(s["rows"], ROW)
        s["mask"] = _tree_masks(rnd, B, Q).to(dev)
        s["n_tokens"] = ints(_tokens(case, Q))
        if op == "tree":
            s["out"] = torch.zeros(B, Q, H, LATENT, device=dev, dtype=torch.bfloat16)
            s["lse"] = torch.zeros(B, Q, H, device=dev)
        else:
            # the attention's own log-sum-exp, which a step has before it asks for the weights
            s["lse"] = torch.cat([_scores(s, b0, b0 + 1)[1] for b0 in range(B)])
            s["weights"] = torch.rand(s["rows"], generator=g, device=dev)
    elif op == "commit":
        Q = case["Q"]
        s["kv"] = normal(s["rows"], ROW)
        paths, counts = [], []
        for _ in range(B):
            k = rnd.randint(0, Q)
            path = sorted(rnd.sample(range(Q), k))
            paths.append(path + [0] * (Q - k))
            counts.append(k)
        s["accept"], s["n_accept"] = ints(paths), ints(counts)
        s["d_pos_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    else:
        s["kv"] = normal(s["rows"], ROW)
        # heavy-tailed sums, many rows that got next to nothing, some ties
        w = torch.rand(s["rows"], generator=g, device=dev).pow(-0.5) - 1
        s["weights"] = torch.where(torch.rand(s["rows"], generator=g, device=dev) < 0.1, torch.zeros_like(w), w)
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in room])
        s["positions"] = pos.to(dev)
        s["next_pos"] = s["d_pos"].clone()
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["positions_out"] = torch.zeros_like(s["positions"])
        s["d_pos_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


def _visible(s, b0, b1, T):
    """[b, Q, T]: whether token i of request b attends row t."""
    d = s["d_pos"][b0:b1, None, None].long()
    Q = s["mask"].shape[1]
    t = torch.arange(T, device=d.device)
    j = t - d                                                   # [b, 1, T]
    drafted = (j >= 0) & (j < s["n_tokens"][b0:b1, None, None])
    bit = (s["mask"][b0:b1, :, None] >> j.clamp(0, Q - 1)) & 1  # [b, Q, T]
    return (t < d) | (drafted & (bit != 0))


def _scores(s, b0, b1):
    """Masked scores [b, Q, H, T], their log-sum-exp and the rows, of requests b0 .. b1."""
    q = s["q"][b0:b1].float()
    b, Q, H, _ = q.shape
    T = s["longest"]
    rows = s["row_offset"][b0:b1, None] + torch.arange(T, device=q.device)
    kv = s["kv"][rows.clamp(max=s["rows"] - 1)].float()
    x = torch.matmul(q.reshape(b, Q * H, ROW), kv.transpose(1, 2)).view(b, Q, H, T)
    x *= SCALE
    x.masked_fill_(~_visible(s, b0, b1, T)[:, :, None, :], -math.inf)
    m = x.amax(-1)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    lse = torch.log(torch.exp(x - m[..., None]).sum(-1)) + m
    return x, lse, kv


def _run_rope(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    ang = s["positions"].double()[..., None] * s["inv_freq"]
    cos, sin = (s["amplitude"] * torch.cos(ang)).float(), (s["amplitude"] * torch.sin(ang)).float()

    def rotate(x, cos, sin):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    N = s["positions"].shape[1]
    here = torch.arange(N, device=ang.device) < s["n_tokens"][:, None]      # [B, N]
    q_rope = rotate(s["q_proj"][..., 128:], cos[:, :, None], sin[:, :, None]).to(torch.bfloat16)
    s["q"][..., LATENT:] = torch.where(here[..., None, None], q_rope, s["q"][..., LATENT:])
    new = torch.cat([s["kv_proj"][..., :LATENT].float(), rotate(s["kv_proj"][..., LATENT:], cos, sin)], -1)
    if case["kv8"]:
        new = (new / s["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        new = new.to(torch.bfloat16)
    rows = s["row_offset"][:, None] + s["d_pos"][:, None] + torch.arange(N, device=ang.device)
    s["kv"][rows] = torch.where(here[..., None], new, s["kv"][rows])


def _run_tree(s):
    x, lse, kv = _scores(s, 0, s["q"].shape[0])
    b, Q, H, T = x.shape
    x = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    out = torch.matmul(x.view(b, Q * H, T), kv[..., :LATENT]).view(b, Q, H, LATENT)
    here = (torch.arange(Q, device=out.device) < s["n_tokens"][:, None])[..., None]
    return (torch.where(here[..., None], out.to(torch.bfloat16), s["out"]),
            torch.where(here, lse, s["lse"]))


def _run_commit(s):
    Q = s["accept"].shape[1]
    k = torch.arange(Q, device=s["kv"].device)
    first = (s["row_offset"] + s["d_pos"])[:, None]
    here = k < s["n_accept"][:, None]
    s["kv"][first + k] = s["kv"][first + torch.where(here, s["accept"].long(), k)]
    return s["kv"], s["d_pos"] + s["n_accept"]


def _run_weights(s):
    x, _, _ = _scores(s, 0, s["q"].shape[0])
    b, Q, H, T = x.shape
    here = (torch.arange(Q, device=x.device) < s["n_tokens"][:, None])[:, :, None, None]
    x = torch.where(here, torch.exp(x - s["lse"][..., None]), torch.zeros_like(x))
    got = x.sum((1, 2))                                                     # [b, T]
    t = torch.arange(T, device=x.device)
    mine = t < (s["d_pos"] + s["n_tokens"])[:, None]
    rows = (s["row_offset"][:, None] + t).clamp(max=s["rows"] - 1)
    add = torch.zeros_like(s["weights"]).scatter_add_(0, rows.flatten(), torch.where(mine, got, 0).flatten())
    touched = torch.zeros_like(s["weights"]).scatter_add_(0, rows.flatten(), mine.float().flatten()) > 0
    decay = s["case"]["decay"]
    s["weights"].copy_(torch.where(touched, decay * s["weights"] + add, s["weights"]))


def _run_evict(s):
    case = s["case"]
    T, rows_all = s["longest"], s["rows"]
    t = torch.arange(T, device=s["kv"].device)
    n = s["d_pos"][:, None]
    keep = n.clamp(max=case["keep"])
    rows = (s["row_offset"][:, None] + t).clamp(max=rows_all - 1)           # [B, T]
    w, pos = s["weights"][rows], s["positions"][rows]
    fixed = (pos < case["sink"]) | (pos >= s["next_pos"][:, None] - case["recent"])
    rank_by = torch.where(fixed, torch.full_like(w, math.inf), w)
    rank_by = torch.where(t < n, rank_by, torch.full_like(w, -math.inf))
    order = torch.sort(rank_by, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, t.expand_as(order))
    kept = (rank < keep) & (t < n)
    hole, moved = (t < keep) & ~kept, (t >= keep) & kept
    # the k-th moved row of a request goes to its k-th hole
    at = torch.zeros(rows.shape[0], T + 1, dtype=torch.int64, device=t.device)
    at.scatter_(1, torch.where(moved, moved.cumsum(1) - 1, T), t.expand_as(rows))
    src = torch.where(hole, at.gather(1, (hole.cumsum(1) - 1).clamp(min=0)), t)
    src = s["row_offset"][:, None] + src
    live = t < keep
    to = rows[live]
    src = src[live]
    s["weights_out"][to] = s["weights"][src]
    s["positions_out"][to] = s["positions"][src]
    s["kv"][to] = s["kv"][src]
    return s["kv"], s["weights_out"], s["positions_out"], keep[:, 0]


# The state's tensors whose addresses are in a call's arguments.
LAID_OUT = dict(
    rope=itemgetter("positions", "q_proj", "q", "kv_proj", "kv", "n_tokens", "d_pos", "row_offset"),
    tree=itemgetter("q", "kv", "out", "lse", "mask", "n_tokens", "d_pos", "row_offset"),
    weights=itemgetter("q", "kv", "lse", "mask", "n_tokens", "d_pos", "row_offset"),
    evict=itemgetter("kv", "weights", "positions", "next_pos", "weights_out", "positions_out", "d_pos_out", "d_pos",
                     "row_offset"))


def _own(s):
    """The calls a serving loop makes: arguments that stay the same are laid out once, and
    again if one of the state's tensors has been replaced by another."""
    import decode_attention_mla_gb300 as mla
    case, op, h = s["case"], s["case"]["op"], None
    if op != "commit":
        tensors = LAID_OUT[op](s)
        laid_out, h = s.get("handle", (tensors, None))
        if any(map(is_not, laid_out, tensors)):
            h = None
    common = dict(d_pos=s["d_pos"], row_offset=s["row_offset"])
    if op == "rope":
        if h is None:
            yarn = dict(scaling="yarn", factor=40.0, original_ctx=4096, amplitude=s["amplitude"])
            table = mla.rope_table(rot_dim=case["rot"], base=10000.0, interleaved=case["interleaved"],
                                   **(yarn if case["yarn"] else {}))
            h = mla.rope_make_args(
                table, s["positions"], q_rope=s["q_proj"][..., 128:], q=s["q"], c=s["kv_proj"][..., :LATENT],
                k_rope=s["kv_proj"][..., LATENT:], kv=s["kv"], n_tokens=s["n_tokens"], kv_scale=s["kv_scale"],
                **common)
            s["handle"] = tensors, h
        mla.rope_append_args(h)
        return None
    if op in ("tree", "weights"):
        if h is None:
            plan = mla.tree_plan(batch=case["B"], tokens=case["Q"], heads=case["H"], scale=SCALE, pdl=True)
            args = mla.tree_make_args(s["q"], s["kv"], s.get("out"), s["lse"], mask=s["mask"],
                                      n_tokens=s["n_tokens"], **common)
            h = plan, args, mla.tree_alloc_scratch(plan)
            s["handle"] = tensors, h
        if op == "tree":
            mla.tree_forward_args(*h)
            return s["out"], s["lse"]
        mla.tree_weights_args(*h, s["weights"], decay=case["decay"])
        return None
    if op == "commit":
        mla.tree_commit(s["kv"], s["accept"], s["n_accept"], d_pos_out=s["d_pos_out"], **common)
        return s["kv"], s["d_pos_out"]
    if h is None:
        args = mla.evict_make_args(
            s["kv"], s["weights"], s["positions"], next_pos=s["next_pos"], keep=case["keep"], sink=case["sink"],
            recent=case["recent"], max_rows=case["hi"], weights_out=s["weights_out"],
            positions_out=s["positions_out"], d_pos_out=s["d_pos_out"], **common)
        h = args, mla.evict_alloc_scratch(batch=case["B"], keep=case["keep"])
        s["handle"] = tensors, h
    mla.evict_args(*h)
    return s["kv"], s["weights_out"], s["positions_out"], s["d_pos_out"]


def run(s):
    op = s["case"]["op"]
    if own:
        r = _own(s)
    else:
        r = {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit, "weights": _run_weights,
             "evict": _run_evict}[op](s)
    if op == "rope":
        kv = s["kv"].view(torch.float8_e4m3fn) if s["case"]["kv8"] else s["kv"]
        return s["q"][..., LATENT:], kv
    if op == "weights":
        return s["weights"]
    return r


def work(case):
    B, op = case["B"], case["op"]
    lens = _lengths(case)
    if op == "rope":
        n = sum(_tokens(case, case["N"]))
        row = ROW if case["kv8"] else 2 * ROW
        pairs = case["rot"] // 2
        return {"bytes": n * (case["H"] * 64 * 4 + 2 * ROW + row + 4) + B * 16,
                "flops": n * 6 * pairs * (case["H"] + 1) + n * pairs * 20}
    if op in ("tree", "weights"):
        n = _tokens(case, case["Q"])
        H = case["H"]
        rows = sum(d + k for d, k in zip(lens, n))
        pairs = sum((d + k) * k * H for d, k in zip(lens, n))
        q = sum(n) * H
        if op == "tree":
            return {"bytes": rows * 2 * ROW + q * (2 * ROW + 2 * LATENT + 4), "flops": pairs * 2 * (ROW + LATENT)}
        return {"bytes": rows * (2 * ROW + (8 if case["decay"] else 4)) + q * (2 * ROW + 4), "flops": pairs * 2 * ROW}
    if op == "commit":
        moved = sum((case["Q"] + 1) / 2 for _ in lens) * 0.9      # paths of 0 .. Q tokens, some already in place
        return {"bytes": moved * 4 * ROW + B * (8 + 4 * case["Q"]), "flops": 0}
    moved = sum(min(n, case["keep"]) * (1 - case["keep"] / n) for n in lens if n > case["keep"])
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": sum(lens) * 8 + kept * 8 + moved * 4 * ROW, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    lens, offs = s["d_pos"].tolist(), s["row_offset"].tolist()
    if op == "commit":
        kv = s["kv"].clone()
        for b, (path, k) in enumerate(zip(s["accept"].tolist(), s["n_accept"].tolist())):
            at = offs[b] + lens[b]
            for i in range(k):
                kv[at + i] = s["kv"][at + path[i]]
        return [kv, torch.tensor([d + k for d, k in zip(lens, s["n_accept"].tolist())], dtype=torch.int32)]
    if op == "evict":
        wo, po = s["weights_out"].double(), s["positions_out"].clone()
        kept_rows = []
        for b in range(B):
            n, keep = lens[b], min(lens[b], case["keep"])
            w = s["weights"][offs[b]:offs[b] + n].double().cpu()
            pos = s["positions"][offs[b]:offs[b] + n].cpu()
            fixed = (pos < case["sink"]) | (pos >= int(s["next_pos"][b]) - case["recent"])
            value = [(-math.inf if f else -v, t) for t, (v, f) in enumerate(zip(w.tolist(), fixed.tolist()))]
            stays = sorted(t for _, t in sorted(value)[:keep])
            low, behind = {t for t in stays if t < keep}, iter([t for t in stays if t >= keep])
            src = torch.tensor([t if t in low else next(behind) for t in range(keep)], dtype=torch.int64)
            wo[offs[b]:offs[b] + keep] = w[src].to(wo)
            po[offs[b]:offs[b] + keep] = pos[src].to(po)
            kept_rows.append(keep)
        return [None, wo, po, torch.tensor(kept_rows, dtype=torch.int32)]
    if op == "rope":
        n = s["n_tokens"].tolist()
        out, kv = s["q"][..., LATENT:].double(), torch.zeros(s["rows"], ROW, dtype=torch.float64, device="cuda")
        pair = torch.arange(case["rot"] // 2, device="cuda")
        first = 2 * pair if case["interleaved"] else pair
        second = first + (1 if case["interleaved"] else case["rot"] // 2)
        for b in range(B):
            turn = s["positions"][b, :n[b], None].double() * s["inv_freq"]
            unit = s["amplitude"] * torch.polar(torch.ones_like(turn), turn)
            for src, dst in ((s["q_proj"][b, :n[b], :, 128:].double(), "q"), (s["kv_proj"][b, :n[b], None, LATENT:].double(), "k")):
                z = torch.complex(src[..., first], src[..., second]) * unit[:, None]
                y = src.clone()
                y[..., first], y[..., second] = z.real, z.imag
                if dst == "q":
                    out[b, :n[b]] = y
                else:
                    at = offs[b] + lens[b]
                    kv[at:at + n[b], :LATENT] = s["kv_proj"][b, :n[b], :LATENT].double()
                    kv[at:at + n[b], LATENT:] = y[:, 0]
        return [out, (kv / s["kv_scale"]).clamp(-448, 448) if case["kv8"] else kv]
    # tree and weights: one request and a block of query rows at a time
    n, Q, H = s["n_tokens"].tolist(), case["Q"], case["H"]
    if sum((d + k) * k * H for d, k in zip(lens, n)) * 2 * (ROW + LATENT) > 4e12:
        return None
    masks = s["mask"].tolist()
    if op == "tree":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        w = s["weights"].double()
    for b in range(B):
        T = lens[b] + n[b]
        kv = s["kv"][offs[b]:offs[b] + T].double()
        got = torch.zeros(T, dtype=torch.float64, device="cuda")
        block = max(1, int(5e8 / (T * H)))
        for i0 in range(0, n[b], block):
            i1 = min(n[b], i0 + block)
            see = torch.ones(i1 - i0, T, dtype=torch.bool)
            for i in range(i0, i1):
                see[i - i0, lens[b]:] = torch.tensor([bool(masks[b][i] >> j & 1) for j in range(n[b])])
            x = (s["q"][b, i0:i1].double().flatten(0, 1) @ kv.T).view(i1 - i0, H, T) * SCALE
            x[~see[:, None].expand(i1 - i0, H, T).to(x.device)] = -math.inf
            if op == "tree":
                l = torch.logsumexp(x, -1)
                p = torch.exp(x - l[..., None])
                out[b, i0:i1] = (p.flatten(0, 1) @ kv[:, :LATENT]).view(i1 - i0, H, LATENT)
                lse[b, i0:i1] = l
            else:
                got += torch.exp(x - s["lse"][b, i0:i1, :, None].double()).sum((0, 1))
        if op == "weights":
            at = slice(offs[b], offs[b] + T)
            w[at] = (case["decay"] * w[at] if case["decay"] else 0) + got
    return [out, lse] if op == "tree" else w
