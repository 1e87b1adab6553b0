"""The accepted path's commit (mla_tree_commit) and eviction by attention
weight (mla_evict), against plain forms; both move rows bit for bit."""
import math
import random

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref

pytestmark = pytest.mark.gpu
NAN = float("nan")


def ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device="cuda")


def cache(rows, fp8, stride, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fp8:
        return torch.randint(0, 256, (rows, stride), generator=g, device="cuda", dtype=torch.uint8)[:, :576]
    return torch.randint(-2 ** 15, 2 ** 15, (rows, stride), generator=g, device="cuda",
                         dtype=torch.int16).view(torch.bfloat16)[:, :576]


def raw(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


@pytest.mark.parametrize("fp8,stride", [(False, 576), (False, 584), (True, 576), (True, 640)])
@pytest.mark.parametrize("Q", [1, 3, 8, 64])
def test_commit_moves_the_path(Q, fp8, stride):
    rnd = random.Random(Q)
    B = 5
    lens = [0, 17, -1, 100, 5]
    offs, at = [], 2
    for n in lens:
        offs.append(at)
        at += max(n, 0) + Q
    rows = at - Q // 2                                       # the last request's drafts end outside the cache
    kv = cache(rows, fp8, stride)
    paths = [rnd.sample(range(Q), Q) for _ in range(B)]
    paths[1] = sorted(paths[1])
    paths[3] = [Q - 1] * Q                                   # the same draft twice and more
    if Q > 2:
        paths[0][1], paths[0][2] = -1, 64                    # no such draft
    counts = [rnd.randint(0, Q) for _ in range(B)]
    counts[3], counts[4] = Q, Q + 7                          # clamped
    pos, w = ints(list(range(rows))), torch.rand(rows, device="cuda")
    want, wp, ww = raw(kv).clone(), pos.clone(), w.clone()
    for b in range(B):
        for k in range(min(counts[b], Q)):
            j, at = paths[b][k], offs[b] + lens[b]
            if lens[b] >= 0 and 0 <= j < 64 and at + k < rows and at + j < rows:
                want[at + k], wp[at + k], ww[at + k] = raw(kv)[at + j], pos[at + j], w[at + j]
    d = ints(lens)
    mla.tree_commit(kv, ints(paths), ints(counts), d_pos=d, d_pos_out=d, row_offset=ints(offs, torch.int64),
                    row_positions=pos, row_weights=w)
    assert torch.equal(raw(kv), want) and torch.equal(pos, wp) and torch.equal(w, ww)
    assert d.tolist() == [n + min(c, Q) if n >= 0 else n for n, c in zip(lens, counts)]


def test_commit_without_advance_leaves_positions():
    kv = cache(40, False, 576)
    d = ints([10])
    mla.tree_commit(kv, ints([[0, 2]]), ints([2]), d_pos=d)
    assert d.tolist() == [10]


def reference(kv, w, p, lens, offs, keep, sink, recent, nxt):
    want, ww, wp = raw(kv).clone(), w.clone(), p.clone()
    wl, pl = w.tolist(), p.tolist()
    for b, n in enumerate(lens):
        o = offs[b]
        n = max(0, min(n, kv.shape[0] - o))
        src = ref.evict_rows(wl[o:o + n], pl[o:o + n], n, keep, sink, nxt[b] - recent)
        if src:
            s = torch.tensor(src, device="cuda") + o
            want[o:o + len(src)], ww[o:o + len(src)], wp[o:o + len(src)] = raw(kv)[s], w[s], p[s]
    return want, ww, wp


@pytest.mark.parametrize("fp8,stride", [(False, 576), (True, 592)])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([33], 32, 0, 0), ([64, 0, -1, 31, 32], 32, 2, 5), ([1000], 999, 4, 16),
    ([1000, 500, 1024, 1025], 100, 4, 32), ([5000, 8192, 8193], 4096, 0, 500), ([20000, 40000, 7], 3001, 4, 64),
    ([9000, 12000], 11000, 0, 0), ([3000], 50, 0, 3000), ([3000], 50, 3000, 0),
])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict_keeps_the_heaviest_rows(lens, keep, sink, recent, kind, fp8, stride):
    rnd = random.Random(len(lens) + keep)
    offs, at = [], 1
    for n in lens:
        offs.append(at)
        at += max(n, 0) + rnd.randint(0, 3)
    rows = at
    kv = cache(rows, fp8, stride, seed=keep)
    g = torch.Generator(device="cuda").manual_seed(keep)
    w = torch.rand(rows, generator=g, device="cuda").pow(-1.5)
    if kind == "ties":
        w = torch.randint(0, 3, (rows,), generator=g, device="cuda").float()
    elif kind == "special":
        at = torch.randint(0, 8, (rows,), generator=g, device="cuda")
        for k, v in enumerate([NAN, math.inf, -math.inf, -0.0, 0.0, -1.5, 1e-42]):
            w[at == k] = v
    p = torch.cat([torch.randperm(max(n, 0) + 4, device="cuda")[:max(n, 0)].int() for n in lens] +
                  [torch.zeros(rows, dtype=torch.int32, device="cuda")])[:rows].contiguous()
    nxt = [max(n, 0) for n in lens]
    want, ww, wp = reference(kv, w, p, lens, offs, keep, sink, recent, nxt)
    scratch = mla.evict_alloc_scratch(batch=len(lens), keep=keep)
    scratch.fill_(255)
    kv0, w0, p0 = raw(kv).clone(), w.clone(), p.clone()
    common = dict(next_pos=ints(nxt), keep=keep, sink=sink, recent=recent, row_offset=ints(offs, torch.int64))
    # out of place, with the sizes it expects
    wo, po, do = torch.full_like(w, 9), torch.full_like(p, 9), ints([9] * len(lens))
    mla.evict(kv, w, p, scratch, d_pos=ints(lens), weights_out=wo, positions_out=po, d_pos_out=do,
              max_rows=max(max(lens), 1), **common)
    assert torch.equal(raw(kv), want)
    kept = [min(max(n, 0), keep) for n in lens]
    assert do.tolist() == kept
    for o, k in zip(offs, kept):
        assert torch.equal(wo[o:o + k].view(torch.int32), ww[o:o + k].view(torch.int32))
        assert torch.equal(po[o:o + k], wp[o:o + k])
        wo[o:o + k], po[o:o + k] = 9, 9
    assert (wo == 9).all() and (po == 9).all()               # nothing else is written
    assert torch.equal(w.view(torch.int32), w0.view(torch.int32)) and torch.equal(p, p0)
    # in place, with a wrong expectation of the sizes
    raw_view = kv
    raw_view.copy_(kv0.view(kv.dtype))
    d = ints(lens)
    mla.evict(kv, w, p, scratch, d_pos=d, max_rows=1 if max(lens) > 9000 else rows + 100000, **common)
    assert torch.equal(raw(kv), want) and d.tolist() == kept
    for o, k in zip(offs, kept):
        assert torch.equal(w[o:o + k].view(torch.int32), ww[o:o + k].view(torch.int32))
        assert torch.equal(p[o:o + k], wp[o:o + k])


@pytest.mark.parametrize("n,keep", [(3000, 1100), (20000, 9000), (700, 800)])
@pytest.mark.parametrize("own_weights", [True, False])
def test_one_side_array_in_place_and_the_other_not(n, keep, own_weights):
    kv = cache(n + 2, False, 576)
    g = torch.Generator(device="cuda").manual_seed(n)
    w, p = torch.rand(n + 2, generator=g, device="cuda"), torch.randperm(n + 2, device="cuda").int()
    want, ww, wp = reference(kv, w, p, [n], [2], keep, 3, 20, [n])
    wo, po = (torch.full_like(w, 9), p) if own_weights else (w, torch.full_like(p, 9))
    d = ints([n])
    mla.evict(kv, w, p, mla.evict_alloc_scratch(batch=1, keep=keep), d_pos=d, next_pos=ints([n]), keep=keep, sink=3,
              recent=20, row_offset=ints([2], torch.int64), weights_out=wo, positions_out=po)
    k = min(n, keep)
    assert torch.equal(raw(kv), want) and d.tolist() == [k]
    assert torch.equal(wo[2:2 + k], ww[2:2 + k]) and torch.equal(po[2:2 + k], wp[2:2 + k])


def test_rows_behind_the_cache_are_no_rows():
    kv = cache(100, False, 576)
    w, p = torch.rand(100, device="cuda"), ints(list(range(100)))
    want, ww, _ = reference(kv, w, p, [500], [20], 30, 0, 0, [80])
    d = ints([500])
    mla.evict(kv, w, p, mla.evict_alloc_scratch(batch=1, keep=30), d_pos=d, next_pos=ints([80]), keep=30,
              row_offset=ints([20], torch.int64))
    assert torch.equal(raw(kv), want) and torch.equal(w, ww) and d.tolist() == [30]


def test_more_rows_than_the_select_holds_in_shared_memory():
    n = 300000
    kv = cache(n, True, 576)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 5000, (n,), generator=g, device="cuda").float()
    p = torch.arange(n, dtype=torch.int32, device="cuda")
    for expect in (n, 100):
        k, wk, pk, d = kv.clone(), w.clone(), p.clone(), ints([n])
        want, ww, wp = reference(k, w, p, [n], [0], 70001, 4, 1000, [n])
        mla.evict(k, wk, pk, mla.evict_alloc_scratch(batch=1, keep=70001), d_pos=d, next_pos=ints([n]), keep=70001,
                  sink=4, recent=1000, max_rows=expect)
        assert torch.equal(raw(k), want) and torch.equal(wk[:70001], ww[:70001]) and torch.equal(pk[:70001], wp[:70001])


@pytest.mark.parametrize("n,keep", [(3000, 1100), (20000, 9000)])
def test_captured_behind_copies(n, keep):
    # the launches may begin before the work ahead of them has ended: here copies that bring their inputs
    kv = cache(n, False, 576)
    g = torch.Generator(device="cuda").manual_seed(n)
    w, p = torch.rand(n, generator=g, device="cuda"), torch.randperm(n, device="cuda").int()
    want, ww, wp = reference(kv, w, p, [n - 2], [0], keep, 3, 20, [n])
    start = [t.clone() for t in (raw(kv), w, p)]
    d, path, two = ints([n - 2]), ints([[1, 0]]), ints([2])
    d0, nxt, scratch = ints([n - 2]), ints([n]), mla.evict_alloc_scratch(batch=1, keep=keep)
    side = dict(row_positions=p, row_weights=w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for t, s in zip((raw(kv), w, p), start):
            t.copy_(s)
        d.copy_(d0)
        mla.evict(kv, w, p, scratch, d_pos=d, next_pos=nxt, keep=keep, sink=3, recent=20)
        d -= 2
        mla.tree_commit(kv, path, two, d_pos=d, d_pos_out=d, **side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want[keep - 2:keep] = want[keep - 2:keep].flip(0)
    ww[keep - 2:keep], wp[keep - 2:keep] = ww[keep - 2:keep].flip(0), wp[keep - 2:keep].flip(0)
    assert torch.equal(raw(kv)[:keep], want[:keep]) and d.tolist() == [keep]
    assert torch.equal(w[:keep], ww[:keep]) and torch.equal(p[:keep], wp[:keep])


def test_two_evictions_at_once():
    runs = []
    for n, keep in ((30000, 9000), (12000, 5000)):
        kv = cache(n, False, 576, seed=n)
        g = torch.Generator(device="cuda").manual_seed(n)
        w, p = torch.rand(n, generator=g, device="cuda"), torch.randperm(n, device="cuda").int()
        want, ww, wp = reference(kv, w, p, [n], [0], keep, 4, 64, [n])
        runs.append((kv, w, p, ints([n]), ints([n]), keep, mla.evict_alloc_scratch(batch=1, keep=keep),
                     torch.cuda.Stream(), want, ww, wp))
    torch.cuda.synchronize()
    for kv, w, p, d, nxt, keep, scratch, s, *_ in runs:
        mla.evict(kv, w, p, scratch, d_pos=d, next_pos=nxt, keep=keep, sink=4, recent=64, stream=s)
    torch.cuda.synchronize()
    for kv, w, p, d, _, keep, _, _, want, ww, wp in runs:
        assert torch.equal(raw(kv), want) and d.tolist() == [keep]
        assert torch.equal(w[:keep], ww[:keep]) and torch.equal(p[:keep], wp[:keep])


@pytest.mark.parametrize("name", ["keep", "sink", "recent", "max_rows"])
def test_integers_past_32_bits_are_refused(name):
    kv, w, p, d = cache(40, False, 576), torch.rand(40, device="cuda"), ints(list(range(40))), ints([30])
    with pytest.raises(ValueError, match="32-bit"):
        mla.evict_make_args(kv, w, p, d_pos=d, next_pos=ints([30]), **{"keep": 20, name: 2 ** 32 + 5})


@pytest.mark.parametrize("n,keep", [(3000, 1100), (20000, 9000), (60, 90)])
def test_next_positions_in_the_tensor_that_is_rewritten(n, keep):
    """Before the first eviction the next position is the number of rows: one tensor may be both, in place."""
    kv = cache(n, False, 576)
    g = torch.Generator(device="cuda").manual_seed(n)
    w, p = torch.rand(n, generator=g, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    want, ww, wp = reference(kv, w, p, [n], [0], keep, 4, 50, [n])
    d = ints([n])
    mla.evict(kv, w, p, mla.evict_alloc_scratch(batch=1, keep=keep), d_pos=d, next_pos=d, keep=keep, sink=4, recent=50)
    k = min(n, keep)
    assert torch.equal(raw(kv), want) and d.tolist() == [k]
    assert torch.equal(w[:k], ww[:k]) and torch.equal(p[:k], wp[:k])
