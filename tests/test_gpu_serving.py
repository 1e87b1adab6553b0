"""The drafted-token operators together, as a serving loop uses them: rotate and
append the drafts, verify the tree, gather weights, commit the accepted path,
evict when the cache outgrows its budget, and decode on with the dense kernels.
Each step is checked against the plain form on the cache as it stood."""
import math
import random
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import decode_attention_mla_gb300 as mla
import _tree_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(576)


def ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device="cuda")


class Loop:
    B, Q, H, CAP, KEEP = 3, 6, 16, 80, 48

    def __init__(self, seed, out_dtype=torch.float32):
        B, Q, H, CAP = self.B, self.Q, self.H, self.CAP
        self.g = torch.Generator().manual_seed(seed)
        self.rnd = random.Random(seed)
        self.kv = torch.full((B * CAP, 576), float("nan"), device="cuda", dtype=torch.bfloat16)
        self.weights = torch.full((B * CAP,), float("nan"), device="cuda")
        self.positions = torch.full((B * CAP,), -1, device="cuda", dtype=torch.int32)
        self.offs = [b * CAP for b in range(B)]
        self.row_offset = ints(self.offs, torch.int64)
        self.d_pos, self.next_pos = ints([0] * B), ints([0] * B)
        self.table = mla.rope_table(64, scaling="yarn", factor=8.0)
        self.f = ref.inv_freq(64, 10000.0, "yarn", 8.0)
        self.q = torch.zeros(B, Q, H, 576, device="cuda", dtype=torch.bfloat16)
        self.q_rope = torch.zeros(B, Q, H, 64, device="cuda", dtype=torch.bfloat16)
        self.new = torch.zeros(B, Q, 576, device="cuda", dtype=torch.bfloat16)
        self.pos = torch.zeros(B, Q, device="cuda", dtype=torch.int32)
        self.mask = torch.zeros(B, Q, device="cuda", dtype=torch.int64)
        self.n = torch.zeros(B, device="cuda", dtype=torch.int32)
        self.accept, self.n_accept = torch.zeros(B, Q, device="cuda", dtype=torch.int32), ints([0] * B)
        self.out = torch.zeros(B, Q, H, 512, device="cuda", dtype=out_dtype)
        self.lse = torch.zeros(B, Q, H, device="cuda")
        self.plan = mla.tree_plan(batch=B, tokens=Q, heads=H, scale=SCALE, pdl=True)
        self.scratch = mla.tree_alloc_scratch(self.plan)
        self.ev_scratch = mla.evict_alloc_scratch(batch=B, keep=self.KEEP)

    def draw(self, width=None):
        """New inputs of a step, written into the step's tensors."""
        B, Q, H = self.B, self.Q, self.H
        n = [width or self.rnd.randint(0, Q) for _ in range(B)]
        bits = [ref.masks_of_tree(self.rnd, Q) for _ in range(B)]
        nxt = self.next_pos.tolist()
        pos = [[nxt[b] + bin(bits[b][i]).count("1") - 1 for i in range(Q)] for b in range(B)]
        paths, counts = [], []
        for b in range(B):
            leaf = self.rnd.randrange(n[b]) if n[b] else None
            path = [i for i in range(Q) if leaf is not None and bits[b][leaf] >> i & 1]
            paths.append(path + [0] * (Q - len(path)))
            counts.append(len(path))
        r = lambda *s: torch.randn(*s, generator=self.g).bfloat16()  # noqa: E731
        self.q[..., :512] = r(B, Q, H, 512).cuda()
        self.q_rope.copy_(r(B, Q, H, 64))
        self.new.copy_(r(B, Q, 576))
        for dst, v in ((self.pos, pos), (self.n, n), (self.accept, paths), (self.n_accept, counts),
                       (self.mask, [[ref.signed(w) for w in row] for row in bits])):
            dst.copy_(torch.tensor(v, dtype=dst.dtype))
        return n, bits, paths, counts

    def step(self):
        side = dict(row_positions=self.positions, row_weights=self.weights, row_offset=self.row_offset)
        mla.rope_append(self.table, self.pos, q_rope=self.q_rope, q=self.q, c=self.new[..., :512],
                        k_rope=self.new[..., 512:], kv=self.kv, d_pos=self.d_pos, n_tokens=self.n, **side)
        args = mla.tree_make_args(self.q, self.kv, self.out, self.lse, d_pos=self.d_pos, row_offset=self.row_offset,
                                  mask=self.mask, n_tokens=self.n)
        mla.tree_forward_args(self.plan, args, self.scratch)
        mla.tree_weights_args(self.plan, args, self.scratch, self.weights, decay=0.9375)

    def commit(self):
        mla.tree_commit(self.kv, self.accept, self.n_accept, d_pos=self.d_pos, d_pos_out=self.d_pos,
                        row_offset=self.row_offset, row_positions=self.positions, row_weights=self.weights)
        self.next_pos += self.n_accept

    def evict(self):
        mla.evict(self.kv, self.weights, self.positions, self.ev_scratch, d_pos=self.d_pos, next_pos=self.next_pos,
                  keep=self.KEEP, sink=2, recent=10, row_offset=self.row_offset, max_rows=self.CAP)


def test_serving_loop_step_by_step():
    s = Loop(1)
    evictions = 0
    for it in range(80):
        n, bits, paths, counts = s.draw(width=s.Q if it < 20 else None)
        lens, old_kv, old_w = s.d_pos.tolist(), s.kv.clone(), s.weights.cpu()
        s.step()
        torch.cuda.synchronize()
        # rows behind the committed ones: the rotated drafts
        kv = s.kv.cpu()
        for b in range(s.B):
            at = s.offs[b] + lens[b]
            old_w[at:at + n[b]] = 0
            want = ref.rotate(s.new[b, :n[b], 512:].cpu(), s.pos[b, :n[b]].cpu(), s.f, 64, True, 1.0)
            err = (kv[at:at + n[b], 512:].double() - want).abs()
            assert (err <= ref.BF16 * want.abs() + 2.0 ** -18).all()
            assert torch.equal(kv[at:at + n[b], :512], s.new[b, :n[b], :512].cpu())
        common = dict(d_pos=lens, row_offset=s.offs, n_tokens=n, bits=bits, scale=SCALE)
        for (b, i), (ro, rl, to, tl) in ref.tree(s.q.cpu(), kv, **common).items():
            assert ((s.out[b, i].double().cpu() - ro).abs() <= to).all()
            assert ((s.lse[b, i].double().cpu() - rl).abs() <= tl).all()
        new_w, tol = ref.weights(s.q.cpu(), kv, s.lse.cpu(), old_w, decay=0.9375, **common)
        live = ~torch.isnan(new_w)
        assert ((s.weights.double().cpu() - new_w).abs()[live] <= tol[live]).all()
        before = s.kv.clone()
        s.commit()
        for b in range(s.B):
            at = s.offs[b] + lens[b]
            for k in range(counts[b]):
                assert torch.equal(s.kv[at + k].view(torch.int16), before[at + paths[b][k]].view(torch.int16))
        assert s.d_pos.tolist() == [a + c for a, c in zip(lens, counts)]
        if max(s.d_pos.tolist()) > s.CAP - 2 * s.Q:
            before, w, p = s.kv.clone(), s.weights.tolist(), s.positions.tolist()
            lens, nxt = s.d_pos.tolist(), s.next_pos.tolist()
            s.evict()
            evictions += 1
            for b in range(s.B):
                o = s.offs[b]
                src = ref.evict_rows(w[o:o + lens[b]], p[o:o + lens[b]], lens[b], s.KEEP, 2, nxt[b] - 10)
                at = torch.tensor(src, dtype=torch.int64, device="cuda") + o
                assert torch.equal(s.kv[o:o + len(src)].view(torch.int16), before[at].view(torch.int16))
                assert s.positions[o:o + len(src)].tolist() == [p[o + r] for r in src]
                assert int(s.d_pos[b]) == len(src)
                assert set(range(2)) <= set(s.positions[o:o + len(src)].tolist())
    assert evictions >= 2 and mla.status_word(s.plan, s.scratch) == 0
    # the dense decode reads the same cache: append one more row per request, project the latent
    p = mla.plan(batch=s.B, heads=s.H, max_ctx=s.CAP, scale=SCALE)
    row = torch.randn(s.B, 576, generator=s.g).bfloat16().cuda()
    mla.append(s.kv, row, s.d_pos, row_offset=s.row_offset)
    q = torch.randn(s.B, s.H, 576, generator=s.g).bfloat16().cuda()
    o, l = torch.empty(s.B, s.H, 512, device="cuda"), torch.empty(s.B, s.H, device="cuda")
    mla.forward(p, q, s.kv, o, l, mla.alloc_scratch(p), d_pos=s.d_pos, row_offset=s.row_offset)
    want = ref.tree(q.cpu()[:, None], s.kv.cpu(), d_pos=s.d_pos.tolist(), row_offset=s.offs, n_tokens=[1] * s.B,
                    bits=[[1]] * s.B, scale=SCALE)
    for b in range(s.B):
        assert ((o[b].double().cpu() - want[b, 0][0]).abs() <= want[b, 0][2]).all()
    wv = torch.randn(s.H, 32, 512, generator=s.g).bfloat16().cuda()
    y = torch.empty(s.B * s.Q, s.H, 32, device="cuda")
    mla.project(s.out.view(s.B * s.Q, s.H, 512), wv, y)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()


def test_serving_loop_as_one_graph():
    """The whole step captured once and replayed gives what separate calls give, bit for bit."""
    a, b = Loop(2, torch.bfloat16), Loop(2, torch.bfloat16)
    for s in (a, b):
        for _ in range(8):
            s.draw(width=s.Q)
            s.step()
            s.commit()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.step()
        b.commit()
        b.evict()
    for _ in range(40):
        for s in (a, b):
            s.draw(width=s.Q)
        a.step()
        a.commit()
        a.evict()
        graph.replay()
        torch.cuda.synchronize()
        assert a.d_pos.tolist() == b.d_pos.tolist()
        for x, y in ((a.kv, b.kv), (a.out, b.out)):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        for x, y in ((a.weights, b.weights), (a.lse, b.lse)):
            assert torch.equal(x.view(torch.int32), y.view(torch.int32))
        assert torch.equal(a.positions, b.positions)
    assert max(a.d_pos.tolist()) == a.KEEP


FIRST_USE = """
import torch, decode_attention_mla_gb300 as mla
N, KEEP = 20000, 7000
g = torch.Generator(device="cuda").manual_seed(3)
i32 = dict(dtype=torch.int32, device="cuda")
kv = torch.randn(N + 8, 576, device="cuda", generator=g).bfloat16()
w = torch.rand(N + 8, device="cuda", generator=g)
pos = torch.arange(N + 8, **i32)
table = mla.rope_table()
state = dict(kv=kv, w=w, pos=pos, d=torch.tensor([N], **i32), q=torch.zeros(1, 4, 16, 576, device="cuda").bfloat16())
start = {k: v.clone() for k, v in state.items()}
x = torch.randn(1, 4, 16, 64, device="cuda", generator=g).bfloat16()
rows = torch.randn(1, 4, 576, device="cuda", generator=g).bfloat16()
at = torch.arange(N, N + 4, **i32)[None].contiguous()
accept, n_accept, nxt = torch.tensor([[0, 2, 3, 0]], **i32), torch.tensor([3], **i32), torch.tensor([N + 3], **i32)
scratch = mla.evict_alloc_scratch(batch=1, keep=KEEP)
plan = mla.tree_plan(batch=1, tokens=4, heads=16, scale=0.04, num_sms=152)
tree_scratch = mla.tree_alloc_scratch(plan)
lse = torch.zeros(1, 4, 16, device="cuda")
out = torch.zeros(1, 4, 16, 512, device="cuda")

def step(s):
    mla.rope_append(table, at, q_rope=x, q=s["q"], c=rows[..., :512], k_rope=rows[..., 512:], kv=s["kv"],
                    d_pos=s["d"], row_positions=s["pos"], row_weights=s["w"])
    mla.tree_commit(s["kv"], accept, n_accept, d_pos=s["d"], d_pos_out=s["d"], row_positions=s["pos"],
                    row_weights=s["w"])
    mla.evict(s["kv"], s["w"], s["pos"], scratch, d_pos=s["d"], next_pos=nxt, keep=KEEP, sink=4, recent=64)

torch.cuda.synchronize()
refused = False
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(state)                                   # the library's first launches
    try:
        mla.tree_forward(plan, state["q"], state["kv"], out, lse, tree_scratch, d_pos=state["d"])
    except mla.MLADecodeError as e:
        refused = e.status == mla.ENOTREADY
assert refused
for _ in range(2):
    for k, v in start.items():
        state[k].copy_(v)
    graph.replay()
torch.cuda.synchronize()
step(start)
for k, v in start.items():
    assert torch.equal(state[k], v), k
print("same")
"""


def test_first_use_inside_a_capture():
    run = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=Path(mla.__file__).parents[1], capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0 and "same" in run.stdout, run.stderr[-2000:]
