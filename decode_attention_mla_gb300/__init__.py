"""Python binding of ``libmla_decode.so`` (split-KV MLA decode on GB300).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/mla_decode.h``.  Tensors are
PyTorch CUDA tensors; the binding passes their device pointers, sizes and the
current CUDA stream.  If the library is not built, importing works but every
call raises ``RuntimeError`` -- there is no fallback path.

Typical use::

    import decode_attention_mla_gb300 as mla
    plan = mla.plan(batch=1, heads=16, max_ctx=8192, scale=1/24)
    scratch = mla.alloc_scratch(plan)           # before any graph capture
    mla.forward(plan, q, kv, out, lse, scratch, d_pos=d_pos)
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")

D_LATENT = 512
D_ROPE = 64
D_ROW = 576
Q4_ROW = 416                           # bytes of a row of the 4-bit cache
MAX_SPLITS = 256

OK, EINVAL, EUNSUPPORTED, ESCRATCH, EALIGN, ECUDA, EDEVICE, ENOTREADY = 0, -1, -2, -3, -4, -5, -6, -7
ESTATICLIMIT = -8
STATIC_SCRATCH_BYTES = 8 << 20      # scratch of mla_decode_forward_static


class Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("heads", ctypes.c_int), ("d_latent", ctypes.c_int),
                ("d_rope", ctypes.c_int), ("sparse", ctypes.c_int), ("max_ctx", ctypes.c_int),
                ("topk", ctypes.c_int), ("scale", ctypes.c_float), ("num_sms", ctypes.c_int),
                ("splits_override", ctypes.c_int), ("variant", ctypes.c_int), ("pdl", ctypes.c_int),
                ("stall_test", ctypes.c_int), ("kv_fp8", ctypes.c_int)]


class Plan(ctypes.Structure):
    _fields_ = [("shape", Shape), ("magic", ctypes.c_int), ("variant", ctypes.c_int),
                ("splits", ctypes.c_int), ("entries_per_split", ctypes.c_int), ("head_group", ctypes.c_int),
                ("n_head_groups", ctypes.c_int), ("ctas_per_sm", ctypes.c_int), ("num_sms", ctypes.c_int),
                ("grid_x", ctypes.c_int), ("grid_y", ctypes.c_int), ("grid_z", ctypes.c_int),
                ("block", ctypes.c_int), ("smem_bytes", ctypes.c_int), ("combine_grid_x", ctypes.c_int),
                ("combine_grid_y", ctypes.c_int), ("combine_block", ctypes.c_int),
                ("scratch_bytes", ctypes.c_size_t), ("o_part_offset", ctypes.c_size_t),
                ("lse_part_offset", ctypes.c_size_t), ("status_offset", ctypes.c_size_t),
                ("flat_ranges", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {k: getattr(self, k) for k, _ in self._fields_ if k != "shape"}
        d["shape"] = {k: getattr(self.shape, k) for k, _ in Shape._fields_}
        return d


class Args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("kv", ctypes.c_void_p), ("kv_rows", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong), ("d_pos", ctypes.c_void_p), ("row_offset", ctypes.c_void_p),
                ("cache_len", ctypes.c_void_p), ("indices", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("kv_scale", ctypes.c_float)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_ctx", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double)]


class RopeArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float), ("turns", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("n_tokens", ctypes.c_void_p),
                ("q_rope", ctypes.c_void_p), ("q_rope_batch", ctypes.c_longlong), ("q_rope_token", ctypes.c_longlong),
                ("q_rope_head", ctypes.c_longlong),
                ("q_out", ctypes.c_void_p), ("q_out_batch", ctypes.c_longlong), ("q_out_token", ctypes.c_longlong),
                ("q_out_head", ctypes.c_longlong),
                ("c", ctypes.c_void_p), ("c_batch", ctypes.c_longlong), ("c_token", ctypes.c_longlong),
                ("k_rope", ctypes.c_void_p), ("k_rope_batch", ctypes.c_longlong), ("k_rope_token", ctypes.c_longlong),
                ("kv", ctypes.c_void_p), ("kv_rows", ctypes.c_longlong), ("row_stride", ctypes.c_longlong),
                ("kv_fp8", ctypes.c_int), ("kv_scale", ctypes.c_float),
                ("d_pos", ctypes.c_void_p), ("row_offset", ctypes.c_void_p),
                ("row_positions", ctypes.c_void_p), ("row_weights", ctypes.c_void_p)]


class TreeShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("scale", ctypes.c_float),
                ("num_sms", ctypes.c_int), ("pdl", ctypes.c_int), ("stall_test", ctypes.c_int)]


class TreePlan(ctypes.Structure):
    _fields_ = [("shape", TreeShape), ("magic", ctypes.c_int), ("num_sms", ctypes.c_int), ("grid", ctypes.c_int),
                ("scratch_bytes", ctypes.c_size_t), ("status_offset", ctypes.c_size_t),
                ("part_offset", ctypes.c_size_t), ("lse_part_offset", ctypes.c_size_t)]


class TreeArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("q", ctypes.c_void_p), ("kv", ctypes.c_void_p), ("kv_rows", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong), ("d_pos", ctypes.c_void_p), ("row_offset", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("n_tokens", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("out_fp32", ctypes.c_int), ("lse", ctypes.c_void_p)]


class TreeCommitArgs(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("kv_rows", ctypes.c_longlong), ("row_stride", ctypes.c_longlong),
                ("kv_fp8", ctypes.c_int), ("batch", ctypes.c_int), ("tokens", ctypes.c_int),
                ("accept", ctypes.c_void_p), ("n_accept", ctypes.c_void_p), ("d_pos", ctypes.c_void_p),
                ("d_pos_out", ctypes.c_void_p), ("row_offset", ctypes.c_void_p),
                ("row_positions", ctypes.c_void_p), ("row_weights", ctypes.c_void_p)]


# The same layout, packed in one go: tree_commit fills its arguments on every call.
_COMMIT_ARGS = struct.Struct("Pqqiii0P7P")


class EvictArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("kv", ctypes.c_void_p), ("kv_rows", ctypes.c_longlong), ("row_stride", ctypes.c_longlong),
                ("kv_fp8", ctypes.c_int), ("batch", ctypes.c_int), ("keep", ctypes.c_int), ("sink", ctypes.c_int),
                ("recent", ctypes.c_int), ("max_rows", ctypes.c_int), ("weights", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("d_pos", ctypes.c_void_p), ("next_pos", ctypes.c_void_p),
                ("row_offset", ctypes.c_void_p), ("weights_out", ctypes.c_void_p), ("positions_out", ctypes.c_void_p),
                ("d_pos_out", ctypes.c_void_p)]


class PagedCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_stride", ctypes.c_longlong), ("n_pages", ctypes.c_int),
                ("page_rows", ctypes.c_int), ("page_table", ctypes.c_void_p), ("columns", ctypes.c_int),
                ("kv_scale", ctypes.c_float)]


class PagedAppendArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("cache", PagedCache), ("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("heads", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("n_tokens", ctypes.c_void_p),
                ("q_rope", ctypes.c_void_p), ("q_rope_batch", ctypes.c_longlong), ("q_rope_token", ctypes.c_longlong),
                ("q_rope_head", ctypes.c_longlong),
                ("q_out", ctypes.c_void_p), ("q_out_batch", ctypes.c_longlong), ("q_out_token", ctypes.c_longlong),
                ("q_out_head", ctypes.c_longlong),
                ("c", ctypes.c_void_p), ("c_batch", ctypes.c_longlong), ("c_token", ctypes.c_longlong),
                ("k_rope", ctypes.c_void_p), ("k_rope_batch", ctypes.c_longlong), ("k_rope_token", ctypes.c_longlong),
                ("c_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("d_pos", ctypes.c_void_p)]


class PagedReadArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("cache", PagedCache), ("batch", ctypes.c_int), ("rows", ctypes.c_int), ("first", ctypes.c_void_p),
                ("n_rows", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_batch", ctypes.c_longlong),
                ("out_row", ctypes.c_longlong)]


class PagedShape(ctypes.Structure):
    _fields_ = TreeShape._fields_


class PagedPlan(ctypes.Structure):
    _fields_ = [("shape", PagedShape)] + TreePlan._fields_[1:]


class PagedArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = [("cache", PagedCache), ("q", ctypes.c_void_p), ("d_pos", ctypes.c_void_p), ("n_tokens", ctypes.c_void_p),
                ("window", ctypes.c_int), ("sink", ctypes.c_int), ("out", ctypes.c_void_p), ("out_fp32", ctypes.c_int),
                ("lse", ctypes.c_void_p)]


_POOL_FIELDS = [("pages", ctypes.c_void_p), ("page_stride", ctypes.c_longlong), ("n_pages", ctypes.c_int),
                ("page_rows", ctypes.c_int), ("row_bytes", ctypes.c_int), ("batch", ctypes.c_int),
                ("columns", ctypes.c_int), ("page_table", ctypes.c_void_p)]


class PagesForkArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = _POOL_FIELDS + [
        ("d_pos", ctypes.c_void_p), ("parent", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("reserve", ctypes.c_int),
        ("window", ctypes.c_int), ("sink", ctypes.c_int), ("page_table_out", ctypes.c_void_p),
        ("d_pos_out", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("missing", ctypes.c_void_p)]


class PagesCompactArgs(ctypes.Structure):
    _device = None                     # device of the tensors, where a *_make_args call has checked them
    _fields_ = _POOL_FIELDS + [("refs", ctypes.c_void_p), ("page_table_out", ctypes.c_void_p),
                               ("refs_out", ctypes.c_void_p), ("used", ctypes.c_void_p)]


class MLADecodeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


_lock = threading.Lock()
_lib = None

EXPORTED = ("mla_decode_abi_version", "mla_decode_plan", "mla_decode_run", "mla_decode_combine",
            "mla_decode_forward", "mla_decode_append", "mla_decode_advance", "mla_decode_scratch_init",
            "mla_decode_strerror", "mla_decode_forward_static", "mla_decode_project", "mla_decode_forward_step",
            "mla_floor_empty_pair", "mla_floor_read", "mla_floor_gather", "mla_decode_static_status", "mla_decode_static_reset",
            "mla_rope_table", "mla_rope_append", "mla_tree_plan", "mla_tree_forward", "mla_tree_weights",
            "mla_tree_commit", "mla_evict_scratch_bytes", "mla_evict", "mla_paged_append", "mla_paged_read",
            "mla_paged_plan", "mla_paged_forward", "mla_pages_scratch_bytes", "mla_pages_fork", "mla_pages_compact")


def lib():
    """The loaded library; raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m decode_attention_mla_gb300.build` "
                               "(or __graft_entry__.build()); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        P, I, SZ, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
        L.mla_decode_abi_version.restype = I
        L.mla_decode_abi_version.argtypes = []
        L.mla_decode_plan.restype = I
        L.mla_decode_plan.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Plan)]
        for name in ("mla_decode_run", "mla_decode_combine", "mla_decode_forward"):
            fn = getattr(L, name)
            fn.restype = I
            fn.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(Args), P, SZ, P]
        L.mla_decode_forward_step.restype = I
        L.mla_decode_forward_step.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(Args), P, SZ, P, I, P]
        L.mla_decode_forward_static.restype = I
        L.mla_decode_forward_static.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(Args), P]
        L.mla_decode_append.restype = I
        L.mla_decode_append.argtypes = [P, LL, LL, P, P, P, I, P]
        L.mla_decode_project.restype = I
        L.mla_decode_project.argtypes = [P, P, I, I, I, P, I, P]
        L.mla_decode_advance.restype = I
        L.mla_decode_advance.argtypes = [P, I, P]
        L.mla_decode_scratch_init.restype = I
        L.mla_decode_scratch_init.argtypes = [P, SZ, P]
        L.mla_decode_strerror.restype = ctypes.c_char_p
        L.mla_decode_strerror.argtypes = [I]
        L.mla_decode_static_status.restype = I
        L.mla_decode_static_status.argtypes = [P, P]
        L.mla_decode_static_reset.restype = I
        L.mla_decode_static_reset.argtypes = [P]
        L.mla_floor_empty_pair.restype = I
        L.mla_floor_empty_pair.argtypes = [I, I, I, I, I, I, I, P]
        L.mla_floor_read.restype = I
        L.mla_floor_read.argtypes = [P, SZ, I, P, P, I, P]
        L.mla_floor_gather.restype = I
        L.mla_floor_gather.argtypes = [P, LL, LL, I, P, LL, I, P, P, I, P]
        F = ctypes.c_float
        L.mla_rope_table.restype = I
        L.mla_rope_table.argtypes = [ctypes.POINTER(RopeSpec), ctypes.POINTER(ctypes.c_ulonglong)]
        L.mla_rope_append.restype = I
        L.mla_rope_append.argtypes = [ctypes.POINTER(RopeArgs), P]
        L.mla_tree_plan.restype = I
        L.mla_tree_plan.argtypes = [ctypes.POINTER(TreeShape), ctypes.POINTER(TreePlan)]
        L.mla_tree_forward.restype = I
        L.mla_tree_forward.argtypes = [ctypes.POINTER(TreePlan), ctypes.POINTER(TreeArgs), P, SZ, P]
        L.mla_tree_weights.restype = I
        L.mla_tree_weights.argtypes = [ctypes.POINTER(TreePlan), ctypes.POINTER(TreeArgs), P, F, P, SZ, P]
        L.mla_tree_commit.restype = I
        L.mla_tree_commit.argtypes = [P, P]
        L.mla_evict_scratch_bytes.restype = SZ
        L.mla_evict_scratch_bytes.argtypes = [I, I]
        L.mla_evict.restype = I
        L.mla_evict.argtypes = [ctypes.POINTER(EvictArgs), P, SZ, P]
        L.mla_paged_append.restype = I
        L.mla_paged_append.argtypes = [ctypes.POINTER(PagedAppendArgs), P]
        L.mla_paged_read.restype = I
        L.mla_paged_read.argtypes = [ctypes.POINTER(PagedReadArgs), P]
        L.mla_paged_plan.restype = I
        L.mla_paged_plan.argtypes = [ctypes.POINTER(PagedShape), ctypes.POINTER(PagedPlan)]
        L.mla_paged_forward.restype = I
        L.mla_paged_forward.argtypes = [ctypes.POINTER(PagedPlan), ctypes.POINTER(PagedArgs), P, SZ, P]
        L.mla_pages_scratch_bytes.restype = SZ
        L.mla_pages_scratch_bytes.argtypes = [I, I, I]
        L.mla_pages_fork.restype = I
        L.mla_pages_fork.argtypes = [ctypes.POINTER(PagesForkArgs), P, SZ, P]
        L.mla_pages_compact.restype = I
        L.mla_pages_compact.argtypes = [ctypes.POINTER(PagesCompactArgs), P, SZ, P]
        _lib = L
        return L


def strerror(status: int) -> str:
    try:
        return lib().mla_decode_strerror(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise MLADecodeError(rc, what)


def _ptr(t):
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise ValueError("tensors passed to the MLA decode kernels must be CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


_torch = None
_raw_stream = None


def _device():
    """The current device (replaced by torch's own getter on first use)."""
    return _tc().cuda.current_device()


def _tc():
    """The torch module, imported on first use (and the getters of the current stream's address and
    device, where this torch has them: building a Stream object costs as much as a launch)."""
    global _torch, _raw_stream, _device
    if _torch is None:
        import torch
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch = torch
    return _torch


def _stream(stream):
    if stream is None:
        torch = _torch or _tc()
        if _raw_stream is not None:
            return _raw_stream(_device())                      # (every entry point declares the pointer type)
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def plan(*, batch: int, heads: int, scale: float, max_ctx: int = 0, topk: int = 0, sparse: bool = False,
         num_sms: int = 0, splits: int = 0, variant: int = 0, pdl: bool = False, stall_test: bool = False,
         kv_fp8: bool = False) -> Plan:
    """``mla_decode_plan``: derive the split count, grid and scratch layout.

    ``num_sms=0`` queries the current CUDA device and prepares the kernels on it
    (do this before capturing a graph).  ``kv_fp8``: the cache holds E4M3 bytes
    (pass the cache's scale as ``kv_scale`` to :func:`make_args` / :func:`forward`)."""
    s = Shape(batch=batch, heads=heads, d_latent=D_LATENT, d_rope=D_ROPE, sparse=int(bool(sparse)),
              max_ctx=max_ctx, topk=topk, scale=scale, num_sms=num_sms, splits_override=splits,
              variant=variant, pdl=int(bool(pdl)), stall_test=int(bool(stall_test)), kv_fp8=int(bool(kv_fp8)))
    p = Plan()
    _check(lib().mla_decode_plan(ctypes.byref(s), ctypes.byref(p)), "mla_decode_plan")
    return p


def alloc_scratch(p: Plan, device=None):
    """Allocate and zero the caller-owned scratch the plan needs (outside capture)."""
    import torch
    n = (int(p.scratch_bytes) + 255) // 256 * 256
    buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    scratch_init(buf)
    return buf


def scratch_init(scratch, stream=None) -> None:
    _check(lib().mla_decode_scratch_init(_ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)),
           "mla_decode_scratch_init")


def status_word(p: Plan, scratch) -> int:
    """The device status word of a scratch region (0 = healthy); synchronises."""
    import torch
    off = int(p.status_offset)
    return int(scratch[off:off + 4].view(torch.int32).item())


def make_args(q, kv, out, lse, *, d_pos=None, row_offset=None, cache_len=None, indices=None,
              kv_rows: int | None = None, row_stride: int | None = None, kv_scale: float = 1.0) -> Args:
    """Per-call arguments.  ``kv``: bf16 rows, or E4M3 bytes (uint8 / float8_e4m3fn) for plans made
    with ``kv_fp8`` (then ``row_stride`` counts bytes and ``kv_scale`` is the cache's scale)."""
    if row_stride is None:
        row_stride = kv.stride(0) if kv.dim() == 2 else D_ROW
    if kv_rows is None:
        kv_rows = kv.shape[0] if kv.dim() == 2 else kv.numel() // row_stride
    return Args(q=_ptr(q), kv=_ptr(kv), kv_rows=int(kv_rows), row_stride=int(row_stride), d_pos=_ptr(d_pos),
                row_offset=_ptr(row_offset), cache_len=_ptr(cache_len), indices=_ptr(indices), out=_ptr(out),
                lse=_ptr(lse), kv_scale=float(kv_scale))


def _scratch_args(scratch):
    if getattr(scratch, "is_cuda", False):
        return scratch.data_ptr(), scratch.nbytes
    return _ptr(scratch), scratch.numel() * scratch.element_size()


def run(p: Plan, args: Args, scratch, stream=None) -> None:
    """``mla_decode_run``: launch the split partial kernel."""
    sp, sb = _scratch_args(scratch)
    _check(lib().mla_decode_run(ctypes.byref(p), ctypes.byref(args), sp, sb, _stream(stream)), "mla_decode_run")


def combine(p: Plan, args: Args, scratch, stream=None) -> None:
    """``mla_decode_combine``: launch the log-sum-exp merge kernel."""
    sp, sb = _scratch_args(scratch)
    _check(lib().mla_decode_combine(ctypes.byref(p), ctypes.byref(args), sp, sb, _stream(stream)),
           "mla_decode_combine")


def forward_args(p: Plan, args: Args, scratch, stream=None) -> None:
    """``mla_decode_forward``: partial + combine with prebuilt arguments."""
    sp, sb = _scratch_args(scratch)
    _check(lib().mla_decode_forward(ctypes.byref(p), ctypes.byref(args), sp, sb, _stream(stream)),
           "mla_decode_forward")


def forward_step_args(p: Plan, args: Args, scratch, new_rows, *, advance: bool = True, stream=None) -> None:
    """``mla_decode_forward_step``: append ``new_rows`` at d_pos, partial + combine, then (if ``advance``)
    d_pos += 1, in two launches (dense plans)."""
    sp, sb = _scratch_args(scratch)
    _check(lib().mla_decode_forward_step(ctypes.byref(p), ctypes.byref(args), sp, sb, _ptr(new_rows),
                                         int(bool(advance)), _stream(stream)), "mla_decode_forward_step")


def forward_step(p: Plan, q, kv, out, lse, scratch, new_rows, *, d_pos, row_offset=None, advance: bool = True,
                 kv_rows=None, row_stride=None, stream=None) -> None:
    """As :func:`forward`, with the cache append before it and the position advance after it folded in."""
    a = make_args(q, kv, out, lse, d_pos=d_pos, row_offset=row_offset, kv_rows=kv_rows, row_stride=row_stride)
    forward_step_args(p, a, scratch, new_rows, advance=advance, stream=stream)


def forward(p: Plan, q, kv, out, lse, scratch, *, d_pos=None, row_offset=None, cache_len=None, indices=None,
            kv_rows=None, row_stride=None, kv_scale: float = 1.0, stream=None) -> None:
    """Partial + combine: ``out[B,H,512]`` and ``lse[B,H]`` (fp32) from bf16 ``q`` and ``kv``
    (bf16 rows, or E4M3 bytes with ``kv_scale`` for ``kv_fp8`` plans)."""
    a = make_args(q, kv, out, lse, d_pos=d_pos, row_offset=row_offset, cache_len=cache_len, indices=indices,
                  kv_rows=kv_rows, row_stride=row_stride, kv_scale=kv_scale)
    forward_args(p, a, scratch, stream)


def forward_static(p: Plan, q, kv, out, lse, *, d_pos=None, row_offset=None, cache_len=None, indices=None,
                   kv_rows=None, row_stride=None, stream=None) -> None:
    """``mla_decode_forward_static``: as :func:`forward`, with the library's own 8 MiB static scratch."""
    a = make_args(q, kv, out, lse, d_pos=d_pos, row_offset=row_offset, cache_len=cache_len, indices=indices,
                  kv_rows=kv_rows, row_stride=row_stride)
    _check(lib().mla_decode_forward_static(ctypes.byref(p), ctypes.byref(a), _stream(stream)),
           "mla_decode_forward_static")


def static_status(dst, stream=None) -> None:
    """``mla_decode_static_status``: stream-ordered copy of the static scratch's status word into
    ``dst`` (a CUDA int32 tensor of at least one element)."""
    _check(lib().mla_decode_static_status(_ptr(dst), _stream(stream)), "mla_decode_static_status")


def static_reset(stream=None) -> None:
    """``mla_decode_static_reset``: clear the static scratch's status word."""
    _check(lib().mla_decode_static_reset(_stream(stream)), "mla_decode_static_reset")


def append(kv, new_rows, d_pos, *, row_offset=None, kv_rows=None, row_stride=None, stream=None) -> None:
    """``mla_decode_append``: write new_rows[b] at cache row base_b + d_pos[b] (on the device)."""
    if row_stride is None:
        row_stride = kv.stride(0)
    if kv_rows is None:
        kv_rows = kv.shape[0]
    batch = int(d_pos.numel())
    _check(lib().mla_decode_append(_ptr(kv), int(kv_rows), int(row_stride), _ptr(new_rows), _ptr(d_pos),
                                   _ptr(row_offset), batch, _stream(stream)), "mla_decode_append")


def project(latent, wv_b, y, *, pdl: bool = False, stream=None) -> None:
    """``mla_decode_project``: y[B,H,v] = latent[B,H,512] . wv_b[H,v,512]^T per head (fp32 out)."""
    B, H, r = latent.shape
    if r != D_LATENT or tuple(wv_b.shape[:1]) != (H,) or wv_b.shape[-1] != D_LATENT:
        raise ValueError("latent must be [B, H, 512] and wv_b [H, v_dim, 512]")
    v_dim = int(wv_b.shape[1])
    _check(lib().mla_decode_project(_ptr(latent), _ptr(wv_b), int(B), int(H), v_dim, _ptr(y), int(bool(pdl)),
                                    _stream(stream)), "mla_decode_project")


def advance(d_pos, stream=None) -> None:
    """``mla_decode_advance``: d_pos += 1 on the device."""
    _check(lib().mla_decode_advance(_ptr(d_pos), int(d_pos.numel()), _stream(stream)), "mla_decode_advance")


# ---- drafted tokens, their rotation, and a bounded cache ---------------------
# Arguments that stay the same from call to call are laid out once
# (``*_make_args``), which also checks the tensors; the ``*_args`` calls then
# pass them on.  The returned structures keep their tensors alive.

def _need(t, name, dtypes, shape=None, contiguous=True):
    """Check a tensor of a call (CUDA, on the current device, type, shape, layout); its address."""
    torch = _torch or _tc()
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError(f"{name}: a CUDA tensor is needed (tensors passed to the MLA decode kernels must be "
                         "CUDA tensors)")
    if t.get_device() != _device():
        raise ValueError(f"{name} is on {t.device}, the current device is {_device()}")
    if t.dtype is not dtypes and (type(dtypes) is not tuple or t.dtype not in dtypes):
        names = " or ".join(map(str, dtypes)) if type(dtypes) is tuple else dtypes
        raise ValueError(f"{name}: dtype {t.dtype}, expected {names}")
    if shape is not None and t.shape != shape and (
            t.dim() != len(shape) or any(e is not None and e != n for n, e in zip(t.shape, shape))):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple('*' if e is None else e for e in shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _quick(t, name, dtype, shape, device):
    """As _need, for the calls that check their tensors every time: the usual case first."""
    try:
        if t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _need(t, name, dtype, shape)


def _scratch_here(scratch):
    """Address and bytes of a call's scratch (CUDA, on the current device, contiguous)."""
    try:
        if scratch.get_device() == _device() and scratch.is_contiguous():
            return scratch.data_ptr(), scratch.nbytes
    except AttributeError:
        pass
    return _need(scratch, "scratch", getattr(scratch, "dtype", None)), scratch.nbytes


def _stream_of(a, stream):
    """Stream of a call with prebuilt arguments, which were checked against the device that was current then."""
    device = _device()
    if a._device is not None and a._device != device:
        raise ValueError(f"arguments for device {a._device}, the current device is {device}")
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


def _int(v, name):
    """An int argument: a C int would take a larger one modulo 2^32."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} = {v} is no 32-bit integer")
    return v


def _maybe(t, name, dtypes, shape):
    return None if t is None else _need(t, name, dtypes, shape)


def _cache(kv, kv_rows, row_stride, fp8_ok=True):
    """(pointer, rows, row stride, fp8) of a cache tensor [rows, 576] with contiguous rows."""
    torch = _torch or _tc()
    p = _need(kv, "kv", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn) if fp8_ok else torch.bfloat16,
              contiguous=False)
    shape = kv.shape
    if len(shape) != 2 or shape[1] != D_ROW or kv.stride(1) != 1:
        raise ValueError("kv must be [rows, 576] with contiguous rows")
    rows, stride = shape[0], kv.stride(0)
    if rows < 2:
        if rows == 0:
            raise ValueError("kv has no rows")
        stride = max(stride, D_ROW)
    if kv_rows is not None:
        if not 1 <= kv_rows <= rows:
            raise ValueError("kv_rows is outside the tensor")
        rows = int(kv_rows)
    if row_stride is not None and row_stride != stride:
        raise ValueError("row_stride differs from the tensor's")
    return p, rows, stride, 0 if kv.dtype is torch.bfloat16 else 1


def _quick_cache(kv, device, torch):
    """As _cache(kv, None, None) for the usual cache; None if it is not one."""
    try:
        dt, shape, strides = kv.dtype, kv.shape, kv.stride()
        if (kv.get_device() == device and len(shape) == 2 and shape[1] == D_ROW and strides[1] == 1 and shape[0] > 1
                and (dt is torch.bfloat16 or dt is torch.uint8 or dt is torch.float8_e4m3fn)):
            return kv.data_ptr(), shape[0], strides[0], 0 if dt is torch.bfloat16 else 1
    except AttributeError:
        pass
    return None


def _strides(t, name, shape, last):
    """Pointer and leading strides of a bf16 tensor whose last dimension is contiguous."""
    torch = _torch or _tc()
    p = _need(t, name, torch.bfloat16, shape, contiguous=False)
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # the stride of a dimension of one is never used: 0 passes every check
    return [p] + [int(t.stride(i)) if t.shape[i] > 1 else 0 for i in range(last)]


def _apart(t, name, dims):
    """Refuse an output whose entries lie in one place (the strides of its first `dims` dimensions are used)."""
    if any(t.stride(i) == 0 and t.shape[i] > 1 for i in range(dims)):
        raise ValueError(f"{name} is an expanded tensor: its entries would be written to one place")


class RopeTable:
    """Angles per position of the rotated pairs (``mla_rope_table``), on the device."""

    def __init__(self, turns, rot_dim, interleaved, amplitude):
        self.turns, self.rot_dim, self.interleaved, self.amplitude = turns, rot_dim, interleaved, amplitude


ROPE_SCALING = {"none": 0, "linear": 1, "yarn": 2}


def rope_turns(rot_dim: int = D_ROPE, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
               original_ctx: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0) -> list:
    """``mla_rope_table``: angle per position of each pair, as 64-bit fractions of a turn (host integers)."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    spec = RopeSpec(rot_dim=_int(rot_dim, "rot_dim"), scaling=ROPE_SCALING[scaling], base=base, factor=factor,
                    original_ctx=original_ctx, beta_fast=beta_fast, beta_slow=beta_slow)
    buf = (ctypes.c_ulonglong * 32)()
    _check(lib().mla_rope_table(ctypes.byref(spec), buf), "mla_rope_table")
    return list(buf[:rot_dim // 2])


def rope_table(rot_dim: int = D_ROPE, base: float = 10000.0, *, interleaved: bool = True, scaling: str = "none",
               factor: float = 1.0, original_ctx: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
               amplitude: float = 1.0, device=None) -> RopeTable:
    """Rotation table on the device: pairs (2j, 2j+1) if ``interleaved``, else (j, j + rot_dim/2);
    ``scaling``: "none", "linear" or "yarn" (the angles); ``amplitude`` multiplies sines and cosines and is
    the caller's to give: 1 whatever the scaling, where YaRN's usual one is 0.1 ln(factor) + 1."""
    torch = _torch or _tc()
    turns = rope_turns(rot_dim, base, scaling=scaling, factor=factor, original_ctx=original_ctx,
                       beta_fast=beta_fast, beta_slow=beta_slow)
    t = torch.tensor(turns, dtype=torch.int64, device=device or "cuda")       # all below 2^62
    return RopeTable(t, rot_dim, bool(interleaved), float(amplitude))


def rope_make_args(table: RopeTable, positions, *, q_rope=None, q=None, c=None, k_rope=None, kv=None, d_pos=None,
                   row_offset=None, n_tokens=None, kv_scale: float = 1.0, row_positions=None, row_weights=None,
                   kv_rows: int | None = None, row_stride: int | None = None) -> RopeArgs:
    """Arguments of :func:`rope_append_args`.

    ``positions``: int32 [B, N].  Queries: ``q_rope`` bf16 [B, N, H, 64] (any strides, multiples of 8) is
    rotated into ``q[..., 512:]`` of bf16 [B, N, H, 576].  Rows: ``c`` bf16 [B, N, 512] and ``k_rope``
    bf16 [B, N, 64] go to cache row ``row_offset[b] + d_pos[b] + n`` of ``kv`` (bf16, or E4M3 bytes of
    value / ``kv_scale``); ``row_positions`` (int32 [rows]) takes the positions, ``row_weights``
    (fp32 [rows]) zeros.  Either part may be left out."""
    torch = _torch or _tc()
    B, N = positions.shape
    a = RopeArgs(batch=int(B), tokens=int(N), rot_dim=table.rot_dim, interleaved=int(table.interleaved),
                 amplitude=table.amplitude, turns=_need(table.turns, "table", torch.int64),
                 positions=_need(positions, "positions", torch.int32, (B, N)),
                 n_tokens=_maybe(n_tokens, "n_tokens", torch.int32, (B,)), kv_scale=float(kv_scale))
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q go together")
    if q is not None:
        H = q.shape[2] if q.dim() == 4 else -1
        a.heads = int(H)
        a.q_rope, a.q_rope_batch, a.q_rope_token, a.q_rope_head = _strides(q_rope, "q_rope", (B, N, H, D_ROPE), 3)
        _need(q, "q", torch.bfloat16, (B, N, H, D_ROW), contiguous=False)
        part = q[..., D_LATENT:]
        a.q_out, a.q_out_batch, a.q_out_token, a.q_out_head = _strides(part, "q", (B, N, H, D_ROPE), 3)
    if not (c is None) == (k_rope is None) == (kv is None) == (d_pos is None):
        raise ValueError("c, k_rope, kv and d_pos go together")
    if kv is None and not (row_positions is None and row_weights is None):
        raise ValueError("row_positions and row_weights belong to the rows of kv")
    if kv is not None:
        a.c, a.c_batch, a.c_token = _strides(c, "c", (B, N, D_LATENT), 2)
        a.k_rope, a.k_rope_batch, a.k_rope_token = _strides(k_rope, "k_rope", (B, N, D_ROPE), 2)
        a.kv, a.kv_rows, a.row_stride, a.kv_fp8 = _cache(kv, kv_rows, row_stride)
        a.d_pos = _need(d_pos, "d_pos", torch.int32, (B,))
        a.row_offset = _maybe(row_offset, "row_offset", torch.int64, (B,))
        a.row_positions = _side(row_positions, "row_positions", torch.int32, a.kv_rows)
        a.row_weights = _side(row_weights, "row_weights", torch.float32, a.kv_rows)
    a._device = _device()
    a._keep = (table, positions, q_rope, q, c, k_rope, kv, d_pos, row_offset, n_tokens, row_positions, row_weights)
    return a


def _side(t, name, dtype, rows):
    """A per-row array: at least one entry for every cache row."""
    if t is None:
        return None
    if getattr(t, "dtype", None) is dtype and t.dim() == 1 and t.shape[0] >= rows and t.is_contiguous() and (
            t.get_device() == _device()):
        return t.data_ptr()
    p = _need(t, name, dtype, (None,))
    if t.shape[0] < rows:
        raise ValueError(f"{name} needs an entry for each of the {rows} cache rows")
    return p


def rope_append_args(a: RopeArgs, stream=None) -> None:
    """``mla_rope_append`` with prebuilt arguments."""
    _check(lib().mla_rope_append(ctypes.byref(a), _stream_of(a, stream)), "mla_rope_append")


def rope_append(table: RopeTable, positions, *, stream=None, **kw) -> None:
    """Rotate the new tokens' queries and keys by their positions and append their rows to the cache
    (arguments as for :func:`rope_make_args`)."""
    rope_append_args(rope_make_args(table, positions, **kw), stream)


def tree_plan(*, batch: int, tokens: int, heads: int, scale: float, num_sms: int = 0, pdl: bool = False,
              stall_test: bool = False) -> TreePlan:
    """``mla_tree_plan``: up to ``tokens`` (<= 64) drafted tokens per request."""
    s = TreeShape(batch=_int(batch, "batch"), tokens=_int(tokens, "tokens"), heads=_int(heads, "heads"), scale=scale,
                  num_sms=_int(num_sms, "num_sms"), pdl=int(bool(pdl)), stall_test=int(bool(stall_test)))
    p = TreePlan()
    _check(lib().mla_tree_plan(ctypes.byref(s), ctypes.byref(p)), "mla_tree_plan")
    return p


def tree_alloc_scratch(p: TreePlan, device=None):
    """Allocate and zero the scratch of a tree plan (outside capture); :func:`status_word` reads its status."""
    return alloc_scratch(p, device)


def tree_make_args(q, kv, out, lse, *, d_pos, row_offset=None, mask=None, n_tokens=None,
                   kv_rows: int | None = None, row_stride: int | None = None) -> TreeArgs:
    """Arguments of :func:`tree_forward_args` and :func:`tree_weights_args` (which needs no ``out``).

    ``q``: bf16 [B, Q, H, 576]; ``kv``: bf16 [rows, 576]; ``out``: bf16 or fp32 [B, Q, H, 512] (fp32 also takes
    probabilities in 16 bits instead of 8, as the decode does, for up to 1.6 times the time); ``lse``: fp32 [B, Q, H]; ``mask``: int64 [B, Q], bit j of word i: token i attends drafted token j (None: a chain)."""
    torch = _torch or _tc()
    if q.dim() != 4:
        raise ValueError("q must be [B, Q, H, 576]")
    B, Q, H, _ = q.shape
    kvp, rows, stride, _ = _cache(kv, kv_rows, row_stride, fp8_ok=False)
    a = TreeArgs(q=_need(q, "q", torch.bfloat16, (B, Q, H, D_ROW)), kv=kvp, kv_rows=rows, row_stride=stride,
                 d_pos=_need(d_pos, "d_pos", torch.int32, (B,)),
                 row_offset=_maybe(row_offset, "row_offset", torch.int64, (B,)),
                 mask=_maybe(mask, "mask", torch.int64, (B, Q)),
                 n_tokens=_maybe(n_tokens, "n_tokens", torch.int32, (B,)),
                 out=_maybe(out, "out", (torch.bfloat16, torch.float32), (B, Q, H, D_LATENT)),
                 out_fp32=int(out is not None and out.dtype == torch.float32),
                 lse=_need(lse, "lse", torch.float32, (B, Q, H)))
    a._device = _device()
    a._keep = (q, kv, d_pos, row_offset, mask, n_tokens, out, lse)
    a._dims = (int(B), int(Q), int(H))
    return a


def _tree_dims(p: TreePlan, a: TreeArgs):
    """The arguments' [B, Q, H] must be the plan's: the kernels index by the plan."""
    if a._dims != (p.shape.batch, p.shape.tokens, p.shape.heads):
        raise ValueError(f"arguments of shape {a._dims} for a plan of "
                         f"{(p.shape.batch, p.shape.tokens, p.shape.heads)}")


def tree_forward_args(p: TreePlan, a: TreeArgs, scratch, stream=None) -> None:
    """``mla_tree_forward`` with prebuilt arguments."""
    _tree_dims(p, a)
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_tree_forward(ctypes.byref(p), ctypes.byref(a), sp, sb, _stream_of(a, stream)), "mla_tree_forward")


def tree_forward(p: TreePlan, q, kv, out, lse, scratch, *, stream=None, **kw) -> None:
    """Attention of each request's drafted tokens over its committed rows and the drafted rows that their
    masks name (arguments as for :func:`tree_make_args`)."""
    tree_forward_args(p, tree_make_args(q, kv, out, lse, **kw), scratch, stream)


def tree_weights_args(p: TreePlan, a: TreeArgs, scratch, weights, *, decay: float = 1.0, stream=None) -> None:
    """``mla_tree_weights`` with prebuilt arguments: ``weights`` fp32 [rows], one entry per cache row."""
    torch = _torch or _tc()
    _tree_dims(p, a)
    w = _side(weights, "weights", torch.float32, a.kv_rows)
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_tree_weights(ctypes.byref(p), ctypes.byref(a), w, float(decay), sp, sb, _stream_of(a, stream)),
           "mla_tree_weights")


def tree_weights(p: TreePlan, q, kv, lse, scratch, weights, *, decay: float = 1.0, stream=None, **kw) -> None:
    """``weights[row] = decay * weights[row] +`` the attention weight the row got from every token and head,
    given the log-sum-exps that :func:`tree_forward` returned."""
    tree_weights_args(p, tree_make_args(q, kv, None, lse, **kw), scratch, weights, decay=decay, stream=stream)


def tree_commit(kv, accept, n_accept, *, d_pos, d_pos_out=None, row_offset=None, row_positions=None,
                row_weights=None, kv_rows: int | None = None, row_stride: int | None = None, stream=None) -> None:
    """``mla_tree_commit``: rows ``d_pos + accept[b, k]`` move to ``d_pos + k`` for k < n_accept[b]
    (``accept``: int32 [B, Q]); ``d_pos_out`` (may be ``d_pos``) takes d_pos + n_accept."""
    torch = _torch or _tc()
    B, Q = accept.shape
    i32, dev = torch.int32, _device()
    kvp, rows, stride, fp8 = _quick_cache(kv, dev, torch) or _cache(kv, None, None)
    if kv_rows is not None or row_stride is not None:
        kvp, rows, stride, fp8 = _cache(kv, kv_rows, row_stride)
    args = _COMMIT_ARGS.pack(
        kvp, rows, stride, fp8, B, Q, _quick(accept, "accept", i32, (B, Q), dev),
        _quick(n_accept, "n_accept", i32, (B,), dev), _quick(d_pos, "d_pos", i32, (B,), dev),
        0 if d_pos_out is None else _quick(d_pos_out, "d_pos_out", i32, (B,), dev),
        0 if row_offset is None else _quick(row_offset, "row_offset", torch.int64, (B,), dev),
        0 if row_positions is None else _side(row_positions, "row_positions", i32, rows),
        0 if row_weights is None else _side(row_weights, "row_weights", torch.float32, rows))
    _check(lib().mla_tree_commit(args, _stream(stream)), "mla_tree_commit")


def evict_alloc_scratch(*, batch: int, keep: int, device=None):
    """Scratch of :func:`evict` for a batch and a budget."""
    torch = _torch or _tc()
    n = int(lib().mla_evict_scratch_bytes(_int(batch, "batch"), _int(keep, "keep")))
    if n == 0:
        raise ValueError("batch must be 1 .. 65535 and keep at least 1")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def evict_make_args(kv, weights, positions, *, d_pos, next_pos, keep: int, sink: int = 0, recent: int = 0,
                    row_offset=None, max_rows: int | None = None, weights_out=None, positions_out=None,
                    d_pos_out=None, kv_rows: int | None = None, row_stride: int | None = None) -> EvictArgs:
    """Arguments of :func:`evict_args`.  ``weights`` fp32 [rows] and ``positions`` int32 [rows] have an entry
    per cache row; the ``*_out`` tensors default to the inputs (in place).  ``max_rows``: largest ``d_pos``
    expected (sizes the launch; default: the cache's rows)."""
    torch = _torch or _tc()
    B = int(d_pos.shape[0])
    kvp, rows, stride, fp8 = _cache(kv, kv_rows, row_stride)
    wo = weights if weights_out is None else weights_out
    po = positions if positions_out is None else positions_out
    do = d_pos if d_pos_out is None else d_pos_out
    a = EvictArgs(kv=kvp, kv_rows=rows, row_stride=stride, kv_fp8=fp8, batch=B, keep=_int(keep, "keep"),
                  sink=_int(sink, "sink"), recent=_int(recent, "recent"),
                  max_rows=min(rows, 0x7fffffff) if max_rows is None else _int(max_rows, "max_rows"),
                  weights=_side(weights, "weights", torch.float32, rows),
                  positions=_side(positions, "positions", torch.int32, rows),
                  d_pos=_need(d_pos, "d_pos", torch.int32, (B,)),
                  next_pos=_need(next_pos, "next_pos", torch.int32, (B,)),
                  row_offset=_maybe(row_offset, "row_offset", torch.int64, (B,)),
                  weights_out=_side(wo, "weights_out", torch.float32, rows),
                  positions_out=_side(po, "positions_out", torch.int32, rows),
                  d_pos_out=_need(do, "d_pos_out", torch.int32, (B,)))
    a._device = _device()
    a._keep = (kv, weights, positions, d_pos, next_pos, row_offset, wo, po, do)
    return a


def evict_args(a: EvictArgs, scratch, stream=None) -> None:
    """``mla_evict`` with prebuilt arguments."""
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_evict(ctypes.byref(a), sp, sb, _stream_of(a, stream)), "mla_evict")


def evict(kv, weights, positions, scratch, *, stream=None, **kw) -> None:
    """Keep each request's ``keep`` rows of largest weight (the first ``sink`` and the last ``recent``
    positions before all others), compacted in place (arguments as for :func:`evict_make_args`)."""
    evict_args(evict_make_args(kv, weights, positions, **kw), scratch, stream)


# ---- a latent cache in 4 bits, in pages --------------------------------------

def paged_alloc(n_pages: int, page_rows: int, device=None):
    """Pages of a 4-bit cache: uint8 [n_pages, page_rows, 416], zeros (every row then stands for zeros)."""
    torch = _torch or _tc()
    return torch.zeros(n_pages, page_rows, Q4_ROW, dtype=torch.uint8, device=device or "cuda")


def _pool(pages, row_bytes=None):
    """(pointer, page stride in bytes, pages, rows per page, bytes per row) of pages [n, page_rows, ..] whose
    rows are contiguous within a page."""
    torch = _torch or _tc()
    if not isinstance(pages, torch.Tensor) or pages.dim() != 3:
        raise ValueError("pages must be a tensor [n_pages, page_rows, row]")
    p = _need(pages, "pages", pages.dtype, contiguous=False)
    n, rows, width = pages.shape
    size = pages.element_size()
    if n < 1 or rows < 1 or width < 1:
        raise ValueError("pages has no rows")
    if row_bytes is not None and (pages.dtype is not torch.uint8 or width != row_bytes):
        raise ValueError(f"pages: {tuple(pages.shape)} of {pages.dtype}, expected [*, *, {row_bytes}] of torch.uint8")
    if pages.stride(2) != 1 and width > 1 or pages.stride(1) != width and rows > 1:
        raise ValueError("the rows of a page must be contiguous")
    return p, (pages.stride(0) if n > 1 else rows * width) * size, _int(n, "n_pages"), rows, width * size


def _paged_cache(pages, page_table, kv_scale, batch) -> PagedCache:
    torch = _torch or _tc()
    p, stride, n, rows, _ = _pool(pages, Q4_ROW)
    table = _need(page_table, "page_table", torch.int32, (batch, None))
    return PagedCache(pages=p, page_stride=stride, n_pages=n, page_rows=rows, page_table=table,
                      columns=_int(page_table.shape[1], "columns"), kv_scale=float(kv_scale))


def paged_append_make_args(table: RopeTable, positions, *, q_rope=None, q=None, c=None, k_rope=None, pages=None,
                           page_table=None, d_pos=None, n_tokens=None, c_norm=None, k_norm=None, q_norm=None,
                           eps: float = 1e-6, kv_scale: float = 1.0) -> PagedAppendArgs:
    """Arguments of :func:`paged_append_args`.

    ``positions``: int32 [B, N].  Queries: ``q_rope`` bf16 [B, N, H, 64] (any strides, multiples of 8),
    normalised with ``q_norm`` (bf16 [64]) if given, is rotated into ``q[..., 512:]`` of bf16 [B, N, H, 576] (not expanded).
    Rows: ``c`` bf16 [B, N, 512], normalised with ``c_norm`` (bf16 [512]) if given, goes in 4 bits, and ``k_rope``
    bf16 [B, N, 64], normalised with ``k_norm`` if given and rotated, in bf16 to row ``d_pos[b] + n`` of request b
    in ``pages`` (uint8 [n_pages, page_rows, 416]) by ``page_table`` (int32 [B, columns]).  ``kv_scale``: a power
    of two.  Either part may be left out."""
    torch = _torch or _tc()
    B, N = positions.shape
    a = PagedAppendArgs(batch=int(B), tokens=int(N), rot_dim=table.rot_dim, interleaved=int(table.interleaved),
                        amplitude=table.amplitude, turns=_need(table.turns, "table", torch.int64),
                        positions=_need(positions, "positions", torch.int32, (B, N)),
                        n_tokens=_maybe(n_tokens, "n_tokens", torch.int32, (B,)), eps=float(eps))
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q go together")
    if q is not None:
        H = q.shape[2] if q.dim() == 4 else -1
        a.heads = int(H)
        a.q_rope, a.q_rope_batch, a.q_rope_token, a.q_rope_head = _strides(q_rope, "q_rope", (B, N, H, D_ROPE), 3)
        _need(q, "q", torch.bfloat16, (B, N, H, D_ROW), contiguous=False)
        part = q[..., D_LATENT:]
        _apart(part, "q", 3)
        a.q_out, a.q_out_batch, a.q_out_token, a.q_out_head = _strides(part, "q", (B, N, H, D_ROPE), 3)
    elif q_norm is not None:
        raise ValueError("q_norm belongs to q_rope and q")
    rows = (c, k_rope, pages, page_table, d_pos)
    if any(t is None for t in rows) != all(t is None for t in rows):
        raise ValueError("c, k_rope, pages, page_table and d_pos go together")
    if pages is None and not (c_norm is None and k_norm is None):
        raise ValueError("c_norm and k_norm belong to the rows")
    if pages is not None:
        a.c, a.c_batch, a.c_token = _strides(c, "c", (B, N, D_LATENT), 2)
        a.k_rope, a.k_rope_batch, a.k_rope_token = _strides(k_rope, "k_rope", (B, N, D_ROPE), 2)
        a.cache = _paged_cache(pages, page_table, kv_scale, B)
        a.d_pos = _need(d_pos, "d_pos", torch.int32, (B,))
    a.c_norm = _maybe(c_norm, "c_norm", torch.bfloat16, (D_LATENT,))
    a.k_norm = _maybe(k_norm, "k_norm", torch.bfloat16, (D_ROPE,))
    a.q_norm = _maybe(q_norm, "q_norm", torch.bfloat16, (D_ROPE,))
    a._device = _device()
    a._keep = (table, positions, q_rope, q, c, k_rope, pages, page_table, d_pos, n_tokens, c_norm, k_norm, q_norm)
    return a


def paged_append_args(a: PagedAppendArgs, stream=None) -> None:
    """``mla_paged_append`` with prebuilt arguments."""
    _check(lib().mla_paged_append(ctypes.byref(a), _stream_of(a, stream)), "mla_paged_append")


def paged_append(table: RopeTable, positions, *, stream=None, **kw) -> None:
    """Normalise and rotate the new tokens' queries and keys, normalise and quantise their latents, and write
    their rows (arguments as for :func:`paged_append_make_args`)."""
    paged_append_args(paged_append_make_args(table, positions, **kw), stream)


def paged_read_make_args(out, pages, page_table, *, first=None, n_rows=None, kv_scale: float = 1.0) -> PagedReadArgs:
    """Arguments of :func:`paged_read_args`.  ``out``: bf16 [B, N, 576], any strides that are multiples of 8, not expanded;
    ``first``, ``n_rows``: int32 [B] (None: 0, N)."""
    torch = _torch or _tc()
    if out.dim() != 3:
        raise ValueError("out must be [B, N, 576]")
    B, N, _ = out.shape
    _apart(out, "out", 2)
    a = PagedReadArgs(cache=_paged_cache(pages, page_table, kv_scale, B), batch=int(B), rows=int(N),
                      first=_maybe(first, "first", torch.int32, (B,)), n_rows=_maybe(n_rows, "n_rows", torch.int32, (B,)))
    a.out, a.out_batch, a.out_row = _strides(out, "out", (B, N, D_ROW), 2)
    if N == 1:
        a.out_row = D_ROW                  # never used
    a._device = _device()
    a._keep = (out, pages, page_table, first, n_rows)
    return a


def paged_read_args(a: PagedReadArgs, stream=None) -> None:
    """``mla_paged_read`` with prebuilt arguments."""
    _check(lib().mla_paged_read(ctypes.byref(a), _stream_of(a, stream)), "mla_paged_read")


def paged_read(out, pages, page_table, *, stream=None, **kw) -> None:
    """``out[b, n] =`` row ``first[b] + n`` of request b as bf16 values, for n < n_rows[b] (arguments as for
    :func:`paged_read_make_args`)."""
    paged_read_args(paged_read_make_args(out, pages, page_table, **kw), stream)


def paged_plan(*, batch: int, tokens: int, heads: int, scale: float, num_sms: int = 0, pdl: bool = False,
               stall_test: bool = False) -> PagedPlan:
    """``mla_paged_plan``: up to ``tokens`` (<= 64) new tokens per request."""
    s = PagedShape(batch=_int(batch, "batch"), tokens=_int(tokens, "tokens"), heads=_int(heads, "heads"), scale=scale,
                   num_sms=_int(num_sms, "num_sms"), pdl=int(bool(pdl)), stall_test=int(bool(stall_test)))
    p = PagedPlan()
    _check(lib().mla_paged_plan(ctypes.byref(s), ctypes.byref(p)), "mla_paged_plan")
    return p


def paged_alloc_scratch(p: PagedPlan, device=None):
    """Allocate and zero the scratch of a paged plan (outside capture); :func:`status_word` reads its status."""
    return alloc_scratch(p, device)


def paged_make_args(q, pages, page_table, out, lse, *, d_pos, n_tokens=None, window: int = 0, sink: int = 0,
                    kv_scale: float = 1.0) -> PagedArgs:
    """Arguments of :func:`paged_forward_args`.

    ``q``: bf16 [B, Q, H, 576]; ``pages``: uint8 [n_pages, page_rows, 416]; ``page_table``: int32 [B, columns];
    ``out``: bf16 or fp32 [B, Q, H, 512]; ``lse``: fp32 [B, Q, H].  Token i stands in row ``d_pos[b] + i`` and
    attends the rows up to it: all of them, or with a ``window`` the last ``window`` and the first ``sink``."""
    torch = _torch or _tc()
    if q.dim() != 4:
        raise ValueError("q must be [B, Q, H, 576]")
    B, Q, H, _ = q.shape
    a = PagedArgs(cache=_paged_cache(pages, page_table, kv_scale, B),
                  q=_need(q, "q", torch.bfloat16, (B, Q, H, D_ROW)), d_pos=_need(d_pos, "d_pos", torch.int32, (B,)),
                  n_tokens=_maybe(n_tokens, "n_tokens", torch.int32, (B,)), window=_int(window, "window"),
                  sink=_int(sink, "sink"),
                  out=_need(out, "out", (torch.bfloat16, torch.float32), (B, Q, H, D_LATENT)),
                  out_fp32=int(out.dtype == torch.float32), lse=_need(lse, "lse", torch.float32, (B, Q, H)))
    a._device = _device()
    a._keep = (q, pages, page_table, out, lse, d_pos, n_tokens)
    a._dims = (int(B), int(Q), int(H))
    return a


def paged_forward_args(p: PagedPlan, a: PagedArgs, scratch, stream=None) -> None:
    """``mla_paged_forward`` with prebuilt arguments."""
    _tree_dims(p, a)
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_paged_forward(ctypes.byref(p), ctypes.byref(a), sp, sb, _stream_of(a, stream)),
           "mla_paged_forward")


def paged_forward(p: PagedPlan, q, pages, page_table, out, lse, scratch, *, stream=None, **kw) -> None:
    """Attention of each request's new tokens over its rows in the 4-bit cache (arguments as for
    :func:`paged_make_args`)."""
    paged_forward_args(p, paged_make_args(q, pages, page_table, out, lse, **kw), scratch, stream)


def pages_alloc_scratch(pages, page_table, device=None):
    """Scratch of :func:`pages_fork` and :func:`pages_compact` for a pool and a table."""
    torch = _torch or _tc()
    B, columns = page_table.shape
    n = int(lib().mla_pages_scratch_bytes(_int(B, "batch"), _int(columns, "columns"), _int(pages.shape[0], "n_pages")))
    if n == 0:
        raise ValueError("batch must be 1 .. 4096, and the table and the pool below 2^30 entries")
    return torch.empty(n, dtype=torch.uint8, device=device or pages.device)


def _pool_args(cls, pages, page_table, page_table_out, **kw):
    torch = _torch or _tc()
    p, stride, n, rows, row_bytes = _pool(pages)
    t = _need(page_table, "page_table", torch.int32, (None, None))
    B, columns = page_table.shape
    to = t if page_table_out is None else _need(page_table_out, "page_table_out", torch.int32, (B, columns))
    return cls(pages=p, page_stride=stride, n_pages=n, page_rows=rows, row_bytes=_int(row_bytes, "row bytes"),
               batch=_int(B, "batch"), columns=_int(columns, "columns"), page_table=t, page_table_out=to, **kw), B, n


def pages_fork_make_args(pages, page_table, d_pos, refs, *, parent=None, rows=None, reserve: int = 0, window: int = 0,
                         sink: int = 0, page_table_out=None, d_pos_out=None, missing) -> PagesForkArgs:
    """Arguments of :func:`pages_fork_args`.  ``pages``: [n_pages, page_rows, row] of any type, rows of a multiple of
    16 bytes; ``page_table``: int32 [B, columns]; ``d_pos``, ``parent``, ``rows``: int32 [B]; ``refs``: int32
    [n_pages], written; ``missing``: int32 [1], written.  The ``*_out`` tensors default to the inputs (in place)."""
    torch = _torch or _tc()
    a, B, n = _pool_args(PagesForkArgs, pages, page_table, page_table_out, reserve=_int(reserve, "reserve"),
                         window=_int(window, "window"), sink=_int(sink, "sink"))
    a.d_pos = _need(d_pos, "d_pos", torch.int32, (B,))
    a.d_pos_out = a.d_pos if d_pos_out is None else _need(d_pos_out, "d_pos_out", torch.int32, (B,))
    a.parent = _maybe(parent, "parent", torch.int32, (B,))
    a.rows = _maybe(rows, "rows", torch.int32, (B,))
    a.refs = _need(refs, "refs", torch.int32, (n,))
    a.missing = _need(missing, "missing", torch.int32, (1,))
    a._device = _device()
    a._keep = (pages, page_table, page_table_out, d_pos, d_pos_out, parent, rows, refs, missing)
    return a


def pages_fork_args(a: PagesForkArgs, scratch, stream=None) -> None:
    """``mla_pages_fork`` with prebuilt arguments."""
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_pages_fork(ctypes.byref(a), sp, sb, _stream_of(a, stream)), "mla_pages_fork")


def pages_fork(pages, page_table, d_pos, refs, scratch, *, stream=None, **kw) -> None:
    """Every request goes on from the first ``rows[b]`` rows of request ``parent[b]`` (its own rows, all of them, where
    not given; a parent outside 0 .. B - 1 ends it): full pages are shared, a last page that others need is copied,
    pages for ``reserve`` rows more are taken, and all others are free (arguments as for
    :func:`pages_fork_make_args`)."""
    pages_fork_args(pages_fork_make_args(pages, page_table, d_pos, refs, **kw), scratch, stream)


def pages_compact_make_args(pages, page_table, refs, *, page_table_out=None, refs_out=None, used) -> PagesCompactArgs:
    """Arguments of :func:`pages_compact_args` (tensors as for :func:`pages_fork_make_args`; ``used``: int32 [1],
    written).  The ``*_out`` tensors default to the inputs (in place)."""
    torch = _torch or _tc()
    a, _, n = _pool_args(PagesCompactArgs, pages, page_table, page_table_out)
    a.refs = _need(refs, "refs", torch.int32, (n,))
    a.refs_out = a.refs if refs_out is None else _need(refs_out, "refs_out", torch.int32, (n,))
    a.used = _need(used, "used", torch.int32, (1,))
    a._device = _device()
    a._keep = (pages, page_table, page_table_out, refs, refs_out, used)
    return a


def pages_compact_args(a: PagesCompactArgs, scratch, stream=None) -> None:
    """``mla_pages_compact`` with prebuilt arguments."""
    sp, sb = _scratch_here(scratch)
    _check(lib().mla_pages_compact(ctypes.byref(a), sp, sb, _stream_of(a, stream)), "mla_pages_compact")


def pages_compact(pages, page_table, refs, scratch, *, stream=None, **kw) -> None:
    """Move the pages in use (``refs`` above 0) to the front of the pool (arguments as for
    :func:`pages_compact_make_args`)."""
    pages_compact_args(pages_compact_make_args(pages, page_table, refs, **kw), scratch, stream)


def floor_empty_pair(a, b, *, pdl: bool = True, stream=None) -> None:
    """``mla_floor_empty_pair``: two empty kernels with launch shapes a and b,
    each a (grid, block, dynamic shared bytes) triple."""
    _check(lib().mla_floor_empty_pair(int(a[0]), int(a[1]), int(a[2]), int(b[0]), int(b[1]), int(b[2]),
                                      int(bool(pdl)), _stream(stream)), "mla_floor_empty_pair")


def floor_read(src, nbytes: int, ctas: int, sink, status, *, pdl: bool = True, stream=None) -> None:
    """``mla_floor_read``: one kernel of ``ctas`` CTAs reading ``nbytes`` of ``src`` with bulk copies;
    ``sink``: uint32/int32 [ctas], ``status``: int32 [1] (zeroed by the caller)."""
    _check(lib().mla_floor_read(_ptr(src), int(nbytes), int(ctas), _ptr(sink), _ptr(status), int(bool(pdl)),
                                _stream(stream)), "mla_floor_read")


def floor_gather(kv, rows, ctas: int, sink, status, *, row_bytes: int | None = None, pdl: bool = True,
                 stream=None) -> None:
    """``mla_floor_gather``: one kernel of ``ctas`` CTAs gathering the cache rows listed in ``rows``
    (int64) with one bulk copy per row; ``kv``: [kv_rows, row_stride] (bf16 or bytes)."""
    stride = kv.stride(0) * kv.element_size()
    rb = int(row_bytes) if row_bytes is not None else kv.shape[1] * kv.element_size()
    _check(lib().mla_floor_gather(_ptr(kv), int(kv.shape[0]), int(stride), rb, _ptr(rows), int(rows.numel()),
                                  int(ctas), _ptr(sink), _ptr(status), int(bool(pdl)), _stream(stream)),
           "mla_floor_gather")


def abi_version() -> int:
    return int(lib().mla_decode_abi_version())
