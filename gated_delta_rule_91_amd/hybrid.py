"""The operators beside KDA in a hybrid stack, over the C ABI of
``include/kda_hybrid.h``: the plan of a serving step, a paged key/value cache
held in 4 bits with the attention that reads it, and a gated linear
recurrence with its gradients.

As in the package itself this module only checks tensors, passes device
pointers and the stream, and allocates outputs and workspaces; the work is in
the library's HIP kernels.  Everything here is re-exported by the package.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

from . import _check, _cu, _expect, _expect_workspace, _io_code, _ptr, _stream, _torch, lib

__all__ = ["HYBRID_EXPORTS", "Cache4", "plan_requests", "cache4_append", "cache4_read", "cache4_attention",
           "cache4_attention_workspace_size", "recurrence_workspace_size", "recurrence_backward_workspace_size",
           "recurrence_prefill", "recurrence_prefill_for_backward", "recurrence_backward", "recurrence_autograd",
           "recurrence_step"]

HYBRID_EXPORTS = ("kda_plan_requests", "kda_cache4_append", "kda_cache4_read", "kda_cache4_attention_workspace_size",
                  "kda_cache4_attention", "kda_recurrence_workspace_size", "kda_recurrence_backward_workspace_size",
                  "kda_recurrence_prefill", "kda_recurrence_prefill_for_backward", "kda_recurrence_backward",
                  "kda_recurrence_step")
PAGE_SIZES = (16, 32, 64, 128, 256)


class KdaCache4(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class KdaCache4AttentionProblem(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int64), ("tokens", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_q", ctypes.c_int64), ("max_len", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class KdaRecurrenceProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int64),
                ("n_seq", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("log_alpha_min", ctypes.c_float)]


_bound = None


def _hlib() -> ctypes.CDLL:
    """lib() with the signatures of these calls declared."""
    global _bound
    L = lib()
    if _bound is not L:
        P, I64, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        C, A, R = (ctypes.POINTER(t) for t in (KdaCache4, KdaCache4AttentionProblem, KdaRecurrenceProblem))
        L.kda_plan_requests.argtypes = [I64, I64, I32, I32, P, P, P, I64, P, P, P, P, P, P]
        L.kda_cache4_append.argtypes = [C, I64, I32, P, P, P, P]
        L.kda_cache4_read.argtypes = [C, I64, I32, P, P, P, P]
        L.kda_cache4_attention_workspace_size.argtypes = [C, A]
        L.kda_cache4_attention.argtypes = [C, A, P, P, P, P, P, P, P, SZ, P]
        L.kda_recurrence_workspace_size.argtypes = [R]
        L.kda_recurrence_backward_workspace_size.argtypes = [R]
        L.kda_recurrence_prefill.argtypes = [R, P, P, P, P, P, P, P, P, SZ, P]
        L.kda_recurrence_prefill_for_backward.argtypes = [R, P, P, P, P, P, P, P, P, SZ, P]
        L.kda_recurrence_backward.argtypes = [R, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.kda_recurrence_step.argtypes = [I64, I64, I32, F32, P, P, P, P, P, P]
        for f in HYBRID_EXPORTS:
            getattr(L, f).restype = SZ if f.endswith("workspace_size") else I32
        _bound = L
    return L


def _on(device):
    """A call's kernels run on its tensors' device, whichever is current."""
    torch = _torch()
    if not device.type == "cuda" or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _scratch(nbytes: int, device, stream):
    """A workspace of the call's own, in the pool of the stream that uses it:
    it may be handed out again as soon as the call returns, on that stream."""
    torch = _torch()
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(workspace, nbytes: int, device, stream):
    """(tensor to keep alive, pointer, bytes) of the workspace given, or of one made here."""
    if workspace is None:
        workspace = _scratch(nbytes, device, stream)
        if workspace is None:
            return None, None, 0
    else:
        _expect_workspace(workspace, device)
    return workspace, _ptr(workspace), workspace.numel()


def plan_requests(past_lens, new_lens, block_table, free_pages, page_size: int, tokens: int, stream=None):
    """The plan of a serving step from the requests' lengths (kda_plan_requests).

    past_lens, new_lens: int32 [n]; block_table: int32 [n, max_pages], whose
    entries for the pages that the new tokens begin are written in place, off
    free_pages (int32 [m], read only); tokens: rows of the packed batch, the
    sum of new_lens or more.  Returns (cu_seqlens int32 [n+1], total_lens
    int32 [n], slot_map int64 [tokens], pages_taken int32 [1]); the caller
    drops the first pages_taken entries of free_pages."""
    torch = _torch()
    dev = past_lens.device
    n = past_lens.shape[0] if past_lens.dim() == 1 else -1
    _expect("past_lens", past_lens, (max(n, 0),), torch.int32, dev)
    _expect("new_lens", new_lens, (n,), torch.int32, dev)
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [n, max_pages] and free_pages 1-D")
    _expect("block_table", block_table, (n, block_table.shape[1]), torch.int32, dev)
    _expect("free_pages", free_pages, (free_pages.shape[0],), torch.int32, dev)
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {page_size!r}")
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    cu = torch.empty(n + 1, dtype=torch.int32, device=dev)
    total = torch.empty(n, dtype=torch.int32, device=dev)
    taken = torch.empty(1, dtype=torch.int32, device=dev)
    slots = torch.empty(tokens, dtype=torch.int64, device=dev)
    with _on(dev):
        _check("kda_plan_requests", _hlib().kda_plan_requests(
            n, tokens, page_size, block_table.shape[1], _ptr(past_lens), _ptr(new_lens), _ptr(block_table),
            free_pages.shape[0], _ptr(free_pages), _ptr(cu), _ptr(total), _ptr(slots), _ptr(taken),
            _stream(stream, dev)))
    return cu, total, slots, taken


class Cache4:
    """A paged key/value cache held in 4 bits: k, v uint8 [pages, heads,
    page_size, d/2] (two e2m1 values a byte) and k_scale, v_scale uint8
    [pages, heads, page_size, d/32] (a biased power of two for 32 channels)."""

    def __init__(self, k, k_scale, v, v_scale):
        torch = _torch()
        if k.dim() != 4 or k.shape[2] not in PAGE_SIZES or k.shape[3] not in (32, 64):
            raise ValueError(f"k must be [pages, heads, page_size, d/2] with page_size in {PAGE_SIZES} and d 64 or "
                             f"128, got {tuple(k.shape)}")
        pages, heads, page_size, half = k.shape
        scales = (pages, heads, page_size, half // 16)
        _expect("k", k, k.shape, torch.uint8, k.device)
        _expect("k_scale", k_scale, scales, torch.uint8, k.device)
        _expect("v", v, k.shape, torch.uint8, k.device)
        _expect("v_scale", v_scale, scales, torch.uint8, k.device)
        self.k, self.k_scale, self.v, self.v_scale = k, k_scale, v, v_scale
        self.pages, self.heads, self.page_size, self.d = pages, heads, page_size, 2 * half
        self.device = k.device

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, d: int, device="cuda") -> "Cache4":
        """A cache of zeros."""
        torch = _torch()
        codes = [torch.zeros((pages, heads, page_size, d // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros((pages, heads, page_size, d // 32), dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1])

    def _struct(self) -> KdaCache4:
        return KdaCache4(self.pages, self.page_size, self.heads, self.d, _ptr(self.k), _ptr(self.k_scale),
                         _ptr(self.v), _ptr(self.v_scale))


def _expect_slots(slot_map, device) -> int:
    torch = _torch()
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be 1-D")
    _expect("slot_map", slot_map, slot_map.shape, torch.int64, device)
    return slot_map.shape[0]


def cache4_append(cache: Cache4, k, v, slot_map, stream=None) -> None:
    """Round k, v [T, heads, d] (bf16 or fp32) into the cache at slot_map int64
    [T] (page * page_size + offset; slots outside the cache are dropped, and no
    two rows may name one slot)."""
    T = _expect_slots(slot_map, cache.device)
    io = _io_code(k.dtype)
    _expect("k", k, (T, cache.heads, cache.d), k.dtype, cache.device)
    _expect("v", v, (T, cache.heads, cache.d), k.dtype, cache.device)
    with _on(cache.device):
        _check("kda_cache4_append", _hlib().kda_cache4_append(
            cache._struct(), T, io, _ptr(k), _ptr(v), _ptr(slot_map), _stream(stream, cache.device)))


def cache4_read(cache: Cache4, slot_map, dtype, stream=None):
    """(k, v) [T, heads, d] of the rows at slot_map, as the values they stand
    for; zeros for slots outside the cache."""
    torch = _torch()
    T = _expect_slots(slot_map, cache.device)
    io = _io_code(dtype)
    k, v = (torch.empty((T, cache.heads, cache.d), dtype=dtype, device=cache.device) for _ in range(2))
    with _on(cache.device):
        _check("kda_cache4_read", _hlib().kda_cache4_read(
            cache._struct(), T, io, _ptr(slot_map), _ptr(k), _ptr(v), _stream(stream, cache.device)))
    return k, v


def _attention_problem(cache, q, block_table, n_seq, scale, max_q, max_len) -> KdaCache4AttentionProblem:
    T, heads, _ = q.shape
    if heads % cache.heads:
        raise ValueError(f"{heads} query heads over {cache.heads} key/value heads")
    scale = 1.0 / math.sqrt(cache.d) if scale is None else float(scale)
    if max_len is None:
        max_len = block_table.shape[1] * cache.page_size
    return KdaCache4AttentionProblem(n_seq, T, heads, block_table.shape[1], max(int(max_q), 1), max(int(max_len), 0),
                                     _io_code(q.dtype), scale)


def _attention_inputs(q, cache, block_table, total_lens, cu_seqlens, scale, max_q, max_len):
    torch = _torch()
    dev = cache.device
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [T, heads, d] and block_table [n_seq, max_pages]")
    T, heads, d = q.shape
    n_seq = T if cu_seqlens is None else _cu(cu_seqlens, dev)
    _expect("q", q, (T, heads, cache.d), q.dtype, dev)
    _expect("block_table", block_table, (n_seq, block_table.shape[1]), torch.int32, dev)
    _expect("total_lens", total_lens, (n_seq,), torch.int32, dev)
    if max_q is None:
        max_q = 1 if cu_seqlens is None else max(T, 1)
    return _attention_problem(cache, q, block_table, n_seq, scale, max_q, max_len)


def cache4_attention_workspace_size(q, cache: Cache4, block_table, total_lens, cu_seqlens=None, max_q=None,
                                    max_len=None) -> int:
    """Bytes of workspace that cache4_attention needs for these arguments."""
    p = _attention_inputs(q, cache, block_table, total_lens, cu_seqlens, None, max_q, max_len)
    return _hlib().kda_cache4_attention_workspace_size(cache._struct(), p)


def cache4_attention(q, cache: Cache4, block_table, total_lens, cu_seqlens=None, g=None,
                     scale: Optional[float] = None, max_q: Optional[int] = None, max_len: Optional[int] = None,
                     out=None, workspace=None, stream=None):
    """Causal grouped-query attention over the 4-bit cache (kda_cache4_attention).

    q [T, heads, d] (bf16 or fp32), packed by cu_seqlens int32 [n+1], or one
    row for each of T sequences where that is None; block_table int32 [n,
    max_pages]; total_lens int32 [n], the tokens each sequence has, its
    queries the newest of them (append their keys and values first); g
    [T, heads, d]: the read-out gate, out = attention * sigmoid(g); scale
    defaults to 1/sqrt(d).  max_q and max_len, about the most queries and the
    most tokens of a sequence, steer how the work is split, and nothing else.
    Returns out [T, heads, d]."""
    torch = _torch()
    dev = cache.device
    p = _attention_inputs(q, cache, block_table, total_lens, cu_seqlens, scale, max_q, max_len)
    _expect("g", g, q.shape, q.dtype, dev)
    _expect("out", out, q.shape, q.dtype, dev)
    if out is None:
        out = torch.empty_like(q)
    c = cache._struct()
    with _on(dev):
        ws, ws_ptr, nbytes = _workspace(workspace, _hlib().kda_cache4_attention_workspace_size(c, p), dev, stream)
        _check("kda_cache4_attention", _hlib().kda_cache4_attention(
            c, p, _ptr(q), _ptr(block_table), _ptr(total_lens), _ptr(cu_seqlens), _ptr(g), _ptr(out), ws_ptr, nbytes,
            _stream(stream, dev)))
    return out


def _recurrence_problem(x, log_alpha, log_alpha_min, g, cu_seqlens):
    """(problem, rows of the states) of checked inputs."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    io = _io_code(x.dtype)
    _expect("log_alpha", log_alpha, (B, T, D), torch.float32, x.device)
    _expect("g", g, (B, T, D), x.dtype, x.device)
    n_seq = -1
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("a packed batch is [1, T, D]")
        n_seq = _cu(cu_seqlens, x.device)
    return KdaRecurrenceProblem(B, T, D, n_seq, io, float(log_alpha_min)), B if n_seq < 0 else n_seq


def recurrence_workspace_size(p: KdaRecurrenceProblem) -> int:
    return _hlib().kda_recurrence_workspace_size(p)


def recurrence_backward_workspace_size(p: KdaRecurrenceProblem) -> int:
    return _hlib().kda_recurrence_backward_workspace_size(p)


def _recurrence_forward(name, size, x, log_alpha, log_alpha_min, g, state_in, cu_seqlens, out, state_out, want_state,
                        workspace, stream):
    torch = _torch()
    p, n = _recurrence_problem(x, log_alpha, log_alpha_min, g, cu_seqlens)
    dev, D = x.device, x.shape[2]
    _expect("state_in", state_in, (n, D), torch.float32, dev)
    _expect("out", out, x.shape, x.dtype, dev)
    _expect("state_out", state_out, (n, D), torch.float32, dev)
    if out is None:
        out = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty((n, D), dtype=torch.float32, device=dev)
    with _on(dev):
        ws, ws_ptr, nbytes = _workspace(workspace, size(p), dev, stream)
        _check(name, getattr(_hlib(), name)(
            p, _ptr(x), _ptr(log_alpha), _ptr(g), _ptr(state_in), _ptr(cu_seqlens), _ptr(out), _ptr(state_out), ws_ptr,
            nbytes, _stream(stream, dev)))
    return out, state_out, ws


def recurrence_prefill(x, log_alpha, log_alpha_min: float, g=None, state_in=None, cu_seqlens=None, out=None,
                       state_out=None, want_state: bool = True, workspace=None, stream=None):
    """h_t = exp(max(log_alpha_t, log_alpha_min)) h_(t-1) + x_t per channel,
    out_t = h_t * sigmoid(g_t) (or h_t): x, g [B, T, D] bf16 or fp32, log_alpha
    fp32.  A packed batch is [1, T, D] with cu_seqlens int32 [n+1].  States are
    fp32 [B or n, D].  Returns (out, final states)."""
    out, state, _ = _recurrence_forward("kda_recurrence_prefill", recurrence_workspace_size, x, log_alpha,
                                        log_alpha_min, g, state_in, cu_seqlens, out, state_out, want_state, workspace,
                                        stream)
    return out, state


def recurrence_prefill_for_backward(x, log_alpha, log_alpha_min: float, g=None, state_in=None, cu_seqlens=None,
                                    out=None, state_out=None, want_state: bool = True, workspace=None, stream=None):
    """recurrence_prefill that leaves what recurrence_backward continues from.
    Returns (out, final states, workspace)."""
    torch = _torch()
    out, state, ws = _recurrence_forward("kda_recurrence_prefill_for_backward", recurrence_backward_workspace_size, x,
                                         log_alpha, log_alpha_min, g, state_in, cu_seqlens, out, state_out, want_state,
                                         workspace, stream)
    return out, state, torch.empty(0, dtype=torch.uint8, device=x.device) if ws is None else ws


def recurrence_backward(x, log_alpha, log_alpha_min: float, workspace, g=None, state_in=None, cu_seqlens=None,
                        d_out=None, d_state=None, want_dstate: bool = True, stream=None) -> dict:
    """Gradients of <d_out, out> + <d_state, final states>, from the inputs and
    the workspace of recurrence_prefill_for_backward.  Returns a dict with dx,
    dg (dtype of x; dg None without g), dlog_alpha fp32 and dstate0 (None
    unless want_dstate)."""
    torch = _torch()
    p, n = _recurrence_problem(x, log_alpha, log_alpha_min, g, cu_seqlens)
    dev, D = x.device, x.shape[2]
    _expect("state_in", state_in, (n, D), torch.float32, dev)
    _expect("d_out", d_out, x.shape, x.dtype, dev)
    _expect("d_state", d_state, (n, D), torch.float32, dev)
    _expect_workspace(workspace, dev)
    r = dict(dx=torch.empty_like(x), dlog_alpha=torch.empty_like(log_alpha),
             dg=torch.empty_like(g) if g is not None else None,
             dstate0=torch.empty((n, D), dtype=torch.float32, device=dev) if want_dstate else None)
    with _on(dev):
        _check("kda_recurrence_backward", _hlib().kda_recurrence_backward(
            p, _ptr(x), _ptr(log_alpha), _ptr(g), _ptr(state_in), _ptr(cu_seqlens), _ptr(d_out), _ptr(d_state),
            _ptr(r["dx"]), _ptr(r["dlog_alpha"]), _ptr(r["dg"]), _ptr(r["dstate0"]), _ptr(workspace),
            workspace.numel(), _stream(stream, dev)))
    return r


_RECURRENCE_FUNCTION = None


def _recurrence_function():
    """The torch.autograd.Function over the training pair, created on first use."""
    global _RECURRENCE_FUNCTION
    if _RECURRENCE_FUNCTION is None:
        torch = _torch()

        class RecurrenceFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, log_alpha, g, state_in, log_alpha_min, cu_seqlens):
                out, state, ws = recurrence_prefill_for_backward(x, log_alpha, log_alpha_min, g=g, state_in=state_in,
                                                                 cu_seqlens=cu_seqlens)
                ctx.save_for_backward(x, log_alpha, g, state_in, cu_seqlens)
                ctx.workspace, ctx.log_alpha_min = ws, log_alpha_min
                ctx.set_materialize_grads(False)
                return out, state

            @staticmethod
            def backward(ctx, d_out, d_state):
                x, log_alpha, g, state_in, cu_seqlens = ctx.saved_tensors
                r = recurrence_backward(x, log_alpha, ctx.log_alpha_min, ctx.workspace, g=g, state_in=state_in,
                                        cu_seqlens=cu_seqlens, d_out=None if d_out is None else d_out.contiguous(),
                                        d_state=None if d_state is None else d_state.contiguous(),
                                        want_dstate=state_in is not None and ctx.needs_input_grad[3])
                return r["dx"], r["dlog_alpha"], r["dg"], r["dstate0"], None, None

        _RECURRENCE_FUNCTION = RecurrenceFunction
    return _RECURRENCE_FUNCTION


def recurrence_autograd(x, log_alpha, log_alpha_min: float, g=None, state_in=None, cu_seqlens=None):
    """Differentiable recurrence_prefill: returns (out, final states), and
    loss.backward() fills the gradients of x, log_alpha, g and state_in."""
    return _recurrence_function().apply(x, log_alpha, g, state_in, float(log_alpha_min), cu_seqlens)


def recurrence_step(x, log_alpha, state, log_alpha_min: float, g=None, out=None, stream=None):
    """One token of each of N sequences: x, g [N, D], log_alpha fp32; state
    [N, D] fp32, updated in place.  Returns out [N, D]."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    N, D = x.shape
    dev = x.device
    io = _io_code(x.dtype)
    _expect("log_alpha", log_alpha, (N, D), torch.float32, dev)
    _expect("state", state, (N, D), torch.float32, dev)
    _expect("g", g, (N, D), x.dtype, dev)
    _expect("out", out, (N, D), x.dtype, dev)
    if out is None:
        out = torch.empty_like(x)
    with _on(dev):
        _check("kda_recurrence_step", _hlib().kda_recurrence_step(
            N, D, io, float(log_alpha_min), _ptr(x), _ptr(log_alpha), _ptr(g), _ptr(state), _ptr(out),
            _stream(stream, dev)))
    return out
