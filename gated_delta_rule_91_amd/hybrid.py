"""The operators beside KDA in a hybrid stack, over the C ABI of
``include/kda_hybrid.h``: the plan of a serving step, a paged key/value cache
held in 4 bits with the attention that reads it, and a gated linear
recurrence with its gradients.

As in the package itself this module only checks tensors, passes device
pointers and the stream, and allocates outputs and workspaces; the work is in
the library's HIP kernels.  Everything here is re-exported by the package.

Calls run on the current stream, or on `stream`.  A workspace made by a call is
of that stream's pool; outputs are of the current stream's, as everywhere in the
package, so a caller who gives another stream orders the two: the stream waits
for the current one before the call, and the current one for the stream before
it uses or frees the outputs.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

from . import KdaError, _cu, _expect, _expect_workspace, _io_code, _stream, _torch, lib

__all__ = ["HYBRID_EXPORTS", "Cache4", "plan_requests", "cache4_append", "cache4_read", "cache4_attention",
           "cache4_attention_workspace_size", "cache4_shared_attention", "cache4_shared_attention_workspace_size",
           "recurrence_problem", "recurrence_workspace_size",
           "recurrence_backward_workspace_size", "recurrence_prefill", "recurrence_prefill_for_backward",
           "recurrence_backward", "recurrence_autograd", "recurrence_step"]

HYBRID_EXPORTS = ("kda_plan_requests", "kda_cache4_append", "kda_cache4_read", "kda_cache4_attention_workspace_size",
                  "kda_cache4_attention", "kda_cache4_shared_attention_workspace_size",
                  "kda_cache4_shared_attention", "kda_recurrence_workspace_size", "kda_recurrence_backward_workspace_size",
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
        L.kda_cache4_shared_attention_workspace_size.argtypes = [C, A, I64, I64]
        L.kda_cache4_shared_attention.argtypes = [C, A, P, P, P, I64, P, P, I64, P, P, P, P, SZ, P]
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


def _in(name: str, x, shape, dtype, device):
    """The pointer of an argument of the given shape, dtype and device."""
    if x is None:
        return None
    if x.shape != shape or x.dtype != dtype or x.device != device:
        _expect(name, x, shape, dtype, device)
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return x.data_ptr()


def _run(name: str, device, stream, *args) -> None:
    """Call `name` with the stream behind its arguments, on its tensors' device
    whichever is current."""
    torch = _torch()
    if device.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    f = getattr(_hlib(), name)
    if device.index == torch.cuda.current_device():
        # the current stream as the raw handle: a Stream object costs 2 us
        code = f(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            code = f(*args, _stream(stream, device))
    if code != 0:
        raise KdaError(name, code)


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
        if not workspace.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel()


def plan_requests(past_lens, new_lens, block_table, free_pages, page_size: int, tokens: int, stream=None):
    """The plan of a serving step from the requests' lengths (kda_plan_requests).

    past_lens, new_lens: int32 [n]; block_table: int32 [n, max_pages], whose
    entries for the pages that the new tokens begin are written in place, off
    free_pages (int32 [m], read only); tokens: rows of the packed batch, the
    sum of new_lens or more.  Returns (cu_seqlens int32 [n+1], total_lens
    int32 [n], slot_map int64 [tokens], pages_taken int32 [1]); the caller
    drops the first pages_taken entries of free_pages.

    Where the sum of new_lens passes tokens, the last requests are cut off:
    cu_seqlens.diff() is below new_lens there, while total_lens and the pages
    taken go by new_lens.  cache4_attention then takes past_lens +
    cu_seqlens.diff() in the place of total_lens."""
    torch = _torch()
    dev, i32 = past_lens.device, torch.int32
    if past_lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("past_lens and free_pages must be 1-D and block_table [n, max_pages]")
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {page_size!r}")
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    n, max_pages, n_free = past_lens.shape[0], block_table.shape[1], free_pages.shape[0]
    args = (_in("past_lens", past_lens, (n,), i32, dev), _in("new_lens", new_lens, (n,), i32, dev),
            _in("block_table", block_table, (n, max_pages), i32, dev), n_free,
            _in("free_pages", free_pages, (n_free,), i32, dev))
    cu = torch.empty(n + 1, dtype=i32, device=dev)
    total = torch.empty(n, dtype=i32, device=dev)
    taken = torch.empty(1, dtype=i32, device=dev)
    slots = torch.empty(tokens, dtype=torch.int64, device=dev)
    _run("kda_plan_requests", dev, stream, n, tokens, page_size, max_pages, *args, cu.data_ptr(), total.data_ptr(),
         slots.data_ptr(), taken.data_ptr())
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
        scales, dev, u8 = (pages, heads, page_size, half // 16), k.device, torch.uint8
        self._struct = KdaCache4(pages, page_size, heads, 2 * half, _in("k", k, k.shape, u8, dev),
                                 _in("k_scale", k_scale, scales, u8, dev), _in("v", v, k.shape, u8, dev),
                                 _in("v_scale", v_scale, scales, u8, dev))
        self._tensors = (k, k_scale, v, v_scale)
        self.pages, self.heads, self.page_size, self.d = pages, heads, page_size, 2 * half
        self.device = dev

    # the tensors of a cache stay the ones it was made with
    k = property(lambda self: self._tensors[0])
    k_scale = property(lambda self: self._tensors[1])
    v = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, d: int, device="cuda") -> "Cache4":
        """A cache of zeros."""
        torch = _torch()
        codes = [torch.zeros((pages, heads, page_size, d // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros((pages, heads, page_size, d // 32), dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1])


def _rows_of(slot_map) -> int:
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be 1-D")
    return slot_map.shape[0]


def cache4_append(cache: Cache4, k, v, slot_map, stream=None) -> None:
    """Round k, v [T, heads, d] (bf16 or fp32) into the cache at slot_map int64
    [T] (page * page_size + offset; slots outside the cache are dropped, and no
    two rows may name one slot)."""
    T, io, dev = _rows_of(slot_map), _io_code(k.dtype), cache.device
    shape = (T, cache.heads, cache.d)
    args = (_in("k", k, shape, k.dtype, dev), _in("v", v, shape, k.dtype, dev),
            _in("slot_map", slot_map, (T,), _torch().int64, dev))
    _run("kda_cache4_append", dev, stream, cache._struct, T, io, *args)


def cache4_read(cache: Cache4, slot_map, dtype, stream=None):
    """(k, v) [T, heads, d] of the rows at slot_map, as the values they stand
    for; zeros for slots outside the cache."""
    torch = _torch()
    T, io, dev = _rows_of(slot_map), _io_code(dtype), cache.device
    slots = _in("slot_map", slot_map, (T,), torch.int64, dev)
    k = torch.empty((T, cache.heads, cache.d), dtype=dtype, device=dev)
    v = torch.empty_like(k)
    _run("kda_cache4_read", dev, stream, cache._struct, T, io, slots, k.data_ptr(), v.data_ptr())
    return k, v


def _attention_problem(q, cache, block_table, total_lens, cu_seqlens, scale, max_q, max_len):
    """(problem, pointers of q, block_table, total_lens and cu_seqlens) of checked inputs."""
    i32, dev = _torch().int32, cache.device
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [T, heads, d] and block_table [n_seq, max_pages]")
    T, heads, _ = q.shape
    n_seq, max_pages = T if cu_seqlens is None else _cu(cu_seqlens, dev), block_table.shape[1]
    io = _io_code(q.dtype)
    ptrs = (_in("q", q, (T, heads, cache.d), q.dtype, dev),
            _in("block_table", block_table, (n_seq, max_pages), i32, dev),
            _in("total_lens", total_lens, (n_seq,), i32, dev), _in("cu_seqlens", cu_seqlens, (n_seq + 1,), i32, dev))
    if heads % cache.heads:
        raise ValueError(f"{heads} query heads over {cache.heads} key/value heads")
    if max_q is None:
        max_q = 1 if cu_seqlens is None else T
    if max_len is None:
        max_len = max_pages * cache.page_size
    return KdaCache4AttentionProblem(n_seq, T, heads, max_pages, max(int(max_q), 1), max(int(max_len), 0), io,
                                     1.0 / math.sqrt(cache.d) if scale is None else float(scale)), ptrs


def cache4_attention_workspace_size(q, cache: Cache4, block_table, total_lens, cu_seqlens=None, max_q=None,
                                    max_len=None) -> int:
    """Bytes of workspace that cache4_attention needs for these arguments."""
    p, _ = _attention_problem(q, cache, block_table, total_lens, cu_seqlens, None, max_q, max_len)
    return _hlib().kda_cache4_attention_workspace_size(cache._struct, p)


def cache4_attention(q, cache: Cache4, block_table, total_lens, cu_seqlens=None, g=None,
                     scale: Optional[float] = None, max_q: Optional[int] = None, max_len: Optional[int] = None,
                     out=None, workspace=None, stream=None):
    """Causal grouped-query attention over the 4-bit cache (kda_cache4_attention).

    q [T, heads, d] (bf16 or fp32), packed by cu_seqlens int32 [n+1], or one
    row for each of T sequences where that is None; block_table int32 [n,
    max_pages]; total_lens int32 [n], the tokens each sequence has, its
    queries the newest of them (append their keys and values first); g
    [T, heads, d]: the read-out gate, out = attention * sigmoid(g); scale
    defaults to 1/sqrt(d).  bf16 queries have their probabilities rounded to
    bf16, fp32 ones do not.  max_q and max_len, about the most queries and the
    most tokens of a sequence, steer how the work is split, and nothing else.
    Returns out [T, heads, d]."""
    dev = cache.device
    p, ptrs = _attention_problem(q, cache, block_table, total_lens, cu_seqlens, scale, max_q, max_len)
    gate = _in("g", g, q.shape, q.dtype, dev)
    if out is None:
        out = _torch().empty_like(q)
    to = _in("out", out, q.shape, q.dtype, dev)
    c = cache._struct
    ws, ws_ptr, nbytes = _workspace(workspace, _hlib().kda_cache4_attention_workspace_size(c, p), dev, stream)
    _run("kda_cache4_attention", dev, stream, c, p, *ptrs, gate, to, ws_ptr, nbytes)
    return out


def _shared_problem(q, cache, block_table, total_lens, prefix_lens, group_offsets, cu_seqlens, scale, max_q, max_prefix,
                    max_own):
    """(problem, pointers as _attention_problem gives them, groups, max_prefix, pointers of prefix_lens and
    group_offsets) of checked inputs."""
    i32, dev = _torch().int32, cache.device
    if prefix_lens.dim() != 1:
        raise ValueError("prefix_lens must be 1-D")
    p, ptrs = _attention_problem(q, cache, block_table, total_lens, cu_seqlens, scale, max_q, max_own)
    n = prefix_lens.shape[0]
    if max_prefix is None:
        max_prefix = block_table.shape[1] * cache.page_size
    return p, ptrs, n, max(int(max_prefix), 0), (_in("prefix_lens", prefix_lens, (n,), i32, dev),
                                                 _in("group_offsets", group_offsets, (n + 1,), i32, dev))


def cache4_shared_attention_workspace_size(q, cache: Cache4, block_table, total_lens, prefix_lens, group_offsets,
                                           cu_seqlens=None, max_q=None, max_prefix=None, max_own=None) -> int:
    """Bytes of workspace that cache4_shared_attention needs for these arguments."""
    p, _, n, most, _ = _shared_problem(q, cache, block_table, total_lens, prefix_lens, group_offsets, cu_seqlens, None,
                                       max_q, max_prefix, max_own)
    return _hlib().kda_cache4_shared_attention_workspace_size(cache._struct, p, n, most)


def cache4_shared_attention(q, cache: Cache4, block_table, total_lens, prefix_lens, group_offsets, cu_seqlens=None,
                            g=None, scale: Optional[float] = None, max_q: Optional[int] = None,
                            max_prefix: Optional[int] = None, max_own: Optional[int] = None, out=None, workspace=None,
                            stream=None):
    """cache4_attention for groups of sequences that share their first tokens,
    which are read once for a whole group (kda_cache4_shared_attention).

    The sequences [group_offsets[j], group_offsets[j+1]) have the same first
    prefix_lens[j] tokens (int32 [m+1] and [m]), in the pages of the group's first
    sequence; sequences of no group attend by themselves.  total_lens counts all
    tokens of a sequence, those of its prefix among them.  max_q, max_prefix and
    max_own, about the most queries of a sequence, the longest prefix and the most
    tokens of a sequence behind its prefix, steer how the work is split, and
    nothing else.  The rest is as in cache4_attention.  Returns out [T, heads, d]."""
    dev = cache.device
    p, ptrs, n, most, groups = _shared_problem(q, cache, block_table, total_lens, prefix_lens, group_offsets,
                                               cu_seqlens, scale, max_q, max_prefix, max_own)
    gate = _in("g", g, q.shape, q.dtype, dev)
    if out is None:
        out = _torch().empty_like(q)
    to = _in("out", out, q.shape, q.dtype, dev)
    c = cache._struct
    ws, ws_ptr, nbytes = _workspace(workspace, _hlib().kda_cache4_shared_attention_workspace_size(c, p, n, most), dev,
                                    stream)
    _run("kda_cache4_shared_attention", dev, stream, c, p, *ptrs[:3], n, *groups, most, ptrs[3], gate, to, ws_ptr, nbytes)
    return out


def _recurrence_problem(x, log_alpha, log_alpha_min, g, state_in, cu_seqlens):
    """(problem, shape of the states, pointers of x, log_alpha, g, state_in and
    cu_seqlens) of checked inputs."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    (B, T, D), dtype, dev = x.shape, x.dtype, x.device
    io = _io_code(dtype)
    n_seq = -1
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("a packed batch is [1, T, D]")
        n_seq = _cu(cu_seqlens, dev)
    states = (B if n_seq < 0 else n_seq, D)
    ptrs = (_in("x", x, (B, T, D), dtype, dev), _in("log_alpha", log_alpha, (B, T, D), torch.float32, dev),
            _in("g", g, (B, T, D), dtype, dev), _in("state_in", state_in, states, torch.float32, dev),
            _in("cu_seqlens", cu_seqlens, (n_seq + 1,), torch.int32, dev))
    return KdaRecurrenceProblem(B, T, D, n_seq, io, float(log_alpha_min)), states, ptrs


def recurrence_problem(batch: int, seqlen: int, width: int, io_dtype, log_alpha_min: float,
                       n_seq: int = -1) -> KdaRecurrenceProblem:
    """The problem that the workspace sizes go by; n_seq: sequences of a packed batch."""
    return KdaRecurrenceProblem(batch, seqlen, width, n_seq, _io_code(io_dtype), float(log_alpha_min))


def recurrence_workspace_size(p: KdaRecurrenceProblem) -> int:
    """Bytes of workspace that recurrence_prefill needs."""
    return _hlib().kda_recurrence_workspace_size(p)


def recurrence_backward_workspace_size(p: KdaRecurrenceProblem) -> int:
    """Bytes of workspace that the training pair needs."""
    return _hlib().kda_recurrence_backward_workspace_size(p)


def _recurrence_forward(name, size, x, log_alpha, log_alpha_min, g, state_in, cu_seqlens, out, state_out, want_state,
                        workspace, stream):
    torch = _torch()
    p, states, ptrs = _recurrence_problem(x, log_alpha, log_alpha_min, g, state_in, cu_seqlens)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty(states, dtype=torch.float32, device=dev)
    to = (_in("out", out, x.shape, x.dtype, dev), _in("state_out", state_out, states, torch.float32, dev))
    ws, ws_ptr, nbytes = _workspace(workspace, size(p), dev, stream)
    _run(name, dev, stream, p, *ptrs, *to, ws_ptr, nbytes)
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
    unless want_dstate).  Tokens of no sequence are not written."""
    return _recurrence_gradients(_torch().empty_like, x, log_alpha, log_alpha_min, workspace, g, state_in, cu_seqlens,
                                 d_out, d_state, want_dstate, stream)


def _recurrence_gradients(new_like, x, log_alpha, log_alpha_min, workspace, g, state_in, cu_seqlens, d_out, d_state,
                          want_dstate, stream) -> dict:
    """recurrence_backward into arrays made by new_like."""
    torch = _torch()
    p, states, ptrs = _recurrence_problem(x, log_alpha, log_alpha_min, g, state_in, cu_seqlens)
    dev = x.device
    grads = (_in("d_out", d_out, x.shape, x.dtype, dev), _in("d_state", d_state, states, torch.float32, dev))
    r = dict(dx=new_like(x), dlog_alpha=new_like(log_alpha), dg=new_like(g) if g is not None else None,
             dstate0=torch.empty(states, dtype=torch.float32, device=dev) if want_dstate else None)
    to = (None if r[k] is None else r[k].data_ptr() for k in ("dx", "dlog_alpha", "dg", "dstate0"))
    _, ws_ptr, nbytes = _workspace(workspace, 0, dev, stream)
    _run("kda_recurrence_backward", dev, stream, p, *ptrs, *grads, *to, ws_ptr, nbytes)
    return r


_RECURRENCE_FUNCTION = None


def _gradient(d):
    """A gradient as the calls take it: contiguous and 16-byte aligned.  That of
    a concatenated output is a view, which may begin anywhere."""
    if d is None:
        return None
    d = d.contiguous()
    return d if d.data_ptr() % 16 == 0 else d.clone()


def _recurrence_function():
    """The torch.autograd.Function over the training pair, created on first use."""
    global _RECURRENCE_FUNCTION
    if _RECURRENCE_FUNCTION is None:
        torch = _torch()

        class RecurrenceFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, log_alpha, g, state_in, log_alpha_min, cu_seqlens):
                # the kernels leave tokens of no sequence as they are
                out = None if cu_seqlens is None else torch.zeros_like(x)
                out, state, ws = recurrence_prefill_for_backward(x, log_alpha, log_alpha_min, g=g, state_in=state_in,
                                                                 cu_seqlens=cu_seqlens, out=out)
                ctx.save_for_backward(x, log_alpha, g, state_in, cu_seqlens)
                ctx.workspace, ctx.log_alpha_min = ws, log_alpha_min
                ctx.set_materialize_grads(False)
                return out, state

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_out, d_state):
                x, log_alpha, g, state_in, cu_seqlens = ctx.saved_tensors
                r = _recurrence_gradients(torch.empty_like if cu_seqlens is None else torch.zeros_like, x, log_alpha,
                                          ctx.log_alpha_min, ctx.workspace, g, state_in, cu_seqlens, _gradient(d_out),
                                          _gradient(d_state), state_in is not None and ctx.needs_input_grad[3], None)
                return r["dx"], r["dlog_alpha"], r["dg"], r["dstate0"], None, None

        _RECURRENCE_FUNCTION = RecurrenceFunction
    return _RECURRENCE_FUNCTION


def recurrence_autograd(x, log_alpha, log_alpha_min: float, g=None, state_in=None, cu_seqlens=None):
    """Differentiable recurrence_prefill: returns (out, final states), and
    loss.backward() fills the gradients of x, log_alpha, g and state_in.  In a
    packed batch the tokens of no sequence have outputs and gradients of zero,
    for which all are cleared first (1 x 16384 x 2048 in bf16: 300 us a pass,
    231 by the pair above, which leaves those tokens as they are).

    To capture a training pass into a graph, call the pair above, or drop every
    eager result of the same leaves first: while one lives, PyTorch accumulates
    their gradients on the stream it was made on, outside the capture."""
    return _recurrence_function().apply(x, log_alpha, g, state_in, float(log_alpha_min), cu_seqlens)


def recurrence_step(x, log_alpha, state, log_alpha_min: float, g=None, out=None, stream=None):
    """One token of each of N sequences: x, g [N, D], log_alpha fp32; state
    [N, D] fp32, updated in place.  Returns out [N, D]."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    shape, dtype, dev = x.shape, x.dtype, x.device
    io = _io_code(dtype)
    ptrs = (_in("x", x, shape, dtype, dev), _in("log_alpha", log_alpha, shape, torch.float32, dev),
            _in("g", g, shape, dtype, dev), _in("state", state, shape, torch.float32, dev))
    if out is None:
        out = torch.empty_like(x)
    _run("kda_recurrence_step", dev, stream, shape[0], shape[1], io, float(log_alpha_min), *ptrs,
         _in("out", out, shape, dtype, dev))
    return out
