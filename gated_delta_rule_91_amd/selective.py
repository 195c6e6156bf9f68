"""The short causal convolution and the selective state space, over the C ABI of
``include/kda_selective.h``, with their gradients and single-token forms.

As in ``hybrid.py`` this module only checks tensors, passes device pointers and
the stream, and allocates outputs and workspaces; the work is in the library's
HIP kernels.  Everything here is re-exported by the package.  Calls run on the
current stream, or on `stream`, by the rules stated there.
"""
from __future__ import annotations

import ctypes

from . import _cu, _io_code, _torch, lib
from .hybrid import _gradient, _in, _run, _workspace

__all__ = ["SELECTIVE_EXPORTS", "short_conv_prefill", "short_conv_backward", "short_conv_backward_workspace_size",
           "short_conv_step", "short_conv_autograd", "short_conv_problem", "selective_scan_prefill",
           "selective_scan_prefill_for_backward", "selective_scan_backward", "selective_scan_step",
           "selective_scan_autograd", "selective_scan_problem", "selective_scan_workspace_size",
           "selective_scan_backward_workspace_size"]

SELECTIVE_EXPORTS = ("kda_short_conv_prefill", "kda_short_conv_backward_workspace_size", "kda_short_conv_backward",
                     "kda_short_conv_step", "kda_selective_scan_workspace_size",
                     "kda_selective_scan_backward_workspace_size", "kda_selective_scan_prefill",
                     "kda_selective_scan_prefill_for_backward", "kda_selective_scan_backward",
                     "kda_selective_scan_step")


class KdaShortConvProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int64),
                ("n_seq", ctypes.c_int64), ("taps", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


class KdaSelectiveScanProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int64),
                ("n_seq", ctypes.c_int64), ("states", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


class KdaSelectiveScanInputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "state_in",
                                               "cu_seqlens")]


class KdaSelectiveScanGradients(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias",
                                               "d_state_in")]


_bound = None


def _slib() -> ctypes.CDLL:
    """lib() with the signatures of these calls declared."""
    global _bound
    L = lib()
    if _bound is not L:
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        V, S, N, G = (ctypes.POINTER(t) for t in (KdaShortConvProblem, KdaSelectiveScanProblem, KdaSelectiveScanInputs,
                                                  KdaSelectiveScanGradients))
        L.kda_short_conv_prefill.argtypes = [V, P, P, P, P, P, P, P, P]
        L.kda_short_conv_backward_workspace_size.argtypes = [V]
        L.kda_short_conv_backward.argtypes = [V, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.kda_short_conv_step.argtypes = [I64, I64, I32, I32, I32, P, P, P, P, P, P]
        L.kda_selective_scan_workspace_size.argtypes = [S]
        L.kda_selective_scan_backward_workspace_size.argtypes = [S]
        L.kda_selective_scan_prefill.argtypes = [S, N, P, P, P, SZ, P]
        L.kda_selective_scan_prefill_for_backward.argtypes = [S, N, P, P, P, SZ, P]
        L.kda_selective_scan_backward.argtypes = [S, N, P, P, G, P, SZ, P]
        L.kda_selective_scan_step.argtypes = [I64, I64, I32, I32, P, P, P, P, P, P, P, P, P, P, P]
        for f in SELECTIVE_EXPORTS:
            getattr(L, f).restype = SZ if f.endswith("workspace_size") else I32
        _bound = L
    return L


def _call(name, device, stream, *args) -> None:
    _slib()                     # declares what _run calls
    _run(name, device, stream, *args)


def _rows(x, cu_seqlens):
    """(batch, tokens, width, n_seq or -1, sequences, pointer of cu_seqlens) of x [B, T, D]."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    (B, T, D), dev = x.shape, x.device
    if cu_seqlens is None:
        return B, T, D, -1, B, None
    if B != 1:
        raise ValueError("a packed batch is [1, T, D]")
    n = _cu(cu_seqlens, dev)
    return B, T, D, n, n, _in("cu_seqlens", cu_seqlens, (n + 1,), _torch().int32, dev)


# ---- short convolution ----------------------------------------------------------------

def short_conv_problem(batch: int, seqlen: int, width: int, taps: int, io_dtype, silu: bool = True,
                       n_seq: int = -1) -> KdaShortConvProblem:
    """The problem that the workspace size goes by; n_seq: sequences of a packed batch."""
    return KdaShortConvProblem(batch, seqlen, width, n_seq, taps, int(bool(silu)), _io_code(io_dtype))


def short_conv_backward_workspace_size(p: KdaShortConvProblem) -> int:
    """Bytes of workspace that short_conv_backward needs."""
    return _slib().kda_short_conv_backward_workspace_size(p)


def _taps(weight, D) -> int:
    if weight.dim() != 2 or weight.shape[0] != D or weight.shape[1] not in (2, 3, 4):
        raise ValueError(f"weight must be [{D}, taps] with 2, 3 or 4 taps, got {tuple(weight.shape)}")
    return weight.shape[1]


def _conv_inputs(x, weight, bias, silu, state_in, cu_seqlens):
    """(problem, shape of the states, pointers of x, weight, bias, state_in and cu_seqlens) of checked inputs."""
    f32, dev = _torch().float32, x.device
    B, T, D, n_seq, n, cu = _rows(x, cu_seqlens)
    W = _taps(weight, D)
    states = (n, W - 1, D)
    ptrs = (_in("x", x, x.shape, x.dtype, dev), _in("weight", weight, (D, W), f32, dev),
            _in("bias", bias, (D,), f32, dev), _in("state_in", state_in, states, x.dtype, dev), cu)
    return KdaShortConvProblem(B, T, D, n_seq, W, int(bool(silu)), _io_code(x.dtype)), states, ptrs


def short_conv_prefill(x, weight, bias=None, silu: bool = True, state_in=None, cu_seqlens=None, out=None,
                       state_out=None, want_state: bool = True, stream=None):
    """A causal convolution of each channel with its own 2, 3 or 4 weights
    (kda_short_conv_prefill): y_t = bias + sum_j weight[:, j] x_(t - taps + 1 + j),
    out = silu(y) or y.  x [B, T, D] bf16 or fp32, weight [D, taps] and bias [D]
    fp32; the inputs before a sequence's first are state_in [B or n, taps - 1,
    D] (dtype of x; zeros where None).  A packed batch is [1, T, D] with
    cu_seqlens int32 [n+1].  Returns (out, final states); state_out may be
    state_in."""
    torch = _torch()
    p, states, ptrs = _conv_inputs(x, weight, bias, silu, state_in, cu_seqlens)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty(states, dtype=x.dtype, device=dev)
    _call("kda_short_conv_prefill", dev, stream, p, *ptrs, _in("out", out, x.shape, x.dtype, dev),
         _in("state_out", state_out, states, x.dtype, dev))
    return out, state_out


def short_conv_backward(x, weight, d_out=None, bias=None, silu: bool = True, state_in=None, cu_seqlens=None,
                        d_state=None, want_dstate: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of <d_out, out> + <d_state, final states>, from the inputs of
    short_conv_prefill alone.  Returns a dict with dx, dweight, dbias (None
    without bias) and dstate0 (None unless want_dstate).  Tokens of no sequence
    are not written."""
    return _conv_gradients(_torch().empty_like, x, weight, d_out, bias, silu, state_in, cu_seqlens, d_state,
                           want_dstate, workspace, stream)


def _conv_gradients(new_like, x, weight, d_out, bias, silu, state_in, cu_seqlens, d_state, want_dstate, workspace,
                    stream) -> dict:
    """short_conv_backward into a dx made by new_like."""
    torch = _torch()
    p, states, ptrs = _conv_inputs(x, weight, bias, silu, state_in, cu_seqlens)
    dev = x.device
    grads = (_in("d_out", d_out, x.shape, x.dtype, dev), _in("d_state", d_state, states, x.dtype, dev))
    r = dict(dx=new_like(x), dweight=torch.empty_like(weight), dbias=None if bias is None else torch.empty_like(bias),
             dstate0=torch.empty(states, dtype=x.dtype, device=dev) if want_dstate else None)
    to = (None if r[k] is None else r[k].data_ptr() for k in ("dx", "dweight", "dbias", "dstate0"))
    _, ws_ptr, nbytes = _workspace(workspace, 0 if workspace is not None else short_conv_backward_workspace_size(p),
                                   dev, stream)
    _call("kda_short_conv_backward", dev, stream, p, *ptrs, *grads, *to, ws_ptr, nbytes)
    return r


def short_conv_step(x, weight, state, bias=None, silu: bool = True, out=None, stream=None):
    """One token of each of N sequences: x [N, D]; state [N, taps - 1, D] (dtype
    of x), updated in place.  Returns out [N, D]."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    (N, D), dtype, dev = x.shape, x.dtype, x.device
    W, io = _taps(weight, D), _io_code(dtype)
    ptrs = (_in("x", x, (N, D), dtype, dev), _in("weight", weight, (D, W), torch.float32, dev),
            _in("bias", bias, (D,), torch.float32, dev), _in("state", state, (N, W - 1, D), dtype, dev))
    if out is None:
        out = torch.empty_like(x)
    _call("kda_short_conv_step", dev, stream, N, D, W, int(bool(silu)), io, *ptrs,
         _in("out", out, (N, D), dtype, dev))
    return out


# ---- selective scan -------------------------------------------------------------------

def selective_scan_problem(batch: int, seqlen: int, width: int, states: int, io_dtype,
                           n_seq: int = -1) -> KdaSelectiveScanProblem:
    """The problem that the workspace sizes go by; n_seq: sequences of a packed batch."""
    return KdaSelectiveScanProblem(batch, seqlen, width, n_seq, states, _io_code(io_dtype))


def selective_scan_workspace_size(p: KdaSelectiveScanProblem) -> int:
    """Bytes of workspace that selective_scan_prefill needs."""
    return _slib().kda_selective_scan_workspace_size(p)


def selective_scan_backward_workspace_size(p: KdaSelectiveScanProblem) -> int:
    """Bytes of workspace that the training pair needs."""
    return _slib().kda_selective_scan_backward_workspace_size(p)


def _states(A, D) -> int:
    if A.dim() != 2 or A.shape[0] != D or A.shape[1] not in (8, 16, 32):
        raise ValueError(f"A must be [{D}, states] with 8, 16 or 32 states, got {tuple(A.shape)}")
    return A.shape[1]


def _scan_inputs(x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens):
    """(problem, shape of the states, struct of the inputs) of checked inputs."""
    f32, dev, io = _torch().float32, x.device, x.dtype
    rows, T, D, n_seq, n, cu = _rows(x, cu_seqlens)
    N = _states(A, D)
    states, shared = (n, D, N), (rows, T, N)
    s = KdaSelectiveScanInputs(_in("x", x, x.shape, io, dev), _in("dt", dt, x.shape, io, dev),
                               _in("A", A, (D, N), f32, dev), _in("B", B, shared, io, dev),
                               _in("C", C, shared, io, dev), _in("skip", skip, (D,), f32, dev),
                               _in("z", z, x.shape, io, dev), _in("dt_bias", dt_bias, (D,), f32, dev),
                               _in("state_in", state_in, states, f32, dev), cu)
    return KdaSelectiveScanProblem(rows, T, D, n_seq, N, _io_code(io)), states, s


def _scan_forward(name, size, x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens, out, state_out, want_state,
                  workspace, stream):
    torch = _torch()
    p, states, s = _scan_inputs(x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty(states, dtype=torch.float32, device=dev)
    to = (_in("out", out, x.shape, x.dtype, dev), _in("state_out", state_out, states, torch.float32, dev))
    ws, ws_ptr, nbytes = _workspace(workspace, 0 if workspace is not None else size(p), dev, stream)
    _call(name, dev, stream, p, s, *to, ws_ptr, nbytes)
    return out, state_out, ws


def selective_scan_prefill(x, dt, A, B, C, skip=None, z=None, dt_bias=None, state_in=None, cu_seqlens=None, out=None,
                           state_out=None, want_state: bool = True, workspace=None, stream=None):
    """A selective state space (kda_selective_scan_prefill): per channel, with
    delta = softplus(dt + dt_bias), h_n <- exp(delta A[:, n]) h_n + delta x B_n,
    out = (sum_n C_n h_n + skip x) silu(z).  x, dt, z [B, T, D] and B, C [B, T,
    states] bf16 or fp32; A [D, states] (at most 0), skip and dt_bias [D] fp32;
    8, 16 or 32 states.  A packed batch is [1, T, D] with cu_seqlens int32 [n+1].
    States are fp32 [B or n, D, states].  Returns (out, final states); state_out
    may be state_in."""
    out, state, _ = _scan_forward("kda_selective_scan_prefill", selective_scan_workspace_size, x, dt, A, B, C, skip, z,
                                  dt_bias, state_in, cu_seqlens, out, state_out, want_state, workspace, stream)
    return out, state


def selective_scan_prefill_for_backward(x, dt, A, B, C, skip=None, z=None, dt_bias=None, state_in=None,
                                        cu_seqlens=None, out=None, state_out=None, want_state: bool = True,
                                        workspace=None, stream=None):
    """selective_scan_prefill that leaves what selective_scan_backward continues
    from.  Returns (out, final states, workspace)."""
    torch = _torch()
    out, state, ws = _scan_forward("kda_selective_scan_prefill_for_backward", selective_scan_backward_workspace_size,
                                   x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens, out, state_out, want_state,
                                   workspace, stream)
    return out, state, torch.empty(0, dtype=torch.uint8, device=x.device) if ws is None else ws


def selective_scan_backward(x, dt, A, B, C, workspace, skip=None, z=None, dt_bias=None, state_in=None, cu_seqlens=None,
                            d_out=None, d_state=None, want_dstate: bool = True, stream=None) -> dict:
    """Gradients of <d_out, out> + <d_state, final states>, from the inputs and
    the workspace of selective_scan_prefill_for_backward.  Returns a dict with
    dx, ddt, dz, dB, dC (dtype of x), dA, dskip, ddt_bias (fp32) and dstate0;
    None for what was not given, and for dstate0 unless want_dstate.  Tokens of
    no sequence are not written."""
    return _scan_gradients(_torch().empty_like, x, dt, A, B, C, workspace, skip, z, dt_bias, state_in, cu_seqlens,
                           d_out, d_state, want_dstate, stream)


def _scan_gradients(new_like, x, dt, A, B, C, workspace, skip, z, dt_bias, state_in, cu_seqlens, d_out, d_state,
                    want_dstate, stream) -> dict:
    """selective_scan_backward into arrays made by new_like."""
    torch = _torch()
    p, states, s = _scan_inputs(x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens)
    dev = x.device
    grads = (_in("d_out", d_out, x.shape, x.dtype, dev), _in("d_state", d_state, states, torch.float32, dev))
    like = dict(dx=x, ddt=dt, dA=A, dB=B, dC=C, dskip=skip, dz=z, ddt_bias=dt_bias)
    r = {k: None if t is None else new_like(t) for k, t in like.items()}
    r["dstate0"] = torch.empty(states, dtype=torch.float32, device=dev) if want_dstate else None
    to = KdaSelectiveScanGradients(*(None if t is None else t.data_ptr() for t in r.values()))
    _, ws_ptr, nbytes = _workspace(workspace, 0, dev, stream)
    _call("kda_selective_scan_backward", dev, stream, p, s, *grads, to, ws_ptr, nbytes)
    return r


def selective_scan_step(x, dt, A, B, C, state, skip=None, z=None, dt_bias=None, out=None, stream=None):
    """One token of each of n sequences: x, dt, z [n, D], B, C [n, states]; state
    [n, D, states] fp32, updated in place.  Returns out [n, D]."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [n, D]")
    (n, D), io, dev = x.shape, x.dtype, x.device
    N, f32 = _states(A, D), torch.float32
    ptrs = (_in("x", x, (n, D), io, dev), _in("dt", dt, (n, D), io, dev), _in("A", A, (D, N), f32, dev),
            _in("B", B, (n, N), io, dev), _in("C", C, (n, N), io, dev), _in("skip", skip, (D,), f32, dev),
            _in("z", z, (n, D), io, dev), _in("dt_bias", dt_bias, (D,), f32, dev),
            _in("state", state, (n, D, N), f32, dev))
    if out is None:
        out = torch.empty_like(x)
    _call("kda_selective_scan_step", dev, stream, n, D, N, _io_code(io), *ptrs, _in("out", out, (n, D), io, dev))
    return out


# ---- autograd -------------------------------------------------------------------------

_FUNCTIONS = {}


def _conv_function():
    """The torch.autograd.Function over the convolution's two calls, created on first use."""
    if "conv" not in _FUNCTIONS:
        torch = _torch()

        class ShortConvFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, bias, state_in, silu, cu_seqlens):
                # the kernels leave tokens of no sequence as they are
                out = None if cu_seqlens is None else torch.zeros_like(x)
                out, state = short_conv_prefill(x, weight, bias, silu, state_in, cu_seqlens, out=out)
                ctx.save_for_backward(x, weight, bias, state_in, cu_seqlens)
                ctx.silu = silu
                ctx.set_materialize_grads(False)
                return out, state

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_out, d_state):
                x, weight, bias, state_in, cu_seqlens = ctx.saved_tensors
                r = _conv_gradients(torch.empty_like if cu_seqlens is None else torch.zeros_like, x, weight,
                                    _gradient(d_out), bias, ctx.silu, state_in, cu_seqlens, _gradient(d_state),
                                    state_in is not None and ctx.needs_input_grad[3], None, None)
                return r["dx"], r["dweight"], r["dbias"], r["dstate0"], None, None

        _FUNCTIONS["conv"] = ShortConvFunction
    return _FUNCTIONS["conv"]


def short_conv_autograd(x, weight, bias=None, silu: bool = True, state_in=None, cu_seqlens=None):
    """Differentiable short_conv_prefill: returns (out, final states), and
    loss.backward() fills the gradients of x, weight, bias and state_in.  In a
    packed batch the tokens of no sequence have outputs and gradients of zero.

    To capture a training pass into a graph, call the pair above, or drop every
    eager result of the same leaves first: while one lives, PyTorch accumulates
    their gradients on the stream it was made on, outside the capture."""
    return _conv_function().apply(x, weight, bias, state_in, bool(silu), cu_seqlens)


def _scan_function():
    """The torch.autograd.Function over the scan's training pair, created on first use."""
    if "scan" not in _FUNCTIONS:
        torch = _torch()

        class SelectiveScanFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens):
                # the kernels leave tokens of no sequence as they are
                out = None if cu_seqlens is None else torch.zeros_like(x)
                out, state, ws = selective_scan_prefill_for_backward(x, dt, A, B, C, skip, z, dt_bias, state_in,
                                                                     cu_seqlens, out=out)
                ctx.save_for_backward(x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens)
                ctx.workspace = ws
                ctx.set_materialize_grads(False)
                return out, state

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, d_out, d_state):
                x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens = ctx.saved_tensors
                r = _scan_gradients(torch.empty_like if cu_seqlens is None else torch.zeros_like, x, dt, A, B, C,
                                    ctx.workspace, skip, z, dt_bias, state_in, cu_seqlens, _gradient(d_out),
                                    _gradient(d_state), state_in is not None and ctx.needs_input_grad[8], None)
                return (r["dx"], r["ddt"], r["dA"], r["dB"], r["dC"], r["dskip"], r["dz"], r["ddt_bias"],
                        r["dstate0"], None)

        _FUNCTIONS["scan"] = SelectiveScanFunction
    return _FUNCTIONS["scan"]


def selective_scan_autograd(x, dt, A, B, C, skip=None, z=None, dt_bias=None, state_in=None, cu_seqlens=None):
    """Differentiable selective_scan_prefill: returns (out, final states), and
    loss.backward() fills the gradients of every input.  In a packed batch the
    tokens of no sequence have outputs and gradients of zero.  Captured into a
    graph, what short_conv_autograd says holds here too."""
    return _scan_function().apply(x, dt, A, B, C, skip, z, dt_bias, state_in, cu_seqlens)
