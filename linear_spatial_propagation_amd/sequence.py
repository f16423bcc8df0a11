"""The gated linear recurrence over sequences of tokens (gspn_seq_* of
include/gspn.h), the causal form of the scan:

    h_t = a_t h_{t-1} + lam_t x_t   (without lam: + (1 - a_t) x_t),   a_t = sigmoid(gate_t)
    y_t = u_t h_t                   (without u: h_t)

Tensors (float32 or bfloat16, one dtype, on one GPU), in one of two layouts:
  rows of equal length:  x, lam, u [B, L, D], gate [B, L, D // ch_per_weight]
  packed:  x, lam, u [T, D], gate [T, D // ch_per_weight], and offsets [N + 1]
           (int32): sequence n holds rows offsets[n] .. offsets[n + 1] - 1;
           without offsets the T rows are one sequence
Channels lie next to each other (stride 1); rows may lie any distance apart, so
column ranges of one projection's output need no copy.  States (h0, h_last,
the cache of seq_step) are float32, [N, D].

Rows behind offsets[-1] belong to no sequence: nothing of theirs is used, and
their outputs are zero where this module allocates the output, and left as
they were in an ``out`` of the caller's.
"""
from __future__ import annotations

import ctypes

from . import _lib


def _code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return _lib.GSPN_BF16
    if t.dtype == torch.float32:
        return _lib.GSPN_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use torch.bfloat16 or torch.float32")


def _row_stride(name, t):
    """Elements from one row to the next of a [rows, width] or [B, L, width] tensor."""
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if len(shape) == 2:
        return stride[0] if shape[0] > 1 else shape[1]
    B, L = shape[0], shape[1]
    if L == 0:
        return shape[2]
    if B == 1 or L == 1:
        return stride[1] if L > 1 else stride[0] if B > 1 else shape[2]
    if stride[0] != L * stride[1]:
        raise ValueError(f"{name}'s rows must lie at equal distances (a [B, L, D] whose [B * L, D] view exists)")
    return stride[1]


def _like(name, t, x, shape):
    """t's pointer and row stride; checks device, dtype and shape against x's."""
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x is on {x.device}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, x has {x.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr(), _row_stride(name, t)


def _states(name, t, dev, shape):
    import torch
    if t.device != dev or t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 {tuple(shape)} tensor on {dev}")
    return t.data_ptr()


def _index(name, t, dev):
    import torch
    if t.device != dev or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous one-dimensional int32 tensor on {dev}")
    return t.data_ptr()


def _layout(x, offsets):
    """(T, N) of a packed or an equal-rows tensor."""
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU (HIP) device")
    if x.dim() == 3:
        if offsets is not None:
            raise ValueError("offsets go with packed [T, D] tensors; [B, L, D] has rows of equal length")
        if x.shape[0] == 0:
            raise ValueError("there must be a sequence")
        return x.shape[0] * x.shape[1], x.shape[0]
    if x.dim() != 2:
        raise ValueError("x must be [T, D] or [B, L, D]")
    if offsets is None:
        return x.shape[0], 1
    if offsets.numel() < 2:
        raise ValueError("offsets must hold N + 1 numbers, N >= 1")
    return x.shape[0], offsets.numel() - 1


def _call(fn, dev, *args):
    """fn(*args, the current stream of dev), with dev current."""
    import torch
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc:
        _lib.check(rc)


def _sequence(x, gate, lam, u, offsets, h0, ch_per_weight):
    """The gspn_seq of the inputs (outputs and workspace are the caller's to fill in)."""
    T, N = _layout(x, offsets)
    D = x.shape[-1]
    if ch_per_weight < 1 or D % ch_per_weight:
        raise ValueError("ch_per_weight must divide D")
    s = _lib.Seq(T=T, D=D, N=N, ch_per_weight=ch_per_weight, dtype=_code(x))
    s.x, s.x_stride = x.data_ptr(), _row_stride("x", x)
    s.gate, s.gate_stride = _like("gate", gate, x, x.shape[:-1] + (D // ch_per_weight,))
    if lam is not None:
        s.lam, s.lam_stride = _like("lam", lam, x, x.shape)
    if u is not None:
        s.u, s.u_stride = _like("u", u, x, x.shape)
    if offsets is not None:
        s.offsets = _index("offsets", offsets, x.device)
    if h0 is not None:
        s.h0 = _states("h0", h0, x.device, (N, D))
    return s


def _workspace(s, dev, backward):
    """Allocates the workspace that s asks for; the tensor has to live until the call is enqueued."""
    import torch
    need = _lib.load().gspn_seq_workspace(ctypes.byref(s), backward)
    if need < 0:
        _lib.check(need)
    if need == 0:
        return None
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    s.work, s.work_bytes = work.data_ptr(), need
    return work


def _output(name, out, like, shape, s):
    """An output tensor: the caller's, checked, or a new one whose rows behind the last sequence are to be zero."""
    import torch
    if out is None:
        s.flags = _lib.SEQ_ZERO_TAIL
        out = torch.empty(shape, dtype=like.dtype, device=like.device)
    return (out,) + _like(name, out, like, shape)


def seq_scan_fwd(x, gate, *, lam=None, u=None, offsets=None, h0=None, ch_per_weight: int = 1, out=None,
                 return_states: bool = False):
    """Forward recurrence on the current HIP stream; returns (y, h_last).

    y is shaped like x; h_last [N, D] float32 is each sequence's state behind
    its last token (h0's for a sequence of none).  return_states adds what
    seq_scan_bwd needs: the state in front of every 128th token of a sequence.
    """
    import torch
    s = _sequence(x, gate, lam, u, offsets, h0, ch_per_weight)
    y, s.y, s.y_stride = _output("out", out, x, x.shape, s)
    h_last = torch.empty((s.N, s.D), dtype=torch.float32, device=x.device)
    s.h_last = h_last.data_ptr()
    states = None
    if return_states:
        states = torch.empty((_lib.load().gspn_seq_states_rows(s.T, s.N), s.D), dtype=torch.float32, device=x.device)
        s.states = states.data_ptr()
    work = _workspace(s, x.device, 0)   # noqa: F841 -- lives until the call is enqueued
    _call(_lib.load().gspn_seq_fwd, x.device, ctypes.byref(s))
    return (y, h_last, states) if return_states else (y, h_last)


def seq_scan_bwd(x, gate, gy, states, *, lam=None, u=None, offsets=None, gh_last=None, ch_per_weight: int = 1,
                 out=None):
    """Backward recurrence on the current HIP stream.

    Returns (gx, ggate, glam, gu, gh0), the gradients of a loss whose gradient
    with respect to (y, h_last) of seq_scan_fwd is (gy, gh_last); either may
    be None for zeros.  states is what seq_scan_fwd returned for the same
    inputs.  glam and gu are None where lam and u are; gh0 [N, D] float32
    belongs to h0, whether or not the forward had one.  ``out`` may give the
    five tensors.
    """
    return _backward(x, gate, gy, states, lam, u, offsets, gh_last, ch_per_weight, out, (True,) * 5)


def _backward(x, gate, gy, states, lam, u, offsets, gh_last, ch_per_weight, out, want):
    import torch
    s = _sequence(x, gate, lam, u, offsets, None, ch_per_weight)
    g = _lib.SeqGrad()
    lib = _lib.load()
    s.states = _states("states", states, x.device, (lib.gspn_seq_states_rows(s.T, s.N), s.D))
    if gy is not None:
        g.gy, g.gy_stride = _like("gy", gy, x, x.shape)
    if gh_last is not None:
        g.gh_last = _states("gh_last", gh_last, x.device, (s.N, s.D))
    given = (None,) * 5 if out is None else out
    if len(given) != 5:
        raise ValueError("out must hold five tensors: gx, ggate, glam, gu, gh0")
    if out is not None and any((o is None) != (t is None) for o, t in zip(out, (x, gate, lam, u, x))):
        raise ValueError("out must hold a tensor for every gradient: gx, ggate, gh0, and glam and gu with lam and u")
    grads = [None] * 5
    if want[0]:
        grads[0], g.gx, g.gx_stride = _output("gx", given[0], x, x.shape, s)
    if want[1]:
        grads[1], g.ggate, g.ggate_stride = _output("ggate", given[1], x, gate.shape, s)
    if want[2] and lam is not None:
        grads[2], g.glam, g.glam_stride = _output("glam", given[2], x, x.shape, s)
    if want[3] and u is not None:
        grads[3], g.gu, g.gu_stride = _output("gu", given[3], x, x.shape, s)
    if want[4]:
        grads[4] = given[4] if given[4] is not None else torch.empty((s.N, s.D), dtype=torch.float32, device=x.device)
        g.gh0 = _states("gh0", grads[4], x.device, (s.N, s.D))
    work = _workspace(s, x.device, 1)   # noqa: F841 -- lives until the call is enqueued
    _call(lib.gspn_seq_bwd, x.device, ctypes.byref(s), ctypes.byref(g))
    return tuple(grads)


def _autograd_function():
    import torch
    from torch.autograd.function import once_differentiable

    class _SeqScan(torch.autograd.Function):
        """(y, h_last) = seq_scan_fwd(...) with seq_scan_bwd as its backward (both HIP)."""

        @staticmethod
        def forward(ctx, x, gate, lam, u, offsets, h0, ch_per_weight):
            y, h_last, states = seq_scan_fwd(x, gate, lam=lam, u=u, offsets=offsets, h0=h0,
                                             ch_per_weight=ch_per_weight, return_states=True)
            ctx.save_for_backward(x, gate, lam, u, offsets, states)
            ctx.ch_per_weight = ch_per_weight
            ctx.set_materialize_grads(False)
            return y, h_last

        @staticmethod
        @once_differentiable
        def backward(ctx, gy, gh_last):
            if gy is None and gh_last is None:
                return (None,) * 7
            x, gate, lam, u, offsets, states = ctx.saved_tensors
            if gy is not None and not _rows_usable(gy):
                gy = gy.contiguous()
            gx, ggate, glam, gu, gh0 = _backward(x, gate, gy, states, lam, u, offsets,
                                                 None if gh_last is None else gh_last.contiguous(),
                                                 ctx.ch_per_weight, None,
                                                 tuple(ctx.needs_input_grad[i] for i in (0, 1, 2, 3, 5)))
            return gx, ggate, glam, gu, None, gh0, None

    return _SeqScan


def _rows_usable(t):
    try:
        _row_stride("gy", t)
    except ValueError:
        return False
    return True


_SEQ_SCAN = None


def seq_scan(x, gate, *, lam=None, u=None, offsets=None, h0=None, ch_per_weight: int = 1):
    """seq_scan_fwd as a differentiable torch operation: returns (y, h_last),
    and autograd calls seq_scan_bwd for the gradients of x, gate, lam, u and h0."""
    import torch
    if not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in (x, gate, lam, u, h0)):
        return seq_scan_fwd(x, gate, lam=lam, u=u, offsets=offsets, h0=h0, ch_per_weight=ch_per_weight)
    global _SEQ_SCAN
    if _SEQ_SCAN is None:
        _SEQ_SCAN = _autograd_function()
    return _SEQ_SCAN.apply(x, gate, lam, u, offsets, h0, ch_per_weight)


def seq_step(x, gate, state, *, lam=None, u=None, slots=None, ch_per_weight: int = 1, out=None):
    """One token of each of N requests on the current HIP stream; returns y [N, D].

    x, lam, u: [N, D]; gate: [N, D // ch_per_weight]; state: [S, D] float32,
    the cache of states, changed in place.  slots: [N] int32, the cache row of
    each request (None: request n has row n); a request whose slot is outside
    [0, S) is a row of padding, its state stays and its y is left as it was in
    ``out``, zero in a new tensor.  Requests of the same slot are tokens of one
    request and are taken in order.
    """
    import torch
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU (HIP) device")
    if x.dim() != 2 or state.dim() != 2:
        raise ValueError("x must be [N, D] and state [S, D]")
    N, D = x.shape
    if ch_per_weight < 1 or D % ch_per_weight:
        raise ValueError("ch_per_weight must divide D")
    S = state.shape[0]
    t = _lib.SeqToken(N=N, S=S, D=D, ch_per_weight=ch_per_weight, dtype=_code(x))
    t.x, t.x_stride = x.data_ptr(), _row_stride("x", x)
    t.gate, t.gate_stride = _like("gate", gate, x, (N, D // ch_per_weight))
    if lam is not None:
        t.lam, t.lam_stride = _like("lam", lam, x, x.shape)
    if u is not None:
        t.u, t.u_stride = _like("u", u, x, x.shape)
    t.state = _states("state", state, x.device, (S, D))
    if slots is not None:
        if slots.shape != (N,):
            raise ValueError(f"slots must hold {N} numbers")
        t.slots = _index("slots", slots, x.device)
    if out is None:
        # rows of padding are not written by the kernel
        out = (torch.empty if slots is None else torch.zeros)((N, D), dtype=x.dtype, device=x.device)
    t.y, t.y_stride = _like("out", out, x, x.shape)
    _call(_lib.load().gspn_seq_step, x.device, ctypes.byref(t))
    return out
