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

seq_scan is differentiable; seq_scan_fwd and seq_scan_bwd record nothing for
autograd.  Workspaces are new for every call, so calls on several streams and
captured graphs may overlap.
"""
from __future__ import annotations

import functools

from . import _lib

_PACK_SEQ = _lib.packer(_lib.Seq)
_PACK_GRAD = _lib.packer(_lib.SeqGrad)
_PACK_TOKEN = _lib.packer(_lib.SeqToken)


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
    if stride[-1] != 1 and shape[-1] > 1:
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
    """t's pointer and row stride, (0, 0) for None; checks device, dtype and shape against x's."""
    if t is None:
        return 0, 0
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x is on {x.device}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, x has {x.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr(), _row_stride(name, t)


def _new(x, width):
    """A new contiguous tensor like x, its pointer and row stride."""
    import torch
    t = torch.empty_like(x, memory_format=torch.contiguous_format)   # half the host time of empty() with x's dtype and device
    return t, t.data_ptr(), width


def _states(name, t, dev, shape):
    import torch
    if t is None:
        return 0
    if t.device != dev or t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 {tuple(shape)} tensor on {dev}")
    return t.data_ptr()


def _index(name, t, dev):
    import torch
    if t is None:
        return 0
    if t.device != dev or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous one-dimensional int32 tensor on {dev}")
    return t.data_ptr()


def _layout(x, offsets):
    """(T, N) of a packed or an equal-rows tensor."""
    if not x.is_cuda:
        raise ValueError("tensors must be on a GPU (HIP) device")
    shape = x.shape
    if len(shape) == 3:
        if offsets is not None:
            raise ValueError("offsets go with packed [T, D] tensors; [B, L, D] has rows of equal length")
        if shape[0] == 0:
            raise ValueError("there must be a sequence")
        return shape[0] * shape[1], shape[0]
    if len(shape) != 2:
        raise ValueError("x must be [T, D] or [B, L, D]")
    if offsets is None:
        return shape[0], 1
    if offsets.numel() < 2:
        raise ValueError("offsets must hold N + 1 numbers, N >= 1")
    return shape[0], offsets.numel() - 1


def _call(fn, dev, *args):
    """fn(*args, the current stream of dev), with dev current."""
    import torch
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        _lib.check(rc)


def _sizes(x, ch_per_weight, offsets):
    """(T, N, D) of a call."""
    T, N = _layout(x, offsets)
    D = x.shape[-1]
    if ch_per_weight < 1 or D % ch_per_weight:
        raise ValueError("ch_per_weight must divide D")
    return T, N, D


def _gate(gate, x, D, ch_per_weight):
    return _like("gate", gate, x, x.shape if ch_per_weight == 1 else x.shape[:-1] + (D // ch_per_weight,))


@functools.lru_cache(maxsize=4096)
def _work_bytes(T, D, N, packed, ch_per_weight, code, backward):
    need = _lib.load().gspn_seq_workspace(
        _PACK_SEQ(0, 0, 0, 0, int(packed), 0, 0, 0, 0, 0, 0, T, D, N, 0, 0, 0, 0, 0, ch_per_weight, code, 0), backward)
    if need < 0:
        _lib.check(need)
    return need


def _workspace(T, D, N, packed, ch_per_weight, code, backward, dev):
    """(tensor, pointer, bytes) of a new workspace; the tensor has to live until the call is enqueued."""
    import torch
    need = _work_bytes(T, D, N, packed, ch_per_weight, code, backward)
    if need == 0:
        return None, 0, 0
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    return work, work.data_ptr(), need


def seq_scan_fwd(x, gate, *, lam=None, u=None, offsets=None, h0=None, ch_per_weight: int = 1, out=None,
                 return_states: bool = False):
    """Forward recurrence on the current HIP stream; returns (y, h_last).

    y is shaped like x; h_last [N, D] float32 is each sequence's state behind
    its last token (h0's for a sequence of none).  return_states adds what
    seq_scan_bwd starts from: states inside the sequences, float32, some tokens apart.
    """
    import torch
    T, N, D = _sizes(x, ch_per_weight, offsets)
    dev, code, shape = x.device, _code(x), x.shape
    px, sx = x.data_ptr(), _row_stride("x", x)
    pg, sg = _gate(gate, x, D, ch_per_weight)
    pl, sl = _like("lam", lam, x, shape)
    pu, su = _like("u", u, x, shape)
    po = _index("offsets", offsets, dev)
    ph = _states("h0", h0, dev, (N, D))
    # rows behind the last sequence are zero in a new tensor
    flags = 0 if out is not None or offsets is None else _lib.SEQ_ZERO_TAIL
    if out is None:
        out, py, sy = _new(x, D)
    else:
        py, sy = _like("out", out, x, shape)
    h_last = torch.empty(N, D, dtype=torch.float32, device=dev)
    lib, states, ps = _lib.load(), None, 0
    if return_states:
        states = torch.empty(lib.gspn_seq_states_rows(T, N, po != 0), D, dtype=torch.float32, device=dev)
        ps = states.data_ptr()
    work, pw, nw = _workspace(T, D, N, po != 0, ch_per_weight, code, 0, dev)
    _call(lib.gspn_seq_fwd, dev, _PACK_SEQ(px, pg, pl, pu, po, ph, py, h_last.data_ptr(), ps, pw, nw, T, D, N, sx, sg,
                                           sl, su, sy, ch_per_weight, code, flags))
    return (out, h_last, states) if return_states else (out, h_last)


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
    if out is not None:
        if len(out) != 5 or any((o is None) != (t is None) for o, t in zip(out, (x, gate, lam, u, x))):
            raise ValueError("out must hold a tensor for every gradient: gx, ggate, gh0, and glam and gu with lam and u "
                             "(None without)")
    return _backward(x, gate, gy, states, lam, u, offsets, gh_last, ch_per_weight, out, (True,) * 5)


def _backward(x, gate, gy, states, lam, u, offsets, gh_last, ch_per_weight, out, want):
    import torch
    T, N, D = _sizes(x, ch_per_weight, offsets)
    dev, code, shape, lib = x.device, _code(x), x.shape, _lib.load()
    px, sx = x.data_ptr(), _row_stride("x", x)
    pg, sg = _gate(gate, x, D, ch_per_weight)
    pl, sl = _like("lam", lam, x, shape)
    pu, su = _like("u", u, x, shape)
    po = _index("offsets", offsets, dev)
    if states is None:
        raise ValueError("states must be what seq_scan_fwd returned")
    ps = _states("states", states, dev, (lib.gspn_seq_states_rows(T, N, po != 0), D))
    py, sy = _like("gy", gy, x, shape)
    ph = _states("gh_last", gh_last, dev, (N, D))
    flags = 0 if out is not None or offsets is None else _lib.SEQ_ZERO_TAIL
    if out is None:
        none = (None, 0, 0)
        ox, gx, tx = _new(x, D) if want[0] else none
        og, gg, tg = _new(gate, D // ch_per_weight) if want[1] else none
        ol, gl, tl = _new(lam, D) if lam is not None and want[2] else none
        ou, gu, tu = _new(u, D) if u is not None and want[3] else none
        oh = torch.empty(N, D, dtype=torch.float32, device=dev) if want[4] else None
        gh = 0 if oh is None else oh.data_ptr()
        out = (ox, og, ol, ou, oh)
    else:
        gx, tx = _like("gx", out[0], x, shape)
        gg, tg = _like("ggate", out[1], x, gate.shape)
        gl, tl = _like("glam", out[2], x, shape)
        gu, tu = _like("gu", out[3], x, shape)
        gh = _states("gh0", out[4], dev, (N, D))
    work, pw, nw = _workspace(T, D, N, po != 0, ch_per_weight, code, 1, dev)
    _call(lib.gspn_seq_bwd, dev,
          _PACK_SEQ(px, pg, pl, pu, po, 0, 0, 0, ps, pw, nw, T, D, N, sx, sg, sl, su, 0, ch_per_weight, code, flags),
          _PACK_GRAD(py, ph, gx, gg, gl, gu, gh, sy, tx, tg, tl, tu))
    return tuple(out)


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
    and autograd calls seq_scan_bwd for the gradients of x, gate, lam, u and h0
    (first derivatives only).

    To capture a training step into a graph, capture seq_scan_fwd and
    seq_scan_bwd, or a seq_scan with its backward whose leaves have no live
    graph of an eager call: torch ends the process where a captured backward
    meets the gradient accumulators of one.
    """
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
    request and are taken in order (every row looks through all of slots: meant
    for up to some thousands of requests).  There is no backward: the call
    refuses tensors that ask for a gradient.
    """
    import torch
    if not x.is_cuda:
        raise ValueError("tensors must be on a GPU (HIP) device")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, gate, lam, u, state)):
        raise RuntimeError("seq_step has no backward; call it under torch.no_grad()")
    shape = x.shape
    if len(shape) != 2 or state.dim() != 2:
        raise ValueError("x must be [N, D] and state [S, D]")
    N, D = shape
    if ch_per_weight < 1 or D % ch_per_weight:
        raise ValueError("ch_per_weight must divide D")
    dev, code, S = x.device, _code(x), state.shape[0]
    sx = _row_stride("x", x)
    pg, sg = _gate(gate, x, D, ch_per_weight)
    pl, sl = _like("lam", lam, x, shape)
    pu, su = _like("u", u, x, shape)
    pt = _states("state", state, dev, (S, D))
    if slots is not None and slots.shape != (N,):
        raise ValueError(f"slots must hold {N} numbers")
    pi = _index("slots", slots, dev)
    flags = 0
    if out is None:
        flags = _lib.SEQ_ZERO_TAIL
        out, py, sy = _new(x, D)
    else:
        py, sy = _like("out", out, x, shape)
    _call(_lib.load().gspn_seq_step, dev, _PACK_TOKEN(x.data_ptr(), pg, pl, pu, pi, pt, py, N, S, D, sx, sg, sl, su, sy,
                                                      ch_per_weight, code, flags))
    return out
