"""Low-rank adapters of many requests, added to a shared projection's output
(gspn_adapter_add of include/gspn.h)."""
from __future__ import annotations

import ctypes

from . import _lib
from .sequence import _call, _code, _index, _layout, _like, _output, _row_stride


def adapter_add(base, x, a, b, ids, *, scale=None, offsets=None, out=None):
    """out = base + scale[i] * (x a[i]^T) b[i]^T, i the adapter of each row's request, on the current HIP stream.

    base: [T, M], what the shared projection gave for x: [T, K]; a: [R, r, K]
    and b: [R, M, r], contiguous, the adapters' factors (r <= 256); scale: [R]
    float32 or None for 1; ids: [N] int32, the adapter of each request, or a
    number outside [0, R) for none: its rows of base are copied.  Request n
    holds the rows offsets[n] .. offsets[n + 1] - 1 (offsets: [N + 1] int32);
    without offsets every request has T / N of them, and base and x may be
    [N, L, M] and [N, L, K].  float32 or bfloat16, one dtype.  ``out`` may be
    base itself; rows behind the last request are left as they were in an
    ``out`` of the caller's and zero in a new one.  There is no backward: the
    call refuses tensors that ask for a gradient.
    """
    import torch
    T, N = _layout(x, offsets)
    if ids.dim() != 1 or ids.numel() < 1:
        raise ValueError("ids must hold a number for every request")
    if offsets is None and x.dim() == 2:
        N = ids.numel()
        if T % N:
            raise ValueError(f"{T} rows are no equal shares of {N} requests; give offsets")
    if ids.numel() != N:
        raise ValueError(f"ids must hold {N} numbers")
    if a.dim() != 3 or b.dim() != 3 or base.dim() != x.dim():
        raise ValueError("a must be [R, r, K], b [R, M, r], and base laid out like x")
    R, r, K = a.shape
    M = base.shape[-1]
    for name, t, shape in (("a", a, (R, r, x.shape[-1])), ("b", b, (R, M, r))):
        if t.device != x.device or t.dtype != x.dtype:
            raise ValueError(f"{name} must share x's device and dtype")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (base, x, a, b, scale)):
        raise RuntimeError("adapter_add has no backward; call it under torch.no_grad()")
    s = _lib.Adapter(T=T, K=K, M=M, N=N, R=R, r=r, dtype=_code(x))
    s.x, s.x_stride = x.data_ptr(), _row_stride("x", x)
    s.base, s.base_stride = _like("base", base, x, x.shape[:-1] + (M,))
    s.a, s.b = a.data_ptr(), b.data_ptr()
    s.ids = _index("ids", ids, x.device)
    if offsets is not None:
        s.offsets = _index("offsets", offsets, x.device)
    if scale is not None:
        if scale.device != x.device or scale.dtype != torch.float32 or scale.shape != (R,) or not scale.is_contiguous():
            raise ValueError(f"scale must be a contiguous float32 tensor of {R} numbers on {x.device}")
        s.scale = scale.data_ptr()
    out, s.out, s.out_stride = _output("out", out, x, base.shape, s)
    lib = _lib.load()
    need = lib.gspn_adapter_workspace(ctypes.byref(s))
    if need < 0:
        _lib.check(need)
    if need:
        work = torch.empty(need, dtype=torch.uint8, device=x.device)
        s.work, s.work_bytes = work.data_ptr(), need
    _call(lib.gspn_adapter_add, x.device, ctypes.byref(s))
    return out
