"""Low-rank adapters of many requests, added to a shared projection's output
(gspn_adapter_add of include/gspn.h)."""
from __future__ import annotations

import functools

from . import _lib
from .sequence import _call, _code, _index, _layout, _like, _new, _row_stride

_PACK = _lib.packer(_lib.Adapter)


@functools.lru_cache(maxsize=4096)
def _work_bytes(T, K, M, N, R, r, code, packed):
    need = _lib.load().gspn_adapter_workspace(_PACK(0, 0, 0, 0, 0, 0, int(packed), 0, 0, 0, T, K, M, N, R, r, 0, 0, 0,
                                                    code, 0))
    if need < 0:
        _lib.check(need)
    return need


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
    ``out`` of the caller's and zero in a new one.  Infinities in b or scale
    may give NaN for the requests of that adapter.  There is no backward: the
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
    if a.device != x.device or b.device != x.device or a.dtype != x.dtype or b.dtype != x.dtype:
        raise ValueError("a and b must share x's device and dtype")
    if K != x.shape[-1] or b.shape != (R, M, r):
        raise ValueError(f"a and b have shapes {tuple(a.shape)} and {tuple(b.shape)}, expected [R, r, {x.shape[-1]}] and "
                         f"[R, {M}, r]")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    if torch.is_grad_enabled() and (base.requires_grad or x.requires_grad or a.requires_grad or b.requires_grad or
                                    (scale is not None and scale.requires_grad)):
        raise RuntimeError("adapter_add has no backward; call it under torch.no_grad()")
    dev, code = x.device, _code(x)
    px, sx = x.data_ptr(), _row_stride("x", x)
    pb, sb = _like("base", base, x, x.shape[:-1] + (M,))
    pi, po = _index("ids", ids, dev), _index("offsets", offsets, dev)
    ps = 0
    if scale is not None:
        if scale.device != dev or scale.dtype != torch.float32 or scale.shape != (R,) or not scale.is_contiguous():
            raise ValueError(f"scale must be a contiguous float32 tensor of {R} numbers on {dev}")
        ps = scale.data_ptr()
    flags = 0 if out is not None else _lib.SEQ_ZERO_TAIL
    if out is None:
        out, py, sy = _new(base, M)
    else:
        py, sy = _like("out", out, x, base.shape)
    lib = _lib.load()
    need = _work_bytes(T, K, M, N, R, r, code, po != 0)
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(lib.gspn_adapter_add, dev, _PACK(pb, px, a.data_ptr(), b.data_ptr(), ps, pi, po, py, work.data_ptr(), need, T, K,
                                           M, N, R, r, sb, sx, sy, code, flags))
    return out
