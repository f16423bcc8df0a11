"""CPU: the sequence and adapter entry points reject every invalid argument on the host, before any launch."""
import ctypes

import pytest

import linear_spatial_propagation_amd as gspn
from linear_spatial_propagation_amd import _lib

FAKE = 1 << 40   # aligned, never dereferenced: every call below fails validation first
GB = 1 << 32     # between two fake tensors
NULL, SHAPE, CPW, DTYPE, ALIGN, ALIAS, FLAGS, STRIDE, WORK = -1, -2, -5, -6, -7, -8, -11, -13, -14


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from linear_spatial_propagation_amd import build
        build.build()
    return _lib.load()


def at(i):
    return FAKE + i * GB


def seq(**kw):
    v = dict(x=at(0), gate=at(1), lam=at(2), u=at(3), offsets=at(4), h0=at(5), y=at(6), h_last=at(7), states=at(8),
             work=at(9), work_bytes=1 << 30, T=1000, D=64, N=4, x_stride=64, gate_stride=64, lam_stride=64, u_stride=64,
             y_stride=64, ch_per_weight=1, dtype=1, flags=0)
    v.update(kw)
    return _lib.Seq(**v)


SEQ_BAD = [
    (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(N=0), SHAPE), (dict(T=1 << 31), SHAPE), (dict(D=1 << 21), SHAPE),
    (dict(T=1001, N=4, offsets=0), SHAPE), (dict(T=1 << 29, D=1 << 14), SHAPE),
    (dict(ch_per_weight=0), CPW), (dict(ch_per_weight=3), CPW), (dict(dtype=2), DTYPE),
    (dict(flags=2), FLAGS), (dict(x=0), NULL), (dict(gate=0), NULL),
    (dict(x_stride=-1), STRIDE), (dict(lam_stride=-64), STRIDE),
    (dict(x=at(0) + 1), ALIGN), (dict(h0=at(5) + 2), ALIGN), (dict(offsets=at(4) + 2), ALIGN), (dict(work=at(9) + 8), ALIGN),
]


@pytest.mark.parametrize("kw,code", SEQ_BAD + [
    (dict(y=0), NULL), (dict(y_stride=63), STRIDE), (dict(y_stride=-1), STRIDE),
    (dict(y=at(0)), ALIAS), (dict(y=at(2) + 128), ALIAS), (dict(h_last=at(5)), ALIAS), (dict(states=at(6) + 64), ALIAS),
    (dict(y=at(4)), ALIAS), (dict(h_last=at(8) + 4), ALIAS),
], ids=str)
def test_forward_refuses(lib, kw, code):
    assert lib.gspn_seq_fwd(ctypes.byref(seq(**kw)), None) == code


def grad(**kw):
    v = dict(gy=at(20), gh_last=at(21), gx=at(22), ggate=at(23), glam=at(24), gu=at(25), gh0=at(26), gy_stride=64,
             gx_stride=64, ggate_stride=64, glam_stride=64, gu_stride=64)
    v.update(kw)
    return _lib.SeqGrad(**v)


@pytest.mark.parametrize("kw,gkw,code", [(k, {}, c) for k, c in SEQ_BAD] + [
    (dict(states=0), {}, NULL), (dict(lam=0), {}, NULL), (dict(u=0), {}, NULL),
    ({}, dict(gx_stride=10), STRIDE), ({}, dict(gy_stride=-1), STRIDE), ({}, dict(ggate_stride=60), STRIDE),
    ({}, dict(gx=at(22) + 1), ALIGN), ({}, dict(gh0=at(26) + 2), ALIGN),
    ({}, dict(gx=at(0)), ALIAS), ({}, dict(gh0=at(21)), ALIAS), ({}, dict(glam=at(24) - GB), ALIAS),
    ({}, dict(gu=at(20) + 2), ALIAS), ({}, dict(gx=at(8)), ALIAS),
    (dict(ch_per_weight=64 // 2, gate_stride=2, work=0), dict(ggate_stride=2), WORK),
    (dict(ch_per_weight=64 // 2, gate_stride=2, work_bytes=100), dict(ggate_stride=2), WORK),
], ids=str)
def test_backward_refuses(lib, kw, gkw, code):
    assert lib.gspn_seq_bwd(ctypes.byref(seq(**kw)), ctypes.byref(grad(**gkw)), None) == code


def test_null_structs(lib):
    assert lib.gspn_seq_fwd(None, None) == NULL
    assert lib.gspn_seq_bwd(None, None, None) == NULL
    assert lib.gspn_seq_bwd(ctypes.byref(seq()), None, None) == NULL
    assert lib.gspn_seq_step(None, None) == NULL
    assert lib.gspn_adapter_add(None, None) == NULL
    assert lib.gspn_seq_workspace(None, 0) == NULL
    assert lib.gspn_adapter_workspace(None) == NULL


def token(**kw):
    v = dict(x=at(0), gate=at(1), lam=at(2), u=at(3), slots=at(4), state=at(5), y=at(6), N=8, S=16, D=64, x_stride=64,
             gate_stride=64, lam_stride=64, u_stride=64, y_stride=64, ch_per_weight=1, dtype=0, flags=0)
    v.update(kw)
    return _lib.SeqToken(**v)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), SHAPE), (dict(S=0), SHAPE), (dict(D=0), SHAPE), (dict(slots=0, N=17), SHAPE), (dict(N=1 << 21), SHAPE),
    (dict(ch_per_weight=5), CPW), (dict(dtype=9), DTYPE), (dict(flags=2), FLAGS), (dict(state=0), NULL), (dict(x=0), NULL), (dict(y=0), NULL),
    (dict(y_stride=1), STRIDE), (dict(u_stride=-4), STRIDE), (dict(x=at(0) + 2), ALIGN), (dict(state=at(5) + 1), ALIGN),
    (dict(y=at(0)), ALIAS), (dict(state=at(2)), ALIAS), (dict(y=at(5) + 4), ALIAS), (dict(state=at(4)), ALIAS),
], ids=str)
def test_step_refuses(lib, kw, code):
    assert lib.gspn_seq_step(ctypes.byref(token(**kw)), None) == code


def test_step_of_no_rows(lib):
    assert lib.gspn_seq_step(ctypes.byref(token(N=0, x=0, gate=0, lam=0, u=0, y=0, slots=0)), None) == 0


def adapter(**kw):
    v = dict(base=at(0), x=at(1), a=at(2), b=at(3), scale=at(4), ids=at(5), offsets=at(6), out=at(7), work=at(8),
             work_bytes=1 << 30, T=100, K=64, M=96, N=4, R=3, r=8, base_stride=96, x_stride=64, out_stride=96, dtype=1,
             flags=0)
    v.update(kw)
    return _lib.Adapter(**v)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(R=0), SHAPE), (dict(r=0), SHAPE),
    (dict(r=257), SHAPE), (dict(offsets=0, T=101), SHAPE), (dict(T=1 << 30, M=1 << 20), SHAPE), (dict(dtype=3), DTYPE),
    (dict(flags=4), FLAGS), (dict(base=0), NULL), (dict(x=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL),
    (dict(ids=0), NULL), (dict(out=0), NULL), (dict(out_stride=95), STRIDE), (dict(x_stride=-1), STRIDE),
    (dict(a=at(2) + 1), ALIGN), (dict(scale=at(4) + 1), ALIGN), (dict(work=at(8) + 4), ALIGN),
    (dict(out=at(0) + 2), ALIAS), (dict(out=at(0), out_stride=192), ALIAS), (dict(out=at(1)), ALIAS),
    (dict(out=at(3) + 16), ALIAS), (dict(out=at(8)), ALIAS), (dict(work=0), WORK), (dict(work_bytes=3), WORK),
], ids=str)
def test_adapter_refuses(lib, kw, code):
    assert lib.gspn_adapter_add(ctypes.byref(adapter(**kw)), None) == code


def test_sizes(lib):
    for packed in (0, 1):
        assert lib.gspn_seq_states_rows(0, 3, packed) == 3
        assert lib.gspn_seq_states_rows(-2, 2, packed) == SHAPE
        # a row for the start of each sequence, and for every so many tokens
        assert 2 + 1000 // 256 <= lib.gspn_seq_states_rows(1000, 2, packed) <= 2 + 1000 // 32
    assert lib.gspn_seq_states_rows(131, 2, 0) == SHAPE
    assert lib.gspn_seq_workspace(ctypes.byref(seq(N=0)), 0) == SHAPE
    assert lib.gspn_adapter_workspace(ctypes.byref(adapter(r=300))) == SHAPE
    assert lib.gspn_adapter_add(ctypes.byref(adapter(T=0, base=0, x=0, out=0)), None) == 0


def test_wrappers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    ids = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: gspn.seq_scan_fwd(x, x), lambda: gspn.seq_scan(x, x), lambda: gspn.seq_step(x, x, x),
                 lambda: gspn.seq_scan_bwd(x, x, x, x),
                 lambda: gspn.adapter_add(x, x, x.view(1, 4, 8), x.view(1, 8, 4), ids)):
        with pytest.raises(ValueError):
            call()
