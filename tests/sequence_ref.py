"""The gated recurrence and the adapters in 64 bits on the CPU, token by token,
with a bound for what 32-bit arithmetic and one rounding at the end may be off.

Bounds.  eps = 2^-24 is half a step of fp32.  A kernel's sigmoid comes from
exp2 of -|g| log2(e) and a reciprocal: the rounded argument is off by up to
|g| 2^-24 1.45, the two hardware functions by a step each, the sum and the
products by half a step each, so the smaller of a and 1 - a has a relative
error of at most d = (|g| + 8) 2^-23, the larger one less.

With M the recurrence of absolute values (M_t = a M_{t-1} + |in_t|), a token
adds to the state's error
  d (min(a, 1 - a) M_{t-1} + |in_t|)   for the gate's error, and
  12 eps M_t                           for its roundings: two in the step, two
     more where the step is part of a product of gates that carries a state
     over a stretch of tokens, and what joining the stretches adds, fewer than
     eight in all for each token;
the errors before it shrink by a.  Each is added up as the state is:
E_t = a E_{t-1} + (both).  The adjoint has the same recurrence, backwards.
"""
from __future__ import annotations

import torch

EPS = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _gates(gate, cpw):
    g = gate.double().repeat_interleave(cpw, 1)
    a, q = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    d = (g.abs().clamp(max=700) + 8) * 2.0 ** -23
    return a, q, d


def forward(x, gate, lam, u, lens, h0, cpw):
    """y, h_last and their bounds; rows behind the last sequence are zero."""
    T, D = x.shape
    rnd = half_step(x.dtype) + 2 * EPS
    a, q, d = _gates(gate, cpw)
    xd = x.double()
    term = (q if lam is None else lam.double()) * xd
    h, e, m = (torch.zeros(T, D, dtype=torch.float64) for _ in range(3))
    before, e_before, m_before = (torch.zeros(T, D, dtype=torch.float64) for _ in range(3))
    start = torch.zeros(len(lens), D, dtype=torch.float64) if h0 is None else h0.double()
    last, e_last = start.clone(), torch.zeros_like(start)
    t = 0
    for n, count in enumerate(lens):
        s, es, ms = start[n], torch.zeros(D, dtype=torch.float64), start[n].abs()
        for _ in range(count):
            before[t], e_before[t], m_before[t] = s, es, ms
            s = a[t] * s + term[t]
            es = a[t] * es + d[t] * (torch.minimum(a[t], q[t]) * ms + term[t].abs())
            ms = a[t] * ms + term[t].abs()
            es = es + 12 * EPS * ms
            h[t], e[t], m[t] = s, es, ms
            t += 1
        last[n], e_last[n] = s, es
    ud = torch.ones_like(xd) if u is None else u.double()
    y = ud * h
    ey = ud.abs() * e
    y[t:] = 0
    ey = ey + rnd * (y.abs() + ey)
    ey[t:] = 0
    return dict(y=y, ey=ey, last=last, elast=e_last, h=h, e=e, before=before, e_before=e_before, m_before=m_before,
                a=a, q=q, d=d, rows=t)


def backward(x, gate, lam, u, lens, h0, cpw, gy, gh):
    """{name: (gradient, bound)} of gx, ggate, glam, gu, gh0."""
    f = forward(x, gate, lam, u, lens, h0, cpw)
    T, D = x.shape
    rnd = half_step(x.dtype) + 2 * EPS
    a, q, d, xd = f["a"], f["q"], f["d"], x.double()
    gyd = torch.zeros_like(xd) if gy is None else gy.double()
    src = gyd if u is None else gyd * u.double()
    G, EG, MG = (torch.zeros(T, D, dtype=torch.float64) for _ in range(3))
    gh0 = torch.zeros(len(lens), D, dtype=torch.float64) if gh is None else gh.double().clone()
    e0 = torch.zeros_like(gh0)
    t1 = sum(lens)
    for n in range(len(lens) - 1, -1, -1):
        c, ec, mc = gh0[n], torch.zeros(D, dtype=torch.float64), gh0[n].abs()
        for t in range(t1 - 1, t1 - lens[n] - 1, -1):
            G[t] = src[t] + c
            MG[t] = src[t].abs() + mc
            EG[t] = ec + 12 * EPS * MG[t]
            c = a[t] * G[t]
            ec = a[t] * EG[t] + d[t] * torch.minimum(a[t], q[t]) * MG[t]
            mc = a[t] * MG[t]
        gh0[n], e0[n] = c, ec + 3 * EPS * mc
        t1 -= lens[n]
    out = {}

    def put(name, value, err):
        out[name] = (value, err + rnd * (value.abs() + err))

    if lam is None:
        put("gx", q * G, q * (EG + d * MG))
    else:
        put("gx", lam.double() * G, lam.double().abs() * EG)
        put("glam", xd * G, xd.abs() * EG)
    if u is not None:
        put("gu", gyd * f["h"], gyd.abs() * f["e"])
    w = a * q
    p, mp = (f["before"] - xd, f["m_before"] + xd.abs()) if lam is None else (f["before"], f["m_before"])
    mass = w * MG * mp
    err = w * (EG * mp + MG * f["e_before"]) + (2 * d + (8 + cpw) * EPS) * mass

    def sets(v):
        v = v.clone()
        v[f["rows"]:] = 0
        return v.view(T, D // cpw, cpw).sum(2)

    for k in list(out):
        out[k][0][f["rows"]:] = 0
        out[k][1][f["rows"]:] = 0
    put("ggate", sets(w * G * p), sets(err))
    out["gh0"] = (gh0, e0)
    return out


def adapters(base, x, a, b, scale, lens, ids):
    """out and its bound.  Each product is a sum of K (then r) terms in fp32, in any order: off by at most
    K eps (r eps) of the sum of absolute values; 16 eps more for splitting a factor in two parts, the scale and
    joining partial sums."""
    T, M = base.shape
    R, r, K = a.shape
    rnd = half_step(x.dtype) + 2 * EPS
    out, err = torch.zeros(T, M, dtype=torch.float64), torch.zeros(T, M, dtype=torch.float64)
    t = 0
    for n, count in enumerate(lens):
        rows, i = slice(t, t + count), ids[n]
        out[rows] = base[rows].double()
        if 0 <= i < R and count:
            ad, bd, xd = a[i].double(), b[i].double(), x[rows].double()
            s = 1.0 if scale is None else float(scale[i])
            out[rows] += s * (xd @ ad.t()) @ bd.t()
            mass = abs(s) * (xd.abs() @ ad.abs().t()) @ bd.abs().t()
            err[rows] = (K + r + 16) * EPS * mass
            err[rows] += rnd * (out[rows].abs() + err[rows])
        t += count
    return out, err
