"""GPU: the gated recurrence, its backward and its step against the 64-bit reference, within the bounds that the
reference derives from the arithmetic."""
import pytest
import torch

import sequence_ref as ref
from parity import say
from sequence_cases import close, make, offsets_of, strided, up

pytestmark = pytest.mark.gpu


def call(c, dev="cuda", **kw):
    import linear_spatial_propagation_amd as gspn
    return gspn.seq_scan_fwd(up(c["x"], dev), up(c["gate"], dev), lam=up(c["lam"], dev), u=up(c["u"], dev),
                             offsets=up(offsets_of(c["lens"]), dev), h0=up(c["h0"], dev), ch_per_weight=c["cpw"], **kw)


def check(c, got):
    f = ref.forward(c["x"], c["gate"], c["lam"], c["u"], c["lens"], c["h0"], c["cpw"])
    close("y", got[0], f["y"], f["ey"])
    close("h_last", got[1], f["last"], f["elast"])


LENS = [[1], [63, 65, 64], [0, 0, 7, 0, 130, 1, 0], [700], [1] * 70, [255, 1, 257, 129]]
WIDTHS = [(1, 1), (3, 1), (37, 1), (64, 2), (66, 3), (130, 1), (130, 13), (256, 128), (320, 160), (96, 8), (192, 192)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}seq{sum(v)}")
@pytest.mark.parametrize("D,cpw", [(130, 1), (96, 8)])
def test_forward_lengths(dtype, lens, D, cpw):
    say(f"forward {dtype} lens {lens[:8]} D {D} cpw {cpw}")
    c = make(lens, D, dtype=dtype, cpw=cpw, pad=3, seed=len(lens) + D)
    check(c, call(c))


@pytest.mark.parametrize("N", [62, 63, 64, 65, 127, 4095, 4096, 5000])
def test_numbers_of_sequences(N):
    """Finding a tile's sequence among 64, 64 x 64 and more, empty ones among them."""
    say(f"{N} sequences of 0 to 3 tokens and one of 200")
    lens = [(7 * i + i // 5) % 4 for i in range(N)]
    lens[N // 3] = 200
    c = make(lens, 6, dtype="f32", pad=3, seed=N)
    check(c, call(c))
    check_grads(c, grads(c))


# many tiles behind one another: one sequence, one among single tokens, a few, many of a middling length
LONG = [[5003], [1] * 150 + [3001], [2, 0, 2500, 1000, 1], [90, 0, 45, 200] * 18]


@pytest.mark.parametrize("dtype,D,cpw", [("f32", 8, 2), ("bf16", 134, 2), ("bf16", 35, 5)])
@pytest.mark.parametrize("lens", LONG, ids=lambda v: f"{len(v)}seq{sum(v)}")
def test_long_sequences(dtype, D, cpw, lens):
    say(f"long {dtype} {len(lens)} sequences, {sum(lens)} tokens, D {D}")
    c = make(lens, D, dtype=dtype, cpw=cpw, pad=2, seed=sum(lens))
    check(c, call(c))
    check_grads(c, grads(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L", [(2, 1800), (70, 40), (8, 530)])
@pytest.mark.parametrize("D,cpw", [(40, 8), (21, 7)])
def test_many_equal_rows(dtype, B, L, D, cpw):
    import linear_spatial_propagation_amd as gspn
    say(f"equal rows {dtype} {B} x {L}, D {D}, both directions")
    c = make([L] * B, D, dtype=dtype, cpw=cpw, lam=False, seed=B)
    x, gate, u, gy = (up(c[k]).view(B, L, -1) for k in ("x", "gate", "u", "gy"))
    y, last, st = gspn.seq_scan_fwd(x, gate, u=u, h0=up(c["h0"]), ch_per_weight=cpw, return_states=True)
    check(c, (y.view(B * L, D), last))
    g = gspn.seq_scan_bwd(x, gate, gy, st, u=u, gh_last=up(c["gh"]), ch_per_weight=cpw)
    check_grads(c, [None if t is None else t.reshape(-1, t.shape[-1]) for t in g])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,cpw", WIDTHS)
@pytest.mark.parametrize("lam,u,h0", [(True, True, True), (False, False, False), (True, False, False), (False, True, True)])
def test_forward_widths(dtype, D, cpw, lam, u, h0):
    say(f"forward {dtype} D {D} cpw {cpw} lam {lam} u {u} h0 {h0}")
    c = make([70, 0, 129], D, dtype=dtype, cpw=cpw, lam=lam, u=u, h0=h0, seed=D + cpw)
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L", [(3, 1), (2, 64), (5, 200), (1, 65), (4, 0)])
def test_equal_rows(dtype, B, L):
    import linear_spatial_propagation_amd as gspn
    say(f"equal rows {dtype} {B} x {L}")
    c = make([L] * B, 72, dtype=dtype, seed=B + L)
    t = [up(c[k]).view(B, L, 72) for k in ("x", "gate", "lam", "u")]
    y, last = gspn.seq_scan_fwd(t[0], t[1], lam=t[2], u=t[3], h0=up(c["h0"]))
    assert y.shape == (B, L, 72)
    check(c, (y.reshape(B * L, 72), last))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("extra", [4, 5])
def test_strided_rows(dtype, extra):
    """Rows that are column ranges of wider tensors, at aligned and at odd distances."""
    say(f"strided {dtype} {extra}")
    c = make([70, 3, 0, 150], 66, dtype=dtype, seed=5)
    want = call(c)
    s = dict(c, **{k: strided(c[k], extra) for k in ("x", "gate", "lam", "u")})
    s = {k: v for k, v in s.items()}
    import linear_spatial_propagation_amd as gspn
    t = {k: strided(up(c[k]), extra) for k in ("x", "gate", "lam", "u")}
    got = gspn.seq_scan_fwd(t["x"], t["gate"], lam=t["lam"], u=t["u"], offsets=up(offsets_of(c["lens"])), h0=up(c["h0"]))
    check(c, got)
    check(c, want)


def test_repeated_row():
    """A stride of 0: one row of gates for every token."""
    import linear_spatial_propagation_amd as gspn
    c = make([90, 5], 40, seed=3)
    c["gate"] = c["gate"][:1].expand(95, 40)
    got = gspn.seq_scan_fwd(up(c["x"]), up(c["gate"][:1]).expand(95, 40), lam=up(c["lam"]), u=up(c["u"]),
                            offsets=up(offsets_of(c["lens"])), h0=up(c["h0"]))
    check(c, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_their_ends(dtype):
    """Gates of -inf (the state starts over), +inf (it stays), the type's lowest and highest, +-200 and 0."""
    c = make([150], 70, dtype=dtype, seed=9)
    g = torch.Generator().manual_seed(1)
    pick = torch.randint(0, 8, c["gate"].shape, generator=g)
    top = torch.finfo(c["gate"].dtype).max
    for i, v in enumerate((float("-inf"), float("inf"), -top, top, -200.0, 200.0, 0.0)):
        c["gate"][pick == i] = v
    c["lam"] = None
    got = call(c)
    a = torch.sigmoid(c["gate"].double())
    h, bound, m = c["h0"][0].double(), torch.zeros(70, dtype=torch.float64), c["h0"][0].double().abs()
    ys, es = [], []
    for t in range(150):
        x = c["x"][t].double()
        q = torch.sigmoid(-c["gate"][t].double())
        h = a[t] * h + q * x
        d = (c["gate"][t].double().abs().clamp(max=100) + 8) * 2.0 ** -23
        bound = a[t] * bound + d * (torch.minimum(a[t], q) * m + q * x.abs())
        m = a[t] * m + q * x.abs()
        bound = bound + 12 * ref.EPS * m
        ys.append(h * c["u"][t].double())
        es.append(bound * c["u"][t].double())
    y, e = torch.stack(ys), torch.stack(es)
    close("y", got[0], y, e + (ref.half_step(c["x"].dtype) + 2 * ref.EPS) * (y.abs() + e) + 1e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_passes_between_sequences(dtype):
    """NaN and Inf in one sequence, its h0 and the padding stay there; rows behind the last are zero, or as they were."""
    import linear_spatial_propagation_amd as gspn
    lens = [40, 70, 0, 130, 20]
    c = make(lens, 66, dtype=dtype, pad=9, seed=11)
    off = offsets_of(lens)
    bad = dict(c, x=c["x"].clone(), gate=c["gate"].clone(), lam=c["lam"].clone(), u=c["u"].clone(), h0=c["h0"].clone())
    for k, v in (("x", float("inf")), ("gate", float("nan")), ("lam", float("nan")), ("u", float("-inf"))):
        bad[k][off[1] + 3:off[2]] = v
        bad[k][off[-1]:] = float("nan")
    bad["h0"][1] = float("nan")
    want, got = call(c), call(bad)
    mine = torch.ones(c["x"].shape[0], dtype=torch.bool)
    mine[off[1]:off[2]] = False
    assert torch.equal(want[0].cpu()[mine], got[0].cpu()[mine])
    assert float(got[0][off[-1]:].float().abs().sum()) == 0
    keep = [0, 2, 3, 4]
    assert torch.equal(want[1].cpu()[keep], got[1].cpu()[keep])
    out = torch.full_like(up(c["x"]), 7.0)
    y, _ = call(bad, out=out)
    assert y is out and bool((out[off[-1]:] == 7).all())
    assert torch.equal(out.cpu()[mine][:-9], want[0].cpu()[mine][:-9])
    # gradients of the rows behind the last, and of the others
    st = call(bad, return_states=True)[2]
    gr = gspn.seq_scan_bwd(up(bad["x"]), up(bad["gate"]), up(c["gy"]), st, lam=up(bad["lam"]), u=up(bad["u"]),
                           offsets=up(off))
    st = call(c, return_states=True)[2]
    gw = gspn.seq_scan_bwd(up(c["x"]), up(c["gate"]), up(c["gy"]), st, lam=up(c["lam"]), u=up(c["u"]), offsets=up(off))
    for a, b in zip(gr[:4], gw[:4]):
        assert torch.equal(a.cpu()[mine], b.cpu()[mine])
        assert float(a[off[-1]:].float().abs().sum()) == 0
    assert torch.equal(gr[4].cpu()[keep], gw[4].cpu()[keep])


def test_offsets_that_describe_no_rows():
    """Offsets that are no ascending row numbers: no access leaves the tensors, the call ends, other calls are unharmed."""
    c = make([200, 56], 70, seed=2)
    want = call(c)
    import linear_spatial_propagation_amd as gspn
    for bad in ([0, 300, 256], [-5, 400, 7], [200, 100, 0], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]):
        gspn.seq_scan_fwd(up(c["x"]), up(c["gate"]), lam=up(c["lam"]), u=up(c["u"]), h0=up(c["h0"]),
                          offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    got = call(c)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def grads(c, **kw):
    import linear_spatial_propagation_amd as gspn
    st = call(c, return_states=True)[2]
    return gspn.seq_scan_bwd(up(c["x"]), up(c["gate"]), up(c["gy"]), st, lam=up(c["lam"]), u=up(c["u"]),
                             offsets=up(offsets_of(c["lens"])), gh_last=up(c["gh"]), ch_per_weight=c["cpw"], **kw)


def check_grads(c, got):
    want = ref.backward(c["x"], c["gate"], c["lam"], c["u"], c["lens"], c["h0"], c["cpw"], c["gy"], c["gh"])
    for name, t in zip(("gx", "ggate", "glam", "gu", "gh0"), got):
        assert (t is None) == (name not in want), name
        if t is not None:
            close(name, t, *want[name])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}seq{sum(v)}")
@pytest.mark.parametrize("D,cpw", [(130, 1), (96, 8)])
def test_backward_lengths(dtype, lens, D, cpw):
    say(f"backward {dtype} lens {lens[:8]} D {D} cpw {cpw}")
    c = make(lens, D, dtype=dtype, cpw=cpw, pad=3, seed=len(lens) + D + 1)
    check_grads(c, grads(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,cpw", WIDTHS)
@pytest.mark.parametrize("lam,u", [(True, True), (False, False), (True, False), (False, True)])
def test_backward_widths(dtype, D, cpw, lam, u):
    say(f"backward {dtype} D {D} cpw {cpw} lam {lam} u {u}")
    c = make([70, 0, 129], D, dtype=dtype, cpw=cpw, lam=lam, u=u, seed=D + cpw + 1)
    check_grads(c, grads(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_of_many_shared_gates(dtype):
    """More gate gradients (2100 x 512) than the launch that adds their parts has lanes."""
    say(f"backward {dtype} 2100 tokens, 512 gates of 3 channels")
    c = make([2000, 100], 1536, dtype=dtype, cpw=3, pad=1, seed=77)
    check_grads(c, grads(c))


def test_backward_into_given_tensors_and_strides():
    import linear_spatial_propagation_amd as gspn
    c = make([70, 3, 150], 66, dtype="bf16", cpw=3, pad=4, seed=8)
    t = {k: strided(up(c[k])) for k in ("x", "gate", "lam", "u", "gy")}
    off = up(offsets_of(c["lens"]))
    st = gspn.seq_scan_fwd(t["x"], t["gate"], lam=t["lam"], u=t["u"], offsets=off, h0=up(c["h0"]), ch_per_weight=3,
                           return_states=True)[2]
    out = [strided(torch.full_like(up(c[k]), 7.0)) for k in ("x", "gate", "lam", "u")] + [torch.empty_like(up(c["h0"]))]
    got = gspn.seq_scan_bwd(t["x"], t["gate"], t["gy"], st, lam=t["lam"], u=t["u"], offsets=off, gh_last=up(c["gh"]),
                            ch_per_weight=3, out=out)
    for a, b in zip(got, out):
        assert a is b
    for a in out[:4]:
        assert bool((a[-4:] == 7).all())
        a[-4:] = 0
    check_grads(c, got)


@pytest.mark.parametrize("lam", [True, False])
def test_autograd(lam):
    """seq_scan under autograd: all gradients; of y alone; of h_last alone; of some inputs; broadcast inputs."""
    import linear_spatial_propagation_amd as gspn
    c = make([70, 0, 33], 48, cpw=4, lam=lam, seed=21)
    off = up(offsets_of(c["lens"]))

    def leaves():
        return {k: up(c[k]).requires_grad_() for k in ("x", "gate", "lam", "u", "h0") if c[k] is not None}

    def run(v):
        return gspn.seq_scan(v["x"], v["gate"], lam=v.get("lam"), u=v["u"], offsets=off, h0=v["h0"], ch_per_weight=4)

    for use_y, use_h in ((True, True), (True, False), (False, True)):
        v = leaves()
        y, last = run(v)
        loss = 0
        if use_y:
            loss = loss + (y * up(c["gy"])).sum()
        if use_h:
            loss = loss + (last * up(c["gh"])).sum()
        loss.backward()
        want = ref.backward(c["x"], c["gate"], c["lam"], c["u"], c["lens"], c["h0"], 4, c["gy"] if use_y else None,
                            c["gh"] if use_h else None)
        for k, t in v.items():
            close("g" + k, t.grad, *want["g" + k])
    v = leaves()
    part = {k: t if k == "gate" else t.detach() for k, t in v.items()}
    (g,) = torch.autograd.grad(run(part)[0].sum(), [v["gate"]])
    w = ref.backward(c["x"], c["gate"], c["lam"], c["u"], c["lens"], c["h0"], 4, torch.ones_like(c["gy"]), None)
    close("ggate", g, *w["ggate"])
    # one row of u for every token: its gradient is the sum over them
    row = up(c["u"][:1]).requires_grad_()
    y, _ = gspn.seq_scan(up(c["x"]), up(c["gate"]), lam=up(c["lam"]), u=row.expand(103, 48), offsets=off,
                         h0=up(c["h0"]), ch_per_weight=4)
    (y * up(c["gy"])).sum().backward()
    w = ref.backward(c["x"], c["gate"], c["lam"], c["u"][:1].expand(103, 48), c["lens"], c["h0"], 4, c["gy"], None)["gu"]
    close("gu", row.grad, w[0].sum(0, keepdim=True), w[1].sum(0, keepdim=True) + 103 * ref.EPS * w[0].abs().sum(0, keepdim=True))
    with pytest.raises(RuntimeError):
        v = leaves()
        y, _ = run(v)
        (gx,) = torch.autograd.grad(y.sum(), [v["x"]], create_graph=True)
        gx.sum().backward()


def test_gradients_of_a_projection():
    """The four inputs as column ranges of one projection's output, as a layer has them: the weight's gradient against
    the reference's, in fp32."""
    import linear_spatial_propagation_amd as gspn
    D, cpw, lens = 24, 3, [50, 17]
    g = torch.Generator().manual_seed(4)
    tok, W = torch.randn(67, 16, generator=g), torch.randn(16, 3 * D + D // cpw, generator=g)
    w = up(W).requires_grad_()
    p = up(tok) @ w
    x, lam, u, gate = p.split([D, D, D, D // cpw], 1)
    y, _ = gspn.seq_scan(x, gate, lam=lam, u=u, offsets=up(offsets_of(lens)), ch_per_weight=cpw)
    gy = torch.randn(67, D, generator=g)
    (y * up(gy)).sum().backward()
    pc = p.detach().cpu()
    xc, lc, uc, gc = pc.split([D, D, D, D // cpw], 1)
    r = ref.backward(xc, gc, lc, uc, lens, None, cpw, gy, None)
    cols = [r[k] for k in ("gx", "glam", "gu", "ggate")]
    want, err = torch.cat([v[0] for v in cols], 1), torch.cat([v[1] for v in cols], 1)
    mass = tok.double().abs().t() @ (want.abs() + err)
    close("gw", w.grad, tok.double().t() @ want, tok.double().abs().t() @ err + (67 + 4) * ref.EPS * mass)


def step_ref(c, state, slots):
    """Row by row: y, state and their bounds."""
    state, y, ey = state.double().clone(), torch.zeros(c["x"].shape, dtype=torch.float64), None
    es, ey = torch.zeros_like(state), torch.zeros_like(y)
    a, q, d = ref._gates(c["gate"], c["cpw"])
    rnd = ref.half_step(c["x"].dtype) + 2 * ref.EPS
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            continue
        term = (q[i] if c["lam"] is None else c["lam"][i].double()) * c["x"][i].double()
        es[s] = a[i] * es[s] + d[i] * (torch.minimum(a[i], q[i]) * state[s].abs() + term.abs())
        m = a[i] * state[s].abs() + term.abs()
        es[s] += 12 * ref.EPS * m
        state[s] = a[i] * state[s] + term
        u = 1.0 if c["u"] is None else c["u"][i].double()
        y[i] = u * state[s]
        ey[i] = u * es[s] + rnd * (y[i].abs() + u * es[s])
    return y, ey, state, es


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,cpw", WIDTHS + [(1032, 1)])
@pytest.mark.parametrize("lam,u", [(True, True), (False, False)])
def test_step(dtype, D, cpw, lam, u):
    import linear_spatial_propagation_amd as gspn
    say(f"step {dtype} D {D} cpw {cpw}")
    c = make([9], D, dtype=dtype, cpw=cpw, lam=lam, u=u, seed=D)
    g = torch.Generator().manual_seed(D)
    for slots, S in ((None, 11), ([3, 0, 11, 7, 1, 12, 5, 2, 9], 13)):
        state = torch.randn(S, D, generator=g)
        st = up(state)
        y = gspn.seq_step(up(c["x"]), up(c["gate"]), st, lam=up(c["lam"]), u=up(c["u"]), ch_per_weight=cpw,
                          slots=None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda"))
        wy, ey, ws, es = step_ref(c, state, slots or range(9))
        close("y", y, wy, ey)
        close("state", st, ws, es)


@pytest.mark.parametrize("rows", [5, 300, 700])
def test_step_padding_and_repeated_slots(rows):
    """Slots out of range are skipped; rows of one slot are taken in order, wherever they stand."""
    import linear_spatial_propagation_amd as gspn
    c = make([rows], 34, cpw=2, seed=rows)
    g = torch.Generator().manual_seed(rows)
    S = rows // 2 + 1
    slots = torch.randint(-2, S + 2, (rows,), generator=g, dtype=torch.int32)
    slots[0], slots[-1] = 1, 1
    slots[1] = -2 ** 31
    state = torch.randn(S, 34, generator=g)
    wy, ey, ws, es = step_ref(c, state, slots.tolist())
    for out in (None, torch.full((rows, 34), 7.0, device="cuda")):
        st = up(state)
        y = gspn.seq_step(up(c["x"]), up(c["gate"]), st, lam=up(c["lam"]), u=up(c["u"]), slots=up(slots),
                          ch_per_weight=2, out=out)
        skipped = (slots < 0) | (slots >= S)
        assert bool((y.cpu()[skipped] == (0 if out is None else 7)).all())
        got = y.cpu().clone()
        got[skipped] = 0
        close("y", got, wy, ey)
        close("state", st, ws, es)
        untouched = torch.tensor([s not in set(slots.tolist()) for s in range(S)])
        assert torch.equal(st.cpu()[untouched], state[untouched])


def test_step_refuses_gradients():
    import linear_spatial_propagation_amd as gspn
    x, state = torch.ones(2, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    gate = torch.zeros(2, 8, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no backward"):
        gspn.seq_step(x, gate, state)
    with torch.no_grad():
        assert torch.equal(gspn.seq_step(x, gate, state), torch.full_like(x, 0.5))
    # torch.no_grad is not needed for tensors that ask for none
    gspn.seq_step(x, gate.detach(), state)


def test_step_of_no_rows():
    import linear_spatial_propagation_amd as gspn
    st = torch.ones(3, 8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    assert gspn.seq_step(e, e, st).shape == (0, 8) and bool((st == 1).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(dtype):
    """T = 0: h_last is h0, and its gradient passes straight through."""
    import linear_spatial_propagation_amd as gspn
    c = make([0, 0, 0], 20, dtype=dtype, seed=1)
    y, last, st = call(c, return_states=True)
    assert y.shape == (0, 20) and torch.equal(last.cpu(), c["h0"])
    got = grads(c)
    assert torch.equal(got[4].cpu(), c["gh"]) and got[0].shape == (0, 20)


def test_rows_behind_32_bits():
    """Row distances that put the last rows past 2^31 elements, bf16 and fp32, forward, backward and step."""
    import linear_spatial_propagation_amd as gspn
    for dtype, far in (("bf16", 2 ** 30), ("f32", 2 ** 29 + 2)):
        say(f"far rows {dtype}")
        c = make([3, 3], 40, dtype=dtype, seed=6)
        wide = torch.empty(5 * far + 200, dtype=c["x"].dtype, device="cuda")
        t = {}
        for i, k in enumerate(("x", "gate", "lam", "u")):
            t[k] = wide.as_strided((6, 40), (far, 1), 40 * i)
            t[k].copy_(up(c[k]))
        y, last, st = gspn.seq_scan_fwd(t["x"], t["gate"], lam=t["lam"], u=t["u"], offsets=up(offsets_of(c["lens"])),
                                        h0=up(c["h0"]), return_states=True)
        check(c, (y, last))
        got = gspn.seq_scan_bwd(t["x"], t["gate"], up(c["gy"]), st, lam=t["lam"], u=t["u"],
                                offsets=up(offsets_of(c["lens"])), gh_last=up(c["gh"]))
        check_grads(c, got)
        state = torch.randn(6, 40)
        s = up(state)
        y = gspn.seq_step(t["x"], t["gate"], s, lam=t["lam"], u=t["u"])
        wy, ey, ws, es = step_ref(c, state, range(6))
        close("y", y, wy, ey)
        close("state", s, ws, es)
        del wide, t


@pytest.mark.parametrize("cpw", [1, 8])
def test_capture_and_replay(cpw):
    """Forward, backward and step captured into a graph and replayed: each replay equals the eager call, bit for bit,
    with eager work between."""
    import linear_spatial_propagation_amd as gspn
    c = make([300, 0, 500, 1], 136, dtype="bf16", cpw=cpw, seed=13)
    t = {k: up(c[k]) for k in ("x", "gate", "lam", "u", "h0", "gy", "gh")}
    off = up(offsets_of(c["lens"]))
    state0 = torch.randn(10, 136, device="cuda")

    def once(state):
        y, last, st = gspn.seq_scan_fwd(t["x"], t["gate"], lam=t["lam"], u=t["u"], offsets=off, h0=t["h0"],
                                        ch_per_weight=cpw, return_states=True)
        g = gspn.seq_scan_bwd(t["x"], t["gate"], t["gy"], st, lam=t["lam"], u=t["u"], offsets=off, gh_last=t["gh"],
                              ch_per_weight=cpw)
        z = gspn.seq_step(t["x"][:10], t["gate"][:10], state, lam=t["lam"][:10], u=t["u"][:10], ch_per_weight=cpw)
        return [y, last, *g, z, state]

    want = [v.clone() for v in once(state0.clone())]
    state = state0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(state.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once(state)
    for _ in range(4):
        state.copy_(state0)
        for v in got[:-1]:
            v.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        float(torch.ones(1 << 16, device="cuda").cumsum(0)[-1])
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs():
    """Two captured calls replayed side by side on two streams: each has a workspace of its own."""
    cases = [make([900, 300, 1, 0, 400], 160, dtype="bf16", cpw=8, seed=17), make([2000, 3], 96, seed=18)]
    want = [grads(c) for c in cases]
    import linear_spatial_propagation_amd as gspn
    dev = [({k: up(c[k]) for k in ("x", "gate", "lam", "u", "h0", "gy", "gh")}, up(offsets_of(c["lens"]))) for c in cases]

    def once(i):
        t, off = dev[i]
        st = gspn.seq_scan_fwd(t["x"], t["gate"], lam=t["lam"], u=t["u"], offsets=off, h0=t["h0"],
                               ch_per_weight=cases[i]["cpw"], return_states=True)[2]
        return gspn.seq_scan_bwd(t["x"], t["gate"], t["gy"], st, lam=t["lam"], u=t["u"], offsets=off, gh_last=t["gh"],
                                 ch_per_weight=cases[i]["cpw"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for i in range(2):
            once(i)
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            got.append(once(i))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for g in got:
            for t in g:
                t.fill_(7)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_two_streams():
    """The same inputs on two streams at once: bitwise the same results."""
    c = make([900, 300, 1, 0, 400], 160, dtype="bf16", cpw=8, seed=17)
    want = grads(c)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        res = []
        for s in streams:
            with torch.cuda.stream(s):
                res.append(grads(c))
        torch.cuda.synchronize()
        for r in res:
            for a, b in zip(r, want):
                assert torch.equal(a, b)


def test_wrapper_refusals():
    import linear_spatial_propagation_amd as gspn
    x = torch.zeros(6, 8, device="cuda")
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    bad = [
        lambda: gspn.seq_scan_fwd(x, x[:, :4]), lambda: gspn.seq_scan_fwd(x, x.bfloat16()), lambda: gspn.seq_scan_fwd(x.half(), x.half()),
        lambda: gspn.seq_scan_fwd(x, x, lam=x[:5]), lambda: gspn.seq_scan_fwd(x, x, offsets=off.long()),
        lambda: gspn.seq_scan_fwd(x, x, offsets=off[:1]), lambda: gspn.seq_scan_fwd(x, x, offsets=off.cpu()),
        lambda: gspn.seq_scan_fwd(x.t(), x.t()), lambda: gspn.seq_scan_fwd(x, x, h0=torch.zeros(2, 8, device="cuda")),
        lambda: gspn.seq_scan_fwd(x, x, h0=torch.zeros(1, 8, device="cuda").bfloat16()), lambda: gspn.seq_scan_fwd(x, x, ch_per_weight=3),
        lambda: gspn.seq_scan_fwd(x.view(2, 3, 8), x.view(2, 3, 8), offsets=off), lambda: gspn.seq_scan_fwd(x[0], x[0]),
        lambda: gspn.seq_scan_fwd(x.view(2, 3, 8).transpose(0, 1), x.view(3, 2, 8)), lambda: gspn.seq_scan_fwd(x, x, out=x),
        lambda: gspn.seq_scan_fwd(x, x, out=x[:1].expand(6, 8)), lambda: gspn.seq_step(x, x, x, out=x[:3]),
        lambda: gspn.seq_step(x, x, x[:3]), lambda: gspn.seq_step(x, x, x.bfloat16()),
        lambda: gspn.seq_step(x, x, torch.zeros(6, 8, device="cuda"), slots=off),
        lambda: gspn.seq_scan_bwd(x, x, x, torch.zeros(2, 8, device="cuda")),
        lambda: gspn.seq_scan_bwd(x, x, x, torch.zeros(1, 8, device="cuda"), out=(x, x, None, None)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
            raise AssertionError(f"call {i} was not refused")
