"""GPU: low-rank adapters of many requests against the 64-bit reference, and the run of adapters and recurrence
together as a layer of a server has them."""
import pytest
import torch

import sequence_ref as ref
from parity import say
from sequence_cases import DT, close, make, offsets_of, strided, up

pytestmark = pytest.mark.gpu


def inputs(lens, K, M, r, R, dtype, *, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    T, dt = sum(lens) + pad, DT[dtype]
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    return dict(base=rn(T, M).to(dt), x=rn(T, K).to(dt), a=(rn(R, r, K) / K ** 0.5).to(dt), b=rn(R, M, r).to(dt),
                scale=0.5 + torch.rand(R, generator=g), lens=lens,
                ids=torch.randint(-1, R + 1, (len(lens),), generator=g, dtype=torch.int32))


def call(c, scale=True, **kw):
    import linear_spatial_propagation_amd as gspn
    return gspn.adapter_add(up(c["base"]), up(c["x"]), up(c["a"]), up(c["b"]), up(c["ids"]),
                            scale=up(c["scale"]) if scale else None, offsets=up(offsets_of(c["lens"])), **kw)


def check(c, got, scale=True):
    want, err = ref.adapters(c["base"], c["x"], c["a"], c["b"], c["scale"] if scale else None, c["lens"],
                             c["ids"].tolist())
    close("out", got, want, err)


LENS = [[1], [1] * 33, [16, 17, 15], [0, 5, 0, 0, 90, 1, 0], [200], [64, 1, 1, 130, 3]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}req{sum(v)}")
@pytest.mark.parametrize("K,M,r", [(64, 64, 8), (200, 136, 16)])
def test_lengths(dtype, lens, K, M, r):
    say(f"adapters {dtype} {lens[:6]} {K} -> {r} -> {M}")
    c = inputs(lens, K, M, r, 5, dtype, pad=3, seed=sum(lens))
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,M,r", [(1, 1, 1), (3, 5, 2), (31, 33, 3), (64, 96, 4), (321, 963, 12), (1152, 130, 16),
                                   (129, 257, 17), (520, 72, 32), (96, 1000, 33), (256, 192, 64), (264, 200, 100),
                                   (128, 128, 128), (72, 136, 200), (512, 64, 256), (2304, 64, 8), (4104, 40, 5)])
def test_widths(dtype, K, M, r):
    say(f"adapters {dtype} {K} -> {r} -> {M}")
    c = inputs([5, 1, 0, 40, 1], K, M, r, 3, dtype, pad=2, seed=K + M + r)
    check(c, call(c))
    check(c, call(c, scale=False), scale=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("extra", [8, 5])
def test_strides_and_places(dtype, extra):
    """Rows of wider tensors; into base itself; rows behind the last request as they were, or zero."""
    import linear_spatial_propagation_amd as gspn
    c = inputs([3, 40, 0, 1], 72, 88, 8, 4, dtype, pad=4, seed=extra)
    dev = {k: up(c[k]) for k in ("a", "b", "ids", "scale")}
    off = up(offsets_of(c["lens"]))
    x, base = strided(up(c["x"]), extra), strided(up(c["base"]), extra)
    args = (x, dev["a"], dev["b"], dev["ids"])
    got = gspn.adapter_add(base, *args, scale=dev["scale"], offsets=off)
    check(c, got)
    out = strided(torch.full_like(up(c["base"]), 7.0), extra)
    gspn.adapter_add(base, *args, scale=dev["scale"], offsets=off, out=out)
    assert bool((out[-4:] == 7).all())
    assert torch.equal(out[:-4], got[:-4])
    again = gspn.adapter_add(base, *args, scale=dev["scale"], offsets=off, out=base)
    assert again is base and torch.equal(base[:-4], got[:-4]) and torch.equal(base[-4:].cpu(), c["base"][-4:])


def test_equal_rows_and_repeated_adapters():
    import linear_spatial_propagation_amd as gspn
    for B, L in ((4, 1), (3, 20), (2, 64), (1, 130)):
        c = inputs([L] * B, 64, 80, 8, 2, "bf16", seed=B)
        c["ids"] = torch.tensor([1] * B, dtype=torch.int32)
        got = gspn.adapter_add(up(c["base"]).view(B, L, 80), up(c["x"]).view(B, L, 64), up(c["a"]), up(c["b"]),
                               up(c["ids"]), scale=up(c["scale"]))
        assert got.shape == (B, L, 80)
        check(c, got.view(B * L, 80))
        flat = gspn.adapter_add(up(c["base"]), up(c["x"]), up(c["a"]), up(c["b"]), up(c["ids"]), scale=up(c["scale"]))
        assert torch.equal(flat, got.view(B * L, 80))


def test_no_adapter_copies_base():
    """Rows of requests without an adapter are base's bits, NaN and Inf in their x and in unused adapters included."""
    c = inputs([20, 30, 1, 1], 64, 72, 8, 3, "bf16", pad=2, seed=3)
    c["ids"] = torch.tensor([-1, 0, 3, 1], dtype=torch.int32)
    want = call(c)
    bad = dict(c, x=c["x"].clone(), a=c["a"].clone(), b=c["b"].clone())
    bad["x"][:20] = float("nan")
    bad["x"][50] = float("inf")
    bad["x"][52:] = float("nan")
    bad["a"][2], bad["b"][2] = float("nan"), float("inf")
    got = call(bad)
    assert torch.equal(got, want)
    assert torch.equal(got[:20].cpu(), c["base"][:20]) and torch.equal(got[50].cpu(), c["base"][50])


def test_offsets_that_describe_no_rows():
    import linear_spatial_propagation_amd as gspn
    c = inputs([100, 60], 64, 72, 8, 3, "bf16", seed=3)
    want = call(c)
    for off in ([0, 300, 160], [-5, 400, 7], [160, 100, 0], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]):
        gspn.adapter_add(up(c["base"]), up(c["x"]), up(c["a"]), up(c["b"]), up(c["ids"]),
                         offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(call(c), want)


def test_no_rows():
    import linear_spatial_propagation_amd as gspn
    a, b = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(2, 16, 4, device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = gspn.adapter_add(torch.empty(0, 16, device="cuda"), torch.empty(0, 8, device="cuda"), a, b, ids)
    assert out.shape == (0, 16)


def test_rows_behind_32_bits():
    import linear_spatial_propagation_amd as gspn
    c = inputs([3, 2, 1], 72, 40, 8, 3, "bf16", seed=5)
    far = 2 ** 30
    wide = torch.empty(5 * far + 200, dtype=torch.bfloat16, device="cuda")
    x, base = wide.as_strided((6, 72), (far, 1), 0), wide.as_strided((6, 40), (far, 1), 80)
    x.copy_(up(c["x"]))
    base.copy_(up(c["base"]))
    got = gspn.adapter_add(base, x, up(c["a"]), up(c["b"]), up(c["ids"]), scale=up(c["scale"]),
                           offsets=up(offsets_of(c["lens"])))
    check(c, got)


def test_capture_and_replay():
    import linear_spatial_propagation_amd as gspn
    c = inputs([100, 1, 1, 0, 37], 264, 200, 24, 3, "bf16", seed=7)
    t = {k: up(c[k]) for k in ("base", "x", "a", "b", "ids", "scale")}
    off = up(offsets_of(c["lens"]))

    def once():
        return gspn.adapter_add(t["base"], t["x"], t["a"], t["b"], t["ids"], scale=t["scale"], offsets=off)

    want = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    for _ in range(4):
        got.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        float(torch.ones(1 << 16, device="cuda").cumsum(0)[-1])
        assert torch.equal(got, want)


def test_wrapper_refusals():
    import linear_spatial_propagation_amd as gspn
    z = lambda *s: torch.zeros(*s, device="cuda")   # noqa: E731
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    ok = dict(base=z(6, 16), x=z(6, 8), a=z(3, 4, 8), b=z(3, 16, 4), ids=ids)
    gspn.adapter_add(**ok)
    for kw in (dict(base=z(5, 16)), dict(x=z(6, 9)), dict(a=z(3, 4, 8).bfloat16()), dict(b=z(3, 15, 4)), dict(b=z(2, 16, 4)),
               dict(a=z(3, 8, 4).transpose(1, 2)), dict(ids=ids.long()), dict(ids=ids[:0]), dict(offsets=off.long()),
               dict(offsets=off[:2]), dict(scale=z(2)), dict(scale=z(3).double()), dict(out=z(6, 15)), dict(out=z(6, 1).expand(6, 16)),
               dict(a=z(3, 300, 8), b=z(3, 16, 300)), dict(x=z(6, 8).requires_grad_()), dict(ids=torch.zeros(4, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            gspn.adapter_add(**{**ok, **kw})
            raise AssertionError(f"{list(kw)} was not refused")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_of_a_server(dtype):
    """A recurrent layer for several requests with adapters of their own: packed prefill, then single tokens on the
    cache of states, against the same tokens as whole sequences in 64 bits."""
    import linear_spatial_propagation_amd as gspn
    E, D, cpw, r, R = 48, 64, 4, 8, 3
    g = torch.Generator().manual_seed(31)
    dt = DT[dtype]
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    widths = [D, D, D, D // cpw]
    w_in, a_in, b_in = (rn(E, sum(widths)) / E ** 0.5).to(dt), (rn(R, r, E) / E ** 0.5).to(dt), (rn(R, sum(widths), r) / 4).to(dt)
    w_out, a_out, b_out = (rn(D, E) / D ** 0.5).to(dt), (rn(R, r, D) / D ** 0.5).to(dt), (rn(R, E, r) / 4).to(dt)
    prompt, more, ids = [70, 5, 133], 3, torch.tensor([2, -1, 0], dtype=torch.int32)
    tokens = [rn(n + more, E).to(dt) for n in prompt]

    def project(x, w, a, b, ids, offsets=None):
        return gspn.adapter_add(x @ w, x, a, b, ids, offsets=offsets)

    dev = [up(t) for t in (w_in, a_in, b_in, w_out, a_out, b_out, ids)]
    off = up(offsets_of(prompt))
    p = project(torch.cat([up(t[:n]) for t, n in zip(tokens, prompt)]), dev[0], dev[1], dev[2], dev[6], off)
    x, lam, u, gate = p.split(widths, 1)
    y, last = gspn.seq_scan_fwd(x, gate, lam=lam, u=u, offsets=off, ch_per_weight=cpw)
    z = project(y, dev[3], dev[4], dev[5], dev[6], off)
    cache = torch.full((7, D), 7.0, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    cache[slots.long()] = last
    zs, ps, ys = [z], [p], [y]
    for i in range(more):
        p = project(torch.stack([up(t[n + i]) for t, n in zip(tokens, prompt)]), dev[0], dev[1], dev[2], dev[6])
        x, lam, u, gate = p.split(widths, 1)
        y = gspn.seq_step(x, gate, cache, lam=lam, u=u, slots=slots, ch_per_weight=cpw)
        zs.append(project(y, dev[3], dev[4], dev[5], dev[6]))
        ps.append(p)
        ys.append(y)
    assert bool((cache[[1, 2, 3, 5]] == 7).all())
    # the recurrence of the projections that the calls saw, as whole sequences, in 64 bits
    order = [list(range(sum(prompt[:n]), sum(prompt[:n + 1]))) + [sum(prompt) + 3 * i + n for i in range(more)] for n in range(3)]
    flat = [k for o in order for k in o]
    pc = torch.cat(ps).cpu()[flat]
    xc, lc, uc, gc = pc.split(widths, 1)
    lens = [n + more for n in prompt]
    f = ref.forward(xc, gc, lc, uc, lens, None, cpw)
    close("y", torch.cat(ys).cpu()[flat], f["y"], f["ey"])
    close("states", cache[slots.long()], f["last"], f["elast"])
    # and the adapters on what the projections gave
    yc = torch.cat(ys).cpu()[flat]
    base = (torch.cat(ys) @ dev[3]).cpu()[flat]
    want, err = ref.adapters(base, yc, a_out, b_out, None, lens, ids.tolist())
    # the library's product of the same rows in another batch may round differently: a half step of its result,
    # and D + 1 roundings of its sum
    mass = yc.double().abs() @ w_out.double().abs()
    err = err + 2 * (ref.half_step(dt) + (D + 1) * ref.EPS) * mass
    close("z", torch.cat(zs).cpu()[flat], want, err)
