"""The sequence operators and the request adapters as cases to be timed.

Four operators of the package: the gated linear recurrence over packed
sequences (forward), its training pass (forward and backward), its step for
single tokens on a cache of states, and the low-rank adapters of many requests
beside a shared projection.  ``run`` makes the package's calls where ``own`` is
true and computes the same from elementary torch operations where it is false;
``exact`` computes them in 64 bits, token by token and request by request.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's next token in one layer: the smallest call, all latency
        dict(name="step, one request", op="step", dtype="bf16", N=1, S=4, D=1152, cpw=1, lam=True, u=True),
        # a decode batch: 256 of 512 cached states, gates shared by 8 channels as in the compact mode
        dict(name="step, 256 requests", op="step", dtype="bf16", N=256, S=512, D=2560, cpw=8, lam=True, u=True),
        # three short prompts of odd sizes, in 32 bits
        dict(name="forward, short prompts", op="fwd", dtype="f32", T=37, N=3, pad=0, D=96, cpw=1, lam=False, u=False,
             h0=True),
        # a server's packed prefill: prompts of uneven lengths, continued states, rows of padding behind the last
        dict(name="forward, packed prompts", op="fwd", dtype="bf16", T=8192, N=24, pad=75, D=2048, cpw=1, lam=True,
             u=True, h0=True),
        # one long document: the work is along the sequence alone
        dict(name="forward, long document", op="fwd", dtype="bf16", T=131072, N=1, pad=0, D=1024, cpw=1, lam=False,
             u=False, h0=False),
        # pretraining: equal rows of 2048 tokens, gates shared by 8 channels
        dict(name="train, equal rows", op="train", dtype="bf16", T=16 * 2048, N=16, pad=0, D=1152, cpw=8, lam=True,
             u=True, h0=False),
        # long-context training of a narrow model in 32 bits
        dict(name="train, long row", op="train", dtype="f32", T=32768, N=1, pad=0, D=320, cpw=1, lam=False, u=False,
             h0=True),
        # fine-tuning on packed conversations, one gate for a head of 128 channels
        dict(name="train, packed rows", op="train", dtype="bf16", T=12001, N=40, pad=33, D=2048, cpw=128, lam=True,
             u=False, h0=False),
        # one token of one request with its adapter: all latency
        dict(name="adapters, one token", op="adapt", dtype="bf16", T=1, N=1, pad=0, K=1152, M=1152, r=8, R=4),
        # continuous batching: four prompts and sixty single tokens, an adapter each
        dict(name="adapters, mixed batch", op="adapt", dtype="bf16", T=2560, N=64, pad=20, K=4096, M=4096, r=16, R=48),
        # an evaluation of a small model in 32 bits, an odd rank and odd widths
        dict(name="adapters, odd sizes", op="adapt", dtype="f32", T=1003, N=9, pad=0, K=321, M=963, r=12, R=5),
        # prefill of long prompts at the largest usual rank
        dict(name="adapters, long prompts", op="adapt", dtype="bf16", T=16384, N=8, pad=0, K=4096, M=4096, r=64, R=8),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("step", "fwd", "train", "adapt"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "adapt":
        K, M = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        if rng.random() < 0.7:      # widths are multiples of 64 more often than not
            K, M = K // 64 * 64, M // 64 * 64
        r = rng.choice((4, 8, 16, 32, 64, 128, rng.randint(1, 100)))
        # no more tokens than the largest listed case reads and writes bytes for
        T = _spread(rng, 1, max(1, min(16384, 16384 * 4096 * 3 // ((K + 2 * M) * (1 if dtype == "bf16" else 2)))))
        N = _spread(rng, 1, min(T, 256))
        # nor more adapters than its plain form, which multiplies by all of them, has operations for
        R = min(_spread(rng, 1, 64), max(1, 16384 * 8 * 64 * 8192 // (T * r * (K + M))))
        return dict(op=op, dtype=dtype, T=T, N=N, pad=rng.choice((0, min(T - 1, 17))), K=K, M=M, r=r, R=R)
    cpw = rng.choice((1, 1, 1, 8, 128, rng.choice((2, 3, 16, 64, 160))))
    D = _spread(rng, 32, 4096)
    D = max(cpw, D // cpw * cpw)
    lam, u = rng.random() < 0.5, rng.random() < 0.5
    if op == "step":
        N = _spread(rng, 1, 1024)
        return dict(op=op, dtype=dtype, N=N, S=N + rng.randint(0, N), D=D, cpw=cpw, lam=lam, u=u)
    most = 131072 * 1024 // 4 // (2 if dtype == "f32" else 1) // (2 if op == "train" else 1)
    T = _spread(rng, 1, max(1, min(131072, most // D)))
    N = _spread(rng, 1, min(T, 512))
    return dict(op=op, dtype=dtype, T=T, N=N, pad=rng.choice((0, 0, min(T - 1, 19))), D=D, cpw=cpw, lam=lam, u=u,
                h0=rng.random() < 0.5)


def _lengths(case, seed):
    """Lengths of the N requests: equal where they divide the tokens and nothing is padded (a dense batch), else
    uneven, as requests are: a few long ones, many short, single tokens and now and then an empty one."""
    T, N = case["T"] - case["pad"], case["N"]
    if case["pad"] == 0 and T % N == 0:
        return None
    rng = random.Random(seed * 7 + 1)
    share = [rng.random() ** 6 + 1e-9 for _ in range(N)]
    cuts, total, at = [0], sum(share), 0.0
    for s in share[:-1]:
        at += s
        cuts.append(min(T, int(T * at / total)))
    cuts.append(T)
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    st = {"case": case, "op": case["op"]}
    if case["op"] != "step":
        lens = _lengths(case, seed)
        st["lens"] = lens or [(case["T"] - case["pad"]) // case["N"]] * case["N"]
        offs = [0]
        for n in st["lens"]:
            offs.append(offs[-1] + n)
        st["offsets_host"] = offs
        st["offsets"] = None if lens is None else torch.tensor(offs, dtype=torch.int32, device=dev)
        # first and last rows of the sequences that have any, and which sequences those are
        some = [n for n, k in enumerate(st["lens"]) if k]
        st["first"] = torch.tensor([offs[n] for n in some], device=dev)
        st["last"] = torch.tensor([offs[n + 1] - 1 for n in some], device=dev)
        st["some"] = torch.tensor(some, device=dev)
    if case["op"] == "adapt":
        T, K, M, r, R = (case[k] for k in ("T", "K", "M", "r", "R"))
        st["base"], st["x"] = normal(T, M).to(dt), normal(T, K).to(dt)
        st["a"] = (normal(R, r, K) / math.sqrt(K)).to(dt)
        st["b"] = (normal(R, M, r) / math.sqrt(r)).to(dt)
        st["scale"] = 0.5 + 1.5 * uniform(R)
        rng = random.Random(seed * 11 + 3)
        # one request in sixteen has no adapter
        st["ids_host"] = [-1 if case["N"] > 1 and rng.random() < 1 / 16 else rng.randrange(R) for _ in range(case["N"])]
        st["ids"] = torch.tensor(st["ids_host"], dtype=torch.int32, device=dev)
        return st
    rows, D, cpw = case["N"] if case["op"] == "step" else case["T"], case["D"], case["cpw"]
    st["x"] = normal(rows, D).to(dt)
    # each gate has a bias of its own: memories from a few tokens to some hundreds
    st["gate"] = (normal(rows, D // cpw) + 6 * uniform(D // cpw)).to(dt)
    st["lam"] = uniform(rows, D).to(dt) if case["lam"] else None
    st["u"] = uniform(rows, D).to(dt) if case["u"] else None
    if case["op"] == "step":
        st["state"] = normal(case["S"], D)
        slots = random.Random(seed * 13 + 5).sample(range(case["S"]), case["N"])
        st["slots"] = torch.tensor(slots, dtype=torch.int32, device=dev)
        return st
    st["h0"] = normal(case["N"], D) if case["h0"] else None
    if case["op"] == "train":
        st["gy"] = normal(rows, D).to(dt)
        st["gh"] = normal(case["N"], D) if case["h0"] else None
        st["leaves"] = [t.requires_grad_() for t in (st["x"], st["gate"], st["lam"], st["u"], st["h0"])
                        if t is not None]
    return st


# ------------------------------------------------------------------ plain forms
def _gates(gate, cpw):
    """a and 1 - a of every channel, each with its own relative precision."""
    g = gate.float()
    a, c = torch.sigmoid(g), torch.sigmoid(-g)
    if cpw > 1:
        a, c = a.repeat_interleave(cpw, 1), c.repeat_interleave(cpw, 1)
    return a, c


def _scan(a, b, longest):
    """h with h[t] = a[t] h[t-1] + b[t], by doubling: after a step of s each row holds the last 2 s of its terms."""
    s = 1
    while s < longest:
        b = torch.cat([b[:s], torch.addcmul(b[s:], a[s:], b[:-s])])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _plain_forward(st):
    c = st["case"]
    T, D, used = c["T"], c["D"], st["offsets_host"][-1]
    a, rest = _gates(st["gate"][:used], c["cpw"])
    x = st["x"][:used].float()
    b = rest * x if st["lam"] is None else st["lam"][:used].float() * x
    first, last, some = st["first"], st["last"], st["some"]
    a_open = a.clone()
    a_open[first] = 0
    if st["h0"] is not None:
        b[first] += a[first] * st["h0"][some]
    h = _scan(a_open, b, max(st["lens"]))
    y = torch.zeros(T, D, dtype=st["x"].dtype, device=x.device)
    y[:used] = (h if st["u"] is None else st["u"][:used].float() * h).to(y.dtype)
    h_last = torch.zeros(c["N"], D, device=x.device) if st["h0"] is None else st["h0"].detach().clone()
    h_last[some] = h[last]
    return y, h_last, (a, rest, x, h)


def _plain_train(st):
    c = st["case"]
    T, used, dt, cpw = c["T"], st["offsets_host"][-1], st["x"].dtype, c["cpw"]
    first, last, some = st["first"], st["last"], st["some"]
    y, h_last, (a, rest, x, h) = _plain_forward(st)
    gy = st["gy"][:used].float()
    src = gy.clone() if st["u"] is None else st["u"][:used].float() * gy
    if st["gh"] is not None:
        src[last] += st["gh"][some]
    # the adjoint runs backwards: a row's factor is the gate of the row behind it in its sequence
    behind = torch.cat([a[1:], torch.zeros_like(a[:1])])
    behind[last] = 0
    G = _scan(behind.flip(0), src.flip(0), max(st["lens"])).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0 if st["h0"] is None else st["h0"][some]

    def whole(t):
        out = torch.zeros(T, t.shape[1], dtype=dt, device=t.device)
        out[:used] = t.to(dt)
        return out

    lam = None if st["lam"] is None else st["lam"][:used].float()
    ga = a * rest * G * (before if lam is not None else before - x)
    grads = [whole(G * (rest if lam is None else lam)), whole(ga.view(used, -1, cpw).sum(2))]
    if lam is not None:
        grads.append(whole(G * x))
    if st["u"] is not None:
        grads.append(whole(gy * h))
    if st["h0"] is not None:
        gh0 = st["gh"].clone()
        gh0[some] = (a * G)[first]
        grads.append(gh0)
    return [y, h_last] + grads


def _plain_step(st):
    a, rest = _gates(st["gate"], st["case"]["cpw"])
    x, slots = st["x"].float(), st["slots"].long()
    h = a * st["state"][slots] + (rest * x if st["lam"] is None else st["lam"].float() * x)
    st["state"][slots] = h
    y = h if st["u"] is None else st["u"].float() * h
    return [y.to(st["x"].dtype), st["state"]]


def _plain_adapt(st):
    c = st["case"]
    T, r, R, M, used = c["T"], c["r"], c["R"], c["M"], st["offsets_host"][-1]
    dev = st["x"].device
    row = torch.arange(used, device=dev)
    ids = st["ids"][row // (T // c["N"]) if st["offsets"] is None else
                    torch.searchsorted(st["offsets"][1:], row, right=True)]
    # every adapter's first product for every row; the row's own is kept, and the second product adds it up
    v = st["x"][:used].float() @ st["a"].float().reshape(R * r, -1).t()
    mine = (ids[:, None] == torch.arange(R, device=dev)[None]) * st["scale"][None]
    v = (v.view(used, R, r) * mine[:, :, None]).reshape(used, R * r)
    out = torch.zeros(T, M, dtype=st["x"].dtype, device=dev)
    out[:used] = (st["base"][:used].float() + v @ st["b"].float().transpose(1, 2).reshape(R * r, M)).to(out.dtype)
    return out


def run(st):
    op = st["op"]
    if own:
        import linear_spatial_propagation_amd as gspn
        if op == "adapt":
            if st["offsets"] is None:
                N = st["case"]["N"]
                rows = gspn.adapter_add(st["base"].view(N, -1, st["case"]["M"]), st["x"].view(N, -1, st["case"]["K"]),
                                        st["a"], st["b"], st["ids"], scale=st["scale"])
                return rows.view(-1, st["case"]["M"])
            return gspn.adapter_add(st["base"], st["x"], st["a"], st["b"], st["ids"], scale=st["scale"],
                                    offsets=st["offsets"])
        cpw = st["case"]["cpw"]
        if op == "step":
            y = gspn.seq_step(st["x"], st["gate"], st["state"], lam=st["lam"], u=st["u"], slots=st["slots"],
                              ch_per_weight=cpw)
            return [y, st["state"]]
        x, gate, lam, u = (None if t is None else t if st["offsets"] is not None else
                           t.view(st["case"]["N"], -1, t.shape[1]) for t in
                           (st["x"], st["gate"], st["lam"], st["u"]))
        if op == "fwd":
            y, h_last = gspn.seq_scan_fwd(x, gate, lam=lam, u=u, offsets=st["offsets"], h0=st["h0"], ch_per_weight=cpw)
            return [y.view(st["x"].shape), h_last]
        y, h_last = gspn.seq_scan(x, gate, lam=lam, u=u, offsets=st["offsets"], h0=st["h0"], ch_per_weight=cpw)
        outs, grads = [y.view(st["x"].shape)], [st["gy"]]
        if st["gh"] is not None:
            outs.append(h_last)
            grads.append(st["gh"])
        return [outs[0].detach(), h_last.detach()] + list(torch.autograd.grad(outs, st["leaves"], grads))
    with torch.no_grad():
        if op == "adapt":
            return _plain_adapt(st)
        if op == "step":
            return _plain_step(st)
        if op == "fwd":
            return list(_plain_forward(st)[:2])
        return _plain_train(st)


def work(case):
    s = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "adapt":
        rows, K, M, r = case["T"] - case["pad"], case["K"], case["M"], case["r"]
        used = min(case["N"], case["R"])
        return {"bytes": s * (rows * (K + 2 * M) + used * r * (K + M)) + 8 * case["N"] + 4 * used,
                "flops": 2 * rows * r * (K + M) + rows * M}
    D, extra = case["D"], int(case["lam"]) + int(case["u"])
    if case["op"] == "step":
        E = case["N"] * D
        return {"bytes": 8 * E + s * E * (2 + extra) + s * E // case["cpw"] + 4 * case["N"], "flops": 10 * E}
    E = (case["T"] - case["pad"]) * D
    ends = 4 * case["N"] * D
    forward = s * E * (2 + extra) + s * E // case["cpw"] + ends * (1 + int(case["h0"]))
    if case["op"] == "fwd":
        return {"bytes": forward, "flops": 10 * E}
    # the gradient of y is read, one gradient for each input written
    return {"bytes": forward + s * E * (2 + extra) + s * E // case["cpw"] + ends * 2 * int(case["h0"]), "flops": 40 * E}


# ------------------------------------------------------------------ in 64 bits
def _exact_sequence(st):
    """Token by token; the lists hold one row each."""
    c = st["case"]
    T, D, N, cpw = c["T"], c["D"], c["N"], c["cpw"]
    dev, off, train = st["x"].device, st["offsets_host"], c["op"] == "train"
    x = st["x"].detach().double()
    p = 1 / (1 + torch.exp(-st["gate"].detach().double()))
    q = 1 / (1 + torch.exp(st["gate"].detach().double()))
    p, q = (t[:, :, None].expand(T, D // cpw, cpw).reshape(T, D) for t in (p, q))
    lam = None if st["lam"] is None else st["lam"].detach().double()
    u = None if st["u"] is None else st["u"].detach().double()
    h0 = torch.zeros(N, D, device=dev).double() if st["h0"] is None else st["h0"].detach().double()
    term = q * x if lam is None else lam * x
    h = torch.zeros(T, D, dtype=torch.float64, device=dev)
    h_last, prev = h0.clone(), torch.zeros(T, D, dtype=torch.float64, device=dev)
    for n in range(N):
        state = h0[n]
        for t in range(off[n], off[n + 1]):
            prev[t] = state
            torch.addcmul(term[t], p[t], state, out=h[t])
            state = h[t]
        h_last[n] = state
    y = h if u is None else u * h
    if not train:
        return [y, h_last]
    gy = st["gy"].double()
    S = gy if u is None else u * gy
    S = S.clone()
    gh = torch.zeros(N, D, device=dev).double() if st["gh"] is None else st["gh"].double()
    G, gh0 = torch.zeros_like(S), torch.zeros_like(gh)
    for n in range(N):
        carry = gh[n]
        for t in range(off[n + 1] - 1, off[n] - 1, -1):
            torch.add(S[t], carry, out=G[t])
            carry = p[t] * G[t]
        gh0[n] = carry
    da = G * (prev - x) if lam is None else G * prev
    gate = (da * p * q).view(T, D // cpw, cpw).sum(2)
    out = [y, h_last, G * (q if lam is None else lam), gate]
    if lam is not None:
        out.append(G * x)
    if u is not None:
        out.append(gy * h)
    if st["h0"] is not None:
        out.append(gh0)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("fwd", "train"):
            return _exact_sequence(st)
        if case["op"] == "step":
            g = st["gate"].double()
            state, y = st["state"].double(), []
            p = (1 / (1 + torch.exp(-g))).repeat_interleave(case["cpw"], 1)
            q = (1 / (1 + torch.exp(g))).repeat_interleave(case["cpw"], 1)
            for i, slot in enumerate(st["slots"].tolist()):
                x = st["x"][i].double()
                state[slot] = p[i] * state[slot] + (q[i] if st["lam"] is None else st["lam"][i].double()) * x
                y.append(state[slot] * (1 if st["u"] is None else st["u"][i].double()))
            return [torch.stack(y), state]
        out = torch.zeros(case["T"], case["M"], dtype=torch.float64, device=st["x"].device)
        at = 0
        for n, count in enumerate(st["lens"]):
            rows, i = slice(at, at + count), st["ids_host"][n]
            out[rows] = st["base"][rows].double()
            if i >= 0:
                v = st["x"][rows].double() @ st["a"][i].double().t()
                out[rows] += st["scale"][i].double() * (v @ st["b"][i].double().t())
            at += count
        return out
