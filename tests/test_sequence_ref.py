"""CPU: the 64-bit reference of the sequence operators is the definition: the closed form of the recurrence, and
gradients that central differences give."""
import pytest
import torch

import sequence_ref as ref
from sequence_cases import make

SHAPES = [dict(lens=[5, 0, 3], D=4, cpw=2), dict(lens=[7], D=3, lam=False), dict(lens=[1, 4], D=6, cpw=3, u=False, pad=2),
          dict(lens=[2, 3], D=2, lam=False, u=False, h0=False)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_closed_form(shape):
    """h_t = sum_s (prod of a between s and t) in_s + (prod of a) h0, term by term."""
    c = make(**shape)
    f = ref.forward(c["x"], c["gate"], c["lam"], c["u"], c["lens"], c["h0"], c["cpw"])
    t = 0
    for n, count in enumerate(c["lens"]):
        for i in range(count):
            for d in range(c["x"].shape[1]):
                a = torch.sigmoid(c["gate"][t:t + i + 1, d // c["cpw"]].double())
                take = 1 - a if c["lam"] is None else c["lam"][t:t + i + 1, d].double()
                h = a.prod() * (0 if c["h0"] is None else c["h0"][n, d].double())
                for s in range(i + 1):
                    h = h + a[s + 1:].prod() * take[s] * c["x"][t + s, d].double()
                y = h * (1 if c["u"] is None else c["u"][t + i, d].double())
                assert abs(float(y - f["y"][t + i, d])) < 1e-12
        t += count
    assert float(f["y"][t:].abs().sum()) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_are_differences(shape):
    c = make(**shape, spread=0.5)
    names = [k for k in ("x", "gate", "lam", "u", "h0") if c[k] is not None]
    v = {k: c[k].double() for k in names}

    def loss(**kw):
        z = {**{k: None for k in ("x", "gate", "lam", "u", "h0")}, **v, **kw}
        f = ref.forward(z["x"], z["gate"], z["lam"], z["u"], c["lens"], z["h0"], c["cpw"])
        return float((f["y"] * c["gy"].double()).sum() + (f["last"] * c["gh"].double()).sum())

    z = {**{k: None for k in ("x", "gate", "lam", "u", "h0")}, **v}
    got = ref.backward(z["x"], z["gate"], z["lam"], z["u"], c["lens"], z["h0"], c["cpw"], c["gy"].double(),
                       c["gh"].double())
    step = 1e-5
    for k in names:
        grad = got["g" + k][0]
        for i in range(v[k].numel()):
            hi, lo = v[k].clone(), v[k].clone()
            hi.view(-1)[i] += step
            lo.view(-1)[i] -= step
            # the third derivative's part of a central difference is below step^2 times a few units
            assert abs((loss(**{k: hi}) - loss(**{k: lo})) / (2 * step) - float(grad.reshape(-1)[i])) < 1e-8, (k, i)


def test_a_wrong_gradient_is_seen():
    """A planted mistake, the gate's gradient with h_t in place of h_{t-1}, leaves the bound by far."""
    c = make([9], 4, lam=True, u=False)
    g = ref.backward(c["x"], c["gate"], c["lam"], None, c["lens"], c["h0"], 1, c["gy"], c["gh"])
    f = ref.forward(c["x"], c["gate"], c["lam"], None, c["lens"], c["h0"], 1)
    wrong = g["ggate"][0] / f["before"] * f["h"]
    assert float(((wrong - g["ggate"][0]).abs() - g["ggate"][1]).max()) > 1e-3
