"""The norms and their gradients in 64 bits and by their definitions, with the
bounds of the errors that the comparisons use."""
import torch

from tests.linear_ref import BF16, F32

# A row's sum: a lane adds at most 40 terms one after the other and the lanes'
# sums meet in 10 steps; each addition is half a step (F32 / 2) off.
SUM = 25 * F32


def stats_ref(x, kind, eps):
    """(x - mu, r, bound of x - mu's error, bound of r's relative error) of a
    float64 matrix.

    layer: mu is off by SUM of the mean magnitude at first (em).  The rest of it
    is the mean of the differences (each rounded once), which is off by SUM of
    their mean magnitude, and taking it off rounds once more.  v is off by SUM
    and a product's rounding relative to the sum it comes from, its square root
    by half of that, and one step for the reciprocal root, three for the
    products around it."""
    c = x.shape[1]
    if kind == "layer":
        mu = x.sum(1, keepdim=True) / c
        em = SUM * x.abs().mean(1, keepdim=True)
        d = x - mu
        ed = 2 * F32 * (d.abs() + em) + (SUM + F32) * (d.abs().mean(1, keepdim=True) + em)
    else:
        d, em, ed = x, 0.0, torch.zeros_like(x)
    v = (d * d).sum(1, keepdim=True) / c
    r = (v + eps) ** -0.5
    er = (SUM + 2 * F32) * (v + em * em) / (v + eps) + 4 * F32
    return d, r, ed, er


def forward_ref(x, w, bias, kind, eps):
    """(y, bound of the error before the rounding to bf16) in float64."""
    w = w.double()
    d, r, ed, er = stats_ref(x.double(), kind, eps)
    y = d * r * w
    e = w.abs() * r * ed * (1 + er) + y.abs() * (er + 3 * F32)
    if bias is not None:
        y = y + bias.double()
        e = e + F32 * y.abs()
    return y, e


def rounded(y, e):
    """The bound after one rounding to bf16."""
    return e + BF16 * (y.abs() + e)


def backward_ref(dy, w, x, add, kind, eps):
    """{name: (gradient, bound of its error)} in float64.

    The two means: their sums' error, and that of n in the second.  dx: those
    through the formula, a handful of roundings of its terms, r's error, the
    addition, one rounding.  dw and db: each addition a step relative to the sum
    of magnitudes, n's error, one rounding."""
    T = dy.shape[0]
    dy, w = dy.double(), w.double()
    d, r, ed, er = stats_ref(x.double(), kind, eps)
    n, en = d * r, r * ed * (1 + er) + (d * r).abs() * (er + F32)
    c = dy * w
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    m2 = mean(c * n)
    e2 = (SUM + 4 * F32) * mean((c * n).abs()) + mean(c.abs() * en) + 2 * er * m2.abs()
    m1 = mean(c) if kind == "layer" else torch.zeros_like(m2)
    e1 = (SUM + 2 * F32) * mean(c.abs()) if kind == "layer" else torch.zeros_like(m2)
    dx = r * (c - m1 - n * m2)
    e = r * (4 * F32 * (c.abs() + m1.abs() + (n * m2).abs()) + e1 + n.abs() * e2 + m2.abs() * en
             + en * e2) * (1 + er) + dx.abs() * er
    if add is not None:
        dx = dx + add.double()
        e = e + F32 * dx.abs()
    out = {"dx": (dx, rounded(dx, e))}
    dw = (dy * n).sum(0)
    e = (T + 8) * F32 * (dy * n).abs().sum(0) + (dy.abs() * en).sum(0)
    out["dw"] = dw, rounded(dw, e)
    db = dy.sum(0)
    e = (T + 8) * F32 * dy.abs().sum(0)
    out["db"] = db, rounded(db, e)
    return out
