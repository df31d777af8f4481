"""The gated block and its gradients in 64 bits and by their definitions, with
the bounds of the errors that the comparisons use."""
from tests.linear_ref import BF16, F32, act_ref, slope_ref


def projection_ref(x, w, bias):
    """(z, bound of |z|'s error): K products and the additions of their sums, one
    binary32 step each, relative to the sum of magnitudes."""
    x, w = x.double(), w.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, (x.shape[1] + 8) * F32 * mag


def forward_ref(x, wg, wu, bg, bu, act):
    """{name: (value, bound of its error before any rounding to fewer bits)}.
    act(g): g's error through the slope (below 1.2), act's own operations (16
    steps relative to |g|); h: both factors' errors and one product."""
    g, eg = projection_ref(x, wg, bg)
    u, eu = projection_ref(x, wu, bu)
    a = act_ref(g, act)
    ea = 1.2 * eg + 16 * F32 * (g.abs() + a.abs())
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + F32 * h.abs()
    return {"g": (g, eg), "u": (u, eu), "h": (h, eh)}


def rounded(v, e):
    """The bound after one rounding to bf16."""
    return e + BF16 * (v.abs() + e)


def backward_ref(dh, wg, wu, x, g, u, act):
    """{name: (gradient, bound of its error)} from the values of the checkpoints
    x, g and u.

    dg, du: the slope's operations (24 steps relative to 1.2 + g^2, which bounds
    the terms of its formulas) and the value's (16 relative to |g|), the products
    around them, and one rounding to bf16.  The products: each addition a step
    relative to the sum of magnitudes, dg's and du's errors through the other
    operand, one rounding."""
    dh, T, N = dh.double(), dh.shape[0], dh.shape[1]
    a = act_ref(g, act)
    dg, du = dh * u * slope_ref(g, act), dh * a
    og = (dh * u).abs() * 24 * F32 * (1.2 + g.abs().clamp(max=16) ** 2) + 3 * F32 * dg.abs()
    ou = dh.abs() * 16 * F32 * (g.abs() + a.abs()) + F32 * du.abs()
    rg, ru = og + BF16 * (dg.abs() + og), ou + BF16 * (du.abs() + ou)
    out = {}
    wg, wu = wg.double(), wu.double()
    dx = dg @ wg + du @ wu
    through = rg @ wg.abs() + ru @ wu.abs()
    e = (2 * N + 8) * F32 * (dg.abs() @ wg.abs() + du.abs() @ wu.abs() + through) + through
    out["dx"] = dx, rounded(dx, e)
    for name, d, o, r in (("g", dg, og, rg), ("u", du, ou, ru)):
        dw = d.T @ x
        e = (T + 8) * F32 * ((d.abs() + r).T @ x.abs()) + r.T @ x.abs()
        out["dw" + name] = dw, rounded(dw, e)
        db = d.sum(0)
        e = (T + 8) * F32 * (d.abs() + o).sum(0) + o.sum(0)
        out["db" + name] = db, rounded(db, e)
    return out
