"""The 8-bit checkpoint and a layer's product and gradients, in 64 bits and by
their definitions: what the kernels are compared with.  Also the bounds that
the comparisons use."""
import math

import torch

BLOCK, E4M3_MAX, MIN_EXP = 32, 448.0, -110
# Roundings: half a step relative to the value (bf16 2^-8, e4m3 2^-4), and what
# an e4m3 subnormal is off by (half of 2^-9 steps of the scale).
BF16, E4M3, E4M3_SUB = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
# One binary32 operation; the matrix instruction's additions are allowed a
# whole step (2^-23) each, whatever their order.
F32 = 2.0 ** -23


def e4m3_grid():
    """The finite non-negative e4m3 values in order, by code."""
    vals = []
    for code in range(0x7f):
        ex, man = code >> 3, code & 7
        vals.append(man * 2.0 ** -9 if ex == 0 else (8 + man) * 2.0 ** (ex - 10))
    return torch.tensor(vals, dtype=torch.float64)


def pack_ref(x):
    """(codes uint8 [rows, pitch], scale bytes uint8 [rows, pitch / 32]) of a
    float64 matrix: the nearest e4m3 value, the even code in the middle."""
    rows, cols = x.shape
    pitch = -(-cols // BLOCK) * BLOCK
    v = torch.zeros(rows, pitch, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, pitch // BLOCK, BLOCK)
    finite = v.isfinite()
    amax = torch.where(finite, v.abs(), 0.0).amax(-1)
    e = torch.full_like(amax, MIN_EXP)
    for cand in range(MIN_EXP, 121):  # the smallest of which 448 * 2^e reaches amax
        e = torch.where(amax > E4M3_MAX * 2.0 ** cand, float(cand + 1), e)
    u = torch.where(finite, v, 0.0) / torch.exp2(e)[..., None]
    grid = e4m3_grid().to(x.device)
    hi = torch.searchsorted(grid, u.abs().contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = u.abs() - grid[lo], grid[hi] - u.abs()
    code = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    code = code + 128 * torch.signbit(v).long()
    code = torch.where(finite, code, 0x7f)
    return code.to(torch.uint8).view(rows, pitch), (e + 127).to(torch.uint8)


def unpack_ref(codes, scales, cols):
    """float64 values of a checkpoint's bytes."""
    grid = torch.cat([e4m3_grid(), torch.tensor([math.nan], dtype=torch.float64)]).to(codes.device)
    c = codes.long()
    v = grid[c & 0x7f] * (1 - 2 * (c >> 7)).double()
    s = torch.exp2(scales.double() - 127)
    rows, pitch = codes.shape
    return (v.view(rows, -1, BLOCK) * s[..., None]).view(rows, pitch)[:, :cols]


def act_ref(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope_ref(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "none":
        return torch.ones_like(z)
    c = math.sqrt(8 / math.pi)
    g, dg = (z, 1.0) if act == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2))
    s = torch.sigmoid(g)
    return s + z * s * torch.sigmoid(-g) * dg


def forward_ref(x, w, bias, res, act):
    """(y, z, bound of |z|'s error, bound of |y|'s error) in float64.

    z: K products and the additions of their sums, one binary32 step each,
    relative to the sum of magnitudes.  y: z's error through act (slopes lie
    below 1.2), act's own operations (16 steps relative to |z|, its value's
    bound), the residual's addition, one rounding to bf16."""
    x, w = x.double(), w.double()
    mag = x.abs() @ w.abs().T
    z = x @ w.T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    dz = (x.shape[1] + 8) * F32 * mag
    y = act_ref(z, act)
    r = 0.0 if res is None else res.double()
    y = y + r
    dy = 1.2 * dz + 16 * F32 * (z.abs() + y.abs() + (0.0 if res is None else r.abs()))
    return y, z, dz, dy + BF16 * (y.abs() + dy)


def backward_ref(dy, w, x, z, act):
    """{name: (gradient, bound of its error)} in float64 from the values of the
    checkpoints x and z (None for act none).

    dz: the slope's operations (24 steps relative to 1.2 + |z|, which bounds the
    terms of its formulas), and one rounding to bf16 for the products.  The
    products: each addition a step relative to the sum of magnitudes, dz's
    error through the other operand, one rounding."""
    dy, T, N = dy.double(), dy.shape[0], dy.shape[1]
    dz, off = dy, torch.zeros_like(dy)
    if act != "none":
        dz = dy * slope_ref(z, act)
        # z^3's terms in the tanh form matter only where the sigmoid is not 0 or 1 yet
        off = dy.abs() * 24 * F32 * (1.2 + z.abs().clamp(max=16) ** 2)
    rounded = off + (BF16 * (dz.abs() + off) if act != "none" else 0.0)
    out = {}
    w64 = w.double()
    dx, mag = dz @ w64, (dz.abs() + rounded) @ w64.abs()
    e = (N + 8) * F32 * mag + rounded @ w64.abs()
    out["dx"] = dx, e + BF16 * (dx.abs() + e)
    dw, mag = dz.T @ x, (dz.abs() + rounded).T @ x.abs()
    e = (T + 8) * F32 * mag + rounded.T @ x.abs()
    out["dw"] = dw, e + BF16 * (dw.abs() + e)
    db, mag = dz.sum(0), (dz.abs() + off).sum(0)
    e = (T + 8) * F32 * mag + off.sum(0)
    out["db"] = db, e + BF16 * (db.abs() + e)
    return out
