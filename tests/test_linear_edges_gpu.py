"""GPU tests of the layer products where their arithmetic is most easily lost:
activation functions far from zero, values at the ends of the checkpoint's
range.  Bounds and references as in tests/linear_ref.py."""
import math

import pytest
import torch

from shard_placement_amd.linear import Act8, Linear
from tests import linear_ref as ref
from tests.test_linear_gpu import BF, DEV, gen, kept_of, normal, test_forward as check_forward, within

pytestmark = pytest.mark.gpu

# What exp2's argument is off by: z^2 and its product with the constant, a binary32
# step together, which the exponential multiplies by z^2 / 2.
def _bell(z):
    return z * z * ref.F32


@pytest.mark.parametrize("lo,hi", [(-13.0, -8.0), (-8.0, -4.0), (-4.0, 0.0), (0.0, 6.0)])
def test_gelu_relative(lo, hi):
    """gelu is z Phi(z) to a bf16 rounding relative to itself, in its negative
    tail too: a fit within 6 binary32 steps, 10 operations, and the exponential's
    argument."""
    z = torch.linspace(lo, hi, 1500, dtype=torch.float64, device=DEV).to(BF)
    w = torch.zeros(z.numel(), 8, dtype=BF, device=DEV)
    x = torch.zeros(6, 8, dtype=BF, device=DEV)  # z = bias
    want = ref.act_ref(z.double(), "gelu").expand(6, -1)
    off = 16 * ref.F32 + _bell(z.double())
    within(Linear(w, bias=z, act="gelu").forward(x), want, want.abs() * (ref.BF16 * (1 + off) + off), "y")


def test_gelu_slope_relative():
    """The slope Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi), relative to its two terms."""
    grid = ref.e4m3_grid().to(DEV)
    z = torch.cat([-grid[(grid >= 2.0 ** -4) & (grid <= 13.0)], grid[(grid >= 2.0 ** -4) & (grid <= 13.0)]])
    z = torch.cat([z, z.new_zeros(-z.numel() % 32)])
    N = z.numel()
    z8, zv = kept_of(z.expand(5, N).contiguous())
    assert torch.equal(zv, z.expand(5, N))
    dy = normal(gen(4), 5, N)
    w = torch.eye(N, dtype=BF, device=DEV)  # dx = dz
    dx = Linear(w, act="gelu").backward(dy, z=z8)
    terms = torch.special.erfc(-z / math.sqrt(2)) / 2 + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = dy.double() * ref.slope_ref(z, "gelu")
    e = dy.double().abs() * terms * (24 * ref.F32 + _bell(z))
    within(dx, want, 2 * ref.BF16 * (want.abs() + e) + e, "dx")


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [3, 70])
def test_slope_of_a_value_that_reads_back_as_infinity(act, T):
    """The largest bf16 numbers round up to 2^128 in a checkpoint; their slope is
    1 or 0, and only a z that was not finite makes NaN."""
    N = 64
    z = torch.full((T, N), 0.5, dtype=BF, device=DEV)
    top = torch.finfo(BF).max
    z[1, 4], z[1, 40], z[2, 7], z[2, 8] = top, -top, math.inf, math.nan
    z8 = Act8(T, N, device=DEV).pack(z)
    back = z8.unpack()
    assert back[1, 4] == math.inf and back[1, 40] == -math.inf
    assert back[2, 7].isnan() and back[2, 8].isnan()
    dy = torch.full((T, N), 3.0, dtype=BF, device=DEV)
    db = torch.empty(N, dtype=BF, device=DEV)
    dx = Linear(torch.eye(N, dtype=BF, device=DEV), act=act, bias_grad=db).backward(dy, z=z8)
    # a NaN of dz reaches its token's whole row of dx, and its column's dbias
    assert dx[2].isnan().all() and db[7].isnan() and db[8].isnan()
    assert dx[1, 4] == 3.0 and dx[1, 40] == 0.0
    keep = torch.ones(T, N, dtype=torch.bool, device=DEV)
    keep[2] = False
    assert dx[keep].isfinite().all() and db[[4, 40]].isfinite().all()


# Two to four tokens on both sides of the rule that sends them by the weight's
# rows or through tiles: widths that are no multiples of 8, narrow and wide
# weights, short and long contractions, a weight of more than 192 MB.
@pytest.mark.parametrize("T,N,K", [(2, 33, 512), (2, 511, 2048), (2, 513, 2048), (2, 40, 1024), (2, 33, 1001),
                                   (3, 33, 1001), (3, 300, 4096), (4, 1030, 520), (4, 256, 28672),
                                   (4, 33, 20), (3, 12291, 8200), (4, 12291, 8200)])
@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("gelu", True, True)])
def test_forward_of_two_to_four_tokens(T, N, K, act, bias, res):
    g = gen(T + N + K)
    x, w = normal(g, T, K), normal(g, N, K, scale=2 / math.sqrt(K))
    b = normal(g, N) if bias else None
    r = normal(g, T, N) if res else None
    want, _, _, bound = ref.forward_ref(x, w, b, r, act)
    within(Linear(w, bias=b, act=act).forward(x, residual=r), want, bound, "y")
    if N < 2000:  # rows of x that start anywhere
        xs = torch.full((T, K + 3), math.nan, dtype=BF, device=DEV)[:, 1:K + 1]
        xs.copy_(x)
        within(Linear(w, bias=b, act=act).forward(xs, residual=r), want, bound, "y of strided x")


@pytest.mark.parametrize("rows,cols,depth", [(40, 22030, 1291), (20, 28673, 2048), (64, 22000, 1030)])
def test_narrow_tiles_by_two_sets_of_waves(rows, cols, depth):
    """Forward, dx and dW with few rows of outputs, whole, in two halves of a
    contraction whose steps are odd in number or end inside."""
    check_forward(rows, cols, depth, "silu", True, True, True)
    g = gen(rows)
    for T, N, K in ((rows, depth, cols), (depth, rows, cols)):
        w, dy = normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, T, N, scale=1e-3)
        x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
        want = ref.backward_ref(dy, w, x, None, "none")
        within(Linear(w).backward(dy), *want["dx"], "dx")
        layer = Linear(w, weight_grad=torch.full_like(w, 9))
        layer.backward(dy, x=x8, input_grad=False)
        within(layer.weight_grad, *want["dw"], "dw")
