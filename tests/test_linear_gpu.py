"""GPU tests of the 8-bit checkpoint, the layer product with its epilogue and
its gradients, against tests/linear_ref.py (64 bits, element by element)."""
import math

import pytest
import torch

from shard_placement_amd import api, configs, harness
from shard_placement_amd._lib import TideError
from shard_placement_amd.linear import Act8, Linear
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
ACTS = list(api.ACTS)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def strided(t, ld, shift=0):
    """t's values in rows `ld` apart that start `shift` elements into a buffer
    of NaN: (view, buffer)."""
    rows, cols = t.shape
    buf = torch.full((rows * ld + shift + 8,), math.nan, dtype=BF, device=DEV)
    v = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v, buf


def kept_of(x, cols=None):
    """A checkpoint of the reference's bytes."""
    rows, cols = x.shape
    k = Act8(rows, cols, device=DEV)
    codes, scales = ref.pack_ref(x.double())
    k.data.view(torch.uint8).copy_(codes)
    k.scales.view(torch.uint8).copy_(scales)
    return k, ref.unpack_ref(codes, scales, cols)


def within(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError("%s at %s: got %r, want %r, bound %r (%d off)" % (
            what, i, got[i].item(), want[i].item(), bound[i].item(), int(bad.sum())))


# ---- the checkpoint ----------------------------------------------------------------------------

SIZES = [(1, 1), (1, 31), (2, 32), (3, 33), (1, 8192), (77, 1001), (5, 40), (1000, 64), (33, 5120),
         (4099, 96), (2, 28672)]


def spread(g, rows, cols):
    """Values over many powers of two, zeros, a whole zero block, and values
    that are not finite."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())
    x = x * torch.exp2(torch.randint(-6, 6, (rows, cols), generator=g, device=DEV).float())
    x[torch.rand(rows, cols, generator=g, device=DEV) < 0.05] = 0
    x[rows // 2, :32] = 0
    for v in (math.inf, -math.inf, math.nan):
        x[torch.rand(rows, cols, generator=g, device=DEV) < 0.002] = v
    return x.to(BF)


@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack_bits(rows, cols):
    x = spread(gen(rows * 31 + cols), rows, cols)
    k = Act8(rows, cols, device=DEV)
    k.buffer.fill_(0xAB)
    k.pack(x)
    codes, scales = ref.pack_ref(x.double())
    assert torch.equal(k.scales.view(torch.uint8), scales)
    got = k.data.view(torch.uint8)
    nan = (codes & 0x7f) == 0x7f
    assert torch.equal((got & 0x7f) == 0x7f, nan)
    assert torch.equal(got[~nan], codes[~nan])
    y = k.unpack()
    want = ref.unpack_ref(codes, scales, cols)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.double()[~want.isnan()], want[~want.isnan()])  # exact in bf16


@pytest.mark.parametrize("rows,cols,ld,shift", [(7, 64, 64, 1), (9, 40, 47, 0), (5, 33, 72, 3),
                                                (64, 256, 264, 8), (3, 1, 5, 1)])
def test_checkpoint_strides(rows, cols, ld, shift):
    g = gen(ld)
    x = spread(g, rows, cols)
    xs, _ = strided(x, ld, shift)
    a, b = Act8(rows, cols, device=DEV).pack(x), Act8(rows, cols, device=DEV).pack(xs)
    assert torch.equal(a.buffer, b.buffer)
    out, buf = strided(torch.zeros_like(x), ld, shift)
    before = buf.clone()
    a.unpack(out)
    assert torch.equal(out.view(torch.int16), a.unpack().view(torch.int16))
    out.zero_()  # nothing but the rows was written
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


def test_checkpoint_extremes():
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    x[0, 3], x[0, 40] = 3.3895e38, 9.2e-41            # the largest bf16; a subnormal
    x[1, :] = torch.tensor(float(2.0 ** -118), dtype=BF)
    x[2, 0], x[2, 1] = 448.0, 2.0 ** -10              # half of the smallest e4m3 value: to 0
    x[3, :32] = math.inf
    k = Act8(4, 64, device=DEV).pack(x)
    codes, scales = ref.pack_ref(x.double())
    assert torch.equal(k.scales.view(torch.uint8), scales)
    assert torch.equal(k.data.view(torch.uint8) & 0x7f, codes & 0x7f)
    assert k.unpack()[3, :32].isnan().all() and (k.unpack()[3, 32:] == 0).all()


def test_empty_calls():
    for rows, cols in ((0, 64), (5, 0), (0, 0)):
        k = Act8(rows, cols, device=DEV)
        x = torch.zeros(rows, cols, dtype=BF, device=DEV)
        assert k.pack(x).unpack().shape == (rows, cols)
    w = torch.zeros(8, 0, dtype=BF, device=DEV)
    b, r = normal(gen(1), 8), normal(gen(2), 3, 8)
    # no input feature: y = act(bias) + residual
    y = Linear(w, bias=b, act="silu").forward(torch.zeros(3, 0, dtype=BF, device=DEV), residual=r)
    want, _, _, bound = ref.forward_ref(torch.zeros(3, 0, device=DEV), w, b, r, "silu")
    within(y, want, bound)
    # no token: gradients are empty sums
    w = normal(gen(3), 8, 16)
    layer = Linear(w, bias=b, act="relu", weight_grad=torch.full_like(w, 7), bias_grad=torch.full_like(b, 7))
    none = torch.zeros(0, 8, dtype=BF, device=DEV)
    assert layer.forward(torch.zeros(0, 16, dtype=BF, device=DEV)).shape == (0, 8)
    dx = layer.backward(none, x=Act8(0, 16, device=DEV), z=Act8(0, 8, device=DEV))
    assert dx.shape == (0, 16) and (layer.weight_grad == 0).all() and (layer.bias_grad == 0).all()
    # no output feature: dx is an empty sum
    layer = Linear(torch.zeros(0, 16, dtype=BF, device=DEV))
    dx = torch.full((3, 16), 7.0, dtype=BF, device=DEV)
    layer.backward(torch.zeros(3, 0, dtype=BF, device=DEV), dx=dx)
    assert (dx == 0).all()


# ---- the product -------------------------------------------------------------------------------

# (T, N, K): one token to many, both sides of every tile's edge, odd widths,
# contractions that end inside a staged tile and ones that are split
PRODUCTS = [(1, 1, 1), (1, 8, 8), (1, 1000, 2048), (2, 33, 64), (3, 70, 65), (16, 256, 1024),
            (17, 300, 264), (32, 128, 4096), (33, 64, 72), (64, 513, 130), (65, 129, 128),
            (100, 130, 1544), (127, 255, 63), (128, 128, 64), (129, 257, 520), (300, 1001, 1000),
            (257, 31, 4100), (513, 520, 8), (2100, 4100, 136), (3500, 3500, 192)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("act,bias,res,keep", [("none", False, False, False),
                                               ("silu", True, True, True),
                                               ("gelu", True, False, True),
                                               ("gelu_tanh", False, True, False),
                                               ("relu", True, True, True)])
def test_forward(T, N, K, act, bias, res, keep):
    g = gen(T * 7 + N * 3 + K)
    x, w = normal(g, T, K), normal(g, N, K, scale=2 / math.sqrt(K))
    b = normal(g, N) if bias else None
    r = normal(g, T, N) if res else None
    z = Act8(T, N, device=DEV) if keep else None
    if keep:
        z.buffer.fill_(0xCD)
    y = Linear(w, bias=b, act=act).forward(x, residual=r, z=z)
    want, z64, zerr, bound = ref.forward_ref(x, w, b, r, act)
    within(y, want, bound, "y")
    if keep:
        # the values: half a step from a z that is off by zerr
        scales = z.scales.view(torch.uint8)
        got = ref.unpack_ref(z.data.view(torch.uint8), scales, N)
        step = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :N]
        off = torch.maximum(ref.E4M3 * (z64.abs() + zerr), ref.E4M3_SUB * step) + zerr
        within(got, z64, off, "z")
        # the scales: those of the largest |z| give or take zerr
        pad = torch.nn.functional.pad
        lo = pad((z64.abs() - zerr).clamp(min=0), (0, -N % 32))
        hi = pad(z64.abs() + zerr, (0, -N % 32))
        assert (scales >= ref.pack_ref(lo)[1]).all() and (scales <= ref.pack_ref(hi)[1]).all()
        assert (z.data.view(torch.uint8)[:, N:] == 0).all()


@pytest.mark.parametrize("T,N,K,lds,shifts", [
    (5, 40, 64, (64, 40, 40), (0, 0, 1)), (5, 40, 64, (72, 48, 56), (8, 8, 8)),
    (5, 40, 64, (67, 43, 41), (1, 3, 5)), (70, 264, 136, (136, 264, 264), (4, 0, 0)),
    (130, 261, 77, (80, 264, 300), (0, 1, 2)), (1, 64, 128, (500, 64, 64), (0, 0, 0))])
def test_forward_strides(T, N, K, lds, shifts):
    g = gen(T + N)
    x, w, r = normal(g, T, K), normal(g, N, K), normal(g, T, N)
    xs, _ = strided(x, lds[0], shifts[0])
    rs, _ = strided(r, lds[1], shifts[1])
    ys, buf = strided(torch.zeros(T, N, dtype=BF, device=DEV), lds[2], shifts[2])
    before = buf.clone()
    layer = Linear(w, act="silu")
    assert layer.forward(xs, residual=rs, out=ys) is ys
    want, _, _, bound = ref.forward_ref(x, w, None, r, "silu")
    within(ys, want, bound)
    ys.zero_()
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


def test_forward_of_unaligned_weight():
    """A placed tensor may start on any element."""
    g = gen(5)
    buf = normal(g, 64 * 72 + 8)
    x = normal(g, 20, 72)
    for shift in (1, 2, 4, 8):
        w = buf[shift:shift + 64 * 72].view(64, 72)
        want, _, _, bound = ref.forward_ref(x, w, None, None, "none")
        within(Linear(w).forward(x), want, bound, "shift %d" % shift)


@pytest.mark.parametrize("T,N,K", [(1, 64, 2048), (70, 300, 128), (3000, 4200, 64)])
def test_residual_in_place(T, N, K):
    g = gen(T)
    x, w, r = normal(g, T, K), normal(g, N, K), normal(g, T, N)
    want, _, _, bound = ref.forward_ref(x, w, None, r, "gelu")
    y = r.clone()
    Linear(w, act="gelu").forward(x, residual=y, out=y)
    within(y, want, bound)


def test_rows_of_nan_stay_alone():
    """NaN and infinities of one token or weight row reach their own outputs only."""
    g = gen(9)
    x, w = normal(g, 150, 200), normal(g, 300, 200)
    x[7, 3], x[149, 199], w[5, 0] = math.nan, math.inf, -math.inf
    y = Linear(w).forward(x)
    bad = torch.zeros(150, 300, dtype=torch.bool, device=DEV)
    bad[7], bad[149], bad[:, 5] = True, True, True
    assert torch.equal(~y.isfinite(), bad)
    dy = normal(g, 150, 300)
    dy[11, 2] = math.nan
    x8, z8 = Act8(150, 200, device=DEV).pack(x), Act8(150, 300, device=DEV)
    layer = Linear(w, act="silu", weight_grad=torch.empty_like(w))
    layer.forward(torch.nan_to_num(x, 0, 0, 0), z=z8)  # z is NaN in column 5 only
    dx = layer.backward(dy, x=x8, z=z8)
    dw = layer.weight_grad
    # every dz[t, 5] is NaN, so every dx is; dW: row 5, row 2 (dy), columns 3 and 199 (x)
    assert dx.isnan().all()
    bad = torch.zeros(300, 200, dtype=torch.bool, device=DEV)
    bad[5], bad[2], bad[:, 3], bad[:, 199] = True, True, True, True
    assert torch.equal(~dw.isfinite(), bad)


@pytest.mark.parametrize("T,N,K", [(1, 40, 64), (3, 70, 65), (24, 40, 2048), (150, 300, 200)])
def test_act_of_infinities(T, N, K):
    """relu of minus infinity is 0, so what masks a column out adds nothing; plus
    infinity stays, and the other activations of minus infinity are NaN."""
    g = gen(T + N)
    x, w, r = normal(g, T, K), normal(g, N, K), normal(g, T, N)
    b = torch.zeros(N, dtype=BF, device=DEV)
    b[3], b[N - 1], b[7], b[9] = -math.inf, -math.inf, math.inf, math.nan
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y = Linear(w, bias=b, act=act).forward(x, residual=r)
        for c in (3, N - 1):
            assert torch.equal(y[:, c], r[:, c]) if act == "relu" else y[:, c].isnan().all()
        assert (y[:, 7] == math.inf).all() and y[:, 9].isnan().all()
        assert y[:, [0, 1, 2, 4, 5, 6, 8]].isfinite().all()


# ---- the gradients -----------------------------------------------------------------------------

@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("act,bias", [("none", False), ("none", True), ("silu", True),
                                      ("gelu", False), ("gelu_tanh", True), ("relu", True)])
def test_backward(T, N, K, act, bias):
    g = gen(T * 5 + N + K * 3)
    w, dy = normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, T, N, scale=1e-3)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    z8, z = kept_of(3 * torch.randn(T, N, generator=g, device=DEV)) if act != "none" else (None, None)
    layer = Linear(w, bias=dy[0] if bias else None, act=act, weight_grad=torch.full_like(w, 9),
                   bias_grad=torch.full((N,), 9.0, dtype=BF, device=DEV) if bias else None)
    dx = layer.backward(dy, x=x8, z=z8)
    want = ref.backward_ref(dy, w, x, z, act)
    within(dx, *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    if bias:
        within(layer.bias_grad, *want["db"], "db")


@pytest.mark.parametrize("T,N,K,lds,shifts", [(33, 40, 64, (48, 72), (8, 0)), (33, 40, 64, (41, 67), (1, 3)),
                                              (130, 264, 72, (264, 72), (2, 1))])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_strides(T, N, K, lds, shifts, act):
    g = gen(T + K)
    w, dy = normal(g, N, K), normal(g, T, N)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    z8, z = kept_of(torch.randn(T, N, generator=g, device=DEV))
    ds, _ = strided(dy, lds[0], shifts[0])
    dx, buf = strided(torch.zeros(T, K, dtype=BF, device=DEV), lds[1], shifts[1])
    before = buf.clone()
    layer = Linear(w, act=act, weight_grad=torch.empty_like(w),
                   bias_grad=torch.empty(N, dtype=BF, device=DEV))
    assert layer.backward(ds, x=x8, z=z8, dx=dx) is dx
    want = ref.backward_ref(dy, w, x, z, act)
    within(dx, *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    within(layer.bias_grad, *want["db"], "db")
    dx.zero_()
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


def test_each_gradient_alone_and_what_it_needs():
    g = gen(77)
    T, N, K = 90, 136, 200
    w, dy = normal(g, N, K), normal(g, T, N)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    z8, z = kept_of(torch.randn(T, N, generator=g, device=DEV))
    want = ref.backward_ref(dy, w, x, z, "silu")
    dx, dw, db = torch.empty(T, K, dtype=BF, device=DEV), torch.empty_like(w), torch.empty(N, dtype=BF, device=DEV)
    api.tide_linear_backward(dy, K, weight=w, z_kept=z8.buffer, act="silu", dx=dx)
    api.tide_linear_backward(dy, K, x_kept=x8.buffer, z_kept=z8.buffer, act="silu", dweight=dw)
    api.tide_linear_backward(dy, K, z_kept=z8.buffer, act="silu", dbias=db)
    for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
        within(got, *want[name], name)
    assert Linear(w, act="silu").backward(dy, z=z8, input_grad=False) is None
    with pytest.raises(TideError, match="needs the checkpoint of x"):
        Linear(w, weight_grad=dw).backward(dy)
    with pytest.raises(TideError, match="needs the checkpoint of its argument"):
        Linear(w, act="silu").backward(dy)
    with pytest.raises(TideError, match="rows that share memory"):
        Linear(w).backward(dy[:1].expand(T, N))
    with pytest.raises(TideError, match="not contiguous"):
        Linear(w).backward(torch.empty(N, T, dtype=BF, device=DEV).t())


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """dx and dbias of loss = sum(dy * y) against central differences of the
    forward definition in 64 bits, at a z that the checkpoint holds exactly."""
    g = gen(13)
    T, N, K = 6, 8, 8
    w = torch.eye(8, dtype=BF, device=DEV)  # z = x + bias
    grid = ref.e4m3_grid().to(DEV)
    x = grid[torch.randint(40, 80, (T, K), generator=g, device=DEV)] / 8
    x = torch.where(torch.rand(T, K, generator=g, device=DEV) < 0.5, -x, x)
    dy = normal(g, T, N)
    x8, xv = kept_of(x)
    assert torch.equal(xv, x)
    bias = torch.zeros(N, dtype=BF, device=DEV)
    z8 = Act8(T, N, device=DEV)
    layer = Linear(w, bias=bias, act=act, weight_grad=torch.empty_like(w), bias_grad=torch.empty_like(bias))
    layer.forward(x.to(BF), z=z8)
    dx = layer.backward(dy, x=x8, z=z8)
    h = 2.0 ** -20
    slope = (ref.act_ref(x + h, act) - ref.act_ref(x - h, act)) / (2 * h)
    want = dy.double() * slope
    # two roundings (dz, dx), and the differences' own error
    within(dx, want, 2 * ref.BF16 * want.abs() + 1e-6, "dx")
    within(layer.bias_grad, want.sum(0), ref.BF16 * want.sum(0).abs() + 1e-5 * want.abs().sum(0) + 1e-6, "db")
    dw = want.T @ x
    within(layer.weight_grad, dw, ref.BF16 * (dw.abs() + 1.01 * (want.abs().T @ x.abs())) + 1e-5, "dw")


# ---- every tile, whole and split ---------------------------------------------------------------

# Shapes that between them take each form of the three products: 256 x 256, 256 x
# 192, 256 x 128, 128 x 128 tiles (by one and by two sets of waves) and the narrow
# ones, each with a whole and a split contraction, and dx and dW in one launch
# with each tile of dx, by one and by two sets of waves.
TILES = [(2500, 1550, 260), (1300, 1000, 4001), (5001, 1551, 24), (130, 8201, 2508), (8200, 1303, 25),
         (2500, 1032, 5000), (24, 1032, 5001), (1550, 260, 2500), (1300, 4000, 1000), (1550, 24, 5000),
         (8208, 2501, 130), (8200, 24, 1301), (2501, 5001, 1032), (260, 777, 5000), (4000, 1301, 1001),
         (24, 5003, 1551), (2500, 130, 8200), (24, 8203, 1303), (5000, 2500, 1032), (12, 1040, 200),
         (24, 1035, 24), (40, 1032, 25), (70, 1032, 25), (513, 518, 27), (40, 2051, 2508), (10, 24, 2000),
         (25, 24, 1040), (40, 24, 1040), (1032, 40, 24), (1035, 24, 24), (1030, 12, 40), (4, 40, 5000),
         (517, 2345, 3152), (5407, 153, 4043), (1343, 1450, 3975), (683, 5450, 3587), (273, 134, 6549),
         (7, 387, 6579), (6, 5489, 390), (18, 397, 6590), (18, 5617, 396), (33, 389, 6905),
         (33, 4375, 516), (2425, 130, 5401), (3907, 5428, 148), (4074, 1328, 1412), (3713, 645, 5490),
         (258, 2310, 3592), (5485, 3928, 166), (1342, 3934, 1414), (1210, 4191, 3203), (24, 300, 1000),
         (40, 520, 1001), (24, 1001, 300), (40, 777, 520), (700, 24, 300), (1000, 40, 520)]


@pytest.mark.parametrize("T,N,K", TILES)
def test_every_tile(T, N, K):
    test_forward(T, N, K, "silu", True, True, True)
    test_backward(T, N, K, "gelu_tanh", True)
    test_backward(T, N, K, "none", False)


# dx and dW in one launch of 256-wide tiles: every combination of 256 and 192
# columns, with the tiles of either product first.
PAIRS = [(657, 560, 5536), (771, 969, 6265), (869, 1038, 6478), (785, 660, 7642), (1014, 809, 6607),
         (1489, 528, 7182), (1163, 579, 7954), (1605, 1288, 2524)]


@pytest.mark.parametrize("T,N,K", PAIRS)
def test_both_gradients_in_one_launch(T, N, K):
    test_backward(T, N, K, "silu", True)
    test_backward(T, N, K, "none", False)


@pytest.mark.parametrize("T,N,K", TILES + PAIRS)
def test_each_gradient_alone(T, N, K):
    """dx without dW and dW without dx: each product's own form."""
    g = gen(T + 3 * N + K)
    w, dy = normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, T, N, scale=1e-3)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    want = ref.backward_ref(dy, w, x, None, "none")
    within(Linear(w).backward(dy), *want["dx"], "dx")
    layer = Linear(w, weight_grad=torch.full_like(w, 9))
    assert layer.backward(dy, x=x8, input_grad=False) is None
    within(layer.weight_grad, *want["dw"], "dw")


@pytest.mark.parametrize("T", [5, 12, 16, 30])
def test_forward_of_a_weight_past_the_cache(T):
    """Few tokens through a weight of more than 256 MB: deep tiles, split and,
    with an odd number of rows and a ragged contraction, to its last element."""
    test_forward(T, 16403, 8216, "gelu", True, True, T != 12)


# ---- streams, graphs, repeats, memory ----------------------------------------------------------

def step(layer, x, r, dy, x8, z8):
    x8.pack(x)
    y = layer.forward(x, residual=r, z=z8)
    dx = layer.backward(dy, x=x8, z=z8)
    return y, dx


def make(seed, T=70, N=300, K=200, act="gelu"):
    g = gen(seed)
    w = normal(g, N, K)
    layer = Linear(w, bias=normal(g, N), act=act, weight_grad=torch.empty_like(w),
                   bias_grad=torch.empty(N, dtype=BF, device=DEV))
    return layer, normal(g, T, K), normal(g, T, N), normal(g, T, N), Act8(T, K, device=DEV), Act8(T, N, device=DEV)


def bits(*ts):
    return [t.view(torch.int16 if t.dtype == BF else torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (70, 300, 200), (600, 520, 1000)])
def test_repeats_give_the_same_bits(T, N, K):
    args = make(3, T, N, K)
    layer, x8, z8 = args[0], args[4], args[5]
    first = bits(*step(*args), layer.weight_grad, layer.bias_grad, x8.buffer, z8.buffer)
    for _ in range(3):
        again = bits(*step(*args), layer.weight_grad, layer.bias_grad, x8.buffer, z8.buffer)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams_side_by_side():
    """Two layers' steps issued on two streams at once, by argument and by
    context, against each alone."""
    one, two = make(1, 300, 520, 333), make(2, 300, 520, 333)
    want = [bits(*step(*m), m[0].weight_grad, m[0].bias_grad) for m in (one, two)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        layer, x, r, dy, x8, z8 = one
        x8.pack(x, stream=s[0])
        y1 = layer.forward(x, residual=r, z=z8, stream=s[0])
        dx1 = layer.backward(dy, x=x8, z=z8, stream=s[0])
        with torch.cuda.stream(s[1]):
            y2, dx2 = step(*two)
    torch.cuda.synchronize()
    got = [bits(y1, dx1, one[0].weight_grad, one[0].bias_grad),
           bits(y2, dx2, two[0].weight_grad, two[0].bias_grad)]
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_host_threads():
    """Two threads' steps, each on its own stream with its own layer."""
    import threading

    ms = [make(11, 300, 520, 333), make(12, 40, 1032, 200, act="silu")]
    want = [bits(*step(*m), m[0].weight_grad, m[0].bias_grad, m[4].buffer) for m in ms]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    out = step(*ms[k])
                s.synchronize()
                got[k] = bits(*out, ms[k][0].weight_grad, ms[k][0].bias_grad, ms[k][4].buffer)
                s.synchronize()
        except Exception as e:  # shown by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and not any(t.is_alive() for t in threads)
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_steps():
    """Two captured steps replayed in turn and side by side, with other work
    and synchronisations between, each replay against the eager step on new
    inputs."""
    ms = [make(4, 70, 300, 200), make(5, 257, 136, 512, act="silu")]
    graphs, outs = [], []
    for m in ms:
        step(*m)
    torch.cuda.synchronize()
    for m in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*m))
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for k, m in enumerate(ms):
            for t in (m[1], m[2], m[3]):
                t.copy_(normal(gen(100 * rep + 10 * k + t.shape[1]), *t.shape))
        torch.cuda.synchronize()
        for k in (0, 1):
            with torch.cuda.stream(s[k] if rep % 2 else torch.cuda.current_stream()):
                graphs[k].replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device=DEV).sum()
        got = [bits(*outs[k], m[0].weight_grad, m[0].bias_grad, m[4].buffer, m[5].buffer)
               for k, m in enumerate(ms)]
        for k, m in enumerate(ms):
            want = bits(*step(*m), m[0].weight_grad, m[0].bias_grad, m[4].buffer, m[5].buffer)
            assert all(torch.equal(a, b) for a, b in zip(want, got[k])), (rep, k)
        assert junk.isfinite()


def test_checkpoints_in_caller_memory():
    """Checkpoints carved out of a vacated gathered buffer: nothing else of it
    is written, and no checkpoint memory is allocated."""
    layer, x, r, dy, x8, z8 = make(6)
    want = bits(*step(layer, x, r, dy, x8, z8), layer.weight_grad)
    vacated = torch.full((1 << 16,), -1, dtype=torch.int16, device=DEV).view(BF)
    n1, n2 = Act8.bytes(70, 200), Act8.bytes(70, 300)
    o1, o2 = 64, 64 + -(-n1 // 32) * 16 + 16
    k1 = Act8(70, 200, buffer=vacated[o1:])
    k2 = Act8(70, 300, buffer=vacated[o2 // 8 * 8:])
    got = bits(*step(layer, x, r, dy, k1, k2), layer.weight_grad)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    raw = vacated.view(torch.uint8)
    k1.buffer.fill_(255)
    k2.buffer.fill_(255)
    assert (raw == 255).all()
    with pytest.raises(TideError, match="aligned"):
        Act8(70, 200, buffer=vacated[1:]).pack(x)


# ---- a layer between the collectives -----------------------------------------------------------

def test_layer_step_between_placement_and_reduce_scatter():
    """Place two weights and a bias, run every simulated rank's tokens through
    the two products forward and backward with checkpoints, reduce-scatter the
    gradients: the shards against 64 bits."""
    R, T = 4, 45
    shapes = ((200, 136), (130, 200), (200,))
    w = configs.Workload(key=1, name="two products", R=R, names=("up", "down", "up.bias"),
                         shapes=shapes, sigma=0.05)
    st = harness.setup(w, device=DEV)
    st.plan.ag()
    up, down, bias = st.full[0], st.full[1], st.full[2]
    sums = [0, 0, 0]
    bounds = [0, 0, 0]
    for q in range(R):
        g = gen(50 + q)
        x, res, dy = normal(g, T, 136), normal(g, T, 130), normal(g, T, 130)
        l1 = Linear(up, bias=bias, act="silu", weight_grad=st.grads[q][0], bias_grad=st.grads[q][2])
        l2 = Linear(down, weight_grad=st.grads[q][1])
        x8, z8, h8 = Act8(T, 136, device=DEV), Act8(T, 200, device=DEV), Act8(T, 200, device=DEV)
        x8.pack(x)
        h = l1.forward(x, z=z8)
        h8.pack(h)
        y = l2.forward(h, residual=res)
        dh = l2.backward(dy, x=h8)
        l1.backward(dh, x=x8, z=z8, input_grad=False)
        # each product against 64 bits on what it was given
        want, _, _, b = ref.forward_ref(x, up, bias, None, "silu")
        within(h, want, b, "h")
        want, _, _, b = ref.forward_ref(h, down, None, res, "none")
        within(y, want, b, "y")
        val = lambda k, c: ref.unpack_ref(k.data.view(torch.uint8), k.scales.view(torch.uint8), c)  # noqa: E731
        g2 = ref.backward_ref(dy, down, val(h8, 200), None, "none")
        within(dh, *g2["dx"], "dh")
        g1 = ref.backward_ref(dh, up, val(x8, 136), val(z8, 200), "silu")
        for p, (want, b) in enumerate((g1["dw"], g2["dw"], g1["db"])):
            sums[p], bounds[p] = sums[p] + want, bounds[p] + b
    st.plan.rs()
    for p, shp in enumerate(shapes):
        s = -(-shp[0] // R)
        for r in range(R):
            n = max(0, min(shp[0], (r + 1) * s) - r * s)
            got = st.plan.shard(st.out[r], p)
            want, b = sums[p][r * s:r * s + n], bounds[p][r * s:r * s + n]
            within(got[:n], want, b + R * ref.F32 * (want.abs() + b), "shard %d of %s" % (r, shp))
            assert (got[n:] == 0).all()


# ---- far offsets -------------------------------------------------------------------------------

@pytest.mark.big
def test_offsets_past_32_bits():
    """A checkpoint and operands whose byte (and element) offsets pass 2^32."""
    T, K, N = 140000, 32768, 40
    g = gen(8)
    x = torch.empty(T, K, dtype=BF, device=DEV)
    for t in range(0, T, 20000):
        x[t:t + 20000] = torch.randn(min(20000, T - t), K, generator=g, device=DEV)
    k = Act8(T, K, device=DEV).pack(x)
    w = normal(g, N, K, scale=1 / math.sqrt(K))
    y = Linear(w, act="silu").forward(x)
    rows = torch.tensor([0, 1, 65535, 65536, 131071, 131072, 139998, 139999], device=DEV)
    codes, scales = ref.pack_ref(x[rows].double())
    assert torch.equal(k.data.view(torch.uint8)[rows], codes)
    assert torch.equal(k.scales.view(torch.uint8)[rows], scales)
    want, _, _, bound = ref.forward_ref(x[rows], w, None, None, "silu")
    within(y[rows], want, bound, "y")
    dy = torch.zeros(T, N, dtype=BF, device=DEV)
    dy[rows] = normal(g, len(rows), N)
    layer = Linear(w, weight_grad=torch.empty_like(w))
    dx = layer.backward(dy, x=k, dx=x)
    want = ref.backward_ref(dy[rows], w, ref.unpack_ref(codes, scales, K), None, "none")
    within(dx[rows], *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    assert (dx[70000:70010] == 0).all()
    out = k.unpack(x)
    assert torch.equal(out[rows].double(), ref.unpack_ref(codes, scales, K))


@pytest.mark.big
def test_most_tokens():
    """2^30 tokens of one feature, the most there may be: every product is
    exact (a weight of 2, one non-zero dy), so every element is compared."""
    T = 1 << 30
    x = torch.randint(-64, 65, (T, 1), generator=gen(3), device=DEV, dtype=torch.int8).to(BF)
    w = torch.full((1, 1), 2.0, dtype=BF, device=DEV)
    assert torch.equal(Linear(w).forward(x), x + x)
    last = x[T - 1].item()
    k = Act8(T, 1, device=DEV).pack(x)
    assert torch.equal(k.unpack(), x.clamp(-64, 64).to(torch.float8_e4m3fn).to(BF))
    kept = k.unpack()[T - 1].item()
    assert abs(kept - last) <= abs(last) / 16
    x.zero_()
    x[T - 1] = 3.0
    b = torch.zeros(1, dtype=BF, device=DEV)
    layer = Linear(w, bias=b, weight_grad=torch.empty_like(w), bias_grad=torch.empty_like(b))
    dx = layer.backward(x, x=k)
    assert torch.equal(dx, x + x)
    assert layer.bias_grad.item() == 3.0
    assert layer.weight_grad.item() == torch.tensor(3 * kept).to(BF).item()
