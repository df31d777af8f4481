"""GPU tests of the norms and their gradients against tests/norm_ref.py (64
bits, element by element)."""
import math

import pytest
import torch

from shard_placement_amd import api
from shard_placement_amd._lib import TideError
from shard_placement_amd.linear import Act8
from shard_placement_amd.norm import Norm
from tests import linear_ref as lref
from tests import norm_ref as ref
from tests.test_linear_gpu import BF, DEV, gen, kept_of, normal, strided, within

pytestmark = pytest.mark.gpu
EPS = 1e-5

# one column to the most, both sides of every form's edge and of a vector's; one
# row to several chunks of them
SIZES = [(1, 1), (3, 7), (5, 8), (2, 31), (19, 100), (40, 128), (17, 129), (70, 256), (9, 512),
         (11, 513), (33, 1001), (6, 1024), (5, 1025), (3, 2048), (4, 2049), (5, 4096), (7, 4097),
         (3, 5120), (2, 6144), (3, 6145), (1, 8192), (5, 8192), (4, 8193), (3, 12288), (2, 12289),
         (3, 16384), (2, 16385), (3, 24576), (2, 24577), (3, 28672), (2, 32767), (4, 32768),
         (5000, 72), (1300, 520), (600, 3000), (2100, 2048), (1100, 5121), (515, 28001)]


def rows_of(g, T, C):
    """Rows of unequal size and mean, some of zeros, one constant."""
    x = torch.randn(T, C, generator=g, device=DEV) + torch.randn(T, 1, generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-8, 8, (T, 1), generator=g, device=DEV).float())
    x[T // 2::7] = 0
    if T > 2:
        x[1] = 3.3
    return x.to(BF)


def kept_within(kept, want, err, what):
    """A checkpoint of values that are off by up to err: half a step of its
    own, and the scale of the largest magnitude give or take err."""
    scales = kept.scales.view(torch.uint8)
    cols = want.shape[1]
    got = lref.unpack_ref(kept.data.view(torch.uint8), scales, cols)
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :cols]
    within(got, want, torch.maximum(lref.E4M3 * (want.abs() + err), lref.E4M3_SUB * step) + err, what)
    lo, hi = (want.abs() - err).clamp(min=0), want.abs() + err
    assert (scales >= lref.pack_ref(lo)[1]).all() and (scales <= lref.pack_ref(hi)[1]).all()
    assert (kept.data.view(torch.uint8)[:, cols:] == 0).all()


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("kind,bias,keep", [("rms", False, True), ("layer", True, True),
                                            ("layer", False, False), ("rms", True, False)])
def test_forward(T, C, kind, bias, keep):
    g = gen(T * 7 + C)
    x, w = rows_of(g, T, C), normal(g, C)
    b = normal(g, C) if bias else None
    x8, y8 = Act8(T, C, device=DEV), Act8(T, C, device=DEV)
    for k in (x8, y8):
        k.buffer.fill_(0xCD)
    y = Norm(w, bias=b, kind=kind, eps=EPS).forward(x, **(dict(x8=x8, y8=y8) if keep else {}))
    want, err = ref.forward_ref(x, w, b, kind, EPS)
    within(y, want, ref.rounded(want, err), "y")
    if keep:
        assert torch.equal(x8.buffer, Act8(T, C, device=DEV).pack(x).buffer)
        kept_within(y8, want, err, "y8")
    else:
        assert (x8.buffer == 0xCD).all() and (y8.buffer == 0xCD).all()


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("kind,kept,add,bias", [("rms", True, True, False), ("layer", False, True, True),
                                                ("layer", True, False, True), ("rms", False, False, True),
                                                ("layer", False, False, False)])
def test_backward(T, C, kind, kept, add, bias):
    g = gen(T * 5 + C)
    x = rows_of(g, T, C)
    w, dy = normal(g, C), normal(g, T, C, scale=1e-2)
    a = normal(g, T, C) if add else None
    x8, x64 = kept_of(x) if kept else (x, x.double())
    layer = Norm(w, bias=w if bias else None, kind=kind, eps=EPS, weight_grad=torch.full_like(w, 9),
                 bias_grad=torch.full_like(w, 9) if bias else None)
    dx = layer.backward(dy, x8, add=a)
    want = ref.backward_ref(dy, w, x64, a, kind, EPS)
    within(dx, *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    if bias:
        within(layer.bias_grad, *want["db"], "db")


@pytest.mark.parametrize("T,C,lds,shifts", [(5, 40, (40, 40, 40), (1, 0, 3)), (9, 200, (208, 203, 264), (8, 1, 0)),
                                            (70, 1001, (1001, 1008, 1003), (0, 2, 5)),
                                            (3, 8192, (8200, 8193, 8192), (0, 0, 7))])
@pytest.mark.parametrize("kind", list(api.NORMS))
def test_strides(T, C, lds, shifts, kind):
    g = gen(T + C)
    x, w, dy, add = rows_of(g, T, C), normal(g, C), normal(g, T, C), normal(g, T, C)
    xs, _ = strided(x, lds[0], shifts[0])
    ds, _ = strided(dy, lds[1], shifts[1])
    adds, _ = strided(add, lds[0], shifts[1])
    out, buf = strided(torch.zeros(T, C, dtype=BF, device=DEV), lds[2], shifts[2])
    before = buf.clone()
    layer = Norm(w, kind=kind, eps=EPS, weight_grad=torch.empty_like(w))
    assert layer.forward(xs, out=out) is out
    want, err = ref.forward_ref(x, w, None, kind, EPS)
    within(out, want, ref.rounded(want, err), "y")
    assert layer.backward(ds, xs, add=adds, dx=out) is out
    want = ref.backward_ref(dy, w, x, add, kind, EPS)
    within(out, *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    out.zero_()  # nothing but the rows was written
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


def test_weights_on_any_element():
    g = gen(12)
    buf, gbuf = normal(g, 300), torch.full((300,), 7.0, dtype=BF, device=DEV)
    x, dy = rows_of(g, 6, 201), normal(g, 6, 201)
    for shift in (1, 2, 5, 8):
        w, dw = buf[shift:shift + 201], gbuf[shift:shift + 201]
        layer = Norm(w, bias=w, kind="layer", eps=EPS, weight_grad=dw)
        want, err = ref.forward_ref(x, w, w, "layer", EPS)
        within(layer.forward(x), want, ref.rounded(want, err), "shift %d" % shift)
        layer.backward(dy, x)
        within(dw, *ref.backward_ref(dy, w, x, None, "layer", EPS)["dw"], "shift %d" % shift)
        dw.fill_(7.0)
        assert (gbuf == 7.0).all()


@pytest.mark.parametrize("T,C", [(1, 8192), (33, 128), (70, 1001), (900, 2048)])
def test_gradient_onto_add_in_place(T, C):
    g = gen(T)
    x, w, dy, add = rows_of(g, T, C), normal(g, C), normal(g, T, C), normal(g, T, C)
    want = ref.backward_ref(dy, w, x, add, "rms", EPS)["dx"]
    assert Norm(w, eps=EPS).backward(dy, x, add=add, dx=add) is add
    within(add, *want)


def test_each_gradient_alone():
    g = gen(21)
    T, C = 700, 264
    x, w, dy = rows_of(g, T, C), normal(g, C), normal(g, T, C)
    x8, x64 = kept_of(x)
    for kind in api.NORMS:
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        opt = dict(kind=kind, eps=EPS)
        api.tide_norm_backward(dy, x=x, weight=w, dx=dx, **opt)
        api.tide_norm_backward(dy, x=x, dweight=dw, **opt)
        api.tide_norm_backward(dy, dbias=db, **opt)  # needs no x
        want = ref.backward_ref(dy, w, x, None, kind, EPS)
        for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
            within(got, *want[name], name)
        want = ref.backward_ref(dy, w, x64, None, kind, EPS)
        api.tide_norm_backward(dy, x_kept=x8.buffer, weight=w, dx=dx, dbias=db, **opt)
        api.tide_norm_backward(dy, x_kept=x8.buffer, dweight=dw, **opt)
        for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
            within(got, *want[name], name)
    assert Norm(w, weight_grad=dw).backward(dy, x, input_grad=False) is None


def test_flat_forward_is_the_class_one():
    g = gen(22)
    x, w, b = rows_of(g, 30, 72), normal(g, 72), normal(g, 72)
    x8, y8 = Act8(30, 72, device=DEV), Act8(30, 72, device=DEV)
    y = api.tide_norm_forward(x, w, bias=b, kind="layer", eps=EPS, x_kept=x8.buffer, y_kept=y8.buffer)
    k8 = Act8(30, 72, device=DEV)
    want = Norm(w, bias=b, kind="layer", eps=EPS).forward(x, y8=k8)
    assert torch.equal(y, want) and torch.equal(k8.buffer, y8.buffer)


def test_empty_calls():
    w = normal(gen(1), 8)
    none = torch.zeros(0, 8, dtype=BF, device=DEV)
    layer = Norm(w, bias=w, weight_grad=torch.full_like(w, 7), bias_grad=torch.full_like(w, 7))
    assert layer.forward(none).shape == (0, 8)
    assert layer.backward(none, none).shape == (0, 8)
    assert (layer.weight_grad == 0).all() and (layer.bias_grad == 0).all()
    for C in (200, 2000, 30000):
        v = torch.full((C,), 7.0, dtype=BF, device=DEV)
        Norm(v, kind="layer", weight_grad=v).backward(torch.zeros(0, C, dtype=BF, device=DEV),
                                                      Act8(0, C, device=DEV), input_grad=False)
        assert (v == 0).all()
    flat = Norm(torch.zeros(0, dtype=BF, device=DEV))
    assert flat.forward(torch.zeros(3, 0, dtype=BF, device=DEV)).shape == (3, 0)


def test_a_constant_row_is_its_bias():
    """What binary32 leaves of a large mean does not show next to eps."""
    for C in (96, 1001, 5120, 28672):
        x = torch.full((4, C), 1000.0, dtype=BF, device=DEV)
        x[1], x[2] = -3.3, 3e-3
        w, b = torch.ones(C, dtype=BF, device=DEV), normal(gen(C), C)
        y = Norm(w, bias=b, kind="layer", eps=EPS).forward(x)
        # the differences are off by SUM of the mean at first, by a step of that
        # after it is corrected: times sqrt(1 / eps) below 4e-5
        err = (y.double() - b.double()).abs()
        assert (err <= lref.BF16 * b.double().abs() + 4e-5).all(), (C, err.max())


def test_rows_that_are_not_finite_stay_alone():
    g = gen(9)
    x, w = rows_of(g, 40, 200), torch.ones(200, dtype=BF, device=DEV)
    x[3, 5], x[11, 0], x[12, 199] = math.nan, math.inf, -math.inf
    bad = torch.zeros(40, 200, dtype=torch.bool, device=DEV)
    bad[3], bad[11], bad[12] = True, True, True
    y = Norm(w, kind="layer").forward(x)
    assert torch.equal(y.isnan(), bad)
    y = Norm(w).forward(x)
    bad[11, 1:], bad[12, :199] = False, False
    assert torch.equal(y.isnan(), bad) and (y[11, 1:] == 0).all()
    # the gradient of a bad row is bad, of the others it is not
    dx = Norm(w, kind="layer").backward(normal(g, 40, 200), x)
    bad[11], bad[12] = True, True
    assert torch.equal(dx.isnan(), bad)
    # a sum of squares past binary32: the row is divided by infinity
    x = torch.ones(2, 64, dtype=BF, device=DEV)
    x[1, 3] = 1e30
    y = Norm(w[:64], eps=EPS).forward(x)
    assert (y[0] == 1).all() and (y[1] == 0).all()


@pytest.mark.parametrize("kind", list(api.NORMS))
def test_gradients_against_differences(kind):
    """The sum of y dy along each gradient's own direction, by central differences
    of the kernel's y.  y is rounded to bf16, so the step is large: what the
    difference keeps of the third order is allowed for, and y's roundings."""
    g = gen(31)
    T, C, h = 64, 520, 2.0 ** -4
    x, w, b = normal(g, T, C), normal(g, C), normal(g, C)
    dy = normal(g, T, C)
    layer = Norm(w, bias=b, kind=kind, eps=EPS, weight_grad=torch.empty_like(w), bias_grad=torch.empty_like(b))
    dx = layer.backward(dy, x)

    def loss(x, w, b):
        y = Norm(w, bias=b, kind=kind, eps=EPS).forward(x).double()
        # each y is off by half a step; independent roundings add in squares
        return (y * dy.double()).sum(), ((y * dy.double()) ** 2).sum().sqrt() * lref.BF16

    for name, at, grad in (("dx", x, dx), ("dw", w, layer.weight_grad), ("db", b, layer.bias_grad)):
        v = grad.sign() * h * at.abs().clamp(min=0.25)  # uphill
        parts = [x, w, b]
        k = ("dx", "dw", "db").index(name)
        ends = []
        for sign in (1, -1):
            parts[k] = (at.double() + sign * v.double()).to(BF)
            ends.append((parts[k].double(),) + loss(*parts))
        along = (ends[0][0] - ends[1][0])
        want = (grad.double() * along).sum()
        diff = ends[0][1] - ends[1][1]
        # third order: h^2 of the change; roundings: 6 standard deviations
        assert abs(diff - want) < 4 * h * h * abs(want) + 6 * (ends[0][2] + ends[1][2]), (name, diff, want)


# ---- streams, graphs, repeats ------------------------------------------------------------------

def make(seed, T, C, kind="layer"):
    g = gen(seed)
    w, b = normal(g, C), normal(g, C)
    layer = Norm(w, bias=b, kind=kind, eps=EPS, weight_grad=torch.empty_like(w), bias_grad=torch.empty_like(b))
    return layer, rows_of(g, T, C), normal(g, T, C), Act8(T, C, device=DEV), Act8(T, C, device=DEV)


def step(layer, x, dy, x8, y8):
    y = layer.forward(x, x8=x8, y8=y8)
    return y, layer.backward(dy, x8, add=y)


def bits(m, out):
    return [t.clone().view(torch.uint8) for t in (*out, m[0].weight_grad, m[0].bias_grad, m[3].buffer,
                                                  m[4].buffer)]


@pytest.mark.parametrize("T,C", [(1, 8192), (700, 128), (1200, 1001), (1030, 5120)])
def test_repeats_give_the_same_bits(T, C):
    m = make(T, T, C)
    want = bits(m, step(*m))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, bits(m, step(*m))))


def test_streams_side_by_side():
    ms = [make(1, 1300, 520), make(2, 600, 4097, "rms")]
    want = [bits(m, step(*m)) for m in ms]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for k, m in enumerate(ms):
            with torch.cuda.stream(s[k]):
                out = step(*m)
            outs = outs[-3:] + [out]
    torch.cuda.synchronize()
    for k, m in enumerate(ms):
        assert all(torch.equal(a, b) for a, b in zip(want[k], bits(m, outs[-2 + k])))
    # by the stream argument
    layer, x, dy, x8, y8 = ms[0]
    y = layer.forward(x, stream=s[0])
    dx = layer.backward(dy, x, add=y, stream=s[0])
    s[0].synchronize()
    assert torch.equal(y, layer.forward(x)) and torch.equal(dx, layer.backward(dy, x, add=y))


def test_captured_steps():
    """Two captured steps replayed in turn and side by side, each replay against
    the eager step on new inputs."""
    ms = [make(4, 1100, 264), make(5, 257, 1001, "rms")]
    for m in ms:
        step(*m)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*m))
        graphs.append(g)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for k, m in enumerate(ms):
            m[1].copy_(rows_of(gen(100 * rep + k), *m[1].shape))
            m[2].copy_(normal(gen(200 * rep + k), *m[2].shape))
        torch.cuda.synchronize()
        for k in (0, 1):
            with torch.cuda.stream(s[k] if rep % 2 else torch.cuda.current_stream()):
                graphs[k].replay()
        torch.cuda.synchronize()
        got = [bits(m, outs[k]) for k, m in enumerate(ms)]
        for k, m in enumerate(ms):
            assert all(torch.equal(a, b) for a, b in zip(bits(m, step(*m)), got[k])), (rep, k)


def test_checkpoints_in_caller_memory():
    layer, x, dy, x8, y8 = make(6, 70, 200, "rms")
    want = bits((layer, x, dy, x8, y8), step(layer, x, dy, x8, y8))
    vacated = torch.full((1 << 15,), -1, dtype=torch.int16, device=DEV).view(BF)
    n = -(-Act8.bytes(70, 200) // 32) * 16
    k1, k2 = Act8(70, 200, buffer=vacated[64:]), Act8(70, 200, buffer=vacated[64 + n + 16:])
    got = bits((layer, x, dy, k1, k2), step(layer, x, dy, k1, k2))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    k1.buffer.fill_(255)
    k2.buffer.fill_(255)
    assert (vacated.view(torch.uint8) == 255).all()


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31, and bytes past 2^32."""
    T, C, ld = 520, 64, (1 << 22)
    big = torch.empty(T * ld, dtype=BF, device=DEV)  # 4.4 GB
    x = big.view(T, ld)[:, 100:100 + C]
    x.copy_(rows_of(gen(3), T, C))
    w = normal(gen(4), C)
    y = big.view(T, ld)[:, 1000:1000 + C]
    layer = Norm(w, kind="layer", eps=EPS, weight_grad=torch.empty_like(w))
    layer.forward(x, out=y)
    want, err = ref.forward_ref(x, w, None, "layer", EPS)
    within(y, want, ref.rounded(want, err))
    dx = big.view(T, ld)[:, 2000:2000 + C]
    layer.backward(y, x, add=y, dx=dx)
    want = ref.backward_ref(y, w, x, y, "layer", EPS)
    within(dx, *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")


def test_refusals_on_the_gpu():
    w = normal(gen(1), 64)
    x = normal(gen(2), 4, 64)
    with pytest.raises(TideError, match="TIDE_EOVERLAP"):
        Norm(w).forward(x, out=x)
    with pytest.raises(TideError, match="TIDE_EINVAL"):
        Norm(w, eps=0.0).forward(x)
    wide = torch.zeros(32769, dtype=BF, device=DEV)
    with pytest.raises(TideError, match="TIDE_EUNSUPPORTED"):
        Norm(wide).forward(wide.view(1, -1).clone())
    with pytest.raises(TideError, match="rows that share memory"):
        Norm(w).backward(x[:1].expand(4, 64), x)


@pytest.mark.big
@pytest.mark.parametrize("T,C", [(1 << 27, 2), (299593, 28672)])
def test_most_rows(T, C):
    """The most rows there may be, and the most elements: rows everywhere against
    the reference, the weight's gradient from a few rows that are not zero."""
    g = gen(17)
    w = normal(g, C)
    x = torch.zeros(T, C, dtype=BF, device=DEV)
    rows = torch.tensor([0, 1, T // 3, T // 2 + 1, T - 2, T - 1], device=DEV)
    x[rows] = normal(g, len(rows), C)
    layer = Norm(w, kind="layer", eps=EPS, weight_grad=torch.empty_like(w))
    x8 = Act8(T, C, device=DEV)
    y = layer.forward(x, x8=x8)
    want, err = ref.forward_ref(x[rows], w, None, "layer", EPS)
    within(y[rows], want, ref.rounded(want, err), "y")
    assert (y[T // 4:T // 4 + 9] == 0).all()
    val = lref.unpack_ref(x8.data.view(torch.uint8)[rows], x8.scales.view(torch.uint8)[rows], C)
    y.zero_()
    dy = y
    dy[rows] = normal(g, len(rows), C)
    dx = layer.backward(dy, x8, dx=x)
    want = ref.backward_ref(dy[rows], w, val, None, "layer", EPS)
    within(dx[rows], *want["dx"], "dx")
    within(layer.weight_grad, *want["dw"], "dw")
    assert (dx[T // 4:T // 4 + 9] == 0).all()
