"""GPU tests of the gated block and its gradients against tests/gated_ref.py (64
bits, element by element), and of a feed-forward half of a layer between the
collectives."""
import math
import threading

import pytest
import torch

from shard_placement_amd import api, configs, harness
from shard_placement_amd._lib import TideError
from shard_placement_amd.gated import Gated
from shard_placement_amd.linear import Act8, Linear
from shard_placement_amd.norm import Norm
from tests import gated_ref as ref
from tests import linear_ref as lref
from tests import norm_ref as nref
from tests.test_linear_gpu import BF, DEV, gen, kept_of, normal, strided, within

pytestmark = pytest.mark.gpu
ACTS = list(api.ACTS)

# (T, N, K): one token to many, both sides of every tile's edge, odd widths,
# contractions that end inside a staged tile and ones that are split
PRODUCTS = [(1, 1, 1), (1, 8, 8), (1, 1000, 2048), (2, 33, 64), (3, 70, 65), (4, 2300, 28000), (16, 256, 1024),
            (17, 300, 264), (32, 128, 4096), (33, 64, 72), (64, 513, 130), (65, 129, 128), (100, 130, 1544),
            (127, 255, 63), (128, 128, 64), (129, 257, 520), (300, 1001, 1000), (257, 31, 4100), (513, 520, 8),
            (2100, 2100, 136), (1800, 1700, 192)]
# what else the rules choose; tests/test_gated_cpu.py checks that none is left out
FORMS = [(140, 8848, 2710), (3835, 1644, 1206), (5255, 529, 4096), (35, 258, 6175), (4796, 9572, 170), (393, 1615,
         16293), (2, 525, 11), (424, 332, 25508), (219, 2295, 8229), (107, 2928, 25934), (4538, 3586, 630), (18, 554,
         1), (1, 1, 16817), (19, 13163, 1), (19, 1, 19162), (33, 14137, 1), (66, 1, 18556), (75, 16985, 1), (1, 3257,
         20759), (131, 332, 19254), (18, 3008, 23383), (132, 2405, 4717), (34, 2554, 26228), (795, 465, 6769), (1051,
         1691, 1951), (2201, 6197, 283), (65, 27843, 2500), (65, 9598, 7303), (1434, 543, 5859), (75, 11598, 5865),
         (2211, 4989, 538)]
# few tokens through weights of more than 256 MB together: a ring past the caches, and
# 512 bytes of a row at a time where there are more tiles than compute units
PAST_THE_CACHE = [(5, 8203, 8216), (30, 8203, 8209), (12, 8203, 8216), (64, 8200, 8200), (100, 8200, 8200),
                  (12, 16403, 4104), (30, 16403, 4104)]


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


def check_forward(T, N, K, act, bias, keep):
    g = gen(T * 7 + N * 3 + K)
    x = normal(g, T, K)
    wg, wu = (normal(g, N, K, scale=2 / math.sqrt(K)) for _ in range(2))
    bg, bu = (normal(g, N) if bias else None for _ in range(2))
    kept = {n: Act8(T, N, device=DEV) for n in keep}
    for k in kept.values():
        k.buffer.fill_(0xCD)
    h = Gated(wg, wu, gate_bias=bg, up_bias=bu, act=act).forward(x, **kept)
    want = ref.forward_ref(x, wg, wu, bg, bu, act)
    within(h, want["h"][0], ref.rounded(*want["h"]), "h")
    for n, k in kept.items():
        kept_within(k, *want[n], n)


def backward_case(T, N, K, seed):
    g = gen(seed)
    wg, wu = (normal(g, N, K, scale=1 / math.sqrt(K)) for _ in range(2))
    dh = normal(g, T, N, scale=1e-3)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    g8, gv = kept_of(3 * torch.randn(T, N, generator=g, device=DEV))
    u8, uv = kept_of(torch.randn(T, N, generator=g, device=DEV))
    return wg, wu, dh, (x8, g8, u8), (x, gv, uv)


def check_backward(T, N, K, act, bias):
    wg, wu, dh, (x8, g8, u8), values = backward_case(T, N, K, T * 5 + N + K * 3)
    nine = lambda *s: torch.full(s, 9.0, dtype=BF, device=DEV)  # noqa: E731
    block = Gated(wg, wu, act=act, gate_grad=nine(N, K), up_grad=nine(N, K),
                  gate_bias_grad=nine(N) if bias else None, up_bias_grad=nine(N) if bias else None)
    dx = block.backward(dh, x=x8, g=g8, u=u8)
    want = ref.backward_ref(dh, wg, wu, *values, act)
    within(dx, *want["dx"], "dx")
    within(block.gate_grad, *want["dwg"], "dwg")
    within(block.up_grad, *want["dwu"], "dwu")
    if bias:
        within(block.gate_bias_grad, *want["dbg"], "dbg")
        within(block.up_bias_grad, *want["dbu"], "dbu")


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("act,bias,keep", [("none", False, ""), ("silu", True, "guh"), ("gelu", False, "gu"),
                                           ("gelu_tanh", True, ""), ("relu", False, "h")])
def test_forward(T, N, K, act, bias, keep):
    check_forward(T, N, K, act, bias, keep)


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("act,bias", [("none", True), ("silu", True), ("gelu", False), ("gelu_tanh", True),
                                      ("relu", False)])
def test_backward(T, N, K, act, bias):
    check_backward(T, N, K, act, bias)


@pytest.mark.parametrize("T,N,K", FORMS)
def test_every_form(T, N, K):
    check_forward(T, N, K, "silu", True, "guh")
    check_forward(T, N, K, "gelu", False, "")
    check_backward(T, N, K, "silu", True)


@pytest.mark.parametrize("T,N,K", PRODUCTS[::2] + FORMS)
def test_each_gradient_alone(T, N, K):
    wg, wu, dh, (x8, g8, u8), values = backward_case(T, N, K, T + 3 * N + K)
    want = ref.backward_ref(dh, wg, wu, *values, "silu")
    within(Gated(wg, wu).backward(dh, g=g8, u=u8), *want["dx"], "dx")
    block = Gated(wg, wu, gate_grad=torch.full_like(wg, 9), up_grad=torch.full_like(wg, 9))
    assert block.backward(dh, x=x8, g=g8, u=u8, input_grad=False) is None
    within(block.gate_grad, *want["dwg"], "dwg")
    within(block.up_grad, *want["dwu"], "dwu")
    for name in ("g", "u"):  # one bias without the other
        db = torch.full((N,), 9.0, dtype=BF, device=DEV)
        api.tide_gated_backward(dh, K, g8.buffer, u8.buffer,
                                **{"dgate_bias" if name == "g" else "dup_bias": db})
        within(db, *want["db" + name], "db" + name)


@pytest.mark.parametrize("T,N,K", PAST_THE_CACHE)
def test_forward_of_weights_past_the_cache(T, N, K):
    check_forward(T, N, K, "gelu", True, "guh")
    check_forward(T, N, K, "silu", False, "")


def test_flat_calls_are_the_class_ones():
    g = gen(41)
    T, N, K = 30, 72, 136
    x, wg, wu, bg, bu = normal(g, T, K), normal(g, N, K), normal(g, N, K), normal(g, N), normal(g, N)
    kept = [Act8(T, N, device=DEV) for _ in range(3)]
    h = api.tide_gated_forward(x, wg, wu, gate_bias=bg, up_bias=bu, act="gelu", g_kept=kept[0].buffer,
                               u_kept=kept[1].buffer, h_kept=kept[2].buffer)
    k2 = [Act8(T, N, device=DEV) for _ in range(3)]
    block = Gated(wg, wu, gate_bias=bg, up_bias=bu, act="gelu", gate_grad=torch.empty_like(wg),
                  up_grad=torch.empty_like(wu))
    assert torch.equal(block.forward(x, g=k2[0], u=k2[1], h=k2[2]), h)
    assert all(torch.equal(a.buffer, b.buffer) for a, b in zip(kept, k2))
    x8 = Act8(T, K, device=DEV).pack(x)
    dg, du = torch.empty_like(wg), torch.empty_like(wu)
    dx = api.tide_gated_backward(h, K, kept[0].buffer, kept[1].buffer, gate=wg, up=wu, x_kept=x8.buffer,
                                 act="gelu", dx=True, dgate=dg, dup=du)
    assert torch.equal(dx, block.backward(h, x=x8, g=k2[0], u=k2[1]))
    assert torch.equal(dg, block.gate_grad) and torch.equal(du, block.up_grad)


@pytest.mark.parametrize("T,N,K,lds,shifts", [(5, 40, 64, (72, 48), (8, 8)), (5, 40, 64, (67, 43), (1, 3)),
                                              (70, 264, 136, (136, 264), (4, 0)), (130, 261, 77, (80, 300), (0, 1)),
                                              (1, 64, 128, (500, 64), (0, 0)), (3, 33, 200, (211, 40), (1, 5))])
def test_strides(T, N, K, lds, shifts):
    wg, wu, dh, (x8, g8, u8), values = backward_case(T, N, K, T + N)
    x = normal(gen(T), T, K)
    xs, _ = strided(x, lds[0], shifts[0])
    hs, buf = strided(torch.zeros(T, N, dtype=BF, device=DEV), lds[1], shifts[1])
    before = buf.clone()
    block = Gated(wg, wu, gate_grad=torch.empty_like(wg), up_grad=torch.empty_like(wu))
    assert block.forward(xs, out=hs) is hs
    want = ref.forward_ref(x, wg, wu, None, None, "silu")["h"]
    within(hs, want[0], ref.rounded(*want), "h")
    hs.zero_()  # nothing but the rows was written
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))
    ds, _ = strided(dh, lds[1], shifts[1])
    dx, buf = strided(torch.zeros(T, K, dtype=BF, device=DEV), lds[0], shifts[0])
    before = buf.clone()
    assert block.backward(ds, x=x8, g=g8, u=u8, dx=dx) is dx
    want = ref.backward_ref(dh, wg, wu, *values, "silu")
    within(dx, *want["dx"], "dx")
    within(block.gate_grad, *want["dwg"], "dwg")
    within(block.up_grad, *want["dwu"], "dwu")
    dx.zero_()
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


def test_weights_on_any_element():
    """Placed tensors may start on any element, each on another."""
    g = gen(5)
    buf, grads = normal(g, 4 * 40 * 72), torch.full((4 * 40 * 72,), 7.0, dtype=BF, device=DEV)
    at = lambda b, s: b[s:s + 40 * 72].view(40, 72)  # noqa: E731
    for T in (1, 20):
        x8, x = kept_of(normal(g, T, 72))
        g8, gv = kept_of(normal(g, T, 40))
        u8, uv = kept_of(normal(g, T, 40))
        dh = normal(g, T, 40)
        for s, s2 in ((1, 3000), (8, 3001), (2, 2884), (3, 3008)):
            wg, wu = at(buf, s), at(buf, s2)
            block = Gated(wg, wu, gate_grad=at(grads, s), up_grad=at(grads, s2))
            want = ref.forward_ref(x, wg, wu, None, None, "silu")["h"]
            within(block.forward(x.to(BF)), want[0], ref.rounded(*want), "h %d %d" % (s, s2))
            dx = block.backward(dh, x=x8, g=g8, u=u8)
            want = ref.backward_ref(dh, wg, wu, x, gv, uv, "silu")
            within(dx, *want["dx"], "dx")
            within(block.gate_grad, *want["dwg"], "dwg")
            within(block.up_grad, *want["dwu"], "dwu")
            block.gate_grad.fill_(7.0)
            block.up_grad.fill_(7.0)
            assert (grads == 7.0).all()


def test_one_matrix_twice():
    """gate and up may be the same tensor: h = act(g) g."""
    g = gen(6)
    x, w = normal(g, 50, 64), normal(g, 33, 64, scale=0.1)
    want = ref.forward_ref(x, w, w, None, None, "silu")["h"]
    within(Gated(w, w).forward(x), want[0], ref.rounded(*want), "h")


def test_empty_calls():
    z = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    seven = lambda *s: torch.full(s, 7.0, dtype=BF, device=DEV)  # noqa: E731
    b, c = normal(gen(1), 8), normal(gen(2), 8)
    # no input feature: h = act(bias) bias
    h = Gated(z(8, 0), z(8, 0), gate_bias=b, up_bias=c).forward(z(3, 0))
    want = (lref.act_ref(b.double(), "silu") * c.double()).expand(3, -1)
    within(h, want, want.abs() * (lref.BF16 + 32 * lref.F32) + 1e-6)
    # ... and the biases' gradients are sums all the same
    g8, gv = kept_of(normal(gen(3), 3, 8))
    u8, uv = kept_of(normal(gen(4), 3, 8))
    dh = normal(gen(5), 3, 8)
    block = Gated(z(8, 0), z(8, 0), gate_grad=z(8, 0), up_grad=z(8, 0), gate_bias_grad=seven(8), up_bias_grad=seven(8))
    assert block.backward(dh, x=Act8(3, 0, device=DEV), g=g8, u=u8).shape == (3, 0)
    want = ref.backward_ref(dh, z(8, 0), z(8, 0), torch.zeros(3, 0, dtype=torch.float64, device=DEV), gv, uv, "silu")
    within(block.gate_bias_grad, *want["dbg"])
    within(block.up_bias_grad, *want["dbu"])
    # no token: gradients are empty sums
    w = normal(gen(3), 8, 16)
    block = Gated(w, w, gate_grad=seven(8, 16), up_grad=seven(8, 16), gate_bias_grad=seven(8), up_bias_grad=seven(8))
    assert block.forward(z(0, 16)).shape == (0, 8)
    none = Act8(0, 8, device=DEV)
    assert block.backward(z(0, 8), x=Act8(0, 16, device=DEV), g=none, u=none).shape == (0, 16)
    for t in (block.gate_grad, block.up_grad, block.gate_bias_grad, block.up_bias_grad):
        assert (t == 0).all()
    # no output feature: dx is an empty sum
    dx, none = seven(3, 16), Act8(3, 0, device=DEV)
    Gated(z(0, 16), z(0, 16)).backward(z(3, 0), g=none, u=none, dx=dx)
    assert (dx == 0).all()


def test_rows_that_are_not_finite_stay_alone():
    g = gen(9)
    x, wg, wu = normal(g, 150, 200), normal(g, 300, 200), normal(g, 300, 200)
    x[7, 3], x[149, 199], wg[5, 0], wu[6, 1] = math.nan, math.inf, math.nan, math.nan
    h = Gated(wg, wu).forward(x)
    bad = torch.zeros(150, 300, dtype=torch.bool, device=DEV)
    bad[7], bad[149], bad[:, 5], bad[:, 6] = True, True, True, True
    assert torch.equal(~h.isfinite(), bad)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_gates_at_the_ends(act):
    """A g that reads back as infinity has its limit's value and slope; one that
    was not finite is NaN, and stays in its own row and column."""
    T, N = 6, 40
    g8, gv = kept_of(normal(gen(2), T, N))
    gv = gv.clone()
    # the largest scale's largest values stand for 2^128, infinity in binary32
    scales, codes = g8.scales.view(torch.uint8), g8.data.view(torch.uint8)
    codes[1, :32] = 0
    scales[1, 0] = 120 + 127
    codes[1, 0], codes[1, 1] = 0x78, 0xf8                   # 256 * 2^120 = 2^128, and minus that
    codes[2, 7] = 0x7f
    u8, uv = kept_of(normal(gen(3), T, N))
    dh = normal(gen(4), T, N)
    dbg, dbu = (torch.empty(N, dtype=BF, device=DEV) for _ in range(2))
    eye = torch.eye(N, dtype=BF, device=DEV)
    zero = torch.zeros_like(eye)
    # with unit weights dx is dg or du itself
    dg = Gated(eye, zero, act=act).backward(dh, g=g8, u=u8)
    du = Gated(zero, eye, act=act).backward(dh, g=g8, u=u8)
    assert dg[2].isnan().all() and du[2].isnan().all()
    # plus infinity: slope 1, value infinity
    api.tide_gated_backward(dh, N, g8.buffer, u8.buffer, act=act, dgate_bias=dbg, dup_bias=dbu)
    assert dbg[7].isnan() and dbu[7].isnan() and dbg[0].isfinite() and dbg[1].isfinite()
    assert dbu[0].isinf() and dbu[1].isfinite()
    rows = [0, 3, 4, 5]
    want = ref.backward_ref(dh[rows], eye, zero, torch.zeros(4, N, device=DEV).double(), gv[rows], uv[rows], act)
    within(dg[rows], *want["dx"], "dg")
    # minus infinity: slope and value 0
    alone = dh.clone()
    alone[2:], alone[0] = 0, 0
    alone[1, 0] = 0
    codes[2, 7], codes[1, 0] = 0, 0
    api.tide_gated_backward(alone, N, g8.buffer, u8.buffer, act=act, dgate_bias=dbg, dup_bias=dbu)
    assert dbg[1] == 0 and dbu[1] == 0


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """With unit weights every output has one g and one u: dx is their gradients
    times dh, against central differences in 64 bits."""
    g = gen(13)
    T, N = 40, 64
    grid = lref.e4m3_grid().to(DEV)
    draw = lambda: grid[torch.randint(40, 80, (T, N), generator=g, device=DEV)] / 8  # noqa: E731
    sign = lambda v: torch.where(torch.rand(T, N, generator=g, device=DEV) < 0.5, -v, v)  # noqa: E731
    g8, gv = kept_of(sign(draw()))
    u8, uv = kept_of(sign(draw()))
    x8, xv = kept_of(draw())
    dh = normal(g, T, N)
    h = 2.0 ** -20
    value = lref.act_ref(gv, act)
    slope = (lref.act_ref(gv + h, act) - lref.act_ref(gv - h, act)) / (2 * h)
    dg, du = dh.double() * uv * slope, dh.double() * value
    eye = torch.eye(N, dtype=BF, device=DEV)
    zero = torch.zeros_like(eye)
    block = Gated(eye, zero, act=act, gate_grad=torch.empty_like(eye), up_grad=torch.empty_like(eye),
                  gate_bias_grad=torch.empty(N, dtype=BF, device=DEV))
    # two roundings (dg, dx), and the differences' own error
    within(block.backward(dh, x=x8, g=g8, u=u8), dg, 2 * lref.BF16 * dg.abs() + 1e-5, "dg")
    within(Gated(zero, eye, act=act).backward(dh, g=g8, u=u8), du, 2 * lref.BF16 * du.abs() + 1e-5, "du")
    within(block.gate_bias_grad, dg.sum(0), lref.BF16 * dg.sum(0).abs() + 1e-5 * dg.abs().sum(0) + 1e-5, "dbg")
    for got, d in ((block.gate_grad, dg), (block.up_grad, du)):
        dw = d.T @ xv
        within(got, dw, lref.BF16 * (dw.abs() + 1.01 * (d.abs().T @ xv.abs())) + 1e-4, "dw")


# ---- streams, graphs, repeats, memory ----------------------------------------------------------

def make(seed, T=70, N=300, K=200, act="silu"):
    g = gen(seed)
    new = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
    block = Gated(normal(g, N, K, scale=0.1), normal(g, N, K, scale=0.1), gate_bias=normal(g, N),
                  up_bias=normal(g, N), act=act, gate_grad=new(N, K), up_grad=new(N, K),
                  gate_bias_grad=new(N), up_bias_grad=new(N))
    kept = [Act8(T, K, device=DEV)] + [Act8(T, N, device=DEV) for _ in range(3)]
    return block, normal(g, T, K), normal(g, T, N), kept


def step(block, x, dh, kept):
    kept[0].pack(x)
    h = block.forward(x, g=kept[1], u=kept[2], h=kept[3])
    return h, block.backward(dh, x=kept[0], g=kept[1], u=kept[2])


def bits(m, out):
    b = m[0]
    return [t.clone().view(torch.uint8) for t in (*out, b.gate_grad, b.up_grad, b.gate_bias_grad, b.up_bias_grad,
                                                  *(k.buffer for k in m[3]))]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T,N,K", [(1, 300, 2048), (5, 300, 2048), (70, 300, 200), (600, 700, 3000)])
def test_repeats_give_the_same_bits(T, N, K):
    m = make(T, T, N, K)
    want = bits(m, step(*m))
    for _ in range(3):
        assert same(want, bits(m, step(*m)))


def test_streams_side_by_side():
    ms = [make(1), make(2, 257, 136, 512, "gelu")]
    want = [bits(m, step(*m)) for m in ms]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(10):
        for k, m in enumerate(ms):
            with torch.cuda.stream(s[k]):
                outs[k] = step(*m)
    torch.cuda.synchronize()
    assert all(same(want[k], bits(m, outs[k])) for k, m in enumerate(ms))
    block, x, dh, kept = ms[0]  # by the stream argument
    h = block.forward(x, stream=s[0])
    dx = block.backward(dh, x=kept[0], g=kept[1], u=kept[2], stream=s[0])
    s[0].synchronize()
    assert torch.equal(h.view(torch.uint8), want[0][0]) and torch.equal(dx.view(torch.uint8), want[0][1])


def test_two_host_threads():
    ms = [make(1), make(2, 257, 136, 512)]
    want = [bits(m, step(*m)) for m in ms]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    out = step(*ms[k])
                got[k] = bits(ms[k], out)
                s.synchronize()
        except Exception as e:  # shown by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and not any(t.is_alive() for t in threads)
    assert all(same(a, b) for a, b in zip(want, got))


def test_captured_steps():
    """Two captured steps replayed in turn and side by side, with other work
    and synchronisations between, each replay against the eager step on new
    inputs."""
    ms = [make(4), make(5, 257, 136, 512, "gelu_tanh"), make(6, 1, 520, 1024)]
    for m in ms:
        step(*m)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*m))
        graphs.append(g)
    s = [torch.cuda.Stream() for _ in ms]
    for rep in range(4):
        for k, m in enumerate(ms):
            for t in (m[1], m[2]):
                t.copy_(normal(gen(100 * rep + 10 * k + t.shape[1]), *t.shape))
        torch.cuda.synchronize()
        for k in range(len(ms)):
            with torch.cuda.stream(s[k] if rep % 2 else torch.cuda.current_stream()):
                graphs[k].replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device=DEV).sum()
        got = [bits(m, outs[k]) for k, m in enumerate(ms)]
        for k, m in enumerate(ms):
            assert same(bits(m, step(*m)), got[k]), (rep, k)
        assert junk.isfinite()


def test_checkpoints_in_caller_memory():
    """Checkpoints carved out of a vacated gathered buffer: nothing else of it
    is written."""
    m = make(7)
    want = bits(m, step(*m))
    vacated = torch.full((1 << 17,), -1, dtype=torch.int16, device=DEV).view(BF)
    kept, at = [], 64
    for k in m[3]:
        kept.append(Act8(k.rows, k.cols, buffer=vacated[at:]))
        at += -(-Act8.bytes(k.rows, k.cols) // 32) * 16 + 32
    m2 = m[:3] + (kept,)
    assert same(want, bits(m2, step(*m2)))
    for k in kept:
        k.buffer.fill_(255)
    assert (vacated.view(torch.uint8) == 255).all()


def test_refusals_on_the_gpu():
    g = gen(1)
    x, w = normal(g, 4, 64), normal(g, 32, 64)
    with pytest.raises(TideError, match="TIDE_EOVERLAP"):
        Gated(w, w).forward(x, out=x[:, :32])
    k = Act8(4, 32, device=DEV)
    with pytest.raises(TideError, match="TIDE_EOVERLAP"):
        Gated(w, w).forward(x, g=k, u=k)
    with pytest.raises(TideError, match="TIDE_EOVERLAP"):
        Gated(w, w, gate_grad=w, up_grad=torch.empty_like(w)).backward(x[:, :32], x=Act8(4, 64, device=DEV), g=k, u=k)


# ---- a layer between the collectives -----------------------------------------------------------

def test_feed_forward_half_between_placement_and_reduce_scatter():
    """Place a norm, a gate, an up and a down projection, run every simulated
    rank's tokens through norm, block and product onto the residual stream and
    back with checkpoints, reduce-scatter the gradients: each call against 64
    bits on what it was given, and the shards against the sums."""
    R, T, C, F = 4, 45, 136, 200
    shapes = ((C,), (F, C), (F, C), (C, F))
    w = configs.Workload(key=1, name="feed-forward half", R=R, names=("norm", "gate", "up", "down"),
                         shapes=shapes, sigma=0.05)
    st = harness.setup(w, device=DEV)
    st.plan.ag()
    scale, gate, up, down = st.full
    val = lambda k: lref.unpack_ref(k.data.view(torch.uint8), k.scales.view(torch.uint8), k.cols)  # noqa: E731
    sums, bounds = [0] * 4, [0] * 4
    for q in range(R):
        g = gen(50 + q)
        x, dout = normal(g, T, C), normal(g, T, C)
        grads = st.grads[q]
        norm = Norm(scale, kind="rms", eps=1e-5, weight_grad=grads[0])
        block = Gated(gate, up, gate_grad=grads[1], up_grad=grads[2])
        last = Linear(down, weight_grad=grads[3])
        x8, y8 = Act8(T, C, device=DEV), Act8(T, C, device=DEV)
        g8, u8, h8 = (Act8(T, F, device=DEV) for _ in range(3))
        y = norm.forward(x, x8=x8, y8=y8)
        h = block.forward(y, g=g8, u=u8, h=h8)
        out = last.forward(h, residual=x)
        dh = last.backward(dout, x=h8)
        dy = block.backward(dh, x=y8, g=g8, u=u8)
        dx = norm.backward(dy, x8, add=dout)
        want = nref.forward_ref(x, scale, None, "rms", 1e-5)
        within(y, want[0], nref.rounded(*want), "y")
        kept_within(y8, *want, "y8")
        want = ref.forward_ref(y, gate, up, None, None, "silu")
        within(h, want["h"][0], ref.rounded(*want["h"]), "h")
        for k, n in ((g8, "g"), (u8, "u"), (h8, "h")):
            kept_within(k, *want[n], n)
        want, _, _, b = lref.forward_ref(h, down, None, x, "none")
        within(out, want, b, "out")
        g3 = lref.backward_ref(dout, down, val(h8), None, "none")
        within(dh, *g3["dx"], "dh")
        g2 = ref.backward_ref(dh, gate, up, val(y8), val(g8), val(u8), "silu")
        within(dy, *g2["dx"], "dy")
        g1 = nref.backward_ref(dy, scale, val(x8), dout, "rms", 1e-5)
        within(dx, *g1["dx"], "dx")
        for p, (want, b) in enumerate((g1["dw"], g2["dwg"], g2["dwu"], g3["dw"])):
            sums[p], bounds[p] = sums[p] + want, bounds[p] + b
    st.plan.rs()
    for p, shp in enumerate(shapes):
        s = -(-shp[0] // R)
        for r in range(R):
            n = max(0, min(shp[0], (r + 1) * s) - r * s)
            got = st.plan.shard(st.out[r], p)
            want, b = sums[p][r * s:r * s + n], bounds[p][r * s:r * s + n]
            within(got[:n], want, b + R * lref.F32 * (want.abs() + b), "shard %d of %d" % (r, p))
            assert (got[n:] == 0).all()


# ---- far offsets -------------------------------------------------------------------------------

@pytest.mark.big
@pytest.mark.parametrize("T,N,K", [(140000, 40, 16400), (41000, 53000, 72)])
def test_offsets_past_32_bits(T, N, K):
    """Operands, results and checkpoints whose byte offsets pass 2^32."""
    g = gen(8)
    x = torch.empty(T, K, dtype=BF, device=DEV)
    for t in range(0, T, 20000):
        x[t:t + 20000] = torch.randn(min(20000, T - t), K, generator=g, device=DEV)
    x8, g8, u8, h8 = Act8(T, K, device=DEV).pack(x), *(Act8(T, N, device=DEV) for _ in range(3))
    wg, wu = normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, N, K, scale=1 / math.sqrt(K))
    block = Gated(wg, wu, gate_grad=torch.empty_like(wg), up_grad=torch.empty_like(wu))
    h = block.forward(x, g=g8, u=u8, h=h8)
    rows = torch.tensor([0, 1, T // 3, T // 2, T - 40001 % T, T - 2, T - 1], device=DEV)
    raw = lambda k: (k.data.view(torch.uint8)[rows], k.scales.view(torch.uint8)[rows])  # noqa: E731
    want = ref.forward_ref(x[rows], wg, wu, None, None, "silu")
    within(h[rows], want["h"][0], ref.rounded(*want["h"]), "h")
    val = {}
    for name, k, c in (("x", x8, K), ("g", g8, N), ("u", u8, N), ("h", h8, N)):
        val[name] = lref.unpack_ref(*raw(k), c)
        if name != "x":
            v, err = want[name]
            step = torch.exp2(raw(k)[1].double() - 127).repeat_interleave(32, 1)[:, :c]
            within(val[name], v, torch.maximum(lref.E4M3 * (v.abs() + err), lref.E4M3_SUB * step) + err, name)
    dh = h
    dh.zero_()
    dh[rows] = normal(g, len(rows), N)
    dx = block.backward(dh, x=x8, g=g8, u=u8, dx=x)
    want = ref.backward_ref(dh[rows], wg, wu, val["x"], val["g"], val["u"], "silu")
    within(dx[rows], *want["dx"], "dx")
    within(block.gate_grad, *want["dwg"], "dwg")
    within(block.up_grad, *want["dwu"], "dwu")
    assert (dx[T // 4:T // 4 + 5] == 0).all()


@pytest.mark.big
def test_most_tokens():
    """2^30 tokens of one feature: h = (2 x) (4 x) with act none, every element."""
    T = 1 << 30
    x = torch.zeros(T, 1, dtype=BF, device=DEV)
    at = torch.tensor([0, 1, (1 << 29) + 5, T - 1], device=DEV)
    x[at] = torch.tensor([[1.0], [-2.0], [0.5], [3.0]], dtype=BF, device=DEV)
    w2, w4 = (torch.full((1, 1), v, dtype=BF, device=DEV) for v in (2.0, 4.0))
    h = Gated(w2, w4, act="none").forward(x)
    want = torch.zeros(T, 1, dtype=BF, device=DEV)
    want[at] = torch.tensor([[8.0], [32.0], [2.0], [72.0]], dtype=BF, device=DEV)
    assert torch.equal(h, want)
