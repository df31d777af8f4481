"""GPU tests of the gated block where binary32 ends, and of few tokens on any
element."""
import pytest
import torch

from shard_placement_amd.gated import Gated
from tests import gated_ref as ref
from tests import linear_ref as lref
from tests.test_linear_gpu import BF, DEV, gen, kept_of, normal, strided, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,gate", [("relu", -3.0), ("silu", -48.0), ("gelu", -8.0), ("gelu_tanh", -8.0),
                                      ("gelu", -40.0), ("gelu_tanh", -40.0)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_small_slope_of_large_factors(act, gate, sign):
    """dg = dh u act'(g) where dh u alone would pass binary32: finite, and 0 where
    the slope is."""
    T, N = 5, 40
    fill = lambda v, dt=torch.float64: torch.full((T, N), v, dtype=dt, device=DEV)  # noqa: E731
    g8, gv = kept_of(fill(gate))
    u8, uv = kept_of(fill(sign * 2.0 ** 72))
    dh = fill(2.0 ** 60, BF)
    eye = torch.eye(N, dtype=BF, device=DEV)
    zero = torch.zeros_like(eye)
    dbg = torch.empty(N, dtype=BF, device=DEV)
    # with unit weights dx is dg itself
    dg = Gated(eye, zero, act=act, gate_bias_grad=dbg).backward(dh, g=g8, u=u8)
    slope = lref.slope_ref(gv, act)
    if slope.abs().max() < 1e-40:  # below what binary32 holds next to a normal number: 0
        slope = slope * 0
    want = dh.double() * uv * slope
    assert dg.isfinite().all() and dbg.isfinite().all()
    # the slope's own error, and two roundings
    off = 2.0 ** -7 + 2 * lref.BF16
    within(dg, want, off * want.abs(), "dg")
    within(dbg, want.sum(0), off * want.sum(0).abs(), "dbg")


@pytest.mark.parametrize("act,gate", [("silu", 2.5), ("gelu", 1.375), ("gelu_tanh", 1.375), ("relu", 1.0), ("none", 1.0)])
def test_the_largest_factor(act, gate):
    """u near binary32's end and a slope past 1: dg is finite where a small dh makes
    it so."""
    T, N = 3, 33
    fill = lambda v, dt=torch.float64: torch.full((T, N), v, dtype=dt, device=DEV)  # noqa: E731
    g8, gv = kept_of(fill(gate))
    u8, uv = kept_of(fill(240 * 2.0 ** 120))
    assert act in ("relu", "none") or (lref.slope_ref(gv, act) * uv > 2.0 ** 128).all()
    dh = fill(2.0 ** -20, BF)
    eye = torch.eye(N, dtype=BF, device=DEV)
    dg = Gated(eye, torch.zeros_like(eye), act=act).backward(dh, g=g8, u=u8)
    want = dh.double() * uv * lref.slope_ref(gv, act)
    within(dg, want, (2.0 ** -16 + 2 * lref.BF16) * want.abs(), "dg")


@pytest.mark.parametrize("T,N,K", [(2, 2305, 264), (3, 4096, 512), (3, 40, 64), (4, 300, 2056), (4, 1001, 8)])
@pytest.mark.parametrize("shift,more", [(1, 0), (0, 3), (5, 8)])
def test_few_tokens_on_any_element(T, N, K, shift, more):
    """x on any element before weights that can be read where they lie."""
    g = gen(T * N + K)
    x, wg, wu = normal(g, T, K), normal(g, N, K, scale=K ** -0.5), normal(g, N, K, scale=K ** -0.5)
    bg, bu = normal(g, N), normal(g, N)
    xs, _ = strided(x, K + more, shift)
    want = ref.forward_ref(x, wg, wu, bg, bu, "silu")["h"]
    within(Gated(wg, wu, gate_bias=bg, up_bias=bu).forward(xs), want[0], ref.rounded(*want), "h")
