"""GPU tests of the gated block where binary32 ends."""
import pytest
import torch

from shard_placement_amd.gated import Gated
from tests import linear_ref as lref
from tests.test_linear_gpu import BF, DEV, kept_of, within

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
