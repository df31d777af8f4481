"""CPU tests of the layer products and the 8-bit checkpoints: sizes, refusals
(none reaches the GPU), and the reference in tests/linear_ref.py against
independent values."""
import ctypes
import math

import pytest
import torch

from tests import linear_ref as ref
from shard_placement_amd import _lib, api, linear
from shard_placement_amd._lib import TideLinearBackwardArgs, TideLinearForwardArgs

EINVAL, EALIGN, EOVERLAP, ENOSPACE, EUNSUPPORTED = -1, -2, -3, -4, -6
AT = 1 << 30  # made-up device addresses, far apart


def fwd(**kw):
    a = TideLinearForwardArgs()
    a.tokens, a.out_features, a.in_features = 40, 64, 96
    a.x, a.ldx, a.weight, a.y, a.ldy, a.ldr = AT, 96, 2 * AT, 3 * AT, 64, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def bwd(**kw):
    a = TideLinearBackwardArgs()
    a.tokens, a.out_features, a.in_features, a.act = 40, 64, 96, api.ACTS["silu"]
    a.dy, a.lddy, a.weight, a.x_kept, a.z_kept = AT, 64, 2 * AT, 3 * AT, 4 * AT
    a.dx, a.lddx, a.dweight, a.dbias = 5 * AT, 96, 6 * AT, 7 * AT
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def query(name, args):
    n = ctypes.c_size_t(12345)
    st = getattr(_lib.lib(), name)(ctypes.byref(args), ctypes.byref(n))
    return st, n.value


def test_checkpoint_size():
    assert api.tide_act8_bytes(3, 33) == 3 * (64 + 2)
    assert api.tide_act8_bytes(0, 33) == 0 and api.tide_act8_bytes(5, 0) == 0
    assert api.tide_act8_bytes(2 ** 31 - 1, 32) == (2 ** 31 - 1) * 33
    n = ctypes.c_size_t(0)
    L = _lib.lib()
    assert L.tide_act8_bytes(-1, 4, ctypes.byref(n)) == EINVAL
    assert L.tide_act8_bytes(4, -1, ctypes.byref(n)) == EINVAL
    assert L.tide_act8_bytes(4, 4, None) == EINVAL
    assert L.tide_act8_bytes(2 ** 31, 4, ctypes.byref(n)) == EUNSUPPORTED
    assert L.tide_act8_bytes(4, (1 << 22) + 1, ctypes.byref(n)) == EUNSUPPORTED


@pytest.mark.parametrize("unpack", [False, True])
def test_checkpoint_refusals(unpack):
    L = _lib.lib()

    def call(x, ldx, rows, cols, kept):
        if unpack:
            return L.tide_act8_unpack(kept, rows, cols, x, ldx, None)
        return L.tide_act8_pack(x, ldx, rows, cols, kept, None)

    assert call(None, 64, 4, 64, AT) == EINVAL
    assert call(AT, 64, 4, 64, None) == EINVAL
    assert call(AT, 63, 4, 64, 2 * AT) == EINVAL       # rows share memory
    assert call(AT, 64, -4, 64, 2 * AT) == EINVAL
    assert call(AT + 1, 64, 4, 64, 2 * AT) == EALIGN
    assert call(AT, 64, 4, 64, 2 * AT + 8) == EALIGN   # checkpoints lie on 16 bytes
    assert call(AT, (1 << 22) + 1, 4, 64, 2 * AT) == EUNSUPPORTED
    assert call(AT, 64, 4, 64, AT + 256) == EOVERLAP
    assert call(AT + 4 * 66 - 16 * 2, 64, 4, 64, AT) == EOVERLAP  # the last scales
    assert call(None, 0, 0, 64, None) == 0             # nothing to do
    assert call(None, 0, 4, 0, None) == 0


def test_forward_refusals():
    L = _lib.lib()

    def call(a, ws=None, n=0):
        return L.tide_linear_forward(ctypes.byref(a), ws, n, None)

    assert L.tide_linear_forward(None, None, 0, None) == EINVAL
    assert L.tide_linear_forward_workspace(None, None) == EINVAL
    for bad in (dict(tokens=-1), dict(out_features=-1), dict(in_features=-1), dict(act=5),
                dict(act=-1), dict(reserved=1), dict(x=None), dict(weight=None), dict(y=None),
                dict(ldx=95), dict(ldy=63), dict(residual=8 * AT, ldr=63)):
        assert call(fwd(**bad)) == EINVAL, bad
        assert query("tide_linear_forward_workspace", fwd(**bad))[0] == EINVAL, bad
    for bad in (dict(tokens=1 << 31), dict(out_features=(1 << 22) + 1, ldy=1 << 23),
                dict(in_features=(1 << 22) + 1, ldx=1 << 23), dict(ldx=(1 << 22) + 1)):
        assert call(fwd(**bad)) == EUNSUPPORTED, bad
    # grids that a later launch could not have are refused before the first
    for T, N, K in ((1 << 30, 64, 96), (2049, 1 << 22, 96), (40, 1 << 22, 2049)):
        a = fwd(tokens=T, out_features=N, in_features=K, ldx=1 << 22, ldy=1 << 22)
        assert call(a) == EUNSUPPORTED, (T, N, K)
        b = bwd(tokens=T, out_features=N, in_features=K, lddy=1 << 22, lddx=1 << 22)
        assert L.tide_linear_backward(ctypes.byref(b), None, 0, None) == EUNSUPPORTED
    for bad in (dict(x=AT + 1), dict(weight=2 * AT + 1), dict(y=3 * AT + 1), dict(bias=5 * AT + 1),
                dict(residual=6 * AT + 1), dict(z_kept=7 * AT + 8)):
        assert call(fwd(**bad)) == EALIGN, bad
    for bad in (dict(y=AT), dict(y=2 * AT + 64), dict(y=AT + 40 * 96 * 2 - 2),
                dict(z_kept=3 * AT + 16), dict(z_kept=AT), dict(bias=3 * AT + 2),
                dict(residual=3 * AT, ldr=80), dict(residual=3 * AT + 2)):
        assert call(fwd(**bad)) == EOVERLAP, bad
    # nothing to do: no token, or no output feature
    assert call(fwd(tokens=0)) == 0 and call(fwd(out_features=0)) == 0
    # an operand whose rows do not start on 16 bytes needs its copy in a workspace
    st, n = query("tide_linear_forward_workspace", fwd(ldx=97))
    assert st == 0 and n >= 40 * 96 * 2
    assert call(fwd(ldx=97)) == ENOSPACE
    assert call(fwd(ldx=97), 8 * AT, n - 1) == ENOSPACE
    assert call(fwd(ldx=97), 8 * AT + 8, n) == EALIGN
    assert call(fwd(ldx=97), 3 * AT, n) == EOVERLAP
    assert call(fwd(ldx=97), AT + 2, n) in (EALIGN, EOVERLAP)


def test_backward_refusals():
    L = _lib.lib()

    def call(a, ws=None, n=0):
        return L.tide_linear_backward(ctypes.byref(a), ws, n, None)

    assert L.tide_linear_backward(None, None, 0, None) == EINVAL
    for bad in (dict(tokens=-1), dict(act=9), dict(reserved=2), dict(dy=None), dict(weight=None),
                dict(x_kept=None), dict(z_kept=None), dict(lddy=63), dict(lddx=95)):
        assert call(bwd(**bad)) == EINVAL, bad
        assert query("tide_linear_backward_workspace", bwd(**bad))[0] == EINVAL, bad
    for bad in (dict(dy=AT + 1), dict(weight=2 * AT + 1), dict(x_kept=3 * AT + 8),
                dict(z_kept=4 * AT + 4), dict(dx=5 * AT + 1), dict(dweight=6 * AT + 1),
                dict(dbias=7 * AT + 1)):
        assert call(bwd(**bad)) == EALIGN, bad
    for bad in (dict(dx=AT), dict(dweight=2 * AT), dict(dbias=3 * AT), dict(dx=6 * AT),
                dict(dbias=6 * AT + 2), dict(dweight=4 * AT)):
        assert call(bwd(**bad)) == EOVERLAP, bad
    assert call(bwd(tokens=1 << 31)) == EUNSUPPORTED
    st, n = query("tide_linear_backward_workspace", bwd())
    assert st == 0 and n > 0
    assert call(bwd()) == ENOSPACE and call(bwd(), 8 * AT, n - 1) == ENOSPACE
    assert call(bwd(), 8 * AT + 2, n) == EALIGN
    for a in range(1, 8):
        assert call(bwd(), a * AT, n) == EOVERLAP, a
    # what only an absent gradient needs may be absent
    assert query("tide_linear_backward_workspace", bwd(dx=None, weight=None))[0] == 0
    assert query("tide_linear_backward_workspace", bwd(dweight=None, x_kept=None))[0] == 0
    assert query("tide_linear_backward_workspace", bwd(act=0, z_kept=None))[0] == 0
    # no gradient asked for: nothing is looked at
    assert call(bwd(dx=None, dweight=None, dbias=None, dy=None)) == 0


def test_column_ranges_of_one_buffer_are_apart():
    """x and y as column ranges of one buffer with a common row distance share
    no byte; one column more does."""
    L = _lib.lib()
    ok = fwd(x=AT, ldx=176, y=AT + 2 * 96, ldy=176, weight=None)
    assert L.tide_linear_forward(ctypes.byref(ok), None, 0, None) == EINVAL  # only the weight is missing
    a = fwd(x=AT, ldx=176, y=AT + 2 * 95, ldy=176)
    assert L.tide_linear_forward(ctypes.byref(a), None, 0, None) == EOVERLAP
    a = fwd(x=AT, ldx=176, y=AT + 2 * 96, ldy=180)
    assert L.tide_linear_forward(ctypes.byref(a), None, 0, None) == EOVERLAP


def test_python_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(_lib.TideError, match="expected a GPU"):
        api.tide_act8_pack(x, torch.zeros(1000, dtype=torch.uint8))
    with pytest.raises(_lib.TideError, match="dtype"):
        api.tide_act8_pack(x.float(), torch.zeros(1000, dtype=torch.uint8))
    with pytest.raises(_lib.TideError, match="act is"):
        linear.Linear(x, act="swish")
    with pytest.raises(_lib.TideError, match="expected 2"):
        linear.Linear(x[0])
    with pytest.raises(_lib.TideError, match="holds 100 bytes, need 264"):
        linear.Act8(4, 64, buffer=torch.zeros(100, dtype=torch.uint8))
    kept = linear.Act8(4, 33, buffer=torch.zeros(200, dtype=torch.bfloat16))
    assert kept.data.shape == (4, 64) and kept.scales.shape == (4, 2)
    with pytest.raises(_lib.TideError, match="expected .4, 33."):
        kept.pack(x)
    with pytest.raises(_lib.TideError, match="expected a GPU"):
        kept.unpack()
    with pytest.raises(_lib.TideError, match="expected a GPU"):
        kept.unpack(torch.zeros(4, 33, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        linear.Linear(None)


def test_reference_rounds_like_torch():
    """The reference's e4m3 codes against torch's conversion, at every code,
    every middle between two codes and its neighbours."""
    grid = ref.e4m3_grid()
    mid = (grid[1:] + grid[:-1]) / 2
    v = torch.cat([grid, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    v = torch.cat([v, -v])
    rows = torch.full((v.numel(), 32), 0.0, dtype=torch.float64)
    rows[:, 0], rows[:, 1] = 448.0, v  # the scale is 1
    codes, scales = ref.pack_ref(rows)
    assert (scales == 127).all()
    want = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes[:, 1], want)


def test_reference_scales():
    for amax, e in ((448.0, 0), (448.5, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -110),
                    (2.0 ** -120, -110), (1.99 * 2.0 ** 127, 120)):
        x = torch.zeros(1, 40, dtype=torch.float64)
        x[0, 5], x[0, 6] = -amax, math.inf
        codes, scales = ref.pack_ref(x)
        assert scales[0, 0] == e + 127 and scales[0, 1] == 17, amax
        assert codes[0, 6] == 0x7f
        got = ref.unpack_ref(codes, scales, 40)
        if amax >= 2.0 ** -110:
            assert abs(got[0, 5].item() + amax) <= amax * 2.0 ** -4


@pytest.mark.parametrize("act", list(api.ACTS))
def test_reference_slopes_against_differences(act):
    z = torch.linspace(-6, 6, 97, dtype=torch.float64) + 0.013
    h = 1e-6
    want = (ref.act_ref(z + h, act) - ref.act_ref(z - h, act)) / (2 * h)
    assert (ref.slope_ref(z, act) - want).abs().max() < 1e-8


def test_limits_of_long_narrow_matrices():
    """At the documented limits the workspace can be asked for; past them every
    call is refused before its first launch."""
    L = _lib.lib()
    n = ctypes.c_size_t(0)
    assert api.tide_act8_bytes(1 << 14, 1 << 22) == (1 << 36) // 32 * 33
    assert L.tide_act8_bytes((1 << 14) + 1, 1 << 22, ctypes.byref(n)) == EUNSUPPORTED
    assert L.tide_act8_pack(AT, 1 << 22, (1 << 14) + 1, 1 << 22, 1 << 50, None) == EUNSUPPORTED
    far = dict(out_features=1, in_features=1, weight=1 << 50)
    for T, want in ((1 << 30, 0), ((1 << 30) + 1, EUNSUPPORTED)):
        a = fwd(tokens=T, x=1 << 51, ldx=1, y=1 << 52, ldy=1, **far)
        b = bwd(tokens=T, dy=1 << 51, lddy=1, dx=1 << 52, lddx=1, x_kept=1 << 53, z_kept=1 << 54,
                dweight=1 << 55, dbias=1 << 56, **far)
        assert query("tide_linear_forward_workspace", a)[0] == want
        assert query("tide_linear_backward_workspace", b)[0] == want
