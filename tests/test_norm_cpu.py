"""CPU tests of the norms: refusals (none reaches the GPU), workspaces, and the
reference in tests/norm_ref.py against torch and against differences."""
import ctypes
import math

import pytest
import torch

from shard_placement_amd import _lib, api, linear, norm
from shard_placement_amd._lib import TideError, TideNormBackwardArgs, TideNormForwardArgs
from tests import norm_ref as ref

EINVAL, EALIGN, EOVERLAP, ENOSPACE, EUNSUPPORTED = -1, -2, -3, -4, -6
AT = 1 << 30  # made-up device addresses, far apart


def fwd(**kw):
    a = TideNormForwardArgs()
    a.rows, a.cols, a.kind, a.eps = 40, 96, api.NORMS["layer"], 1e-5
    a.x, a.ldx, a.weight, a.bias, a.y, a.ldy = AT, 96, 2 * AT, 3 * AT, 4 * AT, 96
    a.x_kept, a.y_kept = 5 * AT, 6 * AT
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def bwd(**kw):
    a = TideNormBackwardArgs()
    a.rows, a.cols, a.kind, a.eps = 40, 96, api.NORMS["rms"], 1e-5
    a.dy, a.lddy, a.x, a.ldx, a.weight, a.add, a.ldadd = AT, 96, 2 * AT, 96, 3 * AT, 4 * AT, 96
    a.dx, a.lddx, a.dweight, a.dbias = 5 * AT, 96, 6 * AT, 7 * AT
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def query(args):
    n = ctypes.c_size_t(12345)
    return _lib.lib().tide_norm_backward_workspace(ctypes.byref(args), ctypes.byref(n)), n.value


def test_forward_refusals():
    L = _lib.lib()

    def call(a):
        return L.tide_norm_forward(ctypes.byref(a), None)

    assert L.tide_norm_forward(None, None) == EINVAL
    for bad in (dict(rows=-1), dict(cols=-1), dict(kind=2), dict(kind=-1), dict(eps=0.0),
                dict(eps=-1e-5), dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e-31),
                dict(x=None), dict(weight=None), dict(y=None), dict(ldx=95), dict(ldy=95)):
        assert call(fwd(**bad)) == EINVAL, bad
    for bad in (dict(rows=(1 << 27) + 1), dict(cols=32769, ldx=40000, ldy=40000),
                dict(rows=1 << 20, cols=8193, ldx=8193, ldy=8193), dict(ldx=(1 << 22) + 1),
                dict(ldy=(1 << 22) + 1)):
        assert call(fwd(**bad)) == EUNSUPPORTED, bad
    for bad in (dict(x=AT + 1), dict(weight=2 * AT + 1), dict(bias=3 * AT + 1), dict(y=4 * AT + 1),
                dict(x_kept=5 * AT + 8), dict(y_kept=6 * AT + 2)):
        assert call(fwd(**bad)) == EALIGN, bad
    kept = 40 * 99
    for bad in (dict(y=AT), dict(y=2 * AT + 64), dict(y=3 * AT), dict(y=AT + 40 * 96 * 2 - 2),
                dict(x_kept=AT), dict(x_kept=4 * AT), dict(y_kept=5 * AT),
                dict(y_kept=5 * AT + kept // 16 * 16), dict(y_kept=3 * AT)):
        assert call(fwd(**bad)) == EOVERLAP, bad
    assert call(fwd(rows=0, x=None, y=None)) == 0 and call(fwd(cols=0, weight=None)) == 0


def test_backward_refusals():
    L = _lib.lib()

    def call(a, ws=None, n=0):
        return L.tide_norm_backward(ctypes.byref(a), ws, n, None)

    assert L.tide_norm_backward(None, None, 0, None) == EINVAL
    assert L.tide_norm_backward_workspace(None, None) == EINVAL
    kept = dict(x=None, x_kept=2 * AT)
    for bad in (dict(rows=-1), dict(cols=-1), dict(kind=3), dict(eps=0.0), dict(dy=None),
                dict(weight=None), dict(x=None), dict(x_kept=8 * AT), dict(lddy=95), dict(ldx=95),
                dict(lddx=95), dict(ldadd=95)):
        assert call(bwd(**bad)) == EINVAL, bad
        assert query(bwd(**bad))[0] == EINVAL, bad
    for bad in (dict(rows=(1 << 27) + 1), dict(cols=32769, lddy=40000, ldx=40000, ldadd=40000, lddx=40000),
                dict(lddy=(1 << 22) + 1), dict(lddx=(1 << 22) + 1)):
        assert call(bwd(**bad)) == EUNSUPPORTED, bad
    for bad in (dict(dy=AT + 1), dict(x=2 * AT + 1), dict(x=None, x_kept=2 * AT + 8),
                dict(weight=3 * AT + 1), dict(add=4 * AT + 1), dict(dx=5 * AT + 1),
                dict(dweight=6 * AT + 1), dict(dbias=7 * AT + 1)):
        assert call(bwd(**bad)) == EALIGN, bad
    for bad in (dict(dx=AT), dict(dx=2 * AT), dict(dx=3 * AT), dict(dx=4 * AT + 2),
                dict(dx=4 * AT, lddx=104), dict(dweight=3 * AT), dict(dweight=5 * AT),
                dict(dbias=6 * AT + 2), dict(dbias=2 * AT), dict(dx=2 * AT, **kept)):
        assert call(bwd(**bad)) == EOVERLAP, bad
    st, n = query(bwd())
    assert st == 0 and n > 0
    assert call(bwd()) == ENOSPACE and call(bwd(), 8 * AT, n - 1) == ENOSPACE
    assert call(bwd(), 8 * AT + 2, n) == EALIGN
    for a in range(1, 8):
        assert call(bwd(), a * AT, n) == EOVERLAP, a
    assert call(bwd(dx=4 * AT)) == ENOSPACE  # add in place is no overlap
    # what only an absent gradient needs may be absent; one row needs no workspace
    assert query(bwd(dx=None, weight=None, add=None))[0] == 0
    assert query(bwd(dx=None, dweight=None, weight=None, x=None))[0] == 0
    assert query(bwd(rows=1)) == (0, 0) and query(bwd(rows=0)) == (0, 0)
    assert query(bwd(dweight=None, dbias=None)) == (0, 0)
    assert call(bwd(dx=None, dweight=None, dbias=None, dy=None)) == 0
    assert call(bwd(cols=0)) == 0


def test_column_ranges_of_one_buffer_are_apart():
    L = _lib.lib()
    a = fwd(x=AT, ldx=200, y=AT + 2 * 96, ldy=200, weight=None)
    assert L.tide_norm_forward(ctypes.byref(a), None) == EINVAL  # only the weight is missing
    a = fwd(x=AT, ldx=200, y=AT + 2 * 95, ldy=200)
    assert L.tide_norm_forward(ctypes.byref(a), None) == EOVERLAP


def test_limits():
    """At the documented limits the workspace can be asked for."""
    for T, C in ((1 << 27, 1), (1 << 27, 64), (1 << 18, 32768)):
        a = bwd(rows=T, cols=C, lddy=C, ldx=C, ldadd=C, lddx=C, dy=1 << 50, x=1 << 51, add=1 << 52,
                dx=1 << 53)
        st, n = query(a)
        assert st == 0 and 0 < n < 1 << 31


def test_python_refusals():
    w = torch.zeros(64, dtype=torch.bfloat16)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TideError, match="kind is"):
        norm.Norm(w, kind="batch")
    with pytest.raises(TideError, match="expected 1"):
        norm.Norm(x)
    with pytest.raises(TypeError):
        norm.Norm(None)
    with pytest.raises(TideError, match="expected a GPU"):
        norm.Norm(w)
    with pytest.raises(TideError, match="expected a GPU"):
        api.tide_norm_forward(x, w)
    with pytest.raises(TideError, match="dtype"):
        api.tide_norm_backward(x.float())


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors taken for a GPU's (index -1); the library's calls recorded."""
    ran = []
    monkeypatch.setattr(api, "_index", lambda t, what: -1)
    monkeypatch.setattr(api, "_require", lambda t, dtype, what: None)
    monkeypatch.setattr(api, "_on_device", lambda index, stream, call, *a: ran.append(call.__name__))
    return ran


def test_what_a_norm_refuses_on_the_host(calls):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    leaf = lambda *s: bf(*s).requires_grad_()  # noqa: E731
    layer = norm.Norm(leaf(16), bias=leaf(16), weight_grad=bf(16))
    x8 = linear.Act8(4, 16, buffer=torch.zeros(200, dtype=torch.uint8))
    uses = [lambda f: layer.forward(f(4, 16)), lambda f: layer.forward(bf(4, 16), out=f(4, 16)),
            lambda f: layer.backward(f(4, 16), x8), lambda f: layer.backward(bf(4, 16), f(4, 16)),
            lambda f: layer.backward(bf(4, 16), x8, add=f(4, 16)),
            lambda f: layer.backward(bf(4, 16), x8, dx=f(4, 16)),
            lambda f: api.tide_norm_forward(f(4, 16), bf(16)),
            lambda f: api.tide_norm_backward(f(4, 16), dbias=bf(16)),
            lambda f: api.tide_norm_backward(bf(4, 16), x=f(4, 16), dweight=bf(16))]
    for use in uses:
        with pytest.raises(TideError, match="requires a gradient"):
            use(leaf)
        assert not calls
        use(bf)
        with torch.no_grad():
            use(leaf)
        assert len(calls) == 2
        calls.clear()
    bad = [("need x or its checkpoint", lambda: layer.backward(bf(4, 16))),
           ("not asked for", lambda: layer.backward(bf(4, 16), x8, add=bf(4, 16), input_grad=False)),
           ("not asked for", lambda: layer.backward(bf(4, 16), x8, dx=bf(4, 16), input_grad=False)),
           ("checkpoint of .4, 16., expected .5, 16.", lambda: layer.backward(bf(5, 16), x8)),
           ("expected .4, 16.", lambda: layer.forward(bf(4, 17))),
           ("one of them", lambda: api.tide_norm_backward(bf(4, 16), x=bf(4, 16),
                                                          x_kept=torch.zeros(200, dtype=torch.uint8))),
           ("needs the weight", lambda: api.tide_norm_backward(bf(4, 16), x=bf(4, 16), dx=True)),
           ("not asked for", lambda: api.tide_norm_backward(bf(4, 16), add=bf(4, 16), dbias=bf(16))),
           ("need x or", lambda: api.tide_norm_backward(bf(4, 16), weight=bf(16), dx=True))]
    for text, use in bad:
        with pytest.raises(TideError, match=text):
            use()
    assert not calls


@pytest.mark.parametrize("kind", list(api.NORMS))
def test_reference_against_torch(kind):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, 45, generator=g, dtype=torch.float64) * 3 + 1
    w, b = torch.randn(45, generator=g, dtype=torch.float64), torch.randn(45, generator=g, dtype=torch.float64)
    want = (torch.nn.functional.layer_norm(x, (45,), w, b, 1e-3) if kind == "layer"
            else torch.nn.functional.rms_norm(x, (45,), w, 1e-3) + b)
    y, e = ref.forward_ref(x, w, b, kind, 1e-3)
    assert (y - want).abs().max() < 1e-12 and (e > 0).all()
    assert e.max() < 1e-4


@pytest.mark.parametrize("kind", list(api.NORMS))
def test_reference_gradients_against_differences(kind):
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy, add = rand(5, 11) + 0.5, rand(11), rand(11), rand(5, 11), rand(5, 11)
    out = ref.backward_ref(dy, w, x, add, kind, 1e-2)
    h = 1e-6

    def loss(x, w, b):
        return (ref.forward_ref(x, w, b, kind, 1e-2)[0] * dy).sum() + (x * add).sum()

    for name, at, k in (("dx", x, 0), ("dw", w, 1), ("db", b, 2)):
        for i in range(0, at.numel(), 3):
            t = [x.clone(), w.clone(), b.clone()]
            t[k].view(-1)[i] += h
            up = loss(*t)
            t[k].view(-1)[i] -= 2 * h
            want = (up - loss(*t)) / (2 * h)
            assert abs(out[name][0].view(-1)[i] - want) < 1e-7, (name, i)
