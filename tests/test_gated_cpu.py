"""CPU tests of the gated block: refusals (none reaches the GPU), workspaces,
the rules that choose its launches, and the reference in tests/gated_ref.py
against differences."""
import ctypes
import random

import pytest
import torch

from shard_placement_amd import _lib, api, gated, linear
from shard_placement_amd._lib import TideError, TideGatedBackwardArgs, TideGatedForwardArgs
from tests import gated_ref as ref
from tests import gated_rules as rules

EINVAL, EALIGN, EOVERLAP, ENOSPACE, EUNSUPPORTED = -1, -2, -3, -4, -6
AT = 1 << 30  # made-up device addresses, far apart


def fwd(**kw):
    a = TideGatedForwardArgs()
    a.tokens, a.out_features, a.in_features, a.act = 40, 64, 96, api.ACTS["silu"]
    a.x, a.ldx, a.gate, a.up, a.h, a.ldh = AT, 96, 2 * AT, 3 * AT, 4 * AT, 64
    a.g_kept, a.u_kept, a.h_kept, a.gate_bias, a.up_bias = 5 * AT, 6 * AT, 7 * AT, 8 * AT, 9 * AT
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def bwd(**kw):
    a = TideGatedBackwardArgs()
    a.tokens, a.out_features, a.in_features, a.act = 40, 64, 96, api.ACTS["silu"]
    a.dh, a.lddh, a.gate, a.up, a.x_kept, a.g_kept, a.u_kept = AT, 64, 2 * AT, 3 * AT, 4 * AT, 5 * AT, 6 * AT
    a.dx, a.lddx, a.dgate, a.dup, a.dgate_bias, a.dup_bias = 7 * AT, 96, 8 * AT, 9 * AT, 10 * AT, 11 * AT
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def query(name, args):
    n = ctypes.c_size_t(12345)
    st = getattr(_lib.lib(), name)(ctypes.byref(args), ctypes.byref(n))
    return st, n.value


def test_forward_refusals():
    L = _lib.lib()

    def call(a, ws=None, n=0):
        return L.tide_gated_forward(ctypes.byref(a), ws, n, None)

    assert L.tide_gated_forward(None, None, 0, None) == EINVAL
    assert L.tide_gated_forward_workspace(None, None) == EINVAL
    for bad in (dict(tokens=-1), dict(out_features=-1), dict(in_features=-1), dict(act=5), dict(act=-1),
                dict(reserved=1), dict(x=None), dict(gate=None), dict(up=None), dict(h=None),
                dict(ldx=95), dict(ldh=63)):
        assert call(fwd(**bad)) == EINVAL, bad
        assert query("tide_gated_forward_workspace", fwd(**bad))[0] == EINVAL, bad
    for bad in (dict(tokens=1 << 31), dict(out_features=(1 << 21) + 1, ldh=1 << 22),
                dict(in_features=(1 << 22) + 1, ldx=1 << 23), dict(ldx=(1 << 22) + 1),
                dict(tokens=(1 << 26) + 1), dict(tokens=1 << 20, out_features=4097, ldh=4097)):
        assert call(fwd(**bad)) == EUNSUPPORTED, bad
    for bad in (dict(x=AT + 1), dict(gate=2 * AT + 1), dict(up=3 * AT + 1), dict(h=4 * AT + 1),
                dict(g_kept=5 * AT + 8), dict(u_kept=6 * AT + 1), dict(h_kept=7 * AT + 4),
                dict(gate_bias=8 * AT + 1), dict(up_bias=9 * AT + 1)):
        assert call(fwd(**bad)) == EALIGN, bad
    for bad in (dict(h=AT), dict(h=2 * AT + 64), dict(h=3 * AT), dict(h=AT + 40 * 96 * 2 - 2),
                dict(g_kept=4 * AT + 16), dict(u_kept=5 * AT), dict(h_kept=6 * AT), dict(h_kept=AT),
                dict(gate_bias=4 * AT + 2), dict(up_bias=5 * AT)):
        assert call(fwd(**bad)) == EOVERLAP, bad
    # the two weights may be one matrix
    st, n = query("tide_gated_forward_workspace", fwd(up=2 * AT, ldx=97))
    assert st == 0 and n >= 40 * 96 * 2 and call(fwd(up=2 * AT, ldx=97)) == ENOSPACE
    assert call(fwd(tokens=0)) == 0 and call(fwd(out_features=0)) == 0
    assert call(fwd(ldx=97), 12 * AT, n - 1) == ENOSPACE
    assert call(fwd(ldx=97), 12 * AT + 8, n) == EALIGN
    for a in range(1, 10):
        assert call(fwd(ldx=97), a * AT, n) == EOVERLAP, a


def test_backward_refusals():
    L = _lib.lib()

    def call(a, ws=None, n=0):
        return L.tide_gated_backward(ctypes.byref(a), ws, n, None)

    assert L.tide_gated_backward(None, None, 0, None) == EINVAL
    for bad in (dict(tokens=-1), dict(act=9), dict(reserved=2), dict(dh=None), dict(gate=None),
                dict(up=None), dict(x_kept=None), dict(g_kept=None), dict(u_kept=None), dict(lddh=63),
                dict(lddx=95), dict(dgate=None), dict(dup=None)):
        assert call(bwd(**bad)) == EINVAL, bad
        assert query("tide_gated_backward_workspace", bwd(**bad))[0] == EINVAL, bad
    for bad in (dict(dh=AT + 1), dict(gate=2 * AT + 1), dict(up=3 * AT + 1), dict(x_kept=4 * AT + 8),
                dict(g_kept=5 * AT + 4), dict(u_kept=6 * AT + 4), dict(dx=7 * AT + 1),
                dict(dgate=8 * AT + 1), dict(dup=9 * AT + 1), dict(dgate_bias=10 * AT + 1),
                dict(dup_bias=11 * AT + 1)):
        assert call(bwd(**bad)) == EALIGN, bad
    for bad in (dict(dx=AT), dict(dgate=2 * AT), dict(dup=3 * AT), dict(dup=8 * AT),
                dict(dgate_bias=4 * AT), dict(dx=8 * AT), dict(dup_bias=10 * AT + 2), dict(dgate=5 * AT),
                dict(dup=6 * AT)):
        assert call(bwd(**bad)) == EOVERLAP, bad
    assert call(bwd(tokens=1 << 31)) == EUNSUPPORTED
    st, n = query("tide_gated_backward_workspace", bwd())
    assert st == 0 and n > 0
    assert call(bwd()) == ENOSPACE and call(bwd(), 12 * AT, n - 1) == ENOSPACE
    assert call(bwd(), 12 * AT + 2, n) == EALIGN
    for a in range(1, 12):
        assert call(bwd(), a * AT, n) == EOVERLAP, a
    # what only an absent gradient needs may be absent
    for ok in (dict(dx=None, gate=None, up=None), dict(dgate=None, dup=None, x_kept=None),
               dict(dgate_bias=None), dict(dup_bias=None), dict(gate=2 * AT, up=2 * AT)):
        assert query("tide_gated_backward_workspace", bwd(**ok))[0] == 0, ok
    none = dict(dx=None, dgate=None, dup=None, dgate_bias=None, dup_bias=None, dh=None)
    assert call(bwd(**none)) == 0


def test_limits():
    """At the documented limits the workspace can be asked for."""
    far = dict(gate=1 << 50, up=1 << 51, gate_bias=None, up_bias=None)
    for T, N, K, want in ((1 << 30, 1, 1, 0), ((1 << 30) + 1, 1, 1, EUNSUPPORTED), (4, 1 << 21, 1024, 0),
                          (2048, 1 << 21, 8, 0), (8, 8, 1 << 22, 0)):
        a = fwd(tokens=T, out_features=N, in_features=K, x=1 << 52, ldx=K, h=1 << 53, ldh=N, g_kept=1 << 54,
                u_kept=1 << 55, h_kept=1 << 56, **far)
        assert query("tide_gated_forward_workspace", a)[0] == want
        b = bwd(tokens=T, out_features=N, in_features=K, dh=1 << 52, lddh=N, dx=1 << 53, lddx=K,
                x_kept=1 << 54, g_kept=1 << 55, u_kept=1 << 56, dgate=1 << 57, dup=1 << 58,
                dgate_bias=1 << 59, dup_bias=1 << 60, gate=1 << 50, up=1 << 51)
        assert query("tide_gated_backward_workspace", b)[0] == want


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors taken for a GPU's (index -1); the library's calls recorded."""
    ran = []
    monkeypatch.setattr(api, "_index", lambda t, what: -1)
    monkeypatch.setattr(api, "_require", lambda t, dtype, what: None)
    monkeypatch.setattr(api, "_on_device", lambda index, stream, call, *a: ran.append(call.__name__))
    return ran


def test_what_a_block_refuses_on_the_host(calls):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    leaf = lambda *s: bf(*s).requires_grad_()  # noqa: E731
    act8 = lambda r, c: linear.Act8(r, c, buffer=torch.zeros(400, dtype=torch.uint8))  # noqa: E731
    block = gated.Gated(leaf(8, 16), leaf(8, 16), gate_bias=leaf(8))
    x8, g8, u8 = act8(4, 16), act8(4, 8), act8(4, 8)
    raw = torch.zeros(400, dtype=torch.uint8)
    uses = [lambda f: block.forward(f(4, 16)), lambda f: block.forward(bf(4, 16), out=f(4, 8)),
            lambda f: block.backward(f(4, 8), g=g8, u=u8),
            lambda f: block.backward(bf(4, 8), g=g8, u=u8, dx=f(4, 16)),
            lambda f: api.tide_gated_forward(f(4, 16), bf(8, 16), bf(8, 16)),
            lambda f: api.tide_gated_backward(f(4, 8), 16, raw, raw, dgate_bias=bf(8))]
    for use in uses:
        with pytest.raises(TideError, match="requires a gradient"):
            use(leaf)
        assert not calls
        use(bf)
        with torch.no_grad():
            use(leaf)
        assert len(calls) == 2
        calls.clear()
    train = gated.Gated(bf(8, 16), bf(8, 16), gate_grad=bf(8, 16), up_grad=bf(8, 16))
    bad = [("act is", lambda: gated.Gated(bf(8, 16), bf(8, 16), act="swish")),
           ("up is .8, 17., expected .8, 16.", lambda: gated.Gated(bf(8, 16), bf(8, 17))),
           ("computed together", lambda: gated.Gated(bf(8, 16), bf(8, 16), up_grad=bf(8, 16))),
           ("checkpoints of g and u", lambda: block.backward(bf(4, 8), g=g8)),
           ("checkpoints of g and u", lambda: block.backward(bf(4, 8), u=u8)),
           ("checkpoint of .4, 16., expected .4, 8.", lambda: block.backward(bf(4, 8), g=x8, u=u8)),
           ("need the checkpoint of x", lambda: train.backward(bf(4, 8), g=g8, u=u8)),
           ("not asked for", lambda: block.backward(bf(4, 8), g=g8, u=u8, dx=bf(4, 16), input_grad=False)),
           ("expected .4, 16.", lambda: block.forward(bf(4, 15))),
           ("checkpoint of .4, 8., expected .5, 8.", lambda: block.forward(bf(5, 16), h=g8)),
           ("needs gate and up", lambda: api.tide_gated_backward(bf(4, 8), 16, raw, raw, dx=True)),
           ("computed together", lambda: api.tide_gated_backward(bf(4, 8), 16, raw, raw, dup=bf(8, 16))),
           ("checkpoint of x", lambda: api.tide_gated_backward(bf(4, 8), 16, raw, raw, dgate=bf(8, 16),
                                                               dup=bf(8, 16)))]
    for text, use in bad:
        with pytest.raises(TideError, match=text):
            use()
    assert not calls


def test_cpu_tensors_are_refused():
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(TideError, match="expected a GPU"):
        gated.Gated(w, w)
    with pytest.raises(TideError, match="expected a GPU"):
        api.tide_gated_forward(w, w, w)
    with pytest.raises(TypeError):
        gated.Gated(None, w)


# ---- the rules ---------------------------------------------------------------------------------

def drawn(n, seed):
    rng = random.Random(seed)
    size = lambda hi: int(round(hi ** rng.random()))  # noqa: E731
    return [(size(16384), size(30000), size(30000)) for _ in range(n)]


def threads(s):
    return 512 if s.bi == 256 or (s.halves == 2 and s.bj > 16) else 256


def test_every_choice_is_a_form_and_covers_the_product():
    """What is chosen is compiled: 256-wide tiles, 128 x 128 ones, rings of 128
    contraction elements for up to 64 tokens, and tiles of 256 of them for weights
    past the cache; a split is a whole number of their steps."""
    for T, N, K in drawn(20000, 3):
        I, depth = rules.rows(N), rules.round8(K)
        s = rules.choose(I, T, depth)
        assert (s.tiles_i - 1) * s.bi < I <= s.tiles_i * s.bi
        assert (s.tiles_j - 1) * s.bj < T <= s.tiles_j * s.bj
        assert (s.splits - 1) * s.split_depth < depth <= s.splits * s.split_depth
        assert s.split_depth % 256 == 0
        form = (s.bi, s.bj, s.bk, s.halves)
        if T <= 64:
            assert form in {(128, 16, 128, 2), (128, 32, 128, 2), (128, 64, 128, 2), (128, 32, 256, 1)}
        else:
            assert form in {(256, 256, 64, 1), (256, 192, 64, 1), (256, 128, 64, 1), (128, 128, 64, 1),
                            (128, 128, 64, 2)}


def test_few_tokens_go_by_the_weights_rows():
    by_rows = lambda *a, **kw: rules.forward(*a, **kw) is None  # noqa: E731
    assert all(by_rows(1, N, K) for N in (1, 64, 28672) for K in (8, 512, 28672))
    assert all(by_rows(T, 64, 1001) for T in (1, 2, 3, 4))  # weights that rings would copy
    assert by_rows(2, 1024, 8192) and by_rows(2, 128, 512) and not by_rows(2, 14336, 1024)
    for case in ((3, 28672, 8192), (4, 64, 1024), (5, 64, 1001), (1, 8, 7)):
        assert not by_rows(*case), case
    assert not by_rows(1, 28672, 8192, keep=True)


def test_splits_of_few_tokens():
    for T, N, K, splits in ((16, 4096, 4096, 2), (5, 1001, 8192, 8), (64, 1001, 8192, 8), (24, 768, 2048, 4),
                            (24, 13824, 5120, 1), (40, 768, 1000, 1), (30, 28672, 8192, 1)):
        assert rules.forward(T, N, K, keep=True).splits == splits, (T, N, K)
    assert rules.forward(30, 28672, 8192).bk == 256 and rules.forward(30, 13824, 5120).bk == 128
    assert rules.forward(40, 28672, 8192).bk == 128


def test_the_inputs_gradient_is_split_beside_the_weights():
    """dx's few long tiles in splits, in one launch with the weights' gradients."""
    for T, N, K, pair in ((1003, 13824, 5120, True), (700, 28672, 8192, True), (4096, 28672, 8192, False)):
        x, w, joint, first = rules.gradients(T, N, K)
        assert joint == pair and (not pair or (x.splits > 1 and w.splits == 1 and first))


def test_every_launch_is_tested():
    """No launch that random sizes take is missing from the GPU tests' lists."""
    from tests.test_gated_gpu import FORMS, PAST_THE_CACHE, PRODUCTS

    covered = set().union(*(rules.forms(*s) for s in PRODUCTS + FORMS))
    covered |= {f for s in PAST_THE_CACHE for f in rules.forms(*s) if f[0].startswith("forward")}
    missing = {}
    for s in drawn(60000, 8):
        for f in rules.forms(*s) - covered:
            missing.setdefault(f, s)
    assert not missing, missing


def test_grids_fit_at_the_limits():
    elements = 1 << 33
    for I in [1 << k for k in range(5, 23)]:
        for T in [1 << k for k in range(0, 31)] + [(1 << 30) - 1]:
            for depth in (8, 64, 4096, 1 << 22):
                if I * T > max(elements, 32 * T) or max(I, T) * depth > elements:
                    continue
                s = rules.choose(I, T, depth)
                assert s.tiles_i * s.tiles_j * s.splits * threads(s) < 1 << 32, (I, T, depth, s)


# ---- the reference -----------------------------------------------------------------------------

@pytest.mark.parametrize("act", list(api.ACTS))
def test_reference_gradients_against_differences(act):
    g = torch.Generator().manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, N, K = 4, 6, 5
    parts = {"x": rand(T, K), "wg": rand(N, K), "wu": rand(N, K), "bg": rand(N), "bu": rand(N)}
    dh, h = rand(T, N), 1e-6

    def loss(p):
        return (ref.forward_ref(p["x"], p["wg"], p["wu"], p["bg"], p["bu"], act)["h"][0] * dh).sum()

    f = ref.forward_ref(*parts.values(), act)
    out = ref.backward_ref(dh, parts["wg"], parts["wu"], parts["x"], f["g"][0], f["u"][0], act)
    for name, of in (("dx", "x"), ("dwg", "wg"), ("dwu", "wu"), ("dbg", "bg"), ("dbu", "bu")):
        for i in range(parts[of].numel()):
            p = {k: v.clone() for k, v in parts.items()}
            p[of].view(-1)[i] += h
            up = loss(p)
            p[of].view(-1)[i] -= 2 * h
            want = (up - loss(p)) / (2 * h)
            assert abs(out[name][0].reshape(-1)[i] - want) < 1e-6, (name, i)
