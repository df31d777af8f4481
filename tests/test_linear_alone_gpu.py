"""GPU tests of each gradient alone with an activation, through Linear and
through the flat calls on raw checkpoints, against tests/linear_ref.py."""
import math

import pytest
import torch

from shard_placement_amd import api
from shard_placement_amd.linear import Linear
from tests import linear_ref as ref
from tests.test_linear_gpu import BF, DEV, gen, kept_of, normal, within

pytestmark = pytest.mark.gpu

# One token, a few (whose column sums are one chunk's), the first number of
# tokens past one chunk, many; odd widths; narrow and 256-wide tiles.
SHAPES = [(1, 8, 40), (5, 33, 70), (64, 257, 96), (65, 129, 128), (130, 264, 72), (700, 1001, 333),
          (2500, 1550, 260), (1300, 1000, 4001)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_gradients_alone_with_an_activation(T, N, K, act):
    g = gen(T + 3 * N + 5 * K)
    w, dy = normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, T, N, scale=1e-3)
    x8, x = kept_of(torch.randn(T, K, generator=g, device=DEV))
    z8, z = kept_of(3 * torch.randn(T, N, generator=g, device=DEV))
    want = ref.backward_ref(dy, w, x, z, act)
    for flat in (False, True):
        dw, db = torch.full_like(w, 9), torch.full((N,), 9.0, dtype=BF, device=DEV)
        if flat:
            dx = torch.full((T, K), 9.0, dtype=BF, device=DEV)
            kept = dict(z_kept=z8.buffer, act=act)
            assert api.tide_linear_backward(dy, K, weight=w, dx=dx, **kept) is dx
            assert api.tide_linear_backward(dy, K, x_kept=x8.buffer, dweight=dw, **kept) is None
            assert api.tide_linear_backward(dy, K, dbias=db, **kept) is None
        else:
            dx = Linear(w, act=act).backward(dy, z=z8)
            assert Linear(w, act=act, weight_grad=dw).backward(dy, x=x8, z=z8, input_grad=False) is None
            assert Linear(w, act=act, bias_grad=db).backward(dy, z=z8, input_grad=False) is None
        for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
            within(got, *want[name], "%s, flat %r" % (name, flat))


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_dbias_alone_without_an_activation(T, N, K):
    g = gen(T + N)
    dy = normal(g, T, N)
    db = torch.full((N,), 9.0, dtype=BF, device=DEV)
    assert Linear(torch.zeros(N, 8, dtype=BF, device=DEV), bias_grad=db).backward(dy, input_grad=False) is None
    want = dy.double().sum(0)
    e = (T + 8) * ref.F32 * dy.double().abs().sum(0)
    within(db, want, e + ref.BF16 * (want.abs() + e), "db")


@pytest.mark.parametrize("T,N,K", [(1, 40, 64), (20, 300, 264), (300, 129, 72)])
@pytest.mark.parametrize("act", list(api.ACTS))
def test_flat_forward_and_all_gradients(T, N, K, act):
    """The flat calls with everything they take; dx=True allocates it."""
    g = gen(T + N + K)
    x, w, b, r = normal(g, T, K), normal(g, N, K, scale=1 / math.sqrt(K)), normal(g, N), normal(g, T, N)
    z8 = torch.full((api.tide_act8_bytes(T, N),), 0xEE, dtype=torch.uint8, device=DEV)
    x8 = torch.full((api.tide_act8_bytes(T, K),), 0xEE, dtype=torch.uint8, device=DEV)
    api.tide_act8_pack(x, x8)
    y = api.tide_linear_forward(x, w, bias=b, residual=r, act=act, z_kept=z8)
    want, _, _, bound = ref.forward_ref(x, w, b, r, act)
    within(y, want, bound, "y")
    out = torch.empty_like(y)
    assert api.tide_linear_forward(x, w, y=out, bias=b, residual=r, act=act) is out
    within(out, want, bound, "y into out")

    def values(kept, cols):
        pitch = -(-cols // 32) * 32
        return ref.unpack_ref(kept[:T * pitch].view(T, pitch), kept[T * pitch:].view(T, pitch // 32), cols)

    back = torch.empty_like(x)
    api.tide_act8_unpack(x8, back)
    assert torch.equal(back.double(), values(x8, K))
    dy = normal(g, T, N, scale=1e-3)
    dw, db = torch.full_like(w, 9), torch.full_like(b, 9)
    dx = api.tide_linear_backward(dy, K, weight=w, x_kept=x8, z_kept=z8, act=act, dx=True, dweight=dw, dbias=db)
    grads = ref.backward_ref(dy, w, values(x8, K), values(z8, N), act)
    for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
        within(got, *grads[name], name)
