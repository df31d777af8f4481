"""CPU tests of what linear.py and the flat calls decide on the host: the
device of a call, its stream, what they refuse.  No device is touched: the
library's calls and torch's device contexts are replaced by recorders."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from shard_placement_amd import api, linear
from shard_placement_amd._lib import TideError


@pytest.fixture
def no_gpu(monkeypatch):
    """Device 0 is current; entering a device or a stream changes nothing."""
    entered = []

    def enter(what):
        @contextlib.contextmanager
        def ctx(v):
            entered.append((what, v))
            yield
        return ctx

    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", enter("device"))
    monkeypatch.setattr(torch.cuda, "stream", enter("stream"))
    return entered


def stream(index, handle=77):
    return SimpleNamespace(device_index=index, cuda_stream=handle)


def test_stream_of_a_call(no_gpu):
    call = lambda s, *a: (s, a)  # noqa: E731
    assert api._on_device(0, None, call, 5) == (1000, (5,)) and not no_gpu
    assert api._on_device(1, None, call) == (1001, ()) and no_gpu == [("device", 1)]
    s = stream(0)
    assert api._on_device(0, s, call) == (77, ()) and no_gpu[1:] == [("device", 0), ("stream", s)]


@pytest.mark.parametrize("handle", [0, 77])  # 0: another device's null stream
def test_stream_of_another_device_is_refused(no_gpu, handle):
    ran = []
    for index, other in ((0, 1), (1, 0)):
        with pytest.raises(TideError, match="stream belongs to cuda:%d" % other) as e:
            api._on_device(index, stream(other, handle), ran.append)
        assert e.value.status == -1
    assert not ran and not no_gpu


@pytest.mark.parametrize("device", [0, 1, "cuda:1", torch.device("cuda", 0), None])
def test_device_of_a_new_checkpoint(monkeypatch, device):
    """Device 0 by its index is device 0, not the current one."""
    asked, empty = [], torch.empty

    def record(*shape, device=None, **kw):
        asked.append(device)
        return empty(*shape, **kw)

    monkeypatch.setattr(torch, "empty", record)
    linear.Act8(3, 40, device=device)
    assert asked == ["cuda" if device is None else device]


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors taken for a GPU's (index -1); the library's calls recorded."""
    ran = []
    monkeypatch.setattr(api, "_index", lambda t, what: -1)
    monkeypatch.setattr(api, "_require", lambda t, dtype, what: None)
    monkeypatch.setattr(api, "_on_device", lambda index, stream, call, *a: ran.append(call.__name__))
    return ran


def test_tensors_of_an_autograd_graph_are_refused(calls):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    leaf = lambda *s: bf(*s).requires_grad_()  # noqa: E731
    layer = linear.Linear(leaf(8, 16), bias=leaf(8))  # their gradients have places of their own
    uses = [lambda f: layer.forward(f(4, 16)), lambda f: layer.forward(bf(4, 16), residual=f(4, 8)),
            lambda f: layer.forward(bf(4, 16), out=f(4, 8)), lambda f: layer.backward(f(4, 8)),
            lambda f: layer.backward(bf(4, 8), dx=f(4, 16)),
            lambda f: api.tide_linear_forward(f(4, 16), bf(8, 16)),
            lambda f: api.tide_linear_forward(bf(4, 16), bf(8, 16), residual=f(4, 8)),
            lambda f: api.tide_linear_backward(f(4, 8), 16, dbias=bf(8))]
    for use in uses:
        with pytest.raises(TideError, match="requires a gradient") as e:
            use(leaf)
        assert e.value.status == -6 and not calls
        for plain in (bf, lambda *s: leaf(*s).detach()):
            use(plain)
        with torch.no_grad():
            use(leaf)
        assert len(calls) == 3
        calls.clear()


def test_inside_an_autograd_function(calls):
    """Grad mode is off in a Function's forward and backward."""
    layer = linear.Linear(torch.zeros(8, 16, dtype=torch.bfloat16))

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            layer.forward(x)
            return x[:, :8] * 2

        @staticmethod
        def backward(ctx, dy):
            layer.backward(dy)
            return torch.cat([dy, dy], 1)

    x = torch.zeros(4, 16, dtype=torch.bfloat16, requires_grad=True)
    (Product.apply(x) * 3).sum().backward()
    assert calls == ["_forward_on", "_backward_on"]
