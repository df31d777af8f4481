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
