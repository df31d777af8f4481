"""A layer's products around the collectives, with activations kept in 8 bits.

FSDP2 places a layer's weights, runs the layer and reduce-scatters its
gradients (Abstract of "The Endgame of FSDP Communication",
weekinpapers.com).  ``Linear`` is one product of that layer: its weight is a
full tensor that the placement writes (``Setup.full[p]``), its gradients are
tensors that the reduce-scatter reads (``Setup.grads[q][p]``).  ``Act8`` is
what it keeps between the passes: an activation in 8 bits, in memory of its own
or in the caller's, e.g. a vacated gathered buffer.

    x8, z8 = Act8(T, K, device=dev), Act8(T, N, device=dev)
    layer = Linear(full[p], act="silu", weight_grad=grads[q][p])
    x8.pack(x)
    y = layer.forward(x, z=z8)              # y = silu(x W^T), z kept in 8 bits
    dx = layer.backward(dy, x=x8, z=z8)     # writes grads[q][p]

All work is done by the library (``include/tide.h``); this module only holds
tensors together.  Autograd records none of it: ``backward`` is the gradient, a
weight's goes to ``weight_grad`` and never to ``weight.grad``, and activations
that require a gradient are refused in grad mode.  In a
``torch.autograd.Function`` grad mode is off, so its forward and backward can
call these as they are.

``stream`` (default: the current one of the tensors' device) is a stream of
that device.  What a call allocates belongs to it; the caller orders it against
other streams and keeps the tensors alive until its work is done.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import api
from ._lib import TideError, TideLinearBackwardArgs, TideLinearForwardArgs

BLOCK = 32  # columns of a checkpoint that share a scale


class Act8:
    """The 8-bit checkpoint of a [rows, cols] bf16 matrix.

    ``buffer``: a contiguous GPU tensor of any type with at least
    ``Act8.bytes(rows, cols)`` bytes, 16-byte aligned; allocated on ``device``
    when not given.  ``data`` (e4m3, [rows, cols rounded up to 32]) and
    ``scales`` (e8m0, one for 32 columns) are views of it."""

    def __init__(self, rows: int, cols: int, buffer: Optional[torch.Tensor] = None, device=None):
        self.rows, self.cols = int(rows), int(cols)
        need = self.bytes(self.rows, self.cols)
        if buffer is None:
            buffer = torch.empty(need, dtype=torch.uint8, device="cuda" if device is None else device)
        if not buffer.is_contiguous():
            raise TideError(-6, "buffer is not contiguous")
        flat = buffer.view(-1).view(torch.uint8)
        if flat.numel() < need:
            raise TideError(-1, "buffer holds %d bytes, need %d" % (flat.numel(), need))
        self.buffer = flat[:need]
        self._gpu = buffer.get_device()  # -1: not a GPU
        pitch = -(-self.cols // BLOCK) * BLOCK
        values = self.rows * pitch
        self.data = self.buffer[:values].view(torch.float8_e4m3fn).view(self.rows, pitch)
        self.scales = self.buffer[values:].view(torch.float8_e8m0fnu).view(self.rows, pitch // BLOCK)

    @staticmethod
    def bytes(rows: int, cols: int) -> int:
        return api.tide_act8_bytes(rows, cols)

    def pack(self, x: torch.Tensor, stream=None) -> "Act8":
        """Write the checkpoint of the bf16 matrix x."""
        px, ldx = self._matrix(x, "x")
        api._on_device(self._gpu, stream, api._pack_on, px, ldx, self.rows, self.cols,
                       self.buffer.data_ptr())
        return self

    def unpack(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The bf16 matrix that the checkpoint stands for (allocated when not given)."""
        if self._gpu < 0:
            raise TideError(-6, "the checkpoint is on %s, expected a GPU" % self.buffer.device)
        if out is None:
            return api._on_device(self._gpu, stream, self._unpack_new)
        px, ldx = self._matrix(out, "out")
        api._on_device(self._gpu, stream, api._unpack_on, self.buffer.data_ptr(), self.rows,
                       self.cols, px, ldx)
        return out

    def _unpack_new(self, s):
        out = torch.empty(self.rows, self.cols, dtype=torch.bfloat16, device=self.buffer.device)
        api._unpack_on(s, self.buffer.data_ptr(), self.rows, self.cols, out.data_ptr(), self.cols)
        return out

    def _matrix(self, t, what):
        if not isinstance(t, torch.Tensor) or t.shape != (self.rows, self.cols):
            raise TideError(-1, "%s is %s, expected [%d, %d]"
                            % (what, list(getattr(t, "shape", ())), self.rows, self.cols))
        if api._index(t, what) != self._gpu:
            raise TideError(-6, "%s is on %s, the checkpoint on %s"
                            % (what, t.device, self.buffer.device))
        return api._rows(t, what)

    def _of(self, rows: int, cols: int, gpu: int, what: str) -> int:
        """The address, as the checkpoint of a [rows, cols] matrix on this GPU."""
        if self.rows != rows or self.cols != cols:
            raise TideError(-1, "%s is a checkpoint of [%d, %d], expected [%d, %d]"
                            % (what, self.rows, self.cols, rows, cols))
        if self._gpu != gpu:
            raise TideError(-6, "%s is on %s, expected cuda:%d" % (what, self.buffer.device, gpu))
        return self.buffer.data_ptr()


class Linear:
    """y = act(x weight^T + bias) + residual and its gradients.

    weight [N, K], bias [N]: contiguous bf16 GPU tensors; weight_grad and
    bias_grad, where given, receive the gradients (overwritten by every
    backward).  act: "none", "relu", "gelu", "gelu_tanh" or "silu".  The four
    tensors are checked here and kept; calls use their memory as it is then."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 act: str = "none", weight_grad: Optional[torch.Tensor] = None,
                 bias_grad: Optional[torch.Tensor] = None):
        self._act = api._act(act)
        self._gpu = api._index(weight, "weight")
        self._shape = N, K = tuple(weight.shape)
        for t, shape, what in ((weight, (N, K), "weight"), (bias, (N,), "bias"),
                               (weight_grad, (N, K), "weight_grad"), (bias_grad, (N,), "bias_grad")):
            if t is not None:
                api._whole(t, shape, what, self._gpu)
        self._weight, self._bias, self.act = weight, bias, act
        self._weight_grad, self._bias_grad = weight_grad, bias_grad

    weight = property(lambda self: self._weight)
    bias = property(lambda self: self._bias)
    weight_grad = property(lambda self: self._weight_grad)
    bias_grad = property(lambda self: self._bias_grad)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, z: Optional[Act8] = None,
                stream=None) -> torch.Tensor:
        """z: the checkpoint that receives act's argument (which backward
        needs unless act is "none").  out is allocated when not given."""
        N, K = self._shape
        gpu = self._gpu
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() else 0
        px, ldx = api._matrix(x, T, K, "x", gpu)
        a = TideLinearForwardArgs(T, N, K, self._act, 0, px, ldx, self._weight.data_ptr())
        if self._bias is not None:
            a.bias = self._bias.data_ptr()
        if residual is not None:
            a.residual, a.ldr = api._matrix(residual, T, N, "residual", gpu)
        if out is not None:
            a.y, a.ldy = api._matrix(out, T, N, "out", gpu)
        if z is not None:
            a.z_kept = z._of(T, N, gpu, "z")
        return api._on_device(gpu, stream, api._forward_on, a, out, gpu)

    def backward(self, dy: torch.Tensor, x: Optional[Act8] = None, z: Optional[Act8] = None,
                 dx: Optional[torch.Tensor] = None, input_grad: bool = True,
                 stream=None) -> Optional[torch.Tensor]:
        """Writes weight_grad and bias_grad (where the layer has them) and
        returns dx (None with input_grad=False).  x: the checkpoint of
        forward's x, z: the one forward wrote.  The residual's gradient is dy."""
        N, K = self._shape
        gpu = self._gpu
        T = dy.shape[0] if isinstance(dy, torch.Tensor) and dy.dim() else 0
        pdy, lddy = api._matrix(dy, T, N, "dy", gpu)
        a = TideLinearBackwardArgs(T, N, K, self._act, 0, pdy, lddy)
        if self._act:
            if z is None:
                raise TideError(-1, "act %r needs the checkpoint of its argument" % self.act)
            a.z_kept = z._of(T, N, gpu, "z")
        if input_grad:
            a.weight = self._weight.data_ptr()
            if dx is None:
                dx = True
            else:
                a.dx, a.lddx = api._matrix(dx, T, K, "dx", gpu)
        else:
            dx = None
        if self._weight_grad is not None:
            if x is None:
                raise TideError(-1, "weight_grad needs the checkpoint of x")
            a.x_kept = x._of(T, K, gpu, "x")
            a.dweight = self._weight_grad.data_ptr()
        if self._bias_grad is not None:
            a.dbias = self._bias_grad.data_ptr()
        return api._on_device(gpu, stream, api._backward_on, a, dx, gpu)
