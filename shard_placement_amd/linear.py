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
tensors together.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import api
from ._lib import TideError

_nothing = contextlib.nullcontext()
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
            buffer = torch.empty(need, dtype=torch.uint8, device=device or "cuda")
        if not buffer.is_contiguous():
            raise TideError(-6, "buffer is not contiguous")
        flat = buffer.view(-1).view(torch.uint8)
        if flat.numel() < need:
            raise TideError(-1, "buffer holds %d bytes, need %d" % (flat.numel(), need))
        self.buffer = flat[:need]
        pitch = -(-self.cols // BLOCK) * BLOCK
        values = self.rows * pitch
        self.data = self.buffer[:values].view(torch.float8_e4m3fn).view(self.rows, pitch)
        self.scales = self.buffer[values:].view(torch.float8_e8m0fnu).view(self.rows, pitch // BLOCK)

    @staticmethod
    def bytes(rows: int, cols: int) -> int:
        return api.tide_act8_bytes(rows, cols)

    def pack(self, x: torch.Tensor, stream=None) -> "Act8":
        if x.shape != (self.rows, self.cols):
            raise TideError(-1, "x is %s, expected [%d, %d]" % (list(x.shape), self.rows, self.cols))
        api.tide_act8_pack(x, self.buffer, stream)
        return self

    def unpack(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if out is None:
            with torch.cuda.stream(stream) if stream is not None else _nothing:
                out = torch.empty(self.rows, self.cols, dtype=torch.bfloat16,
                                  device=self.buffer.device)
        elif out.shape != (self.rows, self.cols):
            raise TideError(-1, "out is %s, expected [%d, %d]"
                            % (list(out.shape), self.rows, self.cols))
        api.tide_act8_unpack(self.buffer, out, stream)
        return out


class Linear:
    """y = act(x weight^T + bias) + residual and its gradients.

    weight [N, K], bias [N]: contiguous bf16 tensors; weight_grad and
    bias_grad, where given, receive the gradients (overwritten by every
    backward).  act: "none", "relu", "gelu", "gelu_tanh" or "silu"."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 act: str = "none", weight_grad: Optional[torch.Tensor] = None,
                 bias_grad: Optional[torch.Tensor] = None):
        if weight.dim() != 2:
            raise TideError(-1, "weight has %d dimensions, expected 2" % weight.dim())
        api._act(act)
        self.weight, self.bias, self.act = weight, bias, act
        self.weight_grad, self.bias_grad = weight_grad, bias_grad

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, z: Optional[Act8] = None,
                stream=None) -> torch.Tensor:
        """z: the checkpoint that receives act's argument (which backward
        needs unless act is "none")."""
        if z is not None:
            self._same(z, x.shape[0], self.weight.shape[0], "z")
        return api.tide_linear_forward(x, self.weight, out, self.bias, residual, self.act,
                                       None if z is None else z.buffer, stream)

    def backward(self, dy: torch.Tensor, x: Optional[Act8] = None, z: Optional[Act8] = None,
                 dx: Optional[torch.Tensor] = None, input_grad: bool = True,
                 stream=None) -> Optional[torch.Tensor]:
        """Writes weight_grad and bias_grad (where the layer has them) and
        returns dx (None with input_grad=False).  x: the checkpoint of
        forward's x, z: the one forward wrote.  The residual's gradient is dy."""
        N, K = self.weight.shape
        if x is not None:
            self._same(x, dy.shape[0], K, "x")
        if z is not None:
            self._same(z, dy.shape[0], N, "z")
        if not input_grad:
            dx = None
        elif dx is None:
            dx = True
        return api.tide_linear_backward(dy, K, self.weight, None if x is None else x.buffer,
                                        None if z is None else z.buffer, self.act, dx,
                                        self.weight_grad, self.bias_grad, stream)

    @staticmethod
    def _same(kept: Act8, rows: int, cols: int, what: str) -> None:
        if (kept.rows, kept.cols) != (rows, cols):
            raise TideError(-1, "%s is a checkpoint of [%d, %d], expected [%d, %d]"
                            % (what, kept.rows, kept.cols, rows, cols))
