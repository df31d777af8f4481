"""The norm in front of a layer's products, and its gradients.

``Norm`` stands before ``Linear`` (linear.py) and ``Gated`` (gated.py): its weight
is a full tensor that the placement writes (``Setup.full[p]``), its gradients
are tensors that the reduce-scatter reads (``Setup.grads[q][p]``).  What its
backward pass needs is x, in bf16 or as an 8-bit checkpoint; the statistics are
worked out again.

    x8, y8 = Act8(T, C, device=dev), Act8(T, C, device=dev)
    norm = Norm(full[p], kind="rms", weight_grad=grads[q][p])
    y = norm.forward(x, x8=x8, y8=y8)        # y8: for the next product's weight gradient
    dx = norm.backward(dy, x8, add=dstream)  # plus the gradient that reaches x past the norm

All work is done by the library (``include/tide.h``); autograd, ``stream`` and
memory are as linear.py describes them.
"""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import api
from ._lib import TideError, TideNormBackwardArgs, TideNormForwardArgs
from .linear import Act8


class Norm:
    """y = (x - mean) / sqrt(var + eps) weight + bias over each row
    (kind="layer"), or with mean 0 and the mean square (kind="rms").

    weight, bias [C]: contiguous bf16 GPU tensors, C at most 32768; weight_grad
    and bias_grad, where given, receive the gradients (overwritten by every
    backward).  The four tensors are checked here and kept; calls use their
    memory as it is then."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 kind: str = "rms", eps: float = 1e-6,
                 weight_grad: Optional[torch.Tensor] = None,
                 bias_grad: Optional[torch.Tensor] = None):
        self._kind = api._norm_kind(kind)
        if not isinstance(weight, torch.Tensor):
            raise TypeError("weight must be a torch.Tensor")
        if weight.dim() != 1:
            raise TideError(-1, "weight has %d dimensions, expected 1" % weight.dim())
        self._gpu = weight.get_device()
        self._cols = C = weight.shape[0]
        for t, what in ((weight, "weight"), (bias, "bias"), (weight_grad, "weight_grad"),
                        (bias_grad, "bias_grad")):
            if t is not None:
                api._whole(t, (C,), what, self._gpu)
        self._weight, self._bias, self.kind, self.eps = weight, bias, kind, float(eps)
        self._weight_grad, self._bias_grad = weight_grad, bias_grad

    weight = property(lambda self: self._weight)
    bias = property(lambda self: self._bias)
    weight_grad = property(lambda self: self._weight_grad)
    bias_grad = property(lambda self: self._bias_grad)

    def forward(self, x: torch.Tensor, x8: Optional[Act8] = None, y8: Optional[Act8] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x8, y8: the checkpoints that receive x and y.  out is allocated when
        not given."""
        C, gpu = self._cols, self._gpu
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() else 0
        px, ldx = api._matrix(x, T, C, "x", gpu)
        a = TideNormForwardArgs(T, C, self._kind, self.eps, px, ldx, self._weight.data_ptr())
        if self._bias is not None:
            a.bias = self._bias.data_ptr()
        if out is not None:
            a.y, a.ldy = api._matrix(out, T, C, "out", gpu)
        if x8 is not None:
            a.x_kept = x8._of(T, C, gpu, "x8")
        if y8 is not None:
            a.y_kept = y8._of(T, C, gpu, "y8")
        return api._on_device(gpu, stream, api._norm_forward_on, a, out, gpu)

    def backward(self, dy: torch.Tensor, x: Union[torch.Tensor, Act8, None] = None,
                 add: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 input_grad: bool = True, stream=None) -> Optional[torch.Tensor]:
        """Writes weight_grad and bias_grad (where the norm has them) and returns
        dx plus ``add`` (None with input_grad=False).  x: forward's x, or its
        checkpoint.  dx may be add itself."""
        C, gpu = self._cols, self._gpu
        T = dy.shape[0] if isinstance(dy, torch.Tensor) and dy.dim() else 0
        pdy, lddy = api._matrix(dy, T, C, "dy", gpu)
        a = TideNormBackwardArgs(T, C, self._kind, self.eps, pdy, lddy)
        if isinstance(x, Act8):
            a.x_kept = x._of(T, C, gpu, "x")
        elif x is not None:
            a.x, a.ldx = api._matrix(x, T, C, "x", gpu)
        elif input_grad or self._weight_grad is not None:
            raise TideError(-1, "dx and weight_grad need x or its checkpoint")
        if input_grad:
            a.weight = self._weight.data_ptr()
            if add is not None:
                a.add, a.ldadd = api._matrix(add, T, C, "add", gpu)
            if dx is None:
                dx = True
            else:
                a.dx, a.lddx = api._matrix(dx, T, C, "dx", gpu)
        elif add is not None or dx is not None:
            raise TideError(-1, "add and dx go with the input's gradient, which is not asked for")
        if self._weight_grad is not None:
            a.dweight = self._weight_grad.data_ptr()
        if self._bias_grad is not None:
            a.dbias = self._bias_grad.data_ptr()
        return api._on_device(gpu, stream, api._norm_backward_on, a, dx, gpu)
