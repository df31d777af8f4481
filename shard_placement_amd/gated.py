"""The gated block in front of a layer's last product, and its gradients.

``Gated`` is the gate and up projections of a feed-forward block with the
activation and the product between them in one kernel; ``Linear`` (linear.py) is
the down projection behind it, ``Norm`` (norm.py) what stands before.  Its
weights are full tensors that the placement writes (``Setup.full[p]``), its
gradients are tensors that the reduce-scatter reads (``Setup.grads[q][p]``).

    g8, u8, h8 = (Act8(T, N, device=dev) for _ in range(3))
    block = Gated(full[p], full[p + 1], gate_grad=grads[q][p], up_grad=grads[q][p + 1])
    h = block.forward(x, g=g8, u=u8, h=h8)       # silu(x gate^T) * (x up^T)
    y = down.forward(h, residual=stream)
    dh = down.backward(dy, x=h8)
    dx = block.backward(dh, x=x8, g=g8, u=u8)    # writes both weights' gradients

All work is done by the library (``include/tide.h``); autograd, ``stream`` and
memory are as linear.py describes them.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import api
from ._lib import TideError, TideGatedBackwardArgs, TideGatedForwardArgs
from .linear import Act8


class Gated:
    """h = act(x gate^T + gate_bias) (x up^T + up_bias) and its gradients.

    gate, up [N, K], biases [N]: contiguous bf16 GPU tensors; the gradients'
    tensors, where given (the weights' both or neither), are overwritten by
    every backward.  act: "none", "relu", "gelu", "gelu_tanh" or "silu".  The
    tensors are checked here and kept; calls use their memory as it is then."""

    def __init__(self, gate: torch.Tensor, up: torch.Tensor,
                 gate_bias: Optional[torch.Tensor] = None, up_bias: Optional[torch.Tensor] = None,
                 act: str = "silu", gate_grad: Optional[torch.Tensor] = None,
                 up_grad: Optional[torch.Tensor] = None,
                 gate_bias_grad: Optional[torch.Tensor] = None,
                 up_bias_grad: Optional[torch.Tensor] = None):
        self._act = api._act(act)
        self._gpu = api._index(gate, "gate")
        self._shape = N, K = tuple(gate.shape)
        for t, shape, what in ((gate, (N, K), "gate"), (up, (N, K), "up"),
                               (gate_bias, (N,), "gate_bias"), (up_bias, (N,), "up_bias"),
                               (gate_grad, (N, K), "gate_grad"), (up_grad, (N, K), "up_grad"),
                               (gate_bias_grad, (N,), "gate_bias_grad"),
                               (up_bias_grad, (N,), "up_bias_grad")):
            if t is not None or what == "up":
                api._whole(t, shape, what, self._gpu)
        if (gate_grad is None) != (up_grad is None):
            raise TideError(-1, "gate_grad and up_grad are computed together")
        self._gate, self._up, self.act = gate, up, act
        self._gate_bias, self._up_bias = gate_bias, up_bias
        self._gate_grad, self._up_grad = gate_grad, up_grad
        self._gate_bias_grad, self._up_bias_grad = gate_bias_grad, up_bias_grad

    gate = property(lambda self: self._gate)
    up = property(lambda self: self._up)
    gate_bias = property(lambda self: self._gate_bias)
    up_bias = property(lambda self: self._up_bias)
    gate_grad = property(lambda self: self._gate_grad)
    up_grad = property(lambda self: self._up_grad)
    gate_bias_grad = property(lambda self: self._gate_bias_grad)
    up_bias_grad = property(lambda self: self._up_bias_grad)

    def forward(self, x: torch.Tensor, g: Optional[Act8] = None, u: Optional[Act8] = None,
                h: Optional[Act8] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """g, u: the checkpoints that receive act's argument and the other
        factor (which backward needs); h: the one that receives the result (which
        the next product's backward needs).  out is allocated when not given."""
        N, K = self._shape
        gpu = self._gpu
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() else 0
        px, ldx = api._matrix(x, T, K, "x", gpu)
        a = TideGatedForwardArgs(T, N, K, self._act, 0, px, ldx, self._gate.data_ptr(),
                                 self._up.data_ptr())
        if self._gate_bias is not None:
            a.gate_bias = self._gate_bias.data_ptr()
        if self._up_bias is not None:
            a.up_bias = self._up_bias.data_ptr()
        if out is not None:
            a.h, a.ldh = api._matrix(out, T, N, "out", gpu)
        if g is not None:
            a.g_kept = g._of(T, N, gpu, "g")
        if u is not None:
            a.u_kept = u._of(T, N, gpu, "u")
        if h is not None:
            a.h_kept = h._of(T, N, gpu, "h")
        return api._on_device(gpu, stream, api._gated_forward_on, a, out, gpu)

    def backward(self, dh: torch.Tensor, x: Optional[Act8] = None, g: Optional[Act8] = None,
                 u: Optional[Act8] = None, dx: Optional[torch.Tensor] = None,
                 input_grad: bool = True, stream=None) -> Optional[torch.Tensor]:
        """Writes the gradients that the block has tensors for and returns dx
        (None with input_grad=False).  x: the checkpoint of forward's x; g, u:
        those that forward wrote."""
        N, K = self._shape
        gpu = self._gpu
        T = dh.shape[0] if isinstance(dh, torch.Tensor) and dh.dim() else 0
        pdh, lddh = api._matrix(dh, T, N, "dh", gpu)
        a = TideGatedBackwardArgs(T, N, K, self._act, 0, pdh, lddh)
        if g is None or u is None:
            raise TideError(-1, "the gradients need the checkpoints of g and u")
        a.g_kept, a.u_kept = g._of(T, N, gpu, "g"), u._of(T, N, gpu, "u")
        if input_grad:
            a.gate, a.up = self._gate.data_ptr(), self._up.data_ptr()
            if dx is None:
                dx = True
            else:
                a.dx, a.lddx = api._matrix(dx, T, K, "dx", gpu)
        elif dx is not None:
            raise TideError(-1, "dx is the input's gradient, which is not asked for")
        if self._gate_grad is not None:
            if x is None:
                raise TideError(-1, "gate_grad and up_grad need the checkpoint of x")
            a.x_kept = x._of(T, K, gpu, "x")
            a.dgate, a.dup = self._gate_grad.data_ptr(), self._up_grad.data_ptr()
        if self._gate_bias_grad is not None:
            a.dgate_bias = self._gate_bias_grad.data_ptr()
        if self._up_bias_grad is not None:
            a.dup_bias = self._up_bias_grad.data_ptr()
        return api._on_device(gpu, stream, api._gated_backward_on, a, dx, gpu)
