"""The dense gated FFN as torch modules: 16 bits with gradients while a shared expert or a dense
layer is trained, W8A8 int8 when it is served.

``gated_ffn`` is differentiable (``ops.moe_gated_ffn`` and ``ops.moe_gated_ffn_backward``);
``GatedFFN`` holds its two weights; ``GatedFFN.to_int8`` quantises their rows
(``ops.moe_quant_int8``) for ``Int8GatedFFN``, which runs the routed int8 experts with one expert
(``ops.moe_grouped_ffn_int8``).

All three take their workspaces for one call; ``ops.device_failure`` tells whether a kernel gave up a wait.
"""
from __future__ import annotations

import math

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import ops


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2, activation):
        y, h = ops.moe_gated_ffn(x, w13, w2, activation, save_h=True)
        ctx.save_for_backward(x, w13, w2, h)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w13, w2, h = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:                     # a slice of a larger gradient
            dy = dy.clone()
        grads = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, ctx.activation,
                                           need=ctx.needs_input_grad[:3])
        return (*grads, None)


def gated_ffn(x, w13, w2, activation: str = "silu"):
    """(act(x Wg^T) * (x Wu^T)) W2^T for x [..., d] in bf16 or fp16, with first-order reverse-mode
    gradients for x, w13 [2F, d] and w2 [d, F]; tensors that carry a forward-mode tangent are refused.
    Tokens and weights have one type, under ``torch.autocast`` too. The pre-activations are kept for the
    backward pass when one of them asks for a gradient. (Capturing the backward pass into a CUDA graph
    follows torch's rule: no eager graph of the same leaves may be alive during the capture.)"""
    # (a dual tensor need not require a gradient: without a word its tangent would come back as none,
    # which stands for a derivative of zero)
    if any(forward_ad.unpack_dual(t).tangent is not None for t in (x, w13, w2)):
        raise NotImplementedError("gated_ffn has no forward-mode derivative")
    rows = x.reshape(-1, x.shape[-1]).contiguous()
    # (asked here: inside the function torch reports the leaves' wishes under no_grad as well)
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, w13, w2)):
        y = _GatedFFN.apply(rows, w13, w2, activation)
    else:
        y = ops.moe_gated_ffn(rows, w13, w2, activation)
    return y.reshape(x.shape)


class GatedFFN(torch.nn.Module):
    """A gated FFN of hidden size d and width F; w13 = [gate; up] [2F, d], w2 [d, F]."""

    def __init__(self, d: int, F: int, activation: str = "silu", dtype=torch.bfloat16,
                 device="cuda"):
        super().__init__()
        if activation not in ops.ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ops.ACTIVATIONS)}")
        self.activation = activation
        self.w13 = torch.nn.Parameter(torch.empty(2 * F, d, dtype=dtype, device=device))
        self.w2 = torch.nn.Parameter(torch.empty(d, F, dtype=dtype, device=device))
        with torch.no_grad():
            self.w13.normal_(0.0, 1 / math.sqrt(d))
            self.w2.normal_(0.0, 1 / math.sqrt(F))

    def forward(self, x):
        return gated_ffn(x, self.w13, self.w2, self.activation)

    def to_int8(self) -> "Int8GatedFFN":
        """The serving form: one int8 scale per output channel. SiLU gates only (the routed
        experts' activation)."""
        if self.activation != "silu":
            raise ValueError("the int8 experts are SwiGLU: activation must be 'silu'")
        with torch.no_grad():
            return Int8GatedFFN(*ops.moe_quant_int8(self.w13.detach()),
                                *ops.moe_quant_int8(self.w2.detach()))


class Int8GatedFFN(torch.nn.Module):
    """A W8A8 int8 SwiGLU FFN: codes w13 [2F, d], w2 [d, F] with scales [2F], [d] (buffers that hold them
    as those of one expert); bf16 tokens. It serves: tokens whose gradient is wanted are refused. Casts
    of a model leave the scales in fp32."""

    def __init__(self, w13, w13_scale, w2, w2_scale):
        super().__init__()
        self.d, self.F = w2.shape
        for name, t in zip(("w13", "w13_scale", "w2", "w2_scale"), (w13, w13_scale, w2, w2_scale)):
            self.register_buffer(name, t.detach().unsqueeze(0))

    @property
    def weights(self):
        return self.w13, self.w13_scale, self.w2, self.w2_scale

    def _apply(self, fn, recurse=True):
        scales = {n: getattr(self, n) for n in ("w13_scale", "w2_scale")}
        super()._apply(fn, recurse)
        for name, scale in scales.items():
            now = getattr(self, name)
            if now.dtype != scale.dtype:
                setattr(self, name, scale.to(now.device))
        return self

    def forward(self, x, dtype=torch.bfloat16):
        """y [..., d] of x [..., d] bf16, summed in fp32 and rounded once to ``dtype``."""
        ops._no_derivative("Int8GatedFFN", x)
        rows = x.reshape(-1, x.shape[-1]).contiguous()
        T = rows.shape[0]
        offsets = torch.arange(2, dtype=torch.int32, device=x.device) * T     # one expert's rows
        perm = torch.arange(T, dtype=torch.int32, device=x.device)
        out = ops.moe_grouped_ffn_int8(rows, *self.weights, offsets, perm, 1)
        return out[:T].to(dtype).reshape(x.shape)
