"""Layer norm in front of the expert layer, as an autograd module over the C ABI
(mxgg_layer_norm_fwd / _bwd), in GroupedLinear's manner:

- the gradients of weight and bias are accumulated in place into their fp32
  ``main_grad`` (autograd sees none), or overwrite it when
  ``weight.overwrite_main_grad`` is set (the first microbatch);
- mean and 1/std per row are kept in fp32 between forward and backward.

Every step runs in libmxgg's kernels; tensors must live on the GPU.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _lib as L


def _rows(t):
    """[..., C] as rows with unit inner stride; a copy only where the kernels
    could not read it (a broadcast or transposed gradient, a row stride of 2^31
    or more)."""
    rows = t.reshape(-1, t.shape[-1])
    n, cols = rows.shape
    if (cols > 1 and rows.stride(1) != 1) or (n > 1 and not cols <= rows.stride(0) < 1 << 31):
        rows = rows.contiguous()
    return rows


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, module):
        rows = _rows(x)
        y, mean, rstd = L.mxgg_layer_norm_fwd(rows, weight, bias, module.eps)
        ctx.save_for_backward(rows, weight, mean, rstd)
        ctx.module, ctx.shape = module, x.shape
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, weight, mean, rstd = ctx.saved_tensors
        m = ctx.module
        dw = m.weight.main_grad if ctx.needs_input_grad[1] else False
        db = m.bias.main_grad if ctx.needs_input_grad[2] else False
        # the accumulation mode is the one in force at this backward
        accumulate = not getattr(m.weight, "overwrite_main_grad", False)
        dx, _, _ = L.mxgg_layer_norm_bwd(_rows(dy), rows, weight, mean, rstd, dweight=dw, dbias=db,
                                         accumulate=accumulate)
        return dx.view(ctx.shape), None, None, None


class LayerNorm(torch.nn.Module):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension
    (at most 16384); x bf16 or fp32 [..., features], weight and bias of `dtype`
    with an fp32 main_grad each."""

    def __init__(self, features, eps=1e-5, dtype=torch.bfloat16, device=None):
        super().__init__()
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"dtype must be bf16 or fp32, got {dtype}")
        self.features, self.eps = features, eps
        device = torch.device("cuda") if device is None else torch.device(device)
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(features, dtype=dtype, device=device))
        for p in (self.weight, self.bias):
            p.main_grad = torch.zeros(features, dtype=torch.float32, device=device)
        self.weight.overwrite_main_grad = False

    def forward(self, x):
        if x.dtype not in (torch.bfloat16, torch.float32) or x.shape[-1] != self.features:
            raise ValueError(f"x must be bf16 or fp32 [..., {self.features}], got {tuple(x.shape)} {x.dtype}")
        return _LayerNormFn.apply(x, self.weight, self.bias, self)
