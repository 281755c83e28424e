"""Tokens to their experts and back, as autograd functions over the C ABI
(mxgg_moe_sort / _dispatch / _combine / _combine_bwd): what stands between a
router and the grouped layers.

    plan = TokenPlan(ids, experts)                   # a router's choices
    y = layer(dispatch(x, plan), plan.m_splits())    # GroupedLinear
    out = combine(y, weights, plan)                  # [tokens, features]

Every step runs in libmxgg's kernels; tensors must live on the GPU.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .layer_norm import _rows


class TokenPlan:
    """The choices ids (int32 or int64 [tokens, top_k], any strides) in the order of
    their experts; a choice outside [0, experts) is dropped.

    rows     int32 [tokens, top_k]: the place of each choice, ~place where dropped
    choices  int32 [tokens * top_k]: the choice at each place
    counts   int32 [experts]: the rows of each expert
    """

    def __init__(self, ids, experts):
        if ids.dim() == 2 and ids.numel():
            ids = _rows(ids)
        self.rows, self.choices, self.counts = L.mxgg_moe_sort(ids, experts)
        self._splits = None
        self._captured = torch.cuda.is_current_stream_capturing()   # every replay then counts anew

    def m_splits(self):
        """counts on the host, what the grouped GEMMs take (the first call waits
        for the device, of a captured plan every call)."""
        if self._splits is None or self._captured:
            self._splits = self.counts.tolist()
        return self._splits


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, expert_rows):
        ctx.save_for_backward(rows)
        return L.mxgg_moe_dispatch(_rows(x), rows, expert_rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, = ctx.saved_tensors
        return L.mxgg_moe_combine(_rows(dy), rows), None, None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, rows):
        y, weights = _rows(y), weights.contiguous()
        ctx.save_for_backward(y, weights, rows)
        return L.mxgg_moe_combine(y, rows, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, weights, rows = ctx.saved_tensors
        dy, dweights = L.mxgg_moe_combine_bwd(_rows(dout), y, rows, weights)
        return dy, dweights, None


def dispatch(x, plan, expert_rows=None):
    """x: bf16 or fp32 [tokens, features] -> [expert_rows, features] in the order
    of the experts. expert_rows: sum(plan.m_splits()) by default, without the
    dropped choices; tokens * top_k needs no wait for the device, and holds zeros
    in the dropped choices' rows."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    if expert_rows is None:
        expert_rows = sum(plan.m_splits())
    return _DispatchFn.apply(x, plan.rows, expert_rows)


def combine(y, weights, plan):
    """y: bf16 or fp32 [expert rows, features], weights: fp32 [tokens, top_k] ->
    [tokens, features], each token's rows weighted and summed (zeros where all
    its choices are dropped)."""
    if y.dim() != 2:
        raise ValueError(f"y must be 2-D, got {tuple(y.shape)}")
    return _CombineFn.apply(y, weights, plan.rows)
