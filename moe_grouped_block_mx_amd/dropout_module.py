"""Dropout whose mask is never stored, as an autograd module over the C ABI
(mxgg_dropout): the mask is a function of a seed and a step on the device, of the
call and of the element's place, and the backward pass draws it again.

    state = DropoutState(seed=1)
    drop = Dropout(0.1, state)             # one for each place in the model: a call number of its own
    y = drop(branch, residual=x)
    state.advance()                        # after each forward pass

A forward that is run again in the backward pass (activation checkpointing) reads the
state then. Advance after the backward pass, or give the checkpointed function the
state as an argument, which it gets again:

    y = checkpoint(lambda x, s: drop(x, state=s), x, state.tensor, use_reentrant=False)
"""
import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .layer_norm import _rows


class DropoutState:
    """Seed and step, int64 [2] on the device, shared by a model's dropouts. It is no
    part of the modules' state_dict: a program that goes on from a checkpoint saves
    and loads it beside the model, as it does an optimizer (else the masks of the first
    steps come again)."""

    def __init__(self, seed, step=0, device=None):
        device = torch.device("cuda") if device is None else torch.device(device)
        self.tensor = torch.tensor([seed, step], dtype=torch.int64, device=device)
        self._one = torch.tensor([0, 1], dtype=torch.int64, device=device)
        self._calls, self._given = set(), set()    # the numbers of its dropouts, and those given out here

    def _number(self, call):
        """The caller's number, or for None the first that no dropout has."""
        if call is None:
            call = next(n for n in range(len(self._calls) + 1) if n not in self._calls)
            self._given.add(call)
        elif not 0 <= call < 1 << 32:
            raise ValueError(f"call={call} outside [0, 2^32)")
        elif call in self._given:
            raise ValueError(f"call={call} was given to another dropout of this state, which would draw the same mask")
        self._calls.add(call)
        return call

    def advance(self):
        """New masks from here on. A backward pass still to come keeps the step of
        its forward pass (one that runs the forward again: see above)."""
        self.tensor = self.tensor + self._one

    def advance_(self):
        """The same in place, for a captured graph (each replay then draws new
        masks). A backward pass still to come of an earlier step raises; one that runs
        the forward again has to come first."""
        self.tensor[1:].add_(1)

    def state_dict(self):
        """{"seed", "step"} as ints (waits for the device)."""
        seed, step = self.tensor.tolist()
        return {"seed": seed, "step": step}

    def load_state_dict(self, saved):
        """In place, as advance_: a captured graph goes on from there."""
        self.tensor.copy_(torch.tensor([saved["seed"], saved["step"]], dtype=torch.int64))


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, state, p, call):
        ctx.save_for_backward(state)      # a change of it before the backward pass is an error there
        ctx.p, ctx.call, ctx.shape = p, call, x.shape
        rows = _rows(x)
        res = None if residual is None else _rows(residual)
        return L.mxgg_dropout(rows, p, state, call, residual=res).view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        state, = ctx.saved_tensors
        dx = None
        if ctx.needs_input_grad[0]:
            dx = L.mxgg_dropout(_rows(dy), ctx.p, state, ctx.call).view(ctx.shape)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


class Dropout(torch.nn.Module):
    """residual + x / (1 - p) where kept, residual where dropped; x bf16 or fp32
    [..., features], residual like it or None. p is rounded to a multiple of 2^-16.
    call: the number that tells a state's dropouts apart, by default the first that
    none of them has (by the order in which they are made); two that were given the
    same draw the same mask. forward's state: the int64 [2] to draw from, by default the
    DropoutState's. In eval mode nothing is dropped."""

    def __init__(self, p, state, call=None):
        super().__init__()
        if not 0 <= p <= 1:
            raise ValueError(f"p must be in [0, 1], got {p}")
        self.p, self.state, self.call = p, state, state._number(call)

    def forward(self, x, residual=None, state=None):
        if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
            raise ValueError(f"residual must be {x.dtype} {tuple(x.shape)}, got {residual.dtype} {tuple(residual.shape)}")
        if not self.training or self.p == 0:
            return x if residual is None else residual + x
        return _DropoutFn.apply(x, residual, self.state.tensor if state is None else state, self.p, self.call)
