"""A pre-norm mixture-of-experts block, trained and then served.

    y = x + experts(layer_norm(x))

Training: LayerNorm, a bf16 gate, the experts as two GroupedLinear layers on the
routed rows, the norm of all gradients and clipping, plain SGD. Serving: the
same norm and gate, and the whole expert layer in one call (moe_layer) on the
weights that the grouped layers quantized, for a few tokens at a time.

    python examples/moe_block.py [--steps N] [--hidden H] [--inner I] [--experts E]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_block_mx_amd as mxg  # noqa: E402
from moe_grouped_block_mx_amd.grouped_linear import GroupedLinear  # noqa: E402
from moe_grouped_block_mx_amd.layer_norm import LayerNorm  # noqa: E402


class MoEBlock(torch.nn.Module):
    def __init__(self, hidden, inner, experts, top_k, recipe="a8w4", generator=None):
        super().__init__()
        self.top_k, self.experts = top_k, experts
        self.norm = LayerNorm(hidden)
        self.gate = torch.nn.Parameter(
            (torch.randn((experts, hidden), device="cuda", generator=generator) * hidden ** -0.5).bfloat16())
        # fc1: each expert's gate rows, then its up rows
        self.fc1 = GroupedLinear(experts, hidden, 2 * inner, recipe, weight_std=hidden ** -0.5, generator=generator)
        self.fc2 = GroupedLinear(experts, inner, hidden, recipe, weight_std=inner ** -0.5, generator=generator)

    def forward(self, x):
        """Training: x bf16 [tokens, hidden]."""
        n = self.norm(x)
        top, ids = torch.topk(n @ self.gate.t(), self.top_k, dim=1)
        weights = torch.softmax(top.float(), dim=1)
        # rows in the order of their experts
        flat = ids.reshape(-1)
        order = torch.argsort(flat, stable=True)
        splits = torch.bincount(flat, minlength=self.experts).tolist()
        token = order // self.top_k
        gate, up = self.fc1(n[token], splits).chunk(2, dim=1)
        out = self.fc2(torch.nn.functional.silu(gate) * up, splits)
        y = torch.zeros_like(x, dtype=torch.float32)
        return x + y.index_add(0, token, out.float() * weights.reshape(-1)[order, None]).to(x.dtype)

    @torch.no_grad()
    def decode(self, x):
        """Serving: x bf16 [tokens, hidden], at most MOE_MAX_TOKENS tokens."""
        n, _, _ = mxg.layer_norm_fwd(x, self.norm.weight, self.norm.bias, self.norm.eps)
        w13_q, w13_s, fmt = self.fc1.quantized_weight()
        w2_q, w2_s, w2_fmt = self.fc2.quantized_weight()   # its code layout goes by its own sizes
        y, _, _ = mxg.moe_layer(n, n @ self.gate.t(), w13_q, w13_s, w2_q, w2_s, self.top_k, fmt=fmt, w2_fmt=w2_fmt)
        return x + y

    def gradients(self):
        return [p.main_grad for p in (self.norm.weight, self.norm.bias, self.fc1.weight, self.fc2.weight)] \
            + [self.gate.grad]

    @torch.no_grad()
    def update(self, lr):
        for p in (self.norm.weight, self.norm.bias, self.fc1.weight, self.fc2.weight):
            p.sub_((lr * p.main_grad).view(p.shape).to(p.dtype))
        self.gate.sub_(lr * self.gate.grad)


def train(block, steps, tokens, hidden, lr=0.5, max_norm=1.0, generator=None):
    x = torch.randn((tokens, hidden), device="cuda", generator=generator).bfloat16()
    target = (x.float() + 0.5 * torch.randn((tokens, hidden), device="cuda", generator=generator)).bfloat16()
    history = []
    for step in range(steps):
        for p in (block.norm.weight, block.fc1.weight, block.fc2.weight):
            p.overwrite_main_grad = True       # one microbatch a step: nothing to add to
        block.gate.grad = None
        loss = (block(x).float() - target.float()).square().mean()
        (loss * 1000).backward()
        norm = mxg.clip_grad_norm(block.gradients(), max_norm)
        block.update(lr)
        history.append((float(loss.detach()), float(norm)))
    return history


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=256)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    a = ap.parse_args(argv)
    g = torch.Generator("cuda").manual_seed(0)
    block = MoEBlock(a.hidden, a.inner, a.experts, a.top_k, generator=g)
    history = train(block, a.steps, a.tokens, a.hidden, generator=g)
    for step, (loss, norm) in enumerate(history):
        print(f"step {step}: loss {loss:.5f}, gradient norm {norm:.4f}")
    x = torch.randn((4, a.hidden), device="cuda", generator=g).bfloat16()
    with torch.no_grad():
        trained = block(x).float()
    served = block.decode(x).float()
    off = float((served - trained).norm() / (trained - x.float()).norm())
    print(f"4 tokens served: {off:.4f} of the experts' output from the training path "
          "(whose activations are quantized)")
    return history, off


if __name__ == "__main__":
    main()
