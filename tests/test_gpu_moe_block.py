"""The pre-norm expert block of examples/moe_block.py on the GPU: the layer
norm module against autograd's formula, the block trained for a few steps with
clipped gradients, and served by the few-token layer on the same weights."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import block as ob

from .gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

from moe_grouped_block_mx_amd.grouped_linear import GroupedLinear  # noqa: E402
from moe_grouped_block_mx_amd.layer_norm import LayerNorm  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_norm_module(dtype):
    g = torch.Generator("cuda").manual_seed(1)
    norm = LayerNorm(200, dtype=torch.float32)
    with torch.no_grad():
        norm.weight.copy_(1 + 0.1 * torch.randn(200, device="cuda", generator=g))
        norm.bias.copy_(torch.randn(200, device="cuda", generator=g))
    x = torch.randn((3, 5, 200), device="cuda", generator=g).to(dtype).requires_grad_()
    dy = torch.randn((3, 5, 200), device="cuda", generator=g).to(dtype)
    y = norm(x)
    assert y.shape == x.shape and y.dtype == dtype
    want, mean, rstd = ob.layer_norm_fwd(f64(x).reshape(15, 200), f64(norm.weight), f64(norm.bias))
    # fp32 throughout (see test_gpu_layer_norm.py for the bounds); bf16 results
    # are rounded once
    tol = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -16
    assert (np.abs(f64(y).reshape(15, 200) - want) <= tol * (np.abs(want) + 1e-2)).all()
    y.backward(dy)
    assert norm.weight.grad is None and norm.bias.grad is None
    dx, dw, db = ob.layer_norm_bwd(f64(dy).reshape(15, 200), f64(x).reshape(15, 200), f64(norm.weight), mean, rstd)
    assert (np.abs(f64(x.grad).reshape(15, 200) - dx) <= tol * (np.abs(dx) + 1e-2)).all()
    assert np.allclose(f64(norm.weight.main_grad), dw, rtol=1e-5, atol=1e-4)
    assert np.allclose(f64(norm.bias.main_grad), db, rtol=1e-5, atol=1e-4)
    norm(x).backward(dy)                                   # accumulates
    assert np.allclose(f64(norm.weight.main_grad), 2 * dw, rtol=1e-5, atol=2e-4)
    norm.weight.overwrite_main_grad = True
    norm(x).backward(dy)                                   # and overwrites
    assert np.allclose(f64(norm.weight.main_grad), dw, rtol=1e-5, atol=1e-4)
    assert np.allclose(f64(norm.bias.main_grad), db, rtol=1e-5, atol=1e-4)


def test_layer_norm_module_without_weight_gradients():
    norm = LayerNorm(64)
    norm.requires_grad_(False)
    x = torch.randn((4, 64), device="cuda").bfloat16().requires_grad_()
    norm(x).sum().backward()
    assert x.grad is not None and not norm.weight.main_grad.any()
    with pytest.raises(ValueError):
        norm(torch.zeros((4, 65), device="cuda"))


def test_quantized_weight_is_the_forwards():
    for recipe in ("a4w4", "a8w4", "blockwise"):
        m = GroupedLinear(2, 128, 256, recipe)
        q, s, fmt = m.quantized_weight()
        assert m.quantized_weight()[0] is q               # cached
        with torch.no_grad():
            m.weight.mul_(2)
        q2, s2, fmt2 = m.quantized_weight()
        assert fmt2 == fmt and torch.equal(q2, q) and not torch.equal(s2, s)   # twice the scale


def test_block_trains_and_serves():
    history, off = example().main(["--steps", "6"])
    losses, norms = zip(*history)
    assert losses[-1] < losses[0] and all(np.isfinite(norms))
    # MXFP8 activations (3 significant bits) on the training side, bf16 here
    assert off < 0.1


def test_layer_norm_module_takes_broadcast_and_transposed_gradients():
    norm = LayerNorm(48, dtype=torch.float32)
    g = torch.Generator("cuda").manual_seed(2)
    base = torch.randn((6, 48), device="cuda", generator=g)
    dy = torch.randn((6, 48), device="cuda", generator=g)
    grads = []
    for make in (lambda y: (y * dy).sum(), lambda y: (y.t() * dy.t().contiguous()).sum()):
        x = base.clone().requires_grad_()
        make(norm(x)).backward()
        grads.append(x.grad)
    assert torch.equal(grads[0], grads[1])
    x = base.t().contiguous().t().requires_grad_()        # transposed input
    (norm(x) * dy).sum().backward()
    assert torch.equal(x.grad, grads[0])
    norm.bias.requires_grad_(False)                       # one of the two frozen
    norm.bias.main_grad.zero_()
    norm(base.clone().requires_grad_()).sum().backward()  # dy: one element, expanded
    assert not norm.bias.main_grad.any() and norm.weight.main_grad.any()


@pytest.mark.parametrize("inner,hidden", [(64, 256), (192, 256), (192, 320)])
def test_block_whose_two_layers_have_different_code_layouts(inner, hidden):
    # fc1 is in K blocks where 128 divides hidden, fc2 (inner inputs) in rows
    history, off = example().main(["--steps", "2", "--inner", str(inner), "--hidden", str(hidden)])
    assert all(np.isfinite(norm) for _, norm in history) and off < 0.1
