"""The way through the experts as a user has it: the autograd modules against
plain torch in fp64, a captured training step, the layer in 8-bit integers and the
example's block with dropout and a served prompt."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import tokens as ot

from .gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402
from moe_grouped_block_mx_amd.dropout_module import Dropout, DropoutState  # noqa: E402
from moe_grouped_block_mx_amd.grouped_linear import GroupedLinear  # noqa: E402
from moe_grouped_block_mx_amd.token_plan import TokenPlan, combine, dispatch  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def example():
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return host(t.detach().double())


def inputs(T, k, E, C, dropped, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g)
    ids[torch.rand((T, k), device="cuda", generator=g) < dropped] = -1
    x = torch.randn((T, C), device="cuda", generator=g)
    w = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)
    d = torch.randn((T, C), device="cuda", generator=g)
    return ids, x, w, d


def plain_path(x, w, ids, scale, kept, residual):
    """residual + dropout(sum_j w_j scale[e_j] x) in fp64 torch, with autograd."""
    on = ids >= 0
    s = torch.where(on, w * scale[ids.clamp(min=0)], 0)
    return residual + torch.where(kept, s.sum(1, keepdim=True) * x, 0) / (1 - 16384 / 65536)


@pytest.mark.parametrize("all_rows", [False, True])
def test_gradients_of_the_path(all_rows):
    """dispatch -> a scale for each expert -> combine -> dropout with a residual,
    against fp64 autograd. Everything is fp32: at most 5 choices a token and a few
    products each, so within 32 u of the sums of magnitudes (bounded by those of
    the inputs below)."""
    T, k, E, C = 123, 5, 7, 260
    ids, x, w, d = inputs(T, k, E, C, 0.25)
    scale = torch.linspace(0.5, 2.0, E, device="cuda")
    residual = torch.randn((T, C), device="cuda")
    x, w, residual = (t.clone().requires_grad_() for t in (x, w, residual))
    plan = TokenPlan(ids, E)
    splits = plan.m_splits()
    assert splits == [int((ids == e).sum()) for e in range(E)]
    rows = dispatch(x, plan, T * k if all_rows else None)
    assert rows.shape == (T * k if all_rows else sum(splits), C)
    each = torch.repeat_interleave(scale, torch.tensor(splits, device="cuda"))
    each = torch.cat([each, each.new_ones(rows.shape[0] - each.numel())])
    state = DropoutState(3)
    out = Dropout(0.25, state, call=2)(combine(rows * each[:, None], w, plan), residual=residual)
    out.backward(d)
    kept = torch.from_numpy(ot.dropout(np.zeros((T, C)), 0.25, 3, 0, 2)[1]).cuda()
    px, pw, pr = (t.detach().double().requires_grad_() for t in (x, w, residual))
    want = plain_path(px, pw, ids, scale.double(), kept, pr)
    want.backward(d.double())
    top = 2.0 * 4 / 3 * 5           # the largest scale, dropout's factor, five choices
    assert (np.abs(f64(out) - f64(want)) <= 32 * U * (top * np.abs(f64(x)) + np.abs(f64(residual)))).all()
    assert torch.equal(residual.grad, d)
    assert (np.abs(f64(x.grad) - f64(px.grad)) <= 32 * U * top * np.abs(f64(d))).all()
    # a weight's gradient is a sum over the row
    size = (np.abs(f64(d)) * np.abs(f64(x))).sum(1, keepdims=True) * 2 * 4 / 3
    assert (np.abs(f64(w.grad) - f64(pw.grad)) <= 256 * U * size).all()
    assert not w.grad[ids < 0].any()


def test_rows_that_no_choice_names():
    """More rows than choices: their gradient is zero, not what memory held."""
    ids, x, w, d = inputs(9, 2, 3, 40, 0.0)
    plan = TokenPlan(ids, 3)
    y = torch.randn((25, 40), device="cuda", requires_grad=True)
    combine(y, w, plan).backward(d)
    assert not y.grad[18:].any() and y.grad[:18].any(1).all()
    out = dispatch(x.detach(), plan, 25)
    assert torch.equal(out[:18], dispatch(x.detach(), plan)) and not out[18:].any()


def test_noncontiguous_and_broadcast_gradients():
    ids, x, w, d = inputs(30, 3, 5, 64, 0.1)
    plan = TokenPlan(ids, 5)
    a = x.clone().requires_grad_()
    dispatch(a, plan).sum().backward()                      # a broadcast gradient
    assert torch.equal(a.grad, ((ids >= 0).sum(1, keepdim=True)).float().expand(30, 64))
    b, v = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = combine(dispatch(b, plan), v, plan)
    out.t().backward(d.t())                                 # a transposed one
    want = ot.combine_bwd(f64(d), ot.dispatch(f64(x), host(plan.rows), sum(plan.m_splits())), host(plan.rows), f64(w))
    assert (np.abs(f64(v.grad) - want[1]) <= 256 * U * want[2]).all()


def test_dropout_module():
    x = torch.randn((4, 6, 100), device="cuda", requires_grad=True)
    state = DropoutState(7)
    drop = Dropout(0.5, state, call=1)
    first, again = drop(x), drop(x)
    assert torch.equal(first, again)                        # a function of step and call
    kept = first != 0
    state.advance()
    other = drop(x)
    assert 0.3 < ((other != 0) == kept).double().mean() < 0.7
    first.backward(torch.ones_like(first))                  # keeps its own step
    assert torch.equal(x.grad, 2.0 * kept)
    drop.eval()
    assert drop(x) is x and torch.equal(drop(x, residual=x), x + x)
    drop.train()
    late = drop(x)
    state.advance_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        late.backward(torch.ones_like(late))
    for bad in (dict(p=1.5), dict(p=-0.1), dict(p=0.1, call=-1)):
        with pytest.raises(ValueError):
            Dropout(state=state, **bad)
    with pytest.raises(ValueError):
        drop(x, residual=x[0])


def test_captured_training_step():
    """Forward and backward of the path captured and replayed: new inputs, a new
    mask each time, the same values as eager."""
    T, k, E, C = 64, 3, 6, 200
    ids, x, w, d = inputs(T, k, E, C, 0.2)
    static = [t.clone() for t in (ids, x, w, d)]
    state = DropoutState(1)
    drop = Dropout(0.3, state)

    def step(ids, x, w, d, state_tensor):
        drop.state.tensor = state_tensor
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        plan = TokenPlan(ids, E)
        out = drop(combine(dispatch(x, plan, T * k), w, plan), residual=x)
        return (out, *torch.autograd.grad(out, (x, w), d))
    held = state.tensor
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static, held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static, held)
        held[1:] += 1
    for n in range(3):
        new = inputs(T, k, E, C, 0.2, seed=10 + n)
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*new, torch.tensor([1, n], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


def test_layer_in_int8():
    layer = GroupedLinear(3, 160, 72, weight_std=0.1, generator=torch.Generator("cuda").manual_seed(0))
    x = torch.randn((50, 160), device="cuda").bfloat16()
    for _ in range(2):
        got = layer.forward_int8(x, [20, 0, 30])
        q, s = ot.quantize_int8(f64(x))
        wq, ws = ot.quantize_int8(f64(layer.weight))
        want = ot.grouped_int8(q, s, wq.reshape(3, 72, 160), ws.reshape(3, 72), [20, 0, 30])
        assert (np.abs(f64(got) - want) <= (2.0 ** -8 + 4 * U) * np.abs(want)).all()
        held = layer.int8_weight()
        layer.weight.data.mul_(-2)                           # nothing is kept that misses this
        assert torch.equal(layer.forward_int8(x, [20, 0, 30], held), got)
        assert torch.equal(layer.forward_int8(x, [20, 0, 30]), -2 * got)


def test_example_block():
    """Trained with dropout and served: every step of a served prompt against its
    reference, and the whole equal to its steps."""
    m = example()
    history, off = m.main(["--steps", "3", "--dropout", "0.1"])
    assert len(history) == 3 and all(np.isfinite(history).ravel()) and np.isfinite(off)
    g = torch.Generator("cuda").manual_seed(1)
    block = m.MoEBlock(256, 128, 6, 2, generator=g).eval()
    x = torch.randn((300, 256), device="cuda", generator=g).bfloat16()
    out = block.prefill(x, block.int8_weights())
    n, _, _ = mxg.layer_norm_fwd(x, block.norm.weight, block.norm.bias, block.norm.eps)
    top, ids = torch.topk(n @ block.gate.t(), 2, dim=1)
    rows, choices, counts = mxg.moe_sort(ids, 6)
    for a, b in zip((rows, choices, counts), ot.sort(host(ids), 6)):
        assert np.array_equal(host(a), b)
    splits = counts.tolist()
    y = mxg.moe_dispatch(n, rows)
    assert np.array_equal(f64(y), f64(n)[host(choices) // 2])
    for layer in (block.fc1, block.fc2):
        z = layer.forward_int8(y, splits)
        q, s = ot.quantize_int8(f64(y))
        wq, ws = ot.quantize_int8(f64(layer.weight))
        shape = (6, layer.out_features)
        want = ot.grouped_int8(q, s, wq.reshape(*shape, -1), ws.reshape(shape), splits)
        assert (np.abs(f64(z) - want) <= (2.0 ** -8 + 4 * U) * np.abs(want)).all()
        if layer is block.fc1:
            gate, up = z.chunk(2, dim=1)
            y = torch.nn.functional.silu(gate) * up
    weights = torch.softmax(top.float(), dim=1)
    back = mxg.moe_combine(z, rows, weights)
    want, size = ot.combine(f64(z), host(rows), f64(weights))
    assert (np.abs(f64(back) - want) <= 2.0 ** -8 * np.abs(want) + 8 * U * size).all()
    assert torch.equal(out, x + back)


def test_splits_of_a_captured_plan():
    """Every replay sorts other choices: the counts are read anew."""
    T, k, E, C = 40, 2, 5, 24
    ids, x, _, _ = inputs(T, k, E, C, 0.2)
    TokenPlan(ids, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = TokenPlan(ids, E)
    for seed in range(3):
        ids.copy_(inputs(T, k, E, C, 0.2, seed=seed)[0])
        graph.replay()
        want = [int((ids == e).sum()) for e in range(E)]
        assert plan.m_splits() == want, seed
        assert dispatch(x, plan).shape == (sum(want), C)


@pytest.mark.parametrize("reentrant", [False, True])
def test_dropout_of_a_recomputed_forward(reentrant):
    """A forward that runs again in the backward pass, after the step went on, draws
    the mask of the state that it was given."""
    from torch.utils.checkpoint import checkpoint
    state = DropoutState(5)
    drop = Dropout(0.5, state)
    x = torch.randn((50, 64), device="cuda", requires_grad=True)
    d = torch.randn((50, 64), device="cuda")
    out = checkpoint(lambda x, s: drop(x * 1.0, residual=x, state=s), x, state.tensor, use_reentrant=reentrant,
                     preserve_rng_state=False)
    state.advance()
    out.backward(d)
    kept = torch.from_numpy(ot.dropout(np.zeros((50, 64)), 0.5, 5, 0, 0)[1]).cuda()
    assert torch.equal(x.grad, torch.where(kept, 2 * d, 0) + d)
    assert torch.equal(drop(x, state=torch.tensor([5, 0], device="cuda")) != 0, kept)


def test_dropout_goes_on_where_it_was_saved():
    x, state = torch.ones((64, 64), device="cuda"), DropoutState(2)
    state.advance()
    saved, want = state.state_dict(), Dropout(0.5, state)(x)
    other = DropoutState(9)
    other.load_state_dict(saved)
    assert torch.equal(Dropout(0.5, other)(x), want)


def test_two_dropouts_of_a_state_draw_two_masks():
    x, state = torch.ones((64, 64), device="cuda"), DropoutState(2)
    one, two = Dropout(0.5, state), Dropout(0.5, state)
    assert 0.3 < float(((one(x) == 0) == (two(x) == 0)).double().mean()) < 0.7
    assert torch.equal(one(x), mxg.dropout(x, 0.5, state.tensor, 0))


def test_plan_of_transposed_choices():
    ids, x, _, _ = inputs(30, 3, 5, 16, 0.1)
    plan, turned = TokenPlan(ids, 5), TokenPlan(ids.t().contiguous().t(), 5)
    assert torch.equal(plan.rows, turned.rows) and torch.equal(plan.counts, turned.counts)
    same = TokenPlan(ids[:1].expand(7, 3), 5)
    assert torch.equal(same.rows, TokenPlan(ids[:1].expand(7, 3).contiguous(), 5).rows)
