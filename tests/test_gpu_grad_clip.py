"""The norm of many gradients and clipping on the GPU against the fp64
reference. The norm is an fp64 sum rounded to fp32: 2^-23 of its value; the
factor one fp32 sum and quotient of it: another 2^-22; then each gradient's own
rounding (bf16: 2^-8, and below the normal numbers one step of the type)."""
import math

import numpy as np
import pytest

from oracle import block as ob

from .gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(d).cuda() for n, d in zip(sizes, dtypes)]


def check(grads, max_norm, norm_type=2.0):
    before = [f64(g) for g in grads]
    want = ob.grad_norm(before, norm_type)
    got = mxg.grad_norm(grads, norm_type)
    assert got.shape == () and abs(float(got) - want) <= 2.0 ** -23 * want
    assert all(np.array_equal(f64(g), b) for g, b in zip(grads, before))
    total = mxg.clip_grad_norm(grads, max_norm, norm_type)
    assert torch.equal(total, got)
    f = ob.clip_factor(want, max_norm)
    for g, b in zip(grads, before):
        if f == 1.0:
            assert np.array_equal(f64(g), b)
        else:
            tol = (2.0 ** -8 if g.dtype == BF16 else 0.0) + 2.0 ** -21
            step = 2.0 ** -133 if g.dtype == BF16 else 2.0 ** -149
            assert (np.abs(f64(g) - b * f) <= tol * np.abs(b * f) + step).all()


@pytest.mark.parametrize("norm_type", [2.0, math.inf])
@pytest.mark.parametrize("max_norm", [0.25, 1e9, 0.0])
def test_mixed_types_and_sizes(norm_type, max_norm):
    sizes = [1, 7, 8, 0, 255, 4096, 8191, 8192, 8193, 100_001, 3]
    check(make(sizes, [F32, BF16] * 6, 1), max_norm, norm_type)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 256, 257, 400])
def test_tensor_counts(n):
    rng = np.random.default_rng(n)
    check(make(rng.integers(0, 3000, n).tolist(), [F32 if i % 3 else BF16 for i in range(n)], n), 1.0)


def test_slices_at_every_alignment():
    for dtype in (BF16, F32):
        flat = torch.randn(40_000, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
        keep = flat.clone()
        cuts = [1, 2, 3, 5, 8, 13, 8192, 8193, 20_001]
        parts, at = [], 1
        for c in cuts[:-1]:
            parts.append(flat[at:at + c])
            at += c + 1             # one element between any two stays out
        check(parts, 0.5)
        held = torch.ones(40_000, dtype=torch.bool)
        at = 1
        for c in cuts[:-1]:
            held[at:at + c] = False
            at += c + 1
        assert torch.equal(flat[held.cuda()], keep[held.cuda()])


def test_large_tensor_and_shapes():
    g = [torch.randn((3, 1000, 1024), device="cuda", generator=torch.Generator("cuda").manual_seed(1)),
         torch.randn((1000, 1025), device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()]
    check(g, 5.0)


def test_squares_past_fp32_and_below_it():
    for scale in (1e25, 1e-30):
        check(make([1000, 50], [F32, BF16], 4, scale), scale)


def test_nothing():
    assert float(mxg.grad_norm([])) == 0.0
    e = torch.empty(0, device="cuda")
    assert float(mxg.clip_grad_norm([e], 1.0)) == 0.0
    assert float(mxg.clip_grad_norm([e, torch.zeros(5, device="cuda")], 1.0)) == 0.0


@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_nan_and_infinity(norm_type):
    a, b = make([9000, 20], [F32, BF16], 5)
    a[8999] = float("inf")
    total = mxg.clip_grad_norm([a, b], 1.0, norm_type)
    assert float(total) == math.inf and torch.isnan(a[8999]) and not a[:8999].any() and not b.any()
    a, b = make([9000, 20], [F32, BF16], 5)
    b[0] = float("nan")
    assert math.isnan(float(mxg.clip_grad_norm([a, b], 1.0, norm_type))) and a.isnan().all() and b.isnan().all()


def test_norm_over_ranks():
    # two shards: their norms combined, then each scaled by the whole's norm
    whole = make([5000, 777], [F32, BF16], 6)
    shards = [[g.clone()] for g in whole]
    total = torch.stack([mxg.grad_norm(s) for s in shards]).square().sum().sqrt()
    for s in shards:
        mxg.clip_grads_with_norm(s, 2.0, total)
    want = ob.grad_norm([f64(g) for g in whole])
    f = ob.clip_factor(want, 2.0)
    for s, g in zip(shards, whole):
        tol = (2.0 ** -8 if g.dtype == BF16 else 0.0) + 2.0 ** -20
        assert (np.abs(f64(s[0]) - f64(g) * f) <= tol * np.abs(f64(g) * f)).all()


def test_same_bits_other_stream_poisoned_workspace():
    grads = make([3_000_000, 700_001], [F32, BF16], 7)
    copy = [g.clone() for g in grads]
    first = mxg.clip_grad_norm(grads, 1.0)
    ws = torch.full((mxg.lib.mxgg_grad_norm_workspace(2),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = mxg.clip_grad_norm(copy, 1.0, ws=ws)
    s.synchronize()
    assert torch.equal(first, second) and all(torch.equal(a, b) for a, b in zip(grads, copy))


def test_graph_replays():
    grads = make([10_000, 333], [F32, BF16], 8)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        mxg.clip_grad_norm(grads, 1.0)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        total = mxg.clip_grad_norm(grads, 1.0)
    for seed in (1, 2, 3):
        fresh = make([10_000, 333], [F32, BF16], seed)
        for g, f in zip(grads, fresh):
            g.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = mxg.clip_grad_norm(fresh, 1.0)
        assert torch.equal(total, want) and all(torch.equal(a, b) for a, b in zip(grads, fresh))


def test_more_elements_than_32_bits_count():
    g = torch.zeros(2 ** 31 + 5, dtype=BF16, device="cuda")
    g[0], g[-1] = 3.0, 4.0
    assert float(mxg.clip_grad_norm([g], 1.0)) == 5.0
    assert torch.equal(g[[0, -1]].cpu(), torch.tensor([0.6, 0.8]).bfloat16()) and int(g.count_nonzero()) == 2
