"""The few-token expert layer on the GPU against the fp64 reference (its bound
is derived in oracle/block.py). Weights are quantized by the library's
quantizers, whose codes are bit-exact with the oracle's."""
import functools
import math

import numpy as np
import pytest

from oracle import block as ob
from oracle import blockwise as obw
from oracle import mx as omx
from synth import bf16_normal

from .gpu_util import dev_bf16, have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402

INF = math.inf


def f64(t):
    return t.detach().double().cpu().numpy()


def weights(E, rows, K, fmt, layout, seed):
    """(codes, scales) as the library's quantizer writes them, and the dense
    fp64 [E, rows, K] that they stand for."""
    bits = bf16_normal((E * rows, K), 1.0 / math.sqrt(K), seed)
    if fmt.startswith("fp8_128x128"):
        q, s = mxg.quantize_rowwise(dev_bf16(bits), fmt, flags=mxg.POW2_SCALES if fmt.endswith("p2") else 0)
        dense = obw.dequantize_128x128(*obw.quantize_128x128(bits, pow2=fmt.endswith("p2")))
    else:
        f = mxg.FORMATS[fmt] | (mxg.KBLOCK_ROWS if layout == "kblock" else 0)
        q, s = mxg.quantize_rowwise(dev_bf16(bits), f)
        dense = omx.dequantize_rowwise(*omx.quantize_rowwise(bits, fmt), fmt)
    return q, s, dense.reshape(E, rows, K)


class Layer:
    def __init__(self, E, H, inner, fmt="mxfp4", layout="rows", seed=0):
        self.E, self.H, self.inner = E, H, inner
        self.fmt = mxg.FORMATS[fmt] | (mxg.KBLOCK_ROWS if layout == "kblock" and fmt.startswith("mx") else 0)
        self.w13_q, self.w13_s, self.w13 = weights(E, 2 * inner, H, fmt, layout, seed + 1)
        self.w2_q, self.w2_s, self.w2 = weights(E, H, inner, fmt, layout, seed + 2)

    def run(self, x, logits, k, renormalize=True, **kw):
        return mxg.moe_layer(x, logits, self.w13_q, self.w13_s, self.w2_q, self.w2_s, k, fmt=self.fmt,
                             renormalize=renormalize, **kw)

    def check(self, x, logits, k, renormalize=True):
        out, ids, p = self.run(x, logits, k, renormalize)
        want, wids, wp, bound = ob.moe_layer(f64(x), f64(logits), self.w13, self.w2, k, renormalize)
        assert np.array_equal(ids.cpu().numpy(), wids)
        # exp, a sum of at most 512 terms and a quotient in fp32
        assert (np.abs(f64(p) - wp) <= 64 * 2.0 ** -24 * wp).all()
        err = np.abs(f64(out) - want)
        assert (err <= bound + 64 * 2.0 ** -24 * np.abs(want)).all(), float(np.max(err / np.maximum(bound, 1e-300)))
        return out, ids, p


def tokens(T, H, E, seed=0, pad=0):
    x = dev_bf16(bf16_normal((T, H + pad), 1.0, seed + 10))[:, :H]
    return x, dev_bf16(bf16_normal((T, E), 2.0, seed + 11)).float()


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("fmt,layout,H,inner", [
    ("mxfp4", "rows", 288, 160), ("mxfp4", "kblock", 256, 128), ("mxfp8", "rows", 96, 224), ("mxfp8", "kblock", 384, 128),
    ("fp8_128x128", "kblock", 128, 256), ("fp8_128x128_p2", "kblock", 256, 128)])
def test_token_counts_and_formats(T, fmt, layout, H, inner):
    layer = Layer(6, H, inner, fmt, layout)
    x, logits = tokens(T, H, 6, T)
    layer.check(x, logits, 3)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 1), (16, 16), (65, 8), (130, 5), (512, 4)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_experts_and_choices(E, k, renormalize):
    layer = Layer(E, 64, 32)
    x, logits = tokens(13, 64, E, E)
    layer.check(x, logits, k, renormalize)


def test_all_tokens_on_one_expert():
    for T in (16, 30, 64):
        layer = Layer(4, 128, 64, seed=T)
        x, logits = tokens(T, 128, 4)
        logits[:, 2] = 50.0
        layer.check(x, logits, 1)
        layer.check(x, logits, 2)


@pytest.mark.parametrize("H,inner", [(32, 32), (2080, 32), (32, 992), (1056, 544)])
def test_sizes_that_end_inside_a_piece(H, inner):
    for fmt in ("mxfp4", "mxfp8"):
        layer = Layer(3, H, inner, fmt)
        layer.check(*tokens(5, H, 3, 1), 2)


def test_strided_inputs_and_bf16_logits():
    layer = Layer(10, 128, 64)
    x, logits = tokens(9, 128, 10, pad=24)
    assert x.stride(0) == 152
    big = torch.full((9, 23), 99.0, device="cuda")
    big[:, 3:13] = logits
    a = layer.check(x, big[:, 3:13], 3)
    b = layer.check(x, big.bfloat16()[:, 3:13], 3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_masked_experts_ties_and_extreme_logits():
    layer = Layer(70, 64, 32)
    x, logits = tokens(12, 64, 70)
    low = torch.finfo(torch.float32).min
    logits[0] = -INF                      # nothing to choose
    logits[1] = -INF
    logits[1, 69] = -3.0                  # one of four
    logits[2] = low                       # the type's lowest is a logit like any other
    logits[3] = low
    logits[3, [5, 66]] = 1.0
    logits[4] = 0.0                       # all equal
    logits[5, 64:] = 7.0                  # ties across the wave's slots
    logits[6] = torch.where(torch.arange(70, device="cuda") % 2 == 0, 0.0, -0.0)
    logits[7, 3] = 1e30                   # the others' softmax vanishes
    for renormalize in (True, False):
        out, ids, p = layer.check(x, logits, 4, renormalize)
        assert not out[0].any() and (ids[0] == -1).all() and not p[0].any()
        assert ids[1].tolist() == [69, -1, -1, -1]
        assert ids[2].tolist() == [0, 1, 2, 3] and ids[4].tolist() == [0, 1, 2, 3] and ids[6].tolist() == [0, 1, 2, 3]
        assert ids[3].tolist() == [5, 66, 0, 1]


def test_nothing_chosen_at_all():
    layer = Layer(4, 64, 32)
    x, logits = tokens(3, 64, 4)
    out, ids, p = layer.run(x, torch.full_like(logits, -INF), 2)
    assert not out.any() and (ids == -1).all() and not p.any()


def test_nan_and_infinite_logits_and_tokens_stay_their_own():
    layer = Layer(8, 96, 64)
    x, logits = tokens(20, 96, 8)
    clean = layer.run(x, logits, 3)
    bad, lg = x.clone(), logits.clone()
    bad[4, 7] = float("nan")
    bad[17] = INF
    lg[9, 2] = float("nan")
    lg[11, 5] = INF
    out, ids, p = layer.run(bad, lg, 3)
    keep = [t for t in range(20) if t not in (4, 9, 11, 17)]
    for a, b in zip(clean, (out, ids, p)):
        assert torch.equal(a[keep], b[keep])
    assert out[[4, 9, 11, 17]].isnan().all() and p[[9, 11]].isnan().all()
    assert ids[9, 0] == 2 and ids[11, 0] == 5


def test_a_broken_expert_reaches_only_its_tokens():
    layer = Layer(6, 128, 128, "mxfp8")
    x, logits = tokens(24, 128, 6)
    clean, ids, _ = layer.run(x, logits, 2)
    layer.w13_q.view(6, 256, 128)[3, 5, 7] = 0x7F     # E4M3 NaN
    layer.w2_q.view(6, 128, 128)[3, 9] = 0xFF
    out, ids2, _ = layer.run(x, logits, 2)
    uses = (ids == 3).any(1)
    assert uses.any() and not uses.all() and torch.equal(ids, ids2)
    assert torch.equal(out[~uses], clean[~uses]) and out[uses].isnan().any(1).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "fp8_128x128"])
def test_every_code_and_scale_is_read_exactly(fmt):
    # x[t] = e_t, gate rows 64 e_t (silu(64) is 64 in fp32), up rows e_t / 64:
    # the inner activation of token t is e_t, and the output a column of W2
    n = 64
    H = inner = 128 if fmt.startswith("fp8") else n
    w13 = np.zeros((2 * inner, H), np.float32)
    w13[np.arange(n), np.arange(n)] = 64.0
    w13[inner + np.arange(n), np.arange(n)] = 1.0 / 64
    w13 = torch.from_numpy(w13).cuda().bfloat16()
    f = mxg.FORMATS[fmt]
    w13_q, w13_s = mxg.quantize_rowwise(w13, f)
    rng = np.random.default_rng(1)
    if fmt == "mxfp4":
        q = rng.integers(0, 256, (H, inner // 2), dtype=np.uint8)
    else:
        q = rng.integers(0, 256, (H, inner), dtype=np.uint8)
        q[(q & 0x7F) == 0x7F] = 0x7E                      # no NaN codes
    if fmt == "fp8_128x128":
        s = np.array([[0.0123]], np.float32)
        dense = obw.dequantize_128x128(q, s)
        q = np.ascontiguousarray(q.reshape(H, inner // 64, 64).transpose(1, 0, 2))
        sd = torch.from_numpy(s).cuda()
    else:
        s = rng.integers(20, 240, (H, inner // 32), dtype=np.uint8)
        dense = omx.dequantize_rowwise(q, s, fmt)
        sd = torch.from_numpy(np.ascontiguousarray(s.T)).cuda()
    x = torch.eye(n, H, device="cuda").bfloat16()
    logits = torch.zeros((n, 1), device="cuda")
    out, _, _ = mxg.moe_layer(x, logits, w13_q, w13_s, torch.from_numpy(q).cuda(), sd, 1, fmt=f)
    want = torch.from_numpy(np.ascontiguousarray(dense[:, :n].T)).float().bfloat16()
    assert torch.equal(out.cpu(), want)


def test_kblocked_and_plain_rows_agree():
    rows = Layer(5, 256, 384, "mxfp4", "rows", 3)
    blocks = Layer(5, 256, 384, "mxfp4", "kblock", 3)
    x, logits = tokens(11, 256, 5)
    assert all(torch.equal(a, b) for a, b in zip(rows.run(x, logits, 2), blocks.run(x, logits, 2)))


def test_no_tokens_and_caller_buffers():
    layer = Layer(4, 64, 32)
    x, logits = tokens(6, 64, 4)
    out, ids, p = layer.run(x[:0], logits[:0], 2)
    assert out.shape == (0, 64) and ids.shape == (0, 2)
    a = layer.run(x, logits, 2)
    ws = torch.full((mxg.lib.mxgg_moe_layer_workspace(6, 4, 2, 32),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((6, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    b = layer.run(x, logits, 2, out=out, ws=ws)
    assert b[0] is out and all(torch.equal(u, v) for u, v in zip(a, b))


def test_same_bits_each_run_and_on_another_stream():
    layer = Layer(32, 512, 256, "mxfp4", "kblock")
    x, logits = tokens(40, 512, 32)
    first = layer.run(x, logits, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = layer.run(x, logits, 4)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_graph_replays():
    layer = Layer(16, 256, 128)
    x, logits = tokens(4, 256, 16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.run(x, logits, 4)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = layer.run(x, logits, 4)
    for seed in (1, 2, 3):
        nx, nl = tokens(4, 256, 16, seed)
        x.copy_(nx)
        logits.copy_(nl)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, layer.run(nx, nl, 4)))


def test_output_and_workspace_end_where_they_should():
    layer = Layer(3, 64, 32)
    x, logits = tokens(5, 64, 3)
    need = mxg.lib.mxgg_moe_layer_workspace(5, 3, 2, 32)
    buf = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    outs = torch.full((7, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    layer.run(x, logits, 2, ws=buf[:need], out=outs[:5])
    assert (buf[need:] == 7).all() and (outs[5:] == 3).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_scales_at_the_ends_of_their_range(fmt):
    # as above, one scale for each of 2 x 32 columns: 2^-127 to 2^127, within
    # what bf16 holds of the products (its smallest step is 2^-133)
    n = 64
    w13 = np.zeros((2 * n, n), np.float32)
    w13[np.arange(n), np.arange(n)] = 64.0
    w13[n + np.arange(n), np.arange(n)] = 1.0 / 64
    w13_q, w13_s = mxg.quantize_rowwise(torch.from_numpy(w13).cuda().bfloat16(), mxg.FORMATS[fmt])
    rng = np.random.default_rng(2)
    q = rng.integers(0, 256, (n, n // 2 if fmt == "mxfp4" else n), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x7E
    s = np.zeros((n, 2), np.uint8)
    s[:, 0] = np.resize([0, 1, 2, 3, 8, 9, 10, 20], n)
    s[:, 1] = np.resize([230, 240, 244, 245, 127, 126, 128, 100], n)
    dense = omx.dequantize_rowwise(q, s, fmt)
    x = torch.eye(n, device="cuda").bfloat16()
    out, _, _ = mxg.moe_layer(x, torch.zeros((n, 1), device="cuda"), w13_q, w13_s, torch.from_numpy(q).cuda(),
                              torch.from_numpy(np.ascontiguousarray(s.T)).cuda(), 1, fmt=fmt)
    want = torch.from_numpy(np.ascontiguousarray(dense.T)).float().bfloat16()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("layout", ["rows", "kblock"])
def test_weights_past_32_bit_offsets(layout):
    # 4.4 GB of W1 and W3 codes; only the last expert's are not zero
    E, H, inner = 130, 8192, 2048
    layer = Layer(1, H, inner, "mxfp8", layout, seed=5)

    def last_of(t, rows, at):
        shape = list(t.shape)
        shape[at] = E * rows
        big = torch.zeros(shape, dtype=t.dtype, device="cuda")
        big.narrow(at, (E - 1) * rows, rows).copy_(t)
        return big
    axis = 1 if layout == "kblock" else 0
    w13_q, w2_q = last_of(layer.w13_q, 2 * inner, axis), last_of(layer.w2_q, H, axis)
    w13_s, w2_s = last_of(layer.w13_s, 2 * inner, 1), last_of(layer.w2_s, H, 1)
    assert w13_q.numel() > 2 ** 32
    x, _ = tokens(3, H, 1)
    logits = torch.zeros((3, E), device="cuda")
    logits[:, E - 1] = 1.0
    out, ids, _ = mxg.moe_layer(x, logits, w13_q, w13_s, w2_q, w2_s, 1, fmt=layer.fmt)
    assert (ids == E - 1).all()
    assert torch.equal(out, layer.run(x, logits[:, :1], 1)[0])


@functools.lru_cache(maxsize=None)
def shared_layer(*args):
    return Layer(*args)


# The first product's workgroups (one a CU, 256) take several units of 16 or 32
# inner columns in turn: here each has three or more, some none in the last round.
# `inner` 1120: a last piece that is not whole; `hidden` 256 and 288: fewer pieces
# than waves; 1056: more. One to three token loads a piece.
@pytest.mark.parametrize("E,H,inner,fmt,layout,T,k", [
    (16, 288, 1120, "mxfp4", "rows", 1, 8), (16, 288, 1120, "mxfp4", "rows", 13, 4), (16, 288, 1120, "mxfp4", "rows", 32, 6),
    (16, 288, 1120, "mxfp4", "rows", 64, 4), (16, 256, 1152, "mxfp4", "kblock", 1, 8), (16, 256, 1152, "mxfp4", "kblock", 32, 6),
    (16, 288, 1120, "mxfp8", "rows", 1, 8), (16, 288, 1120, "mxfp8", "rows", 13, 4), (16, 288, 1120, "mxfp8", "rows", 40, 5),
    (16, 256, 1152, "fp8_128x128", "kblock", 1, 8), (16, 256, 1152, "fp8_128x128", "kblock", 13, 4),
    (16, 256, 1152, "fp8_128x128", "kblock", 40, 5),
    (4, 1056, 2272, "mxfp4", "rows", 1, 4), (4, 1056, 2272, "mxfp4", "rows", 26, 4), (4, 1056, 2272, "mxfp8", "rows", 3, 4)])
def test_many_units_a_workgroup(E, H, inner, fmt, layout, T, k):
    x, logits = tokens(T, H, E, T)
    shared_layer(E, H, inner, fmt, layout).check(x, logits, k)


# The second product with 64-row tiles, split over workgroups, for few tokens an
# expert: one token load a piece (T k / E up to about 2 with E2M1 codes, 4 with E4M3)
# or two (up to about 4; with E4M3 8), at most 32 tokens and more.
@pytest.mark.parametrize("fmt,layout,H,inner", [
    ("mxfp4", "rows", 96, 160), ("mxfp4", "kblock", 128, 128), ("mxfp8", "rows", 96, 160), ("mxfp8", "kblock", 128, 128),
    ("fp8_128x128", "kblock", 128, 256)])
@pytest.mark.parametrize("T,k", [(17, 2), (32, 4), (64, 2), (64, 4), (32, 14), (64, 6)])
def test_many_tokens_few_to_an_expert(fmt, layout, H, inner, T, k):
    x, logits = tokens(T, H, 100, T + k)
    shared_layer(100, H, inner, fmt, layout).check(x, logits, k)


@pytest.mark.parametrize("fmt,layout,inner", [("mxfp4", "rows", 96), ("mxfp8", "kblock", 128), ("fp8_128x128", "kblock", 128)])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_wide_outputs_few_tokens(fmt, layout, inner, T):
    # from 6144 outputs on the 64-row tiles serve single tokens too
    x, logits = tokens(T, 6272, 5, T)
    shared_layer(5, 6272, inner, fmt, layout).check(x, logits, 2)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_most_tokens_choices_and_experts(fmt):
    # the largest lists, and the most LDS that the second product asks for
    x, logits = tokens(64, 32, 512, 3)
    shared_layer(512, 32, 32, fmt, "rows").check(x, logits, 16)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("H,inner,layouts", [(256, 128, ("rows", "kblock")), (256, 96, ("kblock", "rows")),
                                             (96, 256, ("rows", "kblock"))])
@pytest.mark.parametrize("T", [2, 40])
def test_code_layout_of_each_matrix(fmt, H, inner, layouts, T):
    layer = Layer(5, H, inner, fmt, "rows", 7)
    x, logits = tokens(T, H, 5, T)
    want = layer.check(x, logits, 2)
    f13, f2 = (mxg.FORMATS[fmt] | (mxg.KBLOCK_ROWS if l == "kblock" else 0) for l in layouts)
    if f13 & mxg.KBLOCK_ROWS:
        layer.w13_q, layer.w13_s, _ = weights(5, 2 * inner, H, fmt, "kblock", 8)
    if f2 & mxg.KBLOCK_ROWS:
        layer.w2_q, layer.w2_s, _ = weights(5, H, inner, fmt, "kblock", 9)
    layer.fmt = f13
    assert all(torch.equal(a, b) for a, b in zip(want, layer.run(x, logits, 2, w2_fmt=f2)))
