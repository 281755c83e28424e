"""The int8 quantizer and the int8 product on the GPU against the fp64 reference,
through the binding. Codes and scales are exact. The product's sum is exact; it is
rounded to fp32, scaled twice in fp32 and rounded to bf16: within
(2^-8 + 4 * 2^-24) of its magnitude."""
import numpy as np
import pytest

from oracle import tokens as ot

from .gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402

TOL = 2.0 ** -8 + 4 * 2.0 ** -24


def f64(t):
    return host(t.double())


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def check_codes(x):
    q, s = mxg.quantize_rowwise(x, "int8")
    wq, ws = ot.quantize_int8(f64(x))
    assert q.dtype == torch.int8 and np.array_equal(host(q), wq)
    assert np.array_equal(host(s), ws, equal_nan=True)


@pytest.mark.parametrize("rows,cols,pad", [(1, 16, 0), (3, 16, 8), (5, 112, 0), (17, 256, 0), (2, 272, 8), (7, 512, 0), (5, 528, 8), (9, 1024, 0),
                                           (4, 1040, 0), (3, 2000, 16), (5, 2048, 0), (3, 2064, 0), (2, 4096, 0), (3, 4112, 0), (2, 7168, 0),
                                           (2, 8208, 0), (1, 16384, 0), (2, 16400, 0), (2, 70000, 0), (1, 131056, 0),
                                           (0, 64, 0), (100001, 16, 0)])
def test_quantizer(rows, cols, pad):
    x = (torch.randn((rows, cols + pad), device="cuda", generator=gen(cols)) * 3).bfloat16()[:, :cols]
    if rows:
        check_codes(x)
    else:
        assert mxg.quantize_rowwise(x, "int8")[0].shape == (0, cols)


def test_quantizer_more_rows_than_workgroups():
    """2^20 workgroups at most, which stay for the rows behind."""
    R = (1 << 20) + 700
    x = torch.empty((R, 2064), dtype=torch.bfloat16, device="cuda").normal_(generator=gen(3))
    q, s = mxg.quantize_rowwise(x, "int8")
    for at in (slice(0, 3), slice((1 << 20) - 2, (1 << 20) + 2), slice(R - 3, R)):
        wq, ws = ot.quantize_int8(f64(x[at]))
        assert np.array_equal(host(q[at]), wq) and np.array_equal(host(s[at]), ws)
    assert bool((q.abs().amax(1) == 127).all())


def test_quantizer_all_ratios():
    """Every mantissa of the largest element, at the ends and in the middle of the
    exponents, against every bf16 value of the 11 binades from it downward, of
    either sign: ties and near ties among them."""
    for e in (1, 2, 60, 64, 100, 127, 190, 191, 254):
        top = np.arange(128, dtype=np.uint16) + (e << 7)
        down = np.minimum(np.arange(11 * 128, dtype=np.int32), (e << 7) + 127)
        bits = np.maximum(top[:, None].astype(np.int32) - down, 0).astype(np.uint16)
        bits[:, 1::3] |= 0x8000
        check_codes(torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16))
    denormal = np.arange(128, dtype=np.uint16)[:, None] * np.ones((1, 16), np.uint16)
    check_codes(torch.from_numpy(denormal.view(np.int16)).cuda().view(torch.bfloat16))


def test_quantizer_special_rows():
    x = torch.randn((6, 1040), device="cuda", generator=gen(0)).bfloat16()
    x[0] = 0
    x[1, 1039], x[2, 5], x[3, 700] = float("inf"), float("nan"), -float("inf")
    x[3, 701] = float("nan")
    x[4] = -x[4].abs()
    check_codes(x)


def weights(g, G, N, K):
    w_q = torch.randint(-127, 128, (G * N, K), dtype=torch.int8, device="cuda", generator=g)
    return w_q, torch.rand(G * N, device="cuda", generator=g) * 1e-3 + 1e-4


def check(splits, N, K, seed=0):
    g, G, M = gen(seed), len(splits), sum(splits)
    a_q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    a_s = torch.rand(M, device="cuda", generator=g) + 0.01
    w_q, w_s = weights(g, G, N, K)
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)[8 * (N % 8 == 0):]              # rows of odd width begin anywhere: a whole buffer of its own
    got = mxg.grouped_fwd(a_q, a_s, w_q, w_s, splits, N, K, "int8", "int8", out=flat[:M * N].view(M, N))
    want = ot.grouped_int8(host(a_q), host(a_s), host(w_q).reshape(G, N, K), host(w_s).reshape(G, N), splits)
    assert (np.abs(f64(got) - want) <= TOL * np.abs(want)).all()
    assert (flat[M * N:] == 7).all()                    # what lies behind the last row stays


@pytest.mark.parametrize("splits,N,K", [
    ([1], 1, 16), ([1], 64, 64), ([3], 33, 48), ([16], 16, 128), ([17], 257, 144), ([64], 256, 256), ([65], 100, 272),
    ([1, 0, 2], 48, 64), ([0, 0, 5, 0], 130, 1040), ([31, 33, 0, 1], 96, 512), ([255, 256, 257], 255, 112),
    ([300, 0, 7], 515, 400), ([1] * 40, 72, 192), ([2000], 1111, 2000), ([513, 1, 700], 520, 4096),
    ([128, 129, 60], 1, 64), ([1], 4096, 7168), ([8], 2048, 8208), ([48, 3, 64], 264, 4112),
    # one shape at least for every form of the kernel: few tokens ...
    ([1], 4100, 160), ([3, 1], 9000, 96), ([30], 1500, 2064), ([64], 4096, 272), ([40], 8200, 80), ([60, 50], 5000, 144),
    ([250], 4100, 96), ([33] * 9, 1030, 592), ([16], 16000, 4096), ([48], 4100, 4096), ([24], 4099, 4096), ([60], 4095, 2000),
    # ... 128 x 128 tiles, and 256 x 256, with rounds of both
    ([1024], 4096, 144), ([700, 0, 1300, 77], 3001, 272), ([100] * 20, 2000, 64), ([4096], 4096, 144),
    ([1300, 0, 2900, 77], 4004, 208), ([257] * 12, 4099, 80), ([9000], 2050, 336),
    ([3000, 1500, 2500], 4099, 176)])
def test_product(splits, N, K):
    check(splits, N, K)


OPTIONS = [(256, 256, 29, 8), (128, 128, 11.5, 2.2), (16, 16, 0, .5), (32, 16, 0, .5), (16, 32, 0, .5), (32, 32, 0, 1.6),
           (32, 64, 0, 1.6), (64, 32, 0, 1.6), (64, 64, 0, 1.6)]


def form(splits, N, K):
    """int8_form restated: the least of rounds times what a workgroup takes."""
    def cost(o):
        pieces = sum(-(-m // o[1]) for m in splits)
        return -(-pieces * -(-N // o[0]) // 256) * ((o[2] or o[0] / 16 + sum(splits) / pieces / 16) + o[3] * 4096 / K)
    return min(OPTIONS, key=cost)[:2]


def test_every_form_is_chosen():
    marks = [m for m in test_product.pytestmark if m.name == "parametrize"][0].args[1]
    assert {form(*m) for m in marks} == {o[:2] for o in OPTIONS}


def test_many_experts():
    rng = np.random.default_rng(0)
    check([int(v) for v in rng.integers(0, 4, 512)], 24, 80)
    check([int(v) for v in rng.integers(0, 90, 100)], 40, 160)
    check([0] * 511 + [300], 40, 160)


def test_longest_contraction():
    """All codes -128, the most that 32 bits have to hold: 2^14 K < 2^31."""
    K = (1 << 17) - 16
    for M in (2, 300):
        a_q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        w_q = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
        w_q[10:] = 127
        one = torch.ones(M, device="cuda"), torch.ones(20, device="cuda")
        got = f64(mxg.grouped_fwd(a_q, one[0], w_q, one[1], [M], 20, K, "int8", "int8"))
        want = np.repeat([[16384.0 * K] * 10 + [-16256.0 * K] * 10], M, 0)
        assert (np.abs(got - want) <= TOL * np.abs(want)).all()


def test_special_rows():
    """A token that holds NaN or infinity comes out as NaN, alone; one of zeros as zeros."""
    x = torch.randn((40, 256), device="cuda", generator=gen(1)).bfloat16()
    x[3], x[7, 9], x[20, 255] = 0, float("nan"), float("inf")
    w_q, w_s = weights(gen(2), 2, 72, 256)
    q, s = mxg.quantize_rowwise(x, "int8")
    for splits in ([10, 30], [40, 0]):
        y = host(mxg.grouped_fwd(q, s, w_q, w_s, splits, 72, 256, "int8", "int8").float())
        bad = np.isnan(y).all(1)
        assert bad[[7, 20]].all() and bad.sum() == 2 and np.isfinite(np.delete(y, [7, 20], 0)).all() and not y[3].any()


def test_linear_layer():
    """Quantized on both sides, the product is near the unquantized one: a code is
    half a step off at most, so a sum is within K (sx |w| + sw |x| + sx sw / 2) / 2."""
    g = gen(5)
    x = torch.randn((70, 512), device="cuda", generator=g).bfloat16()
    w = torch.randn((2 * 96, 512), device="cuda", generator=g).bfloat16()
    xq, xs = mxg.quantize_rowwise(x, "int8")
    wq, ws = mxg.quantize_rowwise(w, mxg.INT8)
    got = f64(mxg.grouped_fwd(xq, xs, wq, ws, [30, 40], 96, 512, "int8", "int8"))
    hx, hw, sx, sw = f64(x), f64(w), f64(xs), f64(ws)
    for g0, lo, hi in ((0, 0, 30), (1, 30, 70)):
        wg, wsg = hw[g0 * 96:(g0 + 1) * 96], sw[g0 * 96:(g0 + 1) * 96]
        want = hx[lo:hi] @ wg.T
        off = (sx[lo:hi, None] * np.abs(wg).sum(1) + np.abs(hx[lo:hi]).sum(1)[:, None] * wsg
               + 256 * sx[lo:hi, None] * wsg) / 2
        assert (np.abs(got[lo:hi] - want) <= off * (1 + 1e-5) + TOL * (np.abs(want) + off)).all()


def test_offsets_past_32_bits():
    """The last experts' codes begin past 2^32 bytes."""
    G, N, K = 70, 4096, 16384
    w_q = torch.empty((G * N, K), dtype=torch.int8, device="cuda")
    w_q.random_(-127, 128, generator=gen(0))
    w_s = torch.full((G * N,), 1e-3, device="cuda")
    for m in (5, 300):
        splits = [0] * G
        splits[G - 1] = m
        a_q = torch.randint(-127, 128, (m, K), dtype=torch.int8, device="cuda", generator=gen(1))
        a_s = torch.ones(m, device="cuda")
        got = f64(mxg.grouped_fwd(a_q, a_s, w_q, w_s, splits, N, K, "int8", "int8"))
        want = ot.grouped_int8(host(a_q), host(a_s), host(w_q[-N:])[None], host(w_s[-N:])[None], [m])
        assert (np.abs(got - want) <= TOL * np.abs(want)).all()


def test_streams_and_graph():
    g = gen(6)
    x = torch.randn((90, 640), device="cuda", generator=g).bfloat16()
    w_q, w_s = weights(g, 3, 200, 640)

    def step(splits):
        q, s = mxg.quantize_rowwise(x, "int8")
        return mxg.grouped_fwd(q, s, w_q, w_s, splits, 200, 640, "int8", "int8")
    for splits in ([90, 0, 0], [2, 0, 88], [30, 30, 30]):
        want = step(splits)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step(splits)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(splits)
        for seed in range(3):
            x.copy_(torch.randn((90, 640), device="cuda", generator=gen(seed)).bfloat16())
            want = step(splits)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), seed


@pytest.mark.parametrize("splits", [[2 ** 31 - 1], [7, 2 ** 31 - 20, 12]])
def test_most_rows(splits):
    """2^31 - 1 rows, nearly all of one expert, whose last tile would end past 2^31."""
    M, K, G = sum(splits), 16, len(splits)
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GiB of memory are not free")
    a_q = torch.empty((M, K), dtype=torch.int8, device="cuda").fill_(2)
    a_q[-300:] = 3
    w_q = torch.ones((G, K), dtype=torch.int8, device="cuda")
    w_s = torch.arange(1.0, G + 1, device="cuda")
    a_s = torch.empty(M, device="cuda").fill_(0.5)
    out = torch.empty((M, 1), dtype=torch.bfloat16, device="cuda").fill_(-1)
    mxg.grouped_fwd(a_q, a_s, w_q, w_s, splits, 1, K, "int8", "int8", out=out)
    at = 0
    for g, m in enumerate(splits):
        plain = min(m, max(M - 300 - at, 0))
        assert bool((out[at:at + plain] == 16 * (g + 1)).all()) and bool((out[at + plain:at + m] == 24 * (g + 1)).all())
        at += m
