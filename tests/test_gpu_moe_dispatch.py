"""Tokens to their experts and back on the GPU against the fp64 reference, through
the binding. Sorting and copying are exact; sums: with u = 2^-24 a sum of n fp32
products in any order whose partial sums add at most 256 terms is within
256 u sum|a b|, a bf16 rounding within 2^-8 |v|."""
import numpy as np
import pytest

from oracle import tokens as ot

from .gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}


def f64(t):
    return host(t.double())


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def choices(g, T, k, E, dropped=0.0, dtype=torch.int32):
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g)
    out = torch.rand((T, k), device="cuda", generator=g) < dropped
    return torch.where(out, torch.randint(-3, 0, (T, k), device="cuda", generator=g), ids).to(dtype)


def rows_of(g, R, C, dt, pad=0, offset=0):
    """[R, C] inside rows of C + pad, `offset` elements into its memory."""
    flat = torch.randn(R * (C + pad) + offset, device="cuda", generator=g).to(dt)
    return flat[offset:].view(R, C + pad)[:, :C]


def check_sort(ids, E):
    got = [host(t) for t in mxg.moe_sort(ids, E)]
    for a, b, name in zip(got, ot.sort(host(ids), E), ("rows", "choices", "counts")):
        assert np.array_equal(a, b), name


# one choice, a wave, one workgroup's chunk and its borders, several chunks, more
# than one launch adds up, ragged ends
@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (1, 16, 512), (9, 7, 3), (256, 8, 128), (257, 8, 512), (2048, 1, 1),
                                   (2049, 1, 64), (5000, 3, 129), (8192, 8, 512), (8193, 8, 9), (32768, 8, 64), (32769, 8, 511),
                                   (100003, 5, 17), (131071, 8, 100), (131072, 8, 3), (140001, 8, 511)])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_sort(T, k, E, itype):
    check_sort(choices(gen(T), T, k, E, 0.1 if T % 2 else 0.0, itype), E)


def test_sort_extremes():
    for T in (300, 3000):
        check_sort(torch.full((T, 4), 6, device="cuda"), 7)                   # one expert, equal choices of a token
        check_sort(torch.full((T, 4), -1, device="cuda"), 7)                  # nothing kept
        check_sort(torch.full((T, 4), 7, device="cuda"), 7)                   # the first number past the experts
        big = torch.tensor([2 ** 32, 2 ** 32 + 1, -2 ** 40, 3], device="cuda").repeat(T, 1)
        check_sort(big, 7)                                                    # outside in 64 bits, inside in 32
        wide = choices(gen(1), T, 9, 7)
        check_sort(wide[:, 2:6], 7)                                           # rows inside wider rows
        check_sort(wide[::3, :5], 7)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,C,pad,offset,dropped", [
    (1, 1, 1, 1, 0, 0, 0.0), (5, 3, 4, 7, 0, 0, 0.4), (3, 2, 4, 8, 3, 1, 0.0), (33, 16, 40, 63, 5, 3, 0.3),
    (17, 8, 32, 1001, 3, 1, 0.2), (64, 8, 16, 2048, 0, 0, 0.0), (11, 5, 9, 2049, 0, 0, 1.0), (6, 4, 8, 7168, 8, 0, 0.3),
    (3, 2, 2, 20001, 0, 1, 0.3), (1025, 2, 6, 96, 0, 0, 0.1), (300, 4, 6, 3, 1, 0, 0.1)])
def test_rows(dt, T, k, E, C, pad, offset, dropped):
    g = gen(T * C)
    rows, _, counts = mxg.moe_sort(choices(g, T, k, E, dropped), E)
    hr, total, n = host(rows), int(counts.sum()), T * k
    x = rows_of(g, T, C, DT[dt], pad, offset)
    # dispatch: copies
    assert np.array_equal(f64(mxg.moe_dispatch(x, rows)), ot.dispatch(f64(x), hr, n))
    # fewer rows, and into rows inside wider ones, whose surroundings stay
    room = rows_of(g, n + 2, C, DT[dt], pad + 2, offset)
    for R in sorted({total, max(total - 1, 0), n}):
        before = f64(room)
        y = mxg.moe_dispatch(x, rows, R, out=room[1:R + 1] if R else None)
        want = ot.dispatch(f64(x), hr, R, before[1:R + 1])
        assert np.array_equal(f64(y), want)
        assert np.array_equal(f64(room), np.concatenate([before[:1], want, before[R + 1:]])) or R == 0
    # combine, with and without weights; what lies at dropped places does not matter
    y = rows_of(g, n, C, DT[dt], pad, offset)
    y[total:] = float("nan")
    w = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)
    hy = f64(y)
    for weights, R in ((w, n), (None, n), (w, total)):
        want, size = ot.combine(hy[:R], hr, None if weights is None else host(weights))
        got = f64(mxg.moe_combine(y[:R], rows, weights))
        assert (np.abs(got - want) <= (k + 2) * U * size + HALF_STEP[dt] * (np.abs(want) + (k + 2) * U * size)).all()
    # gradients
    for R in sorted({n, total}):
        dy, dw = mxg.moe_combine_bwd(x, y[:R], rows, w)
        wy, ww, size = ot.combine_bwd(f64(x), hy[:R], hr, host(w))
        assert not np.isnan(wy).any()
        assert (np.abs(f64(dy) - wy) <= (HALF_STEP[dt] + 2 * U) * np.abs(wy)).all()
        assert (np.abs(f64(dw) - ww) <= 256 * U * size).all()
    # in place of y
    again = y.clone()
    dy2, dw2 = mxg.moe_combine_bwd(x, again, rows, w, dy=again)
    assert torch.equal(dy2, mxg.moe_combine_bwd(x, y, rows, w)[0]) and torch.equal(dw2, mxg.moe_combine_bwd(x, y, rows, w)[1])


def test_combine_special_values():
    """NaN and infinity pass from kept rows only."""
    rows = torch.tensor([[0, 1], [~3, 2], [~4, ~5]], dtype=torch.int32, device="cuda")
    y = torch.ones((6, 16), device="cuda")
    y[1, 3], y[2, 5], y[3:] = float("inf"), float("nan"), float("nan")
    out = host(mxg.moe_combine(y, rows, torch.tensor([[1., 0.], [1., 1.], [1., 1.]], device="cuda")))
    assert np.isnan(out[0, 3]) and np.isnan(out[1, 5]) and not out[2].any()      # 0 * inf; NaN; nothing kept
    assert np.isfinite(np.delete(out, [3], 1)[0]).all() and np.isfinite(np.delete(out, [5], 1)[1]).all()


def test_places_past_the_rows_are_left_out():
    rows = torch.tensor([[0, 5], [2 ** 31 - 1, 1], [-2 ** 31, ~2]], dtype=torch.int32, device="cuda")
    x = torch.arange(1., 4, device="cuda")[:, None].expand(3, 8).contiguous()
    y = mxg.moe_dispatch(x, rows, 4, out=torch.full((4, 8), 9., device="cuda"))
    assert y[:, 0].tolist() == [1, 2, 0, 9]
    assert mxg.moe_combine(y, rows)[:, 0].tolist() == [1, 2, 0]
    dy, dw = mxg.moe_combine_bwd(x, y, rows, torch.ones((3, 2), device="cuda"), dy=torch.full((4, 8), 9., device="cuda"))
    assert dy[:, 0].tolist() == [1, 2, 0, 9] and dw.tolist() == [[8, 0], [0, 32], [0, 0]]


def test_no_tokens_or_rows():
    e = torch.empty((0, 4), device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    rows, choice, counts = mxg.moe_sort(ids, 3)
    assert rows.shape == (0, 2) and choice.numel() == 0 and counts.tolist() == [0, 0, 0]
    assert mxg.moe_dispatch(e, rows).shape == (0, 4) and mxg.moe_combine(e, rows).shape == (0, 4)
    dropped = torch.tensor([[~0, ~1]], dtype=torch.int32, device="cuda")
    assert mxg.moe_combine(e, dropped).tolist() == [[0.0] * 4]
    dy, dw = mxg.moe_combine_bwd(torch.ones((1, 4), device="cuda"), e, dropped, torch.ones((1, 2), device="cuda"))
    assert dy.shape == (0, 4) and dw.tolist() == [[0, 0]]


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart: the last begin past 2^32 elements."""
    T, C, ld = 4200, 40, 1 << 20
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    rows, _, _ = mxg.moe_sort(choices(gen(0), T, 1, 8), 8)
    x = torch.randn((T, C), device="cuda", generator=gen(1)).bfloat16()
    y = mxg.moe_dispatch(x, rows, out=buf[:, 8:8 + C])
    assert torch.equal(y[rows[:, 0].long()], x)
    assert torch.equal(mxg.moe_combine(y, rows), x)
    dy, dw = mxg.moe_combine_bwd(x, y, rows, torch.ones((T, 1), device="cuda"), dy=buf[:, 64:64 + C])
    assert torch.equal(dy, y)
    back = mxg.moe_combine(y, rows, out=buf[:, 128:128 + C])
    assert torch.equal(back, x) and not buf[:, 200:].any()


@pytest.mark.parametrize("T", [700, 2000])                  # one launch of the sort, and two
def test_streams_and_graph(T):
    """Another stream, and a captured sort, dispatch, combine and gradient replayed
    on new inputs with eager work between."""
    k, E, C = 4, 24, 513
    g = gen(3)
    ids, x = choices(g, T, k, E, 0.2), rows_of(g, T, C, torch.bfloat16)
    w = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)

    def step():
        rows, order, counts = mxg.moe_sort(ids, E)
        y = mxg.moe_dispatch(x, rows)
        return (rows, order, counts, y, mxg.moe_combine(y, rows, w), *mxg.moe_combine_bwd(x, y, rows, w))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        g = gen(10 + seed)
        ids.copy_(choices(g, T, k, E, 0.2))
        x.copy_(rows_of(g, T, C, torch.bfloat16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


# Rows whose last chunk is short, its lane in the wave of its neighbour's, in another
# one (513 to 519 bf16 columns, 257 fp32, for few tokens), and at the beginning of the
# next trip over the row (2049); all parts of a chunk are left over once.
@pytest.mark.parametrize("dt,C", [("bf16", c) for c in (9, 130, 257, 513, 514, 515, 516, 517, 518, 519, 1025, 1027, 1031, 1537,
                                                         2049, 2052, 4103)]
                         + [("f32", c) for c in (5, 66, 131, 257, 258, 259, 513, 514, 515, 769, 1025, 2051)])
@pytest.mark.parametrize("T,k", [(1, 16), (40, 8), (300, 3)])
def test_gradient_in_place_of_y(dt, C, T, k):
    """dy over y against the fp64 reference of what y held before: a weight's gradient
    is a sum of at most 64 products a lane."""
    g = gen(C * T)
    rows, _, counts = mxg.moe_sort(choices(g, T, k, 8, 0.1), 8)
    n = T * k
    x = rows_of(g, T, C, DT[dt], 3, 1)
    w = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)
    room = rows_of(g, n + 2, C + 2, DT[dt], 1, 1)
    before = f64(room)
    y = room[1:n + 1, 1:C + 1]
    wy, ww, size = ot.combine_bwd(f64(x), f64(y), host(rows), host(w))
    dy, dw = mxg.moe_combine_bwd(x, y, rows, w, dy=y)
    after = f64(room)
    assert dy.data_ptr() == y.data_ptr() and not np.isnan(wy).any()
    assert (np.abs(after[1:n + 1, 1:C + 1] - wy) <= (HALF_STEP[dt] + 2 * U) * np.abs(wy)).all()
    assert (np.abs(f64(dw) - ww) <= 256 * U * size).all()
    after[1:n + 1, 1:C + 1] = before[1:n + 1, 1:C + 1]
    assert np.array_equal(after, before)                        # what surrounds the rows stays


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [6, 7, 9, 10, 11, 12, 13, 14, 15])
def test_rows_of_any_top_k(dt, k):
    """Numbers of choices between the kernels' own."""
    test_rows(dt, 29, k, 40, 1033, 3, 1, 0.2)
    test_rows(dt, 50, k, 17, 5, 1, 0, 0.1)
