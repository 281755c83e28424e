"""Layer norm on the GPU against the fp64 reference.

Tolerances, with u = 2^-24: a row sum adds at most 100 terms to one partial, so
mean is within 100 u mean|x| and the normalised values within
100 u (mean|x| rstd + |xh|); what follows is a handful of fp32 operations; bf16
outputs add 2^-8 of their value. Column sums add at most 400 terms to one
partial."""
import numpy as np
import pytest

from oracle import block as ob

from .gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

import torch  # noqa: E402

import moe_grouped_block_mx_amd as mxg  # noqa: E402

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def make(rows, cols, dtype, pad=0, seed=0, offset=0.5, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn((rows, cols + pad), generator=g) * scale + offset).to(dtype).cuda()
    return t[:, :cols]


def close(got, want, tol, what):
    err = np.abs(f64(got) - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the bound"


def out_tol(dtype, want):
    return 2.0 ** -8 * np.abs(want) if dtype == BF16 else 2 * U * np.abs(want)


def check_fwd(x, w, b, eps=1e-5):
    y, mean, rstd = mxg.layer_norm_fwd(x, w, b, eps)
    xr, wr = f64(x), None if w is None else f64(w)
    want, m, r = ob.layer_norm_fwd(xr, wr, None if b is None else f64(b), eps)
    mag = np.abs(xr).mean(1)
    close(mean, m, 100 * U * mag, "mean")
    # an error of the mean enters the variance squared, beside its own sum
    close(rstd, r, 100 * U * r + r ** 3 * (100 * U * mag) ** 2, "rstd")
    xh = (xr - m[:, None]) * r[:, None]
    tol = 100 * U * ((mag * r)[:, None] + 2 * np.abs(xh)) + (r ** 2 * (100 * U * mag) ** 2)[:, None] * np.abs(xh)
    tol = tol * (1 if wr is None else np.abs(wr)) + 4 * U * np.abs(want)
    close(y, want, tol + out_tol(x.dtype, want) * (1 + 2.0 ** -7), "y")
    return y, mean, rstd


def check_bwd(dy, x, w, mean, rstd, got, dw0=0.0, db0=0.0):
    dx, dw, db = got
    gr, xr, m, r = f64(dy), f64(x), f64(mean), f64(rstd)
    want, wdw, wdb = ob.layer_norm_bwd(gr, xr, None if w is None else f64(w), m, r)
    wr = 1.0 if w is None else np.abs(f64(w))
    xh = np.abs((xr - m[:, None]) * r[:, None])
    g = np.abs(gr) * wr
    tol = 100 * U * r[:, None] * (g + g.mean(1, keepdims=True) + 2 * xh * (g * xh).mean(1, keepdims=True))
    close(dx, want, tol + out_tol(x.dtype, want) * (1 + 2.0 ** -7), "dx")
    if dw is not None:
        close(dw, wdw + dw0, 400 * U * ((np.abs(gr) * xh).sum(0) + np.abs(dw0)), "dweight")
    if db is not None:
        close(db, wdb + db0, 400 * U * (np.abs(gr).sum(0) + np.abs(db0)), "dbias")


SIZES = [(1, 1), (1, 8), (3, 7), (2, 64), (5, 129), (4, 500), (9, 512), (3, 1000), (2, 1024), (70, 2049), (33, 4096),
         (6, 5001), (5, 7168), (3, 8200), (2, 16383), (2, 16384), (1500, 96), (1100, 1)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,wdtype,pad", [(BF16, BF16, 0), (BF16, F32, 3), (F32, F32, 1), (F32, BF16, 4)])
def test_sizes_types_strides(rows, cols, dtype, wdtype, pad):
    x = make(rows, cols, dtype, pad, 1)
    w, b = make(1, cols, wdtype, 0, 2, 1.0, 0.2)[0].contiguous(), make(1, cols, wdtype, 0, 3, 0.0)[0].contiguous()
    y, mean, rstd = check_fwd(x, w, b)
    dy = make(rows, cols, dtype, 2 * pad, 4, 0.0)
    check_bwd(dy, x, w, mean, rstd, mxg.layer_norm_bwd(dy, x, w, mean, rstd))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_weight_or_bias(dtype):
    x, dy = make(20, 300, dtype, 0, 1), make(20, 300, dtype, 0, 2)
    _, mean, rstd = check_fwd(x, None, None)
    check_fwd(x, make(1, 300, F32, 0, 5)[0].contiguous(), None)
    check_fwd(x, None, make(1, 300, F32, 0, 5)[0].contiguous())
    check_bwd(dy, x, None, mean, rstd, mxg.layer_norm_bwd(dy, x, None, mean, rstd))
    got = mxg.layer_norm_bwd(dy, x, None, mean, rstd, dweight=False)
    assert got[1] is None
    check_bwd(dy, x, None, mean, rstd, got)
    got = mxg.layer_norm_bwd(dy, x, None, mean, rstd, dweight=False, dbias=False)
    assert got[1] is None and got[2] is None
    check_bwd(dy, x, None, mean, rstd, got)


def test_accumulates_into_main_grad():
    x, dy = make(600, 257, BF16, 0, 1), make(600, 257, BF16, 0, 2, 0.0)
    w = make(1, 257, BF16, 0, 3)[0].contiguous()
    _, mean, rstd = mxg.layer_norm_fwd(x, w)
    dw0, db0 = make(1, 257, F32, 0, 4)[0].contiguous(), make(1, 257, F32, 0, 5)[0].contiguous()
    dw, db = dw0.clone(), db0.clone()
    got = mxg.layer_norm_bwd(dy, x, w, mean, rstd, dweight=dw, dbias=db, accumulate=True)
    assert got[1] is dw and got[2] is db
    check_bwd(dy, x, w, mean, rstd, got, f64(dw0), f64(db0))


def test_in_place_and_caller_buffers():
    x, dy = make(40, 777, BF16, 7, 1), make(40, 777, BF16, 0, 2)
    w = make(1, 777, F32, 0, 3)[0].contiguous()
    y, mean, rstd = mxg.layer_norm_fwd(x, w)
    dx, dw, db = mxg.layer_norm_bwd(dy, x, w, mean, rstd)
    dy2 = dy.clone()
    assert mxg.layer_norm_bwd(dy2, x, w, mean, rstd, dx=dy2)[0] is dy2 and torch.equal(dy2, dx)
    big = torch.full((40, 800), 7.0, dtype=BF16, device="cuda")
    xs = x.clone()
    out = mxg.layer_norm_fwd(xs, w, y=big[:, 11:788])[0]
    assert torch.equal(out, y) and (big[:, :11] == 7).all() and (big[:, 788:] == 7).all()
    mxg.layer_norm_fwd(xs, w, y=xs)
    assert torch.equal(xs, y)


def test_rows_that_end_a_buffer_are_not_read_past():
    # NaN around every row: an element too many would poison the row
    big = torch.full((9, 1031), float("nan"), dtype=F32, device="cuda")
    big[:, 5:1006] = make(9, 1001, F32, 0, 1)
    y, mean, rstd = check_fwd(big[:, 5:1006], None, None)
    dyb = torch.full((9, 1031), float("nan"), dtype=F32, device="cuda")
    dyb[:, 1:1002] = make(9, 1001, F32, 0, 2)
    check_bwd(dyb[:, 1:1002], big[:, 5:1006], None, mean, rstd,
              mxg.layer_norm_bwd(dyb[:, 1:1002], big[:, 5:1006], None, mean, rstd))


def test_constant_rows_large_offsets_and_nan():
    x = torch.zeros((6, 640), device="cuda")
    x[1] = 3.0
    x[2] = make(1, 640, F32, 0, 1, 4096.0, 1.0)[0]      # variance far below the square of the mean
    x[3] = make(1, 640, F32, 0, 2, 0.0, 1e18)[0]        # squares near the top of fp32
    x[4, 17] = float("nan")
    x[5, 639] = float("inf")
    y, mean, rstd = mxg.layer_norm_fwd(x)
    assert torch.equal(y[:2], torch.zeros_like(y[:2])) and y[4:].isnan().all()
    check_fwd(x[:4].contiguous(), None, None)
    y, _, rstd = mxg.layer_norm_fwd(x[:1], eps=0.0)      # 0 * inf
    assert y.isnan().all() and torch.isinf(rstd).all()


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 40), generator=g).cuda()
    w, dy = torch.randn(40, generator=g).cuda(), torch.randn((3, 40), generator=g).cuda()
    _, mean, rstd = mxg.layer_norm_fwd(x, w)
    dx, dw, _ = mxg.layer_norm_bwd(dy, x, w, mean, rstd)
    h = 2.0 ** -6   # fp32 values of size 1: rounding 2^-24/h, truncation h^2 times the third derivative
    for r, c in [(0, 0), (1, 17), (2, 39)]:
        e = torch.zeros_like(x)
        e[r, c] = h
        d = ((f64(mxg.layer_norm_fwd(x + e, w)[0]) - f64(mxg.layer_norm_fwd(x - e, w)[0])) * f64(dy)).sum() / (2 * h)
        assert abs(d - float(dx[r, c])) < 5e-3
    e = torch.zeros(40, device="cuda")
    e[5] = h
    d = ((f64(mxg.layer_norm_fwd(x, w + e)[0]) - f64(mxg.layer_norm_fwd(x, w - e)[0])) * f64(dy)).sum() / (2 * h)
    assert abs(d - float(dw[5])) < 1e-3


def test_no_rows():
    x = torch.empty((0, 32), dtype=BF16, device="cuda")
    y, mean, rstd = mxg.layer_norm_fwd(x)
    assert y.shape == (0, 32) and mean.shape == (0,)
    _, dw, db = mxg.layer_norm_bwd(x, x, None, mean, rstd)
    assert not dw.any() and not db.any()
    dw = torch.ones(32, device="cuda")
    assert (mxg.layer_norm_bwd(x, x, None, mean, rstd, dweight=dw, dbias=dw.clone(), accumulate=True)[1] == 1).all()


def test_same_bits_each_run_other_stream_and_poisoned_workspace():
    x, dy = make(3000, 1000, BF16, 0, 1), make(3000, 1000, BF16, 0, 2)
    w = make(1, 1000, BF16, 0, 3)[0].contiguous()
    y, mean, rstd = mxg.layer_norm_fwd(x, w)
    first = mxg.layer_norm_bwd(dy, x, w, mean, rstd)
    ws = torch.full((mxg.lib.mxgg_layer_norm_bwd_workspace(3000, 1000),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, mean2, rstd2 = mxg.layer_norm_fwd(x, w)
        second = mxg.layer_norm_bwd(dy, x, w, mean2, rstd2, ws=ws)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(first, second))


def test_graph_replays():
    x, dy = make(64, 512, BF16, 0, 1), make(64, 512, BF16, 0, 2)
    w = make(1, 512, BF16, 0, 3)[0].contiguous()

    def step():
        y, mean, rstd = mxg.layer_norm_fwd(x, w)
        return (y, *mxg.layer_norm_bwd(dy, x, w, mean, rstd))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for seed in (7, 8, 9):
        x.copy_(make(64, 512, BF16, 0, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_offsets_past_32_bits():
    # row 2 begins 2.4e9 elements into its buffer
    ld = 1_200_000_000
    buf = torch.empty(2 * ld + 1000, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (3, 1000), (ld, 1))
    x.copy_(make(3, 1000, BF16, 0, 1))
    y, mean, rstd = check_fwd(x, None, None)
    dy = make(3, 1000, BF16, 0, 2)
    check_bwd(dy, x, None, mean, rstd, mxg.layer_norm_bwd(dy, x, None, mean, rstd))
    mxg.layer_norm_fwd(x, y=x)
    assert torch.equal(x, y)


def test_mean_of_rows_whose_sum_passes_fp32():
    # powers of two: every partial sum is exact, so the row's deviations are 0
    x = torch.full((3, 4096), 2.0 ** 126, device="cuda")
    x[1] = -(2.0 ** 127)
    y, mean, _ = mxg.layer_norm_fwd(x, None, torch.full((4096,), 0.5, device="cuda"))
    assert torch.equal(mean, x[:, 0]) and (y == 0.5).all()


@pytest.mark.parametrize("rows", [1, 513, 1031])
@pytest.mark.parametrize("cols", [96, 500, 2501, 4096])
def test_dx_over_x_with_a_last_row_that_is_not_finite(rows, cols):
    # the groups of lanes past the last row read it too, maybe after dx is there
    x, dy = make(rows, cols, BF16, 0, 1), make(rows, cols, BF16, 0, 2)
    dy[-1, 5] = float("inf")
    _, mean, rstd = mxg.layer_norm_fwd(x)
    dx, dw, db = mxg.layer_norm_bwd(dy, x, None, mean, rstd)
    assert not dx[-1].isfinite().any() and dx[:-1].isfinite().all()
    assert dw.isfinite().sum() == cols - 1 and db.isfinite().sum() == cols - 1
    got, dw2, db2 = mxg.layer_norm_bwd(dy, x, None, mean, rstd, dx=x)
    assert got is x and torch.equal(got[:-1], dx[:-1]) and not got[-1].isfinite().any()
    assert torch.equal(dw.nan_to_num(), dw2.nan_to_num()) and torch.equal(db, db2)


@pytest.mark.parametrize("rows,cols,dtype", [(3, 5, F32), (3, 5, BF16), (70, 1, F32), (1, 96, BF16), (65, 128, BF16),
                                             (9, 300, F32), (257, 4096, BF16)])
def test_rows_whose_mean_over_their_deviation_passes_fp32(rows, cols, dtype):
    # constant rows: xh is 0, but -mean * rstd (an element of 0 that stands in for
    # one past the row's end, or for a row past the last) is beyond fp32
    x = torch.full((rows, cols), 2.0 ** 123, device="cuda").to(dtype)
    dy = make(rows, cols, dtype, 0, 2)
    _, mean, rstd = mxg.layer_norm_fwd(x)
    assert (mean == 2.0 ** 123).all() and not (mean * rstd).isfinite().any()
    check_bwd(dy, x, None, mean, rstd, mxg.layer_norm_bwd(dy, x, None, mean, rstd))


# Rows enough that a workgroup goes through several (three trips or more, the
# last one with some workgroups or row groups idle), for every number of lanes to
# a row and of row loads ahead: what a trip leaves for the next is compared with
# the reference, on rows that all differ.
@pytest.mark.parametrize("rows,cols,dtype", [
    (140_001, 65, BF16), (33_001, 130, BF16), (33_002, 515, BF16), (16_501, 1026, BF16), (8_300, 2050, BF16),
    (4_200, 4100, BF16), (2_100, 8200, BF16), (140_001, 33, F32), (33_001, 250, F32), (8_300, 1030, F32), (2_100, 4100, F32),
    (2_100, 8200, F32)])
def test_forward_walks_many_rows(rows, cols, dtype):
    x = make(rows, cols, dtype, 3, rows)
    w, b = make(1, cols, F32, 0, 2, 1.0, 0.2)[0].contiguous(), make(1, cols, F32, 0, 3, 0.0)[0].contiguous()
    y, _, _ = check_fwd(x, w, b)
    mxg.layer_norm_fwd(x, w, b, y=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("rows,cols,dtype", [
    (35_001, 96, BF16), (12_301, 500, BF16), (7_003, 600, BF16), (3_501, 1100, BF16), (1_801, 2049, BF16),
    (1_801, 4100, BF16), (901, 6200, BF16), (900, 8200, BF16), (600, 12_300, BF16), (600, 16_384, BF16),
    (35_001, 61, F32), (12_301, 250, F32), (3_501, 1000, F32), (900, 4100, F32), (600, 8000, F32), (600, 8200, F32),
    (520, 16_384, F32)])
def test_backward_walks_many_rows(rows, cols, dtype):
    x, dy = make(rows, cols, dtype, 3, rows), make(rows, cols, dtype, 5, rows + 1, 0.0)
    w = make(1, cols, BF16, 0, 2, 1.0, 0.2)[0].contiguous()
    _, mean, rstd = mxg.layer_norm_fwd(x, w)
    first = mxg.layer_norm_bwd(dy, x, w, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, first)
    dw0, db0 = make(1, cols, F32, 0, 4)[0].contiguous(), make(1, cols, F32, 0, 5)[0].contiguous()
    got = mxg.layer_norm_bwd(dy, x, w, mean, rstd, dweight=dw0.clone(), dbias=db0.clone(), accumulate=True)
    check_bwd(dy, x, w, mean, rstd, got, f64(dw0), f64(db0))
    got = mxg.layer_norm_bwd(dy, x, w, mean, rstd, dx=x)
    assert all(torch.equal(a, b) for a, b in zip(first, got))
