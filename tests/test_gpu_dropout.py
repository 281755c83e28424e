"""Dropout on the GPU against the reference, through the binding: the mask is
exact; a kept value is multiplied in fp32 by a scale rounded to fp32 and added to
the residual in fp32: within 2^-24 (2 |x s| + |out|), then rounded once."""
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


def rows_of(seed, R, C, dt, pad=0, offset=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(R * (C + pad) + offset, device="cuda", generator=g).to(dt)[offset:].view(R, C + pad)[:, :C]


def state_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def check(got, x, dt, p, seed, step, call, residual=None):
    hx = f64(x)
    want, kept = ot.dropout(hx, p, seed, step, call, None if residual is None else f64(residual))
    limit = int(np.rint(np.float64(np.float32(p)) * 65536))
    size = 2 * np.abs(np.where(kept, hx, 0)) * 65536 / max(65536 - limit, 1) + np.abs(want)
    assert (np.abs(f64(got) - want) <= U * size + HALF_STEP[dt] * (np.abs(want) + U * size)).all()
    return kept


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,C,pad,offset", [(1, 1, 0, 0), (3, 7, 2, 1), (2, 8, 0, 0), (5, 9, 0, 1), (70, 63, 1, 0),
                                            (9, 1001, 7, 3), (2, 2048, 0, 0), (3, 2050, 0, 0), (2, 20003, 0, 1),
                                            (3000, 40, 8, 0)])
def test_dropout(dt, R, C, pad, offset):
    x, res = rows_of(R, R, C, DT[dt], pad, offset), rows_of(R + 1, R, C, DT[dt], 2 * pad, offset)
    for p, seed, step, call in ((0.1, 1, 0, 0), (0.5, -2 ** 63, 2 ** 40 + 3, 2 ** 32 - 1), (0.0, 7, 1, 2), (1.0, 7, 1, 2),
                                (2.0 ** -18, 7, 1, 2)):
        state = state_of(seed, step)
        check(mxg.dropout(x, p, state, call), x, dt, p, seed, step, call)
        out = mxg.dropout(x, p, state, call, residual=res)
        check(out, x, dt, p, seed, step, call, res)
        # in place of the residual, and of x, inside wider rows whose other elements stay
        base = rows_of(R + 1, R, C, DT[dt], 2 * pad, offset)
        other = base.as_strided((R, 2 * pad), base.stride(), base.storage_offset() + C) if pad and R > 1 else None
        keep = None if other is None else other[:-1].clone()
        assert torch.equal(mxg.dropout(x, p, state, call, residual=base, out=base), out)
        assert keep is None or torch.equal(other[:-1], keep)
        own = x.clone()
        assert torch.equal(mxg.dropout(own, p, state, call, residual=res, out=own), out)


def test_gradient_is_the_same_call():
    x, d = rows_of(0, 50, 333, torch.float32), rows_of(1, 50, 333, torch.float32)
    state = state_of(11, 4)
    out, dx = mxg.dropout(x, 0.3, state, 5), mxg.dropout(d, 0.3, state, 5)
    kept = ot.dropout(f64(x), 0.3, 11, 4, 5)[1]
    assert ((f64(out) != 0) == kept).all() and ((f64(dx) != 0) == kept).all()
    # differences: the function is linear in x
    e = 2.0 ** -10
    diff = (f64(mxg.dropout(x + e * d, 0.3, state, 5)) - f64(out)) / e
    assert (np.abs(diff - f64(dx)) <= (2 ** 13 * U) * (np.abs(f64(out)) + np.abs(f64(dx)) + np.abs(f64(x)))).all()


def test_dropped_values_are_not_looked_at():
    x = torch.full((64, 256), float("nan"), device="cuda")
    kept = ot.dropout(np.zeros((64, 256)), 0.5, 3, 3, 3)[1]
    out = host(mxg.dropout(x, 0.5, state_of(3, 3), 3))
    assert (np.isnan(out) == kept).all() and not out[~kept].any()
    x.fill_(float("inf"))
    assert not mxg.dropout(x, 1.0, state_of(3, 3)).any()


def test_share_of_dropped():
    """4 million draws: within 5 standard deviations of p."""
    x = torch.ones((2048, 2048), device="cuda")
    for p in (0.1, 0.5, 0.9):
        got = float((mxg.dropout(x, p, state_of(9, 9)) == 0).double().mean())
        assert abs(got - p) < 5 * np.sqrt(p * (1 - p) / 2 ** 22) + 2.0 ** -17


def test_no_rows():
    assert mxg.dropout(torch.empty((0, 8), device="cuda"), 0.1, state_of(0, 0)).shape == (0, 8)


def test_offsets_past_32_bits():
    R, C, ld = 4200, 24, 1 << 20
    buf = torch.zeros(R * ld, dtype=torch.bfloat16, device="cuda").view(R, ld)
    x = buf[:, 8:8 + C]
    x.copy_(rows_of(0, R, C, torch.bfloat16))
    out = mxg.dropout(x, 0.5, state_of(1, 2), 3, residual=x, out=buf[:, 64:64 + C])
    assert torch.equal(out, mxg.dropout(x.contiguous(), 0.5, state_of(1, 2), 3, residual=x.contiguous()))
    assert not buf[:, 100:].any()


def test_graph_draws_new_masks():
    """The step on the device is read at every replay."""
    x, state = rows_of(0, 100, 200, torch.float32), state_of(5, 0)
    mxg.dropout(x, 0.5, state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mxg.dropout(x, 0.5, state)
        state[1:] += 1
    for step in range(4):
        x.copy_(rows_of(step, 100, 200, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, "f32", 0.5, 5, step, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mxg.dropout(x, 0.5, state, 1)
    side.synchronize()
    check(got, x, "f32", 0.5, 5, 4, 1)
