"""The token, int8 and dropout operators without a GPU: their C entry points
refuse bad arguments before any HIP call, and the binding refuses buffers of the
wrong shape, type or layout before the library sees them."""
import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_block_mx_amd as mx
from moe_grouped_block_mx_amd.dropout_module import Dropout, DropoutState
from moe_grouped_block_mx_amd.token_plan import TokenPlan

L = mx.lib
P = ctypes.c_void_p(0x100000)      # a fake aligned device address
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)   # aligned to bf16 only
WORD = ctypes.c_void_p(0x100004)   # aligned to 4 bytes only
OK, NULL, SHAPE, SPLITS, FORMAT, ALIGN, WS, HIP = 0, 1, 2, 3, 4, 5, 6, 9
BIG = 1 << 31


def last():
    return L.mxgg_last_error().decode()


def sort(ids=P, it=0, ldi=8, T=4, k=8, E=16, rows=P, choices=P, counts=P, ws=None, ws_bytes=0):
    return L.mxgg_moe_sort(ids, it, ldi, T, k, E, rows, choices, counts, ws, ws_bytes, None)


def test_sort_rules():
    assert sort() == HIP                                   # valid; no GPU to run it on
    assert sort(it=1) == HIP and sort(ldi=9) == HIP and sort(E=512) == HIP
    assert sort(it=2) == FORMAT and sort(k=0) == SHAPE and sort(k=17, ldi=17) == SHAPE and sort(ldi=7) == SHAPE
    assert sort(T=-1) == SHAPE and sort(T=(BIG >> 4) + 1) == SHAPE and sort(T=1 << 20, ws=P, ws_bytes=BIG) == HIP and sort(E=0) == SHAPE and sort(E=513) == SHAPE
    assert sort(ids=None) == NULL and sort(rows=None) == NULL and sort(choices=None) == NULL and sort(counts=None) == NULL
    assert sort(ids=WORD) == HIP and sort(ids=WORD, it=1) == ALIGN and sort(rows=HALF) == ALIGN
    need = L.mxgg_moe_sort_workspace(4096, 8, 16)
    assert need > 0 and L.mxgg_moe_sort_workspace(4, 8, 16) == 0
    assert sort(T=4096, ws=P, ws_bytes=need) == HIP
    assert sort(T=4096, ws=P, ws_bytes=need - 1) == WS and sort(T=4096, ws_bytes=need) == NULL
    assert L.mxgg_moe_sort_workspace(-1, 8, 16) == 0 and L.mxgg_moe_sort_workspace(BIG, 8, 16) == 0
    sizes = [L.mxgg_moe_sort_workspace(T, 8, 16) for T in (1, 512, 513, 8191, 8192, 8193, 16384, 131071, 131072, 10 ** 6)]
    assert sizes == sorted(sizes)                          # the largest call's does for all
    assert sort(T=0, ids=None, rows=None, choices=None) == HIP   # clears the counts


def dispatch(x=P, ldx=8, dt=0, T=4, C=8, rows=P, k=2, out=P, ldo=8, R=8):
    return L.mxgg_moe_dispatch(x, ldx, dt, T, C, rows, k, out, ldo, R, None)


def combine(y=P, ldy=8, dt=0, R=8, C=8, rows=P, w=P, T=4, k=2, out=P, ldo=8):
    return L.mxgg_moe_combine(y, ldy, dt, R, C, rows, w, T, k, out, ldo, None)


def bwd(d=P, ldd=8, y=P, ldy=8, dt=0, R=8, C=8, rows=P, w=P, T=4, k=2, dy=P, lddy=8, dw=P):
    return L.mxgg_moe_combine_bwd(d, ldd, y, ldy, dt, R, C, rows, w, T, k, dy, lddy, dw, None)


def test_row_rules():
    for f in (dispatch, combine, bwd):
        assert f() == HIP and f(dt=1) == HIP
        assert f(dt=2) == FORMAT and f(C=0) == SHAPE and f(C=9) == SHAPE and f(k=0) == SHAPE and f(k=17) == SHAPE
        assert f(C=(1 << 24) + 1) == SHAPE
        assert f(T=-1) == SHAPE and f(T=(BIG >> 2) + 1) == SHAPE and f(T=BIG >> 2) == HIP and f(R=-1) == SHAPE and f(R=BIG) == SHAPE
        assert f(rows=None) == NULL and f(rows=HALF) == ALIGN
        assert f(T=0, rows=None) == OK
    assert dispatch(ldx=7) == SHAPE and dispatch(ldo=7) == SHAPE and dispatch(ldo=BIG) == SHAPE
    assert dispatch(x=None) == NULL and dispatch(out=None) == NULL and dispatch(x=ODD) == ALIGN and dispatch(x=HALF) == HIP
    assert dispatch(x=HALF, dt=1) == ALIGN and dispatch(R=0, out=None) == OK
    assert combine(ldy=7) == SHAPE and combine(ldo=7) == SHAPE and combine(w=None) == HIP and combine(w=HALF) == ALIGN
    assert combine(y=None) == NULL and combine(y=None, R=0) == HIP and combine(out=None) == NULL
    assert bwd(ldd=7) == SHAPE and bwd(ldy=7) == SHAPE and bwd(lddy=7) == SHAPE
    for name in ("d", "y", "dy", "w", "dw"):
        assert bwd(**{name: None}) == NULL, name
    assert bwd(y=None, dy=None, R=0) == HIP and bwd(dw=HALF) == ALIGN


def drop(x=P, ldx=8, dt=0, R=4, C=8, p=0.1, state=P, call=0, res=P, ldr=8, out=P, ldo=8):
    return L.mxgg_dropout(x, ldx, dt, R, C, p, state, call, res, ldr, out, ldo, None)


def test_dropout_rules():
    assert drop() == HIP and drop(dt=1) == HIP and drop(res=None, ldr=0) == HIP and drop(p=0.0) == HIP and drop(p=1.0) == HIP
    assert drop(p=-0.1) == SHAPE and drop(p=1.5) == SHAPE and drop(p=float("nan")) == SHAPE
    assert drop(dt=3) == FORMAT and drop(C=0) == SHAPE and drop(R=-1) == SHAPE and drop(R=BIG) == SHAPE
    assert drop(ldx=7) == SHAPE and drop(ldr=7) == SHAPE and drop(ldo=7) == SHAPE
    assert drop(x=None) == NULL and drop(out=None) == NULL and drop(state=None) == NULL and drop(state=WORD) == ALIGN
    assert drop(res=HALF, dt=1) == ALIGN
    assert drop(R=0, x=None, out=None, state=None) == OK


def quant(rows=4, cols=64, ldx=64, fmt=6, x=P, q=P, s=P):
    return L.mxgg_quantize_rowwise(x, rows, cols, ldx, fmt, 0, q, s, None)


def fwd(m=(3, 0, 5), M=8, N=33, K=48, af=6, wf=6, a=P, a_s=P, w=P, w_s=P, out=P, G=None):
    arr = (ctypes.c_int64 * len(m))(*m)
    return L.mxgg_grouped_fwd(a, a_s, af, w, w_s, wf, arr, len(m) if G is None else G, M, N, K, out, None, 0, None)


def test_int8_rules():
    assert quant() == HIP and quant(cols=16, ldx=24) == HIP and quant(cols=(1 << 17) - 16, ldx=1 << 17) == HIP
    assert quant(cols=8) == SHAPE and quant(cols=0) == SHAPE and quant(cols=1 << 17, ldx=1 << 17) == SHAPE
    assert quant(ldx=56) == SHAPE and quant(ldx=65) == ALIGN and quant(rows=-1) == SHAPE and quant(rows=BIG) == SHAPE
    assert quant(x=None) == NULL and quant(q=HALF) == ALIGN and quant(rows=0, x=None, q=None, s=None) == OK
    for bits in (0x100, 0x200, 0x1000, 0x2000):
        assert quant(fmt=6 | bits) == FORMAT and "int8" in last()
        assert fwd(af=6 | bits) == FORMAT and fwd(wf=6 | bits) == FORMAT
    assert fwd() == HIP and fwd(N=1) == HIP
    assert fwd(K=40) == SHAPE and fwd(K=1 << 17) == SHAPE and fwd(K=(1 << 17) - 16) == HIP and fwd(N=0) == SHAPE
    assert fwd(N=1 << 23) == SHAPE and fwd(M=7) == SPLITS and fwd(m=(9, -1, 0)) == SPLITS and fwd(G=0) == SHAPE
    assert fwd(M=BIG) == SHAPE
    assert fwd(af=0) == FORMAT and fwd(wf=0) == FORMAT       # both operands or neither
    for name in ("a", "a_s", "w", "w_s", "out"):
        assert fwd(**{name: None}) == NULL and fwd(**{name: HALF}) == ALIGN, name
    assert fwd(m=(0, 0, 0), M=0, a=None, a_s=None, w=None, w_s=None, out=None) == OK
    # no other pass takes the format
    m = (ctypes.c_int64 * 1)(64)
    assert L.mxgg_grouped_dgrad(P, P, P, P, 6, m, 1, 64, 64, 64, P, None, 0, None) == FORMAT
    assert L.mxgg_grouped_wgrad(P, P, P, P, 6, m, 1, 64, 64, 64, P, 0, 1, None, 0, None) == FORMAT
    assert L.mxgg_quantize_colwise_segpad(P, 64, 64, 64, m, 1, 6, 0, P, P, 64, None) == FORMAT
    assert L.mxgg_quantize_dual(P, 64, 64, 64, m, 1, 6, 0, P, P, P, P, 64, None) == FORMAT
    assert L.mxgg_segpad_rows(m, 1, 6) == -1


def refused(call, match=None):
    with pytest.raises(ValueError, match=match):
        call()


def test_binding():
    i32, bf = torch.int32, torch.bfloat16
    ids = torch.zeros(4, 2, dtype=i32)
    refused(lambda: mx.moe_sort(ids.float(), 4), "int32 or int64")
    refused(lambda: mx.moe_sort(ids.t(), 4), "inner stride")
    refused(lambda: mx.moe_sort(ids[0], 4), "2-D")
    for bad in (dict(rows=ids[:3]), dict(choices=ids), dict(counts=torch.zeros(5, dtype=i32)), dict(rows=ids.long())):
        refused(lambda: mx.moe_sort(ids, 4, **bad))
    x, y, w = torch.zeros(4, 8, dtype=bf), torch.zeros(8, 8, dtype=bf), torch.zeros(4, 2)
    for bad in (dict(x=x[:3]), dict(x=x.half()), dict(x=x.t()), dict(rows=ids.long()), dict(rows=ids.t()), dict(rows=ids[0]),
                dict(out=y[:7], expert_rows=8), dict(out=y.float()), dict(out=y[:, :7])):
        refused(lambda: mx.moe_dispatch(**{**dict(x=x, rows=ids), **bad}))
    for bad in (dict(y=y.double()), dict(y=y.t()[:, :3]), dict(weights=w[:3]), dict(weights=w.to(bf)), dict(out=y),
                dict(weights=torch.zeros(2, 4).t())):
        refused(lambda: mx.moe_combine(**{**dict(y=y, rows=ids, weights=w), **bad}))
    for bad in (dict(dout=x[:3]), dict(dout=x.float()), dict(weights=None), dict(dy=x), dict(dweights=w.to(bf)),
                dict(dout=None)):
        refused(lambda: mx.moe_combine_bwd(**{**dict(dout=x, y=y, rows=ids, weights=w), **bad}), "^(?!.*GPU)")
    state = torch.zeros(2, dtype=torch.int64)
    for bad in (dict(state=state.int()), dict(state=state[:1]), dict(residual=x[:3]), dict(out=x.float()), dict(stream=-1),
                dict(stream=1 << 32), dict(x=x.t()), dict(state=None)):
        refused(lambda: mx.dropout(**{**dict(x=x, p=0.1, state=state), **bad}))
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    wq, ws = torch.zeros(2 * 8, 64, dtype=torch.int8), torch.zeros(2 * 8)
    for bad in (dict(a_q=q.view(torch.uint8)), dict(a_s=s[:3]), dict(w_q=wq[:8]), dict(w_s=ws.view(2, 8)), dict(a_fmt="mxfp8"),
                dict(out=torch.zeros(4, 8))):
        args = {**dict(a_q=q, a_s=s, w_q=wq, w_s=ws, m_splits=[3, 1], N=8, K=64, a_fmt="int8", w_fmt="int8"), **bad}
        refused(lambda: mx.grouped_fwd(**args))
    refused(lambda: mx.quantize_rowwise(x[:, :0].float(), "int8"), "bf16")
    refused(lambda: mx.quantize_rowwise(torch.zeros(4, 64, dtype=bf), "int8", q=q.view(torch.uint8)))


def test_host_memory_is_refused():
    ids, x, state = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: mx.moe_sort(ids, 4), lambda: mx.moe_dispatch(x, ids), lambda: mx.moe_combine(torch.zeros(8, 8), ids),
                 lambda: mx.moe_combine_bwd(x, torch.zeros(8, 8), ids, torch.zeros(4, 2)),
                 lambda: mx.dropout(x, 0.1, state)):
        refused(call, "GPU")


def test_gradient_over_y_has_its_strides():
    assert bwd(ldy=8, lddy=9) == SHAPE and "leading dimension" in last()
    assert bwd(ldy=9, lddy=9) == HIP and bwd(ldy=8, lddy=9, R=1) == HIP
    other = ctypes.c_void_p(0x900000)
    assert bwd(ldy=8, lddy=9, dy=other) == HIP


def test_dropout_state_is_saved_and_loaded():
    state = DropoutState(-5, step=2, device="cpu")
    state.advance()
    saved = state.state_dict()
    assert saved == {"seed": -5, "step": 3}
    other = DropoutState(1, device="cpu")
    held = other.tensor
    other.load_state_dict(saved)
    assert other.tensor is held and held.tolist() == [-5, 3]     # in place: a captured graph reads there
    other.advance_()
    assert other.state_dict() == {"seed": -5, "step": 4} and saved["step"] == 3


def test_dropouts_of_a_state_have_numbers_of_their_own():
    state = DropoutState(3, device="cpu")
    assert [Dropout(0.1, state).call for _ in range(3)] == [0, 1, 2]
    other = DropoutState(3, device="cpu")
    assert [Dropout(0.1, other, call=c).call for c in (1, 5, 5)] == [1, 5, 5]    # the caller's may meet
    assert [Dropout(0.1, other).call for _ in range(5)] == [0, 2, 3, 4, 6]
    refused(lambda: Dropout(0.1, other, call=4), "call=4")                       # ... but not one that was given out
    assert Dropout(0.1, other, call=7).call == 7 and Dropout(0.1, other).call == 8
    refused(lambda: Dropout(0.1, other, call=1 << 32), "call")


def test_int8_splits_are_any_numbers():
    """Whatever the other formats take: they all get as far as the check of the memory."""
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    wq, ws = torch.zeros(2 * 8, 64, dtype=torch.int8), torch.zeros(2 * 8)
    for splits in ([3, 1], (3, 1), [3.0, 1.0], (m for m in (3, 1)), (m for m in (3.0, 1.0)), torch.tensor([3, 1]), torch.tensor([3., 1.]),
                   np.array([3, 1]), map(int, "31")):
        refused(lambda: mx.grouped_fwd(q, s, wq, ws, splits, 8, 64, "int8", "int8"), "GPU")
    refused(lambda: mx.grouped_fwd(q, s, wq, ws, (m for m in (3, 1, 0)), 8, 64, "int8", "int8"), "w_q must be")


def test_plan_takes_any_strides():
    ids = torch.zeros(4, 6, dtype=torch.int32)
    for view in (ids.t(), ids[:, ::2], ids[:1].expand(5, 6), ids[:, :1].expand(4, 3)):
        refused(lambda: TokenPlan(view, 4), "GPU")
    for bad in (ids[0], ids.float(), ids[None]):
        refused(lambda: TokenPlan(bad, 4), "^(?!.*GPU)")
