"""The operators around the expert layer without a GPU: their C entry points
refuse bad arguments before any HIP call, and the binding refuses buffers of the
wrong shape, type or layout before the library sees them."""
import ctypes

import pytest
import torch

import moe_grouped_block_mx_amd as mx

L = mx.lib
P = ctypes.c_void_p(0x100000)      # a fake aligned device address
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)   # aligned to bf16 only
OK, NULL, SHAPE, FORMAT, ALIGN, WS, HIP = 0, 1, 2, 4, 5, 6, 9
BIG = 1 << 30


def last():
    return L.mxgg_last_error().decode()


def fwd(x=P, rows=4, cols=8, ldx=8, dt=0, w=P, b=P, wdt=0, eps=1e-5, y=P, ldy=8, mean=P, rstd=P):
    return L.mxgg_layer_norm_fwd(x, rows, cols, ldx, dt, w, b, wdt, eps, y, ldy, mean, rstd, None)


def bwd(dy=P, lddy=8, x=P, ldx=8, rows=4, cols=8, dt=0, w=P, wdt=0, mean=P, rstd=P, dx=P, lddx=8, dw=P, db=P, acc=0,
        ws=P, ws_bytes=BIG):
    return L.mxgg_layer_norm_bwd(dy, lddy, x, ldx, rows, cols, dt, w, wdt, mean, rstd, dx, lddx, dw, db, acc, ws,
                                 ws_bytes, None)


def test_layer_norm_rules():
    assert fwd() == HIP                                    # valid; no GPU to run it on
    assert fwd(w=None, b=None) == HIP
    assert fwd(x=None) == NULL and fwd(mean=None) == NULL and fwd(y=None) == NULL
    assert fwd(rows=-1) == SHAPE and fwd(cols=0) == SHAPE and fwd(cols=16385, ldx=16385, ldy=16385) == SHAPE
    assert fwd(ldx=7) == SHAPE and "ldx" in last()
    assert fwd(ldy=0) == SHAPE and fwd(eps=-1.0) == SHAPE and fwd(eps=float("nan")) == SHAPE
    assert fwd(dt=2) == FORMAT and fwd(wdt=-1) == FORMAT
    assert fwd(x=ODD) == ALIGN and fwd(x=HALF) == HIP and fwd(x=HALF, dt=1) == ALIGN and fwd(w=HALF, wdt=1) == ALIGN
    assert fwd(x=None, y=None, mean=None, rstd=None, rows=0) == OK
    assert bwd() == HIP and bwd(w=None, dw=None, db=None) == HIP
    assert bwd(dx=None) == NULL and bwd(rstd=None) == NULL and bwd(lddx=3) == SHAPE and bwd(acc=2) == FORMAT
    assert bwd(dw=HALF) == ALIGN
    assert bwd(ws_bytes=8) == WS and bwd(ws=None) == NULL
    assert bwd(rows=0, acc=1, ws=None, ws_bytes=0) == OK
    assert bwd(rows=0, dw=None, db=None, ws=None, ws_bytes=0) == OK
    assert L.mxgg_layer_norm_bwd_workspace(4, 0) == 0 and L.mxgg_layer_norm_bwd_workspace(0, 8) == 0
    assert L.mxgg_layer_norm_bwd_workspace(1, 8) >= 64


def clip(ptrs=(0x100000, 0x200000), numels=(8, 8), dtypes=(0, 1), n=None, kind=0, max_norm=1.0, total=P, ws=P,
         ws_bytes=BIG, fn="clip"):
    k = max(1, len(ptrs))
    a = (ctypes.c_void_p * k)(*ptrs)
    m = (ctypes.c_int64 * k)(*numels)
    d = (ctypes.c_int32 * k)(*dtypes)
    n = len(ptrs) if n is None else n
    if fn == "norm":
        return L.mxgg_grad_norm(a, m, d, n, kind, total, ws, ws_bytes, None)
    if fn == "with":
        return L.mxgg_clip_grads_with_norm(a, m, d, n, max_norm, total, None)
    return L.mxgg_clip_grad_norm(a, m, d, n, kind, max_norm, total, ws, ws_bytes, None)


def test_grad_rules():
    for fn in ("norm", "clip", "with"):
        assert clip(fn=fn) == HIP
        assert clip(fn=fn, ptrs=(0x100000, 0x100008)) == SHAPE and "overlap" in last()
        assert clip(fn=fn, ptrs=(0x200000, 0x1FFFFC)) == SHAPE          # in either order
        assert clip(fn=fn, ptrs=(0x100000, 0x100010)) == HIP            # side by side
        assert clip(fn=fn, ptrs=(0x100000, 0x100000), numels=(0, 8)) == HIP   # an empty one overlaps nothing
        assert clip(fn=fn, numels=(8, -1)) == SHAPE and clip(fn=fn, numels=(1 << 42, 1)) == SHAPE
        assert clip(fn=fn, dtypes=(0, 2)) == FORMAT
        assert clip(fn=fn, ptrs=(0x100000, 0x200002)) == ALIGN and clip(fn=fn, ptrs=(0x100000, None)) == NULL
        assert clip(fn=fn, n=-1) == SHAPE and clip(fn=fn, total=None) == NULL
    assert clip(kind=2) == FORMAT and clip(max_norm=-1.0) == SHAPE and clip(max_norm=float("inf")) == SHAPE
    assert clip(max_norm=float("nan")) == SHAPE and clip(fn="with", max_norm=-1.0) == SHAPE
    assert clip(ws_bytes=8) == WS and clip(ws=None) == NULL
    assert clip(fn="with", n=0) == OK                          # nothing to scale
    assert L.mxgg_clip_grad_norm(None, None, None, 1, 0, 1.0, P, P, BIG, None) == NULL
    assert L.mxgg_grad_norm_workspace(0) == 0 and L.mxgg_grad_norm_workspace(-1) == 0
    assert 0 < L.mxgg_grad_norm_workspace(1) < L.mxgg_grad_norm_workspace(1000)


def moe(x=P, ldx=256, lg=P, ldl=8, ldt=1, T=4, H=256, inner=128, E=8, k=2, fmt=0, flags=1, out=P, ids=P, wts=P, ws=P,
        ws_bytes=BIG, q=P):
    return L.mxgg_moe_layer(x, ldx, lg, ldl, ldt, T, H, inner, E, k, q, P, P, P, fmt, flags, out, ids, wts, ws, ws_bytes,
                            None)


def test_moe_rules():
    for fmt in (0, 1, 3, 5, mx.KBLOCK_ROWS, 1 | mx.KBLOCK_ROWS):
        assert moe(fmt=fmt) == HIP, fmt
    for fmt in (2, 4, 6, -1, mx.KBLOCK_COLS, 3 | mx.KBLOCK_ROWS, mx.LAYOUT_MFMA, mx.LAYOUT_ROW_MAJOR):
        assert moe(fmt=fmt) == FORMAT, fmt
    assert moe(T=-1) == SHAPE and moe(T=65) == SHAPE and "64" in last()
    assert moe(T=0, x=None, lg=None, out=None) == OK
    assert moe(E=0) == SHAPE and moe(E=513, ldl=513) == SHAPE and moe(k=0) == SHAPE and moe(k=9) == SHAPE
    assert moe(E=32, ldl=32, k=17) == SHAPE
    assert moe(H=260, ldx=264) == SHAPE and moe(inner=48) == SHAPE and moe(inner=0) == SHAPE and moe(H=65568) == SHAPE
    assert moe(H=288, ldx=288) == HIP and moe(H=288, ldx=288, fmt=mx.KBLOCK_ROWS) == SHAPE
    assert moe(inner=160, fmt=3) == SHAPE
    assert moe(ldx=248) == SHAPE and moe(ldx=260) == ALIGN and moe(ldl=7) == SHAPE
    assert moe(flags=2) == FORMAT and moe(ldt=2) == FORMAT
    assert moe(x=HALF) == ALIGN and moe(lg=HALF) == ALIGN and moe(lg=HALF, ldt=0) == HIP and moe(q=None) == NULL
    assert moe(ids=None) == NULL and moe(wts=HALF) == ALIGN and moe(out=None) == NULL
    assert moe(ws_bytes=16) == WS and moe(ws=None) == NULL
    assert L.mxgg_moe_layer_workspace(65, 8, 2, 128) == 0 and L.mxgg_moe_layer_workspace(1, 8, 9, 128) == 0


def test_layer_norm_binding():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8)
    stat = torch.zeros(4)
    for bad in (dict(x=torch.zeros(4, 8, dtype=torch.float16)), dict(x=torch.zeros(4)), dict(x=torch.zeros(8, 4).t()),
                dict(weight=torch.zeros(7)), dict(weight=torch.zeros(16)[::2]), dict(weight=w, bias=w.bfloat16()),
                dict(y=torch.zeros(4, 8)), dict(y=torch.zeros(4, 9, dtype=torch.bfloat16)), dict(mean=torch.zeros(5)),
                dict(rstd=torch.zeros(4, dtype=torch.float64))):
        with pytest.raises(ValueError):
            mx.layer_norm_fwd(**{"x": x, **bad})
    good = dict(dy=x, x=x, weight=w, mean=stat, rstd=stat)
    for bad in (dict(dy=torch.zeros(4, 8)), dict(dy=x[:3]), dict(mean=stat[:3]), dict(dx=x.float()), dict(accumulate=True),
                dict(dweight=torch.zeros(8, dtype=torch.bfloat16)), dict(dbias=torch.zeros(9)),
                dict(ws=torch.zeros(8192)[::2])):
        with pytest.raises(ValueError):
            mx.layer_norm_bwd(**{**good, **bad})


def test_grad_binding():
    g = torch.zeros(8)
    for bad in ([g.half()], [g[::2]], [g.view(2, 4).t()], [g, torch.zeros(3, dtype=torch.int32)]):
        with pytest.raises(ValueError, match="gradient"):
            mx.clip_grad_norm(bad, 1.0)
    for norm_type in (1.0, 0, 3):
        with pytest.raises(ValueError, match="norm_type"):
            mx.grad_norm([g], norm_type)
    with pytest.raises(ValueError, match="total"):
        mx.clip_grads_with_norm([g], 1.0, torch.zeros(2))
    for call in (lambda: mx.clip_grad_norm([g], 1.0), lambda: mx.grad_norm([g]),
                 lambda: mx.clip_grads_with_norm([g], 1.0, torch.zeros(()))):
        with pytest.raises(ValueError, match="GPU"):       # host memory: refused, never touched
            call()


def test_moe_binding():
    T, H, inner, E, k = 3, 64, 32, 4, 2
    u8 = torch.uint8
    good = dict(x=torch.zeros(T, H, dtype=torch.bfloat16), logits=torch.zeros(T, E),
                w13_q=torch.zeros(E * 2 * inner, H // 2, dtype=u8), w13_s=torch.zeros(H // 32, E * 2 * inner, dtype=u8),
                w2_q=torch.zeros(E * H, inner // 2, dtype=u8), w2_s=torch.zeros(inner // 32, E * H, dtype=u8), top_k=k)
    for bad in (dict(x=torch.zeros(T, H)), dict(logits=torch.zeros(T + 1, E)), dict(logits=torch.zeros(T, E).double()),
                dict(w13_s=torch.zeros(E * 2 * inner, H // 32, dtype=u8)), dict(w2_q=torch.zeros(E * H, inner, dtype=u8)),
                dict(w2_s=torch.zeros(inner // 32, E * H)), dict(fmt="mxfp8"), dict(fmt="fp8_1x128"),
                dict(w13_q=good["w13_q"][:-1]), dict(out=torch.zeros(T, H)), dict(ids=torch.zeros(T, k, dtype=torch.int64)),
                dict(weights=torch.zeros(T, k + 1)), dict(fmt=mx.MXFP4 | mx.KBLOCK_ROWS)):
        with pytest.raises(ValueError):
            mx.moe_layer(**{**good, **bad})


def test_scaling_by_a_norm_needs_one():
    # total is read here, not written: none is refused, not made up
    for grads in ([torch.zeros(8)], []):
        with pytest.raises(ValueError, match="total"):
            mx.clip_grads_with_norm(grads, 1.0, None)


def test_moe_code_layout_of_each_matrix():
    w13, w2 = mx.MOE_W13_KBLOCK, mx.MOE_W2_KBLOCK
    for fmt in (mx.MXFP4, mx.MXFP8):
        assert moe(fmt=fmt, flags=1 | w13) == HIP and moe(fmt=fmt, flags=w2) == HIP and moe(fmt=fmt, flags=w13 | w2) == HIP
        # 64-byte blocks need multiples of 128 along the matrix's own contraction only
        assert moe(fmt=fmt, inner=96, flags=w13) == HIP and moe(fmt=fmt, inner=96, flags=w2) == SHAPE
        assert moe(fmt=fmt, H=288, ldx=288, flags=w2) == HIP and moe(fmt=fmt, H=288, ldx=288, flags=w13) == SHAPE
        assert moe(fmt=fmt | mx.KBLOCK_ROWS, flags=w2) == HIP
        assert moe(fmt=fmt | mx.KBLOCK_ROWS, inner=96, flags=w13) == SHAPE
    assert moe(fmt=mx.FP8_128x128, flags=w13) == FORMAT and moe(flags=16) == FORMAT
    T, H, inner, E = 3, 128, 96, 4
    u8 = torch.uint8
    good = dict(x=torch.zeros(T, H, dtype=torch.bfloat16), logits=torch.zeros(T, E),
                w13_q=torch.zeros(1, E * 2 * inner, 64, dtype=u8), w13_s=torch.zeros(H // 32, E * 2 * inner, dtype=u8),
                w2_q=torch.zeros(E * H, inner // 2, dtype=u8), w2_s=torch.zeros(inner // 32, E * H, dtype=u8), top_k=2,
                fmt=mx.MXFP4 | mx.KBLOCK_ROWS, w2_fmt="mxfp4")
    with pytest.raises(ValueError, match="GPU"):           # the buffers fit their formats; host memory is refused
        mx.moe_layer(**good)
    for bad in (dict(w2_fmt=None), dict(w2_fmt=mx.MXFP4 | mx.KBLOCK_ROWS), dict(fmt="mxfp4"), dict(w2_fmt="mxfp8"),
                dict(w2_fmt=mx.MXFP4 | mx.KBLOCK_COLS), dict(fmt="fp8_128x128", w2_fmt="fp8_128x128_p2")):
        with pytest.raises(ValueError):
            mx.moe_layer(**{**good, **bad})


def test_rows_that_the_kernels_cannot_read_are_copied():
    # the layer norm module takes any strides; the C ABI row strides from the row
    # length up, below 2^31 (a time step out of a long batch has more)
    from moe_grouped_block_mx_amd.layer_norm import _rows
    big = torch.empty((3, 1 << 19, 4096), dtype=torch.bfloat16, device="meta")
    for x, copied in ((big[:, 7], True), (big[:, :2, :], True), (big[:, 7, :100][:1], False), (big[1, :5], False),
                      (big[0, :4, :6].t(), True), (big[0, :1, :6].expand(3, 6), True), (big[0, 5], False)):
        r = _rows(x)
        assert r.shape == (x.numel() // x.shape[-1], x.shape[-1])
        if r.shape[0] > 1:
            assert r.stride(1) == 1 and r.shape[1] <= r.stride(0) < 1 << 31
        assert r.is_contiguous() == copied or not copied
