"""Cases of the operators around the expert layer: layer norm (forward and
backward), the global gradient norm with clipping, and the whole expert layer
for a few tokens.

Every operator has its plain form here (elementary torch operations in 32
bits, rounded once at the end) and, where ``own`` is true, the call that a
user makes of this package. ``exact`` is the same in 64 bits, written from the
definitions.

Sizes: the expert layers are those of the package's workloads (``fc1``: 32
experts, 4096 inputs, 2 x 1536 gated outputs; ``a8w4``: 128 experts, 7168
inputs, 2048 outputs; ``blockwise``: 64 experts, 7168 inputs, 4096 outputs),
the norms and gradients belong to them.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5           # layer norm
CLIP_EPS = 1e-6      # added to the gradient norm before the division
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # decoding: the norm of 8 tokens in flight, all latency
        dict(name="norm_fwd_8x4096", op="norm_fwd", rows=8, cols=4096, dtype="bf16", wdtype="bf16", pad=0),
        # training: 16384 tokens of the widest layer
        dict(name="norm_fwd_16384x7168", op="norm_fwd", rows=16384, cols=7168, dtype="bf16", wdtype="bf16", pad=0),
        # training: the 4096 tokens that fc1 routes to 32768 rows
        dict(name="norm_bwd_4096x4096", op="norm_bwd", rows=4096, cols=4096, dtype="bf16", wdtype="bf16", pad=0),
        # an fp32 residual stream of odd width inside wider rows
        dict(name="norm_bwd_f32_2500x5001", op="norm_bwd", rows=2500, cols=5001, dtype="f32", wdtype="f32", pad=3),
        # the parameters of one gate and one norm: all latency
        dict(name="clip_small", op="clip", tensors=4, total=300_000, bf16_share=0.0, ragged=False, kind="l2"),
        # 150 parameters of all sizes as slices of one fp32 and one bf16 gradient buffer
        dict(name="clip_ragged_150", op="clip", tensors=150, total=30_000_001, bf16_share=0.4, ragged=True, kind="l2"),
        # fc1's fp32 main_grad, 32 experts of 3072 x 4096
        dict(name="clip_main_grad_fc1", op="clip", tensors=1, total=32 * 3072 * 4096, bf16_share=0.0, ragged=False,
             kind="l2"),
        # one token through fc1's experts: latency and 8 experts' weights
        dict(name="moe_fc1_1_token", op="moe", tokens=1, experts=32, hidden=4096, inner=1536, top_k=8, fmt="mxfp4",
             layout="kblock", renormalize=True, masked=0.0),
        # a batch of 8 requests through the 128 small experts of a8w4
        dict(name="moe_a8w4_8_tokens", op="moe", tokens=8, experts=128, hidden=7168, inner=1024, top_k=8, fmt="mxfp4",
             layout="kblock", renormalize=True, masked=0.0),
        # MXFP8 weights in plain rows, sizes that end inside a tile, half of the experts on other ranks
        dict(name="moe_mxfp8_5_tokens", op="moe", tokens=5, experts=24, hidden=2080, inner=992, top_k=4, fmt="mxfp8",
             layout="rows", renormalize=False, masked=0.5),
        # 32 requests: every expert of fc1 is read
        dict(name="moe_fc1_32_tokens", op="moe", tokens=32, experts=32, hidden=4096, inner=1536, top_k=8, fmt="mxfp4",
             layout="kblock", renormalize=True, masked=0.0),
        # the most tokens, the largest weights: blockwise FP8
        dict(name="moe_blockwise_64_tokens", op="moe", tokens=64, experts=64, hidden=7168, inner=2048, top_k=8,
             fmt="fp8_128x128", layout="kblock", renormalize=True, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["norm_fwd", "norm_bwd", "clip", "moe", "moe"])
    if op == "clip":
        return dict(op=op, tensors=_log_int(rng, 1, 200), total=_log_int(rng, 1000, 200_000_000),
                    bf16_share=rng.choice([0.0, 0.5, 1.0]), ragged=rng.random() < 0.5,
                    kind=rng.choice(["l2", "l2", "l2", "max"]))
    if op != "moe":
        cols = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, min(16384, 100_000_000 // cols))
        return dict(op=op, rows=rows, cols=cols + (cols == 3072), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    wdtype=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 8, 5]))
    fmt = rng.choice(["mxfp4", "mxfp4", "mxfp8", "fp8_128x128"])
    layout = "kblock" if fmt == "fp8_128x128" else rng.choice(["rows", "kblock"])
    unit = 128 if layout == "kblock" else 32
    while True:
        hidden = _log_int(rng, 256, 7168) // unit * unit
        inner = max(128, _log_int(rng, 128, 2048) // unit * unit)
        experts = _log_int(rng, 4, 256)
        if experts * hidden * inner <= 64 * 4096 * 2048 and 3072 not in (hidden, inner):
            break
    return dict(op=op, tokens=_log_int(rng, 1, 64), experts=experts, hidden=hidden, inner=inner,
                top_k=rng.randint(1, min(8, experts)), fmt=fmt, layout=layout, renormalize=rng.random() < 0.7,
                masked=rng.choice([0.0, 0.0, 0.5]))


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rows(g, rows, cols, pad, dtype):
    """[rows, cols] inside rows that are `pad` elements longer."""
    return _randn(g, rows, cols + pad).to(dtype)[:, :cols]


def _block_codes(w, fmt):
    """Codes and scales of w [R, K] as a quantizer stores them: E2M1 or E4M3
    with a UE8M0 scale per 32 along K, or E4M3 with an fp32 scale per 128x128
    block. Codes u8 [R, bytes], scales u8 [R, K/32] or f32 [R/128, K/128]."""
    R, K = w.shape
    if fmt == "fp8_128x128":
        b = w.view(R // 128, 128, K // 128, 128)
        s = b.abs().amax((1, 3), keepdim=True) / 448.0
        return (b / s).view(R, K).to(torch.float8_e4m3fn).view(torch.uint8), s.view(R // 128, K // 128)
    b = w.view(R, K // 32, 32)
    e = torch.floor(torch.log2(b.abs().amax(2, keepdim=True))) - (2 if fmt == "mxfp4" else 8)
    v = b * torch.exp2(-e)
    scales = (e.view(R, K // 32) + 127).to(torch.uint8)
    if fmt == "mxfp8":
        return v.clamp(-448, 448).view(R, K).to(torch.float8_e4m3fn).view(torch.uint8), scales
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(R, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales


def _weights(g, experts, rows, K, fmt, layout):
    """The packed weights of all experts, made one expert at a time, in the
    package's layout: codes [E*rows, bytes] or 64-byte K blocks [bytes/64,
    E*rows, 64]; MX scales block-major [K/32, rows rounded up to 4]."""
    R = experts * rows
    nb = K // 2 if fmt == "mxfp4" else K
    q = torch.empty((nb // 64, R, 64) if layout == "kblock" else (R, nb), dtype=torch.uint8, device="cuda")
    if fmt == "fp8_128x128":
        s = torch.empty((R // 128, K // 128), device="cuda")
    else:
        s = torch.zeros((K // 32, (R + 3) // 4 * 4), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        c, sc = _block_codes(_randn(g, rows, K) * (1.0 / math.sqrt(K)), fmt)
        at = slice(e * rows, (e + 1) * rows)
        if layout == "kblock":
            q[:, at] = c.view(rows, nb // 64, 64).transpose(0, 1)
        else:
            q[at] = c
        if fmt == "fp8_128x128":
            s[e * rows // 128:(e + 1) * rows // 128] = sc
        else:
            s[:, at] = sc.t()
    return q, s


def _sizes(case):
    """Element counts of the gradients of a clip case: equal parts, or ragged
    ones from single elements upward; the first `bf16_share` of them bf16."""
    n, total = case["tensors"], case["total"]
    rng = random.Random(n * 1_000_003 + total)
    share = [math.exp(rng.uniform(0, 9)) if case["ragged"] else 1.0 for _ in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    sizes[-1] += max(0, total - sum(sizes))
    return sizes, int(n * case["bf16_share"])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        dt, wdt, C = DTYPES[case["dtype"]], DTYPES[case["wdtype"]], case["cols"]
        x = _rows(g, case["rows"], C, case["pad"], dt)
        x += torch.randn((), device="cuda", generator=g)
        s = dict(case=case, x=x, weight=(1 + 0.1 * _randn(g, C)).to(wdt), bias=(0.1 * _randn(g, C)).to(wdt))
        if op == "norm_bwd":
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = (xf.var(1, unbiased=False) + EPS).rsqrt()
            s["dy"] = _rows(g, case["rows"], C, case["pad"], dt)
        return s
    if op == "clip":
        sizes, n16 = _sizes(case)
        # gradients are slices of one buffer of each type, one behind the other
        flat16 = (1e-3 * _randn(g, sum(sizes[:n16]))).to(torch.bfloat16)
        flat32 = 1e-3 * _randn(g, sum(sizes[n16:]))
        grads = list(flat16.split(sizes[:n16])) if n16 else []
        grads += list(flat32.split(sizes[n16:])) if n16 < len(sizes) else []
        # half of the norm that such values have
        limit = 0.5e-3 * math.sqrt(sum(sizes)) if case["kind"] == "l2" else 2e-3
        return dict(case=case, grads=grads, flat16=flat16, flat32=flat32, limit=limit)
    E, H, inner, T = case["experts"], case["hidden"], case["inner"], case["tokens"]
    x = _randn(g, T, H).to(torch.bfloat16)
    logits = (2 * _randn(g, T, E)).to(torch.bfloat16).float()   # a bf16 gate: equal logits do occur
    if case["masked"]:
        logits[:, torch.rand(E, device="cuda", generator=g) < case["masked"]] = float("-inf")
    w13_q, w13_s = _weights(g, E, 2 * inner, H, case["fmt"], case["layout"])
    w2_q, w2_s = _weights(g, E, H, inner, case["fmt"], case["layout"])
    return dict(case=case, x=x, logits=logits, w13_q=w13_q, w13_s=w13_s, w2_q=w2_q, w2_s=w2_s)


# -------------------------------------------------------------- plain forms

def _norm_fwd(s):
    x = s["x"].float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
    y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    c1 = g.sum(1, keepdim=True) / x.shape[1]
    c2 = (g * xh).sum(1, keepdim=True) / x.shape[1]
    dx = s["rstd"][:, None] * (g - c1 - xh * c2)
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _clip(grads, limit, kind):
    parts = [g.float().abs().amax() if kind == "max" else g.float().square().sum() for g in grads]
    norm = torch.stack(parts)
    norm = norm.amax() if kind == "max" else torch.sqrt(norm.sum())
    coef = (limit / (norm + CLIP_EPS)).clamp(max=1.0)
    for g in grads:
        g.copy_(g.float() * coef)
    return norm


def _unblock(q, at):
    """Rows `at` of a code tensor in either layout: u8 [n, bytes]."""
    if q.dim() == 2:
        return q[at]
    q = q[:, at]
    return q.transpose(0, 1).reshape(q.shape[1], -1)


def _dense(q, s, fmt, rows, experts):
    """fp32 weights [n, rows, K] of the experts (an index tensor)."""
    at = (experts[:, None] * rows + torch.arange(rows, device=q.device)).view(-1)
    c = _unblock(q, at)
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
        v = torch.stack((table[(c & 15).int()], table[(c >> 4).int()]), 2).view(c.shape[0], -1)
    else:
        v = c.view(torch.float8_e4m3fn).float()
    if fmt == "fp8_128x128":
        block = (experts[:, None] * (rows // 128) + torch.arange(rows // 128, device=q.device)).view(-1)
        v = v.view(block.numel(), 128, -1, 128) * s[block][:, None, :, None]
    else:
        v = v.view(c.shape[0], -1, 32) * torch.exp2(s[:, at].t().float() - 127)[:, :, None]
    return v.view(experts.numel(), rows, -1)


def _route(logits, top_k, renormalize):
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :top_k], ids[:, :top_k]
    none = top == float("-inf")
    high = top[:, :1].masked_fill(none[:, :1], 0)
    p = torch.exp(top - high)
    total = (p if renormalize else torch.exp(logits - high)).sum(1, keepdim=True)
    p = torch.where(none, torch.zeros_like(p), p / total)
    return ids.masked_fill(none, -1), p


def _moe(s):
    c = s["case"]
    E, inner, H, T, k = c["experts"], c["inner"], c["hidden"], c["tokens"], c["top_k"]
    x = s["x"].float()
    ids, p = _route(s["logits"], k, c["renormalize"])
    if T * k < E:     # the chosen experts' weights, once for each choice
        w13 = _dense(s["w13_q"], s["w13_s"], c["fmt"], 2 * inner, ids.clamp(min=0).view(-1))
        gu = torch.bmm(w13, x.repeat_interleave(k, 0)[:, :, None]).view(T * k, 2 * inner)
        h = gu[:, :inner] / (1 + torch.exp(-gu[:, :inner])) * gu[:, inner:]
        w2 = _dense(s["w2_q"], s["w2_s"], c["fmt"], H, ids.clamp(min=0).view(-1))
        y = torch.bmm(w2, h[:, :, None]).view(T, k, H)
        y = (y * p[:, :, None]).sum(1)
    else:             # every expert's weights, for all tokens
        every = torch.arange(E, device=x.device)
        w13 = _dense(s["w13_q"], s["w13_s"], c["fmt"], 2 * inner, every).view(E * 2 * inner, H)
        gu = torch.mm(x, w13.t()).view(T, E, 2 * inner)
        del w13
        h = gu[:, :, :inner] / (1 + torch.exp(-gu[:, :, :inner])) * gu[:, :, inner:]
        share = torch.where(ids[:, :, None] == every, p[:, :, None], torch.zeros_like(p[:, :, None])).sum(1)
        h = torch.where(share[:, :, None] == 0, torch.zeros_like(h), h * share[:, :, None])
        w2 = _dense(s["w2_q"], s["w2_s"], c["fmt"], H, every)
        y = torch.bmm(h.transpose(0, 1).contiguous(), w2.transpose(1, 2)).sum(0)
    return y.to(torch.bfloat16), ids.to(torch.int32), p


# ---------------------------------------------------------------------- run

def run(state):
    c = state["case"]
    if c["op"] == "clip":
        # the limit tightens with each pass, so that each has something to scale
        limit = state["limit"]
        state["limit"] = limit * 0.9999
    if own:
        import moe_grouped_block_mx_amd as mxg
        if c["op"] == "norm_fwd":
            return mxg.layer_norm_fwd(state["x"], state["weight"], state["bias"], EPS)
        if c["op"] == "norm_bwd":
            return mxg.layer_norm_bwd(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"])
        if c["op"] == "clip":
            norm = mxg.clip_grad_norm(state["grads"], limit, norm_type=math.inf if c["kind"] == "max" else 2.0)
            return norm, state["flat16"], state["flat32"]
        f = mxg.FORMATS[c["fmt"]]
        if c["fmt"] != "fp8_128x128" and c["layout"] == "kblock":
            f |= mxg.KBLOCK_ROWS
        return mxg.moe_layer(state["x"], state["logits"], state["w13_q"], state["w13_s"], state["w2_q"],
                             state["w2_s"], c["top_k"], fmt=f, renormalize=c["renormalize"])
    if c["op"] == "norm_fwd":
        return _norm_fwd(state)
    if c["op"] == "norm_bwd":
        return _norm_bwd(state)
    if c["op"] == "clip":
        return _clip(state["grads"], limit, c["kind"]), state["flat16"], state["flat32"]
    return _moe(state)


# --------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, size, wsize = case["rows"] * case["cols"], SIZE[case["dtype"]], SIZE[case["wdtype"]]
        if op == "norm_fwd":      # x, y; weight, bias; mean, rstd
            return {"bytes": 2 * n * size + 2 * case["cols"] * wsize + 8 * case["rows"], "flops": 7 * n}
        # x, dy, dx; weight; mean, rstd; dweight, dbias
        return {"bytes": 3 * n * size + case["cols"] * (wsize + 8) + 8 * case["rows"], "flops": 14 * n}
    if op == "clip":
        sizes, n16 = _sizes(case)
        n = 2 * sum(sizes[:n16]) + 4 * sum(sizes[n16:])
        return {"bytes": 2 * n + 4, "flops": 3 * sum(sizes)}
    T, E, H, inner, k = case["tokens"], case["experts"], case["hidden"], case["inner"], case["top_k"]
    open_ = max(1.0, E * (1 - case["masked"]))
    chosen = min(k, open_)
    active = open_ * (1 - (1 - chosen / open_) ** T)     # expected number of experts that any token chooses
    each = {"mxfp4": 17 / 32, "mxfp8": 33 / 32, "fp8_128x128": 1 + 4 / 16384}[case["fmt"]]
    return {"bytes": int(active * 3 * H * inner * each) + T * (4 * H + 4 * E + 8 * k),
            "flops": int(T * chosen * 6 * H * inner)}


# -------------------------------------------------------------------- exact

def _e2m1_64(c):
    """The value of 4-bit codes: sign, two exponent bits, one mantissa bit."""
    c = c.long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(e.double() - 1))
    return torch.where((c >> 3) == 1, -v, v)


def _e4m3_64(c):
    c = c.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where((c >> 7) == 1, -v, v)


def _expert_64(q, s, case, rows, e):
    """Expert e's weights [rows, K] in 64 bits."""
    lo, hi = e * rows, (e + 1) * rows
    c = q[lo:hi] if case["layout"] == "rows" else torch.cat(list(q[:, lo:hi]), 1)
    if case["fmt"] == "mxfp4":
        v = torch.empty((rows, 2 * c.shape[1]), dtype=torch.float64, device=c.device)
        v[:, 0::2], v[:, 1::2] = _e2m1_64(c & 15), _e2m1_64(c >> 4)
    else:
        v = _e4m3_64(c)
    if case["fmt"] == "fp8_128x128":
        sc = s[lo // 128:hi // 128].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        sc = torch.exp2(s[:, lo:hi].double() - 127).t().repeat_interleave(32, 1)
    return v * sc


def _moe_64(s):
    c = s["case"]
    E, inner, T, k = c["experts"], c["inner"], c["tokens"], c["top_k"]
    x, logits = s["x"].double(), s["logits"].double().cpu()
    ids = torch.full((T, k), -1, dtype=torch.int32)
    p = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        row = logits[t].tolist()
        order = sorted((e for e in range(E) if row[e] != -math.inf), key=lambda e: (-row[e], e))
        pick = order[:k]
        if pick:
            total = math.fsum(math.exp(row[e] - row[pick[0]]) for e in (pick if c["renormalize"] else order))
            ids[t, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            p[t, :len(pick)] = torch.tensor([math.exp(row[e] - row[pick[0]]) / total for e in pick])
    y = torch.zeros((T, c["hidden"]), dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        on = t.to(x.device)
        gu = x[on] @ _expert_64(s["w13_q"], s["w13_s"], c, 2 * inner, e).t()
        h = gu[:, :inner] * torch.sigmoid(gu[:, :inner]) * gu[:, inner:]
        out = h @ _expert_64(s["w2_q"], s["w2_s"], c, c["hidden"], e).t()
        y.index_add_(0, on, out * p[t, j].to(x.device)[:, None])
    return y, None, p


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        return _moe_64(s)
    if case["op"] == "clip":
        every = torch.cat([s["flat16"].double(), s["flat32"].double()])
        norm = torch.linalg.vector_norm(every, ord=math.inf if case["kind"] == "max" else 2)
        scale = min(1.0, s["limit"] / (float(norm) + CLIP_EPS))
        return norm, s["flat16"].double() * scale, s["flat32"].double() * scale
    x = s["x"].double()
    w = s["weight"].double()
    if case["op"] == "norm_fwd":
        mean = x.mean(1)
        var = ((x - mean[:, None]) ** 2).mean(1)
        rstd = (var + EPS) ** -0.5
        return (x - mean[:, None]) * rstd[:, None] * w + s["bias"].double(), mean, rstd
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xh = (x - mean) * rstd
    g = dy * w
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd
    return dx, (dy * xh).sum(0), dy.sum(0)
