"""Cases of the operators that bring tokens to their experts and back, of the
expert product in 8-bit integers, and of dropout:

- ``sort``: the choices of a router sorted by expert (stable), the place of every
  choice and the rows of every expert;
- ``dispatch``: the tokens' rows copied to the places of their choices;
- ``combine``: the experts' rows back to their tokens, weighted and summed;
- ``combine_bwd``: its gradients, of the experts' rows and of the weights;
- ``int8``: activations quantized per token, times int8 weights with a scale per
  channel, expert by expert (one expert: a plain linear layer);
- ``dropout``: a counter-based mask, with or without a residual.

Every operator has its plain form here (elementary torch operations in 32
bits, rounded once at the end) and, where ``own`` is true, the call that a
user makes of this package. ``exact`` is the same in 64 bits, written from the
definitions.

Sizes are those of the package's expert layers (``fc1``: 32 experts, 4096
inputs, 1536 inner; ``a8w4``: 128 experts of 7168 inputs; ``blockwise``: 64 experts,
7168 inputs, 4096 outputs) or generic.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ITYPES = {"i32": torch.int32, "i64": torch.int64}
SIZE = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # decoding: 8 tokens' choices among the 128 experts of a8w4, all latency
        dict(name="sort_8_of_128", op="sort", tokens=8, top_k=8, experts=128, itype="i32", dropped=0.0),
        # a long training batch; a tenth of the choices dropped (-1)
        dict(name="sort_32768_of_128", op="sort", tokens=32768, top_k=8, experts=128, itype="i64", dropped=0.1),
        # a few fp32 rows of odd width inside wider rows, a third of the choices dropped
        dict(name="dispatch_f32_7x1001", op="dispatch", tokens=7, top_k=3, experts=16, cols=1001, dtype="f32", pad=3,
             dropped=0.3),
        # fc1's training batch: 4096 tokens to 32768 rows
        dict(name="dispatch_4096x4096", op="dispatch", tokens=4096, top_k=8, experts=32, cols=4096, dtype="bf16",
             pad=0, dropped=0.0),
        # the rows of a8w4's widest layer back to 16384 tokens
        dict(name="combine_16384x7168", op="combine", tokens=16384, top_k=8, experts=128, cols=7168, dtype="bf16",
             pad=0, dropped=0.0, weighted=True),
        # the gradient of fc1's way back
        dict(name="combine_bwd_4096x4096", op="combine_bwd", tokens=4096, top_k=8, experts=32, cols=4096,
             dtype="bf16", pad=0, dropped=0.0),
        # one token through a plain linear layer: latency and 29 MB of weights
        dict(name="int8_1x4096x7168", op="int8", rows=1, experts=1, n=4096, k=7168),
        # 8 tokens with 8 choices each of a8w4's experts
        dict(name="int8_64x2048x7168_of_128", op="int8", rows=64, experts=128, n=2048, k=7168),
        # a prompt over few experts, sizes that end inside every tile
        dict(name="int8_2999x1111x2000_of_5", op="int8", rows=2999, experts=5, n=1111, k=2000),
        # a batch of prompts through blockwise's experts
        dict(name="int8_32768x4096x7168_of_64", op="int8", rows=32768, experts=64, n=4096, k=7168),
        # decoding-sized rows with a residual: all latency
        dict(name="dropout_8x4096", op="dropout", rows=8, cols=4096, dtype="bf16", pad=0, p=0.1, residual=True),
        # training: 16384 tokens of the widest layer
        dict(name="dropout_16384x7168", op="dropout", rows=16384, cols=7168, dtype="bf16", pad=0, p=0.1,
             residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["sort", "dispatch", "combine", "combine_bwd", "int8", "int8", "int8", "dropout"])
    if op == "int8":
        while True:
            rows, experts = _log_int(rng, 1, 16384), rng.choice([1, 1, _log_int(rng, 2, 128)])
            n, k = _log_int(rng, 64, 8192), _log_int(rng, 128, 8192) // 16 * 16
            if rng.random() < 0.5:
                n, k = max(64, n // 64 * 64), max(128, k // 128 * 128)
            if experts * n * k <= 1 << 29 and rows * n * k <= 1 << 38:
                return dict(op=op, rows=rows, experts=experts, n=n, k=k)
    if op == "dropout":
        cols = _log_int(rng, 8, 16384)
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, 100_000_000 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 8, 5]),
                    p=rng.choice([0.1, 0.1, 0.5, 0.02]), residual=rng.random() < 0.5)
    tokens, experts = _log_int(rng, 1, 32768), _log_int(rng, 4, 512)
    top_k = rng.randint(1, min(8, experts))
    dropped = rng.choice([0.0, 0.0, 0.2])
    if op == "sort":
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, itype=rng.choice(["i32", "i64"]),
                    dropped=dropped)
    cols = _log_int(rng, 16, 8192)
    if rng.random() < 0.6:
        cols = max(16, cols // 64 * 64)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    tokens = min(tokens, max(1, 900_000_000 // (cols * top_k * SIZE[dtype])))
    case = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, cols=cols, dtype=dtype,
                pad=rng.choice([0, 0, 8, 3]), dropped=dropped)
    if op == "combine":
        case["weighted"] = rng.random() < 0.7    # without weights: the gradient of dispatch
    return case


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rows(g, rows, cols, pad, dtype):
    """[rows, cols] inside rows that are `pad` elements longer."""
    return _randn(g, rows, cols + pad).to(dtype)[:, :cols]


def _choices(g, case):
    """Top-k choices of a router whose experts are not equally liked, some of
    them dropped (-1); int64 [tokens, top_k]."""
    like = 0.7 * _randn(g, case["experts"])
    ids = torch.topk(_randn(g, case["tokens"], case["experts"]) + like, case["top_k"], dim=1)[1]
    if case["dropped"]:
        ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < case["dropped"], -1, ids)
    return ids


def _row_splits(rows, experts, seed):
    """Rows of each expert, as chance deals them to experts not equally liked."""
    rng = np.random.default_rng(seed)
    like = np.exp(0.7 * rng.standard_normal(experts))
    return [int(v) for v in rng.multinomial(rows, like / like.sum())]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "int8":
        E, N, K = case["experts"], case["n"], case["k"]
        x = _randn(g, case["rows"], K) * (1 + _randn(g, K).square())     # some channels larger than others
        w_q = torch.empty((E * N, K), dtype=torch.int8, device="cuda")
        w_s = torch.empty(E * N, device="cuda")
        for e in range(E):
            w = _randn(g, N, K) * (1.0 / math.sqrt(K))
            top = w.abs().amax(1)
            w_s[e * N:(e + 1) * N] = top / 127
            w_q[e * N:(e + 1) * N] = torch.round(w * (127 / top)[:, None]).to(torch.int8)
        return dict(case=case, x=x.to(torch.bfloat16), w_q=w_q, w_s=w_s, splits=_row_splits(case["rows"], E, seed))
    if op == "dropout":
        dt = DTYPES[case["dtype"]]
        s = dict(case=case, x=_rows(g, case["rows"], case["cols"], case["pad"], dt), residual=None, stream=3)
        if case["residual"]:
            s["residual"] = _rows(g, case["rows"], case["cols"], case["pad"], dt)
        # the generator's state: seed and step
        s["state"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=g)
        return s
    ids = _choices(g, case)
    if op == "sort":
        return dict(case=case, ids=ids.to(ITYPES[case["itype"]]))
    dt, T, C = DTYPES[case["dtype"]], case["tokens"], case["cols"]
    s = dict(case=case, rows=_sort(ids, case["experts"])[0])
    if op in ("dispatch", "combine_bwd"):
        s["x"] = _rows(g, T, C, case["pad"], dt)                 # tokens, or the gradient of the tokens
    if op != "dispatch":
        s["y"] = _rows(g, T * case["top_k"], C, case["pad"], dt)  # the experts' rows
        s["weights"] = torch.softmax(_randn(g, T, case["top_k"]), dim=1) if case.get("weighted", True) else None
    return s


# -------------------------------------------------------------- plain forms

def _sort(ids, experts):
    """(rows, choices, counts): the place of each choice in the order of the
    experts (~place for a dropped one, behind all others), the choice at each
    place, the rows of each expert."""
    key = ids.reshape(-1).long()
    kept = (key >= 0) & (key < experts)
    key = torch.where(kept, key, experts)
    choices = torch.sort(key, stable=True)[1]
    place = torch.empty_like(choices)
    place[choices] = torch.arange(choices.numel(), device=ids.device)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    counts.index_add_(0, key, torch.ones_like(key))
    rows = torch.where(kept, place, -1 - place).view(ids.shape)
    return rows.to(torch.int32), choices.to(torch.int32), counts[:experts].to(torch.int32)


def _dispatch(x, rows):
    out = x.new_zeros((rows.numel(), x.shape[1]))
    kept = rows >= 0
    token = torch.arange(x.shape[0], device=x.device)[:, None].expand_as(rows)
    out[torch.where(kept, rows, -1 - rows).long()] = torch.where(kept[:, :, None], x[token], 0)
    return out


def _combine(y, rows, weights):
    kept = (rows >= 0)[:, :, None]
    v = y[rows.clamp(min=0).long()].float()
    if weights is not None:
        v = v * weights[:, :, None]
    return torch.where(kept, v, 0).sum(1).to(y.dtype)


def _combine_bwd(dout, y, rows, weights):
    kept = rows >= 0
    d = dout.float()
    dw = torch.where(kept, (y[rows.clamp(min=0).long()].float() * d[:, None, :]).sum(2), 0)
    dy = torch.where(kept[:, :, None], weights[:, :, None] * d[:, None, :], 0)
    out = torch.empty((rows.numel(), y.shape[1]), dtype=y.dtype, device=y.device)
    out[torch.where(kept, rows, -1 - rows).long()] = dy.to(y.dtype)
    return out, dw


def _int8(s):
    """Codes are the integers next to 127 x / amax of their row; the products of
    codes are summed, then scaled by row and channel."""
    n = s["case"]["n"]
    x = s["x"].float()
    top = x.abs().amax(1)
    q = torch.round(x * 127 / top[:, None])
    a_s = top / 127
    y = torch.empty((x.shape[0], n), dtype=torch.bfloat16, device=x.device)
    at = 0
    for e, m in enumerate(s["splits"]):
        if m:
            acc = torch.mm(q[at:at + m], s["w_q"][e * n:(e + 1) * n].float().t())
            y[at:at + m] = (acc * a_s[at:at + m, None] * s["w_s"][e * n:(e + 1) * n]).to(torch.bfloat16)
        at += m
    return y


LOW32 = 0xFFFFFFFF


def _philox(counter, key):
    """Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw: Parallel random
    numbers: as easy as 1, 2, 3; 2011). counter: 4 and key: 2 values in 32 bits."""
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57        # 64-bit products, as bits
        c0, c1, c2, c3 = (b >> 32 & LOW32) ^ c1 ^ k0, b & LOW32, (a >> 32 & LOW32) ^ c3 ^ k1, a & LOW32
        k0, k1 = k0 + 0x9E3779B9 & LOW32, k1 + 0xBB67AE85 & LOW32
    return c0, c1, c2, c3


def _dropout(s):
    """Eight columns share one call of the generator: 16 bits each, low half
    first. Columns whose number is below p 2^16 are dropped."""
    c = s["case"]
    x = s["x"]
    rows, cols = x.shape
    groups = (cols + 7) // 8
    at = torch.arange(rows * groups, device=x.device)
    state = s["state"]
    like = torch.zeros_like(at)
    words = _philox((at & LOW32, at >> 32, like + s["stream"], like + (state[1] & LOW32)),
                    (state[0] & LOW32, state[0] >> 32 & LOW32))
    bits = torch.stack([w >> h & 0xFFFF for w in words for h in (0, 16)], 1).view(rows, groups * 8)[:, :cols]
    limit = round(c["p"] * 65536)
    y = torch.where(bits >= limit, x.float() * (65536 / (65536 - limit)), 0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


# ---------------------------------------------------------------------- run

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import moe_grouped_block_mx_amd as mxg
        if op == "sort":
            return mxg.moe_sort(state["ids"], c["experts"])
        if op == "dispatch":
            return mxg.moe_dispatch(state["x"], state["rows"])
        if op == "combine":
            return mxg.moe_combine(state["y"], state["rows"], state["weights"])
        if op == "combine_bwd":
            return mxg.moe_combine_bwd(state["x"], state["y"], state["rows"], state["weights"])
        if op == "int8":
            q, scales = mxg.quantize_rowwise(state["x"], "int8")
            return mxg.grouped_fwd(q, scales, state["w_q"], state["w_s"], state["splits"], c["n"], c["k"],
                                   a_fmt="int8", w_fmt="int8")
        return mxg.dropout(state["x"], c["p"], state["state"], stream=state["stream"], residual=state["residual"])
    if op == "sort":
        return _sort(state["ids"], c["experts"])
    if op == "dispatch":
        return _dispatch(state["x"], state["rows"])
    if op == "combine":
        return _combine(state["y"], state["rows"], state["weights"])
    if op == "combine_bwd":
        return _combine_bwd(state["x"], state["y"], state["rows"], state["weights"])
    return _int8(state) if op == "int8" else _dropout(state)


# --------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "int8":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        used = E * (1 - (1 - 1 / E) ** M) if E > 1 else 1     # about as many experts have a row
        return {"bytes": int(used * N * (K + 4)) + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": (3 if case["residual"] else 2) * n * SIZE[case["dtype"]], "flops": 3 * n}
    choices = case["tokens"] * case["top_k"]
    if op == "sort":
        return {"bytes": choices * (SIZE[case["itype"]] + 8) + 4 * case["experts"], "flops": choices}
    size = SIZE[case["dtype"]]
    token, row = case["tokens"] * case["cols"] * size, choices * case["cols"] * size
    kept = int(row * (1 - case["dropped"]))
    flops = int(2 * choices * case["cols"] * (1 - case["dropped"]))
    if op == "dispatch":
        return {"bytes": token + row + 4 * choices, "flops": 0}
    if op == "combine":
        return {"bytes": kept + token + (8 if case["weighted"] else 4) * choices, "flops": flops}
    return {"bytes": token + kept + row + 12 * choices, "flops": 3 * flops // 2}


# -------------------------------------------------------------------- exact

def _sort_exact(ids, experts):
    key = [e if 0 <= e < experts else experts for e in ids.reshape(-1).tolist()]
    order = sorted(range(len(key)), key=lambda c: (key[c], c))
    rows, counts = [0] * len(key), [0] * experts
    for place, c in enumerate(order):
        rows[c] = place if key[c] < experts else ~place
        if key[c] < experts:
            counts[key[c]] += 1
    as_int = dict(dtype=torch.int32, device=ids.device)
    return torch.tensor(rows, **as_int).view(ids.shape), torch.tensor(order, **as_int), torch.tensor(counts, **as_int)


def _int8_64(s):
    c = s["case"]
    N = c["n"]
    x = s["x"].double()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(127 * x / top)
    y = torch.zeros((c["rows"], N), dtype=torch.float64, device=x.device)
    end = np.cumsum(s["splits"])
    for e in range(c["experts"]):
        lo, hi = int(end[e]) - s["splits"][e], int(end[e])
        if hi > lo:
            w = s["w_q"][e * N:(e + 1) * N].double() * s["w_s"][e * N:(e + 1) * N, None].double()
            y[lo:hi] = (q[lo:hi] * (top[lo:hi] / 127)) @ w.t()
    return y


def _mul32(a, m):
    """High and low 32 bits of a * m, from 16-bit halves of m."""
    low, high = a * (m & 0xFFFF), a * (m >> 16)          # below 2^48 each
    total = (low >> 16) + high
    return total >> 16, (total % 65536) * 65536 + low % 65536


def _dropout_64(s):
    c = s["case"]
    x = s["x"].double()
    rows, cols = x.shape
    per_row = -(-cols // 8)
    seed, step = (int(v) for v in s["state"].tolist())
    block = torch.arange(rows * per_row, dtype=torch.int64, device=x.device)
    word = [block % 2 ** 32, block // 2 ** 32, torch.full_like(block, s["stream"]),
            torch.full_like(block, step % 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        high0, low0 = _mul32(word[0], 0xD2511F53)
        high1, low1 = _mul32(word[2], 0xCD9E8D57)
        word = [high1 ^ word[1] ^ key[0], low1, high0 ^ word[3] ^ key[1], low0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    number = torch.empty((rows * per_row, 8), dtype=torch.int64, device=x.device)
    for i in range(4):
        number[:, 2 * i], number[:, 2 * i + 1] = word[i] % 65536, word[i] // 65536
    number = number.view(rows, per_row * 8)[:, :cols]
    share = round(c["p"] * 65536) / 65536
    y = (number >= share * 65536).double() * x / (1 - share)
    return y if s["residual"] is None else y + s["residual"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return _sort_exact(s["ids"], case["experts"])
    if op == "int8":
        return _int8_64(s)
    if op == "dropout":
        return _dropout_64(s)
    rows, T, k, C = s["rows"].long(), case["tokens"], case["top_k"], case["cols"]
    token = torch.arange(T, device=rows.device)
    if op == "dispatch":
        out = torch.zeros((T * k, C), dtype=torch.float64, device=rows.device)
        for j in range(k):
            on = rows[:, j] >= 0
            out[rows[on, j]] = s["x"][token[on]].double()
        return out
    w = s["weights"].double() if s["weights"] is not None else torch.ones((T, k), dtype=torch.float64, device=rows.device)
    if op == "combine":
        out = torch.zeros((T, C), dtype=torch.float64, device=rows.device)
        for j in range(k):
            on = rows[:, j] >= 0
            out[token[on]] += w[on, j, None] * s["y"][rows[on, j]].double()
        return out
    dy = torch.zeros((T * k, C), dtype=torch.float64, device=rows.device)
    dw = torch.zeros((T, k), dtype=torch.float64, device=rows.device)
    for j in range(k):
        on = rows[:, j] >= 0
        d = s["x"][token[on]].double()
        dy[rows[on, j]] = w[on, j, None] * d
        dw[on, j] = (d * s["y"][rows[on, j]].double()).sum(1)
    return dy, dw
