"""Operators of decoding with an output head in 4 bits, as they are measured: the microscaled 4-bit
quantiser and its inverse, the product of such operands, beam search's selection over the logits
they give, and the reordering of the states that follow the selected beams.

`own` chooses between the plain form (elementary torch operations) and the package's kernels.

4-bit operands: an element has a sign, two bits of exponent and one of mantissa (0, 0.5, 1, 1.5, 2, 3,
4, 6), 32 neighbours of a row share a power of two. A byte holds elements 2 i (its low half) and 2 i + 1,
a scale's byte s stands for 2^(s - 127), 255 for NaN.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a decode batch's activations to 4 bits and back: latency counts
        {"name": "quantize 16x4096 bf16", "op": "quantize", "M": 16, "K": 4096, "ld": 4096,
         "dtype": "bf16"},
        # a weight matrix laid out once, or a prefill's activations, and the values they became
        {"name": "quantize 8192x8192 bf16", "op": "quantize", "M": 8192, "K": 8192, "ld": 8192,
         "dtype": "bf16"},
        # one new token through a square projection: every weight is read for one row
        {"name": "product 1x8192x8192 bf16", "op": "product", "M": 1, "N": 8192, "K": 8192,
         "pad": 0, "out": "bf16", "bias": False},
        # ragged in every dimension: rows that end inside a block, and start off alignment
        {"name": "product 1023x1025x1030 f32", "op": "product", "M": 1023, "N": 1025, "K": 1030,
         "pad": 0, "out": "f32", "bias": True},
        # a long prefill through a square projection: the matrix cores' bound
        {"name": "product 8192x8192x8192 bf16", "op": "product", "M": 8192, "N": 8192, "K": 8192,
         "pad": 0, "out": "bf16", "bias": False},
        # a decode batch of activations through an output head of odd size, in whole
        {"name": "linear 32x50001x4096 bf16", "op": "linear", "M": 32, "N": 50001, "K": 4096,
         "dtype": "bf16", "bias": False},
        # a prompt through a wide projection with a bias, in whole
        {"name": "linear 1000x16384x4096 f16", "op": "linear", "M": 1000, "N": 16384, "K": 4096,
         "dtype": "f16", "bias": True},
        # one request of four beams: latency counts, and rows are long
        {"name": "beams 1x4x131072 f32 top 8", "op": "beams", "B": 1, "W": 4, "V": 131072,
         "ld": 131072, "dtype": "f32", "top": 8, "finished": False, "banned": False},
        # a batch with beams that have ended and tokens that may not follow, padded rows
        {"name": "beams 37x5x50001 f16 top 5", "op": "beams", "B": 37, "W": 5, "V": 50001,
         "ld": 50048, "dtype": "f16", "top": 5, "finished": True, "banned": True},
        # a large batch of wide beams, twice as many candidates as beams
        {"name": "beams 128x8x131072 bf16 top 16", "op": "beams", "B": 128, "W": 8, "V": 131072,
         "ld": 131072, "dtype": "bf16", "top": 16, "finished": False, "banned": False},
        # one request's caches and tokens after a step: many small tensors
        {"name": "reorder 1x4 8 layers 8x100x128 bf16", "op": "reorder", "B": 1, "W": 4,
         "layers": 8, "heads": 8, "length": 100, "capacity": 128, "dim": 128, "dtype": "bf16",
         "place": False},
        # a large batch's caches, the beams that go on staying where they are
        {"name": "reorder 32x8 2 layers 8x1000x128 bf16 in place", "op": "reorder", "B": 32, "W": 8,
         "layers": 2, "heads": 8, "length": 1000, "capacity": 1024, "dim": 128, "dtype": "bf16",
         "place": True},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of them rounded to a multiple of 64 where that fits."""
    n = _log_uniform(rng, lo, hi)
    if n >= 64 and rng.random() < 0.5:
        n -= n % 64
    return n


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "linear", "beams", "beams", "reorder"])
    if op == "quantize":
        M, K = _size(rng, 1, 16384), _size(rng, 32, 16384)
        return {"op": op, "M": min(M, 8192 * 8192 // K), "K": K, "ld": K + rng.choice([0, 0, 0, 8, 13]),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op in ("product", "linear"):
        M, N, K = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
        K += K % 2
        if op == "linear":
            N, K = rng.choice([N, 32001, 50001]), K // 64 * 64
        M = max(1, min(M, 8192 ** 3 // (N * K)))
        case = {"op": op, "M": M, "N": N, "K": K, "bias": rng.random() < 0.5}
        if op == "linear":
            return {**case, "dtype": rng.choice(["f32", "bf16", "f16"])}
        return {**case, "pad": rng.choice([0, 0, 0, 16, 3]), "out": rng.choice(["f32", "bf16", "f16"])}
    if op == "beams":
        W, V = rng.randint(1, 16), _size(rng, 1000, 131072)
        dtype = rng.choice(["f32", "bf16", "f16"])
        rows = (512 if dtype == "f32" else 1024) * 131072 // V
        return {"op": op, "B": max(1, min(_log_uniform(rng, 1, 128), rows // W)), "W": W, "V": V,
                "ld": V + rng.choice([0, 0, 0, 64, 7]), "dtype": dtype,
                "top": rng.choice([W, W, 2 * W]), "finished": rng.random() < 0.4,
                "banned": rng.random() < 0.4}
    B, W, layers, heads = _log_uniform(rng, 1, 64), rng.randint(2, 16), rng.randint(1, 8), rng.randint(1, 16)
    dim, dtype = rng.choice([64, 80, 96, 128]), rng.choice(["f32", "bf16", "f16"])
    most = 2 * 10 ** 9 // (2 * layers * B * W * heads * dim * SIZE[dtype])
    length = max(1, min(_size(rng, 1, 2000), most))
    return {"op": op, "B": B, "W": W, "layers": layers, "heads": heads, "length": length,
            "capacity": length + rng.choice([0, 1, 24, 100]), "dim": dim, "dtype": dtype,
            "place": rng.random() < 0.5}


def _activations(M, K, ld, dtype, gen):
    """Rows of different size, a few channels far larger than the others."""
    x = torch.randn(M, ld, device="cuda", generator=gen)
    x *= torch.exp(torch.randn(M, 1, device="cuda", generator=gen))
    x[:, ::97] *= 8
    return x.to(DTYPES[dtype])[:, :K]


def _operand(rows, K, pad, scale, gen):
    """A quantised matrix in hand: packed rows of K / 2 bytes, `pad` more apart, and their scales."""
    x = torch.randn(rows, K, device="cuda", generator=gen) * scale
    x *= torch.exp(0.5 * torch.randn(rows, 1, device="cuda", generator=gen))
    codes, scales = _quantize(x)
    q = torch.zeros(rows, K // 2 + pad, device="cuda", dtype=torch.uint8)
    q[:, :K // 2] = codes[:, 0::2] + 16 * codes[:, 1::2]
    return q[:, :K // 2], scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state, op = {"case": case}, case["op"]
    if op == "quantize":
        state["x"] = _activations(case["M"], case["K"], case["ld"], case["dtype"], gen)
    elif op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        pad = case.get("pad", 0)
        state["b"], state["sb"] = _operand(N, K, pad, K ** -0.5, gen)
        if op == "product":
            state["a"], state["sa"] = _operand(M, K, pad, 1.0, gen)
        else:
            state["x"] = _activations(M, K, K, case["dtype"], gen)
        state["bias"] = (torch.randn(N, device="cuda", generator=gen) * 0.1
                         if case["bias"] else None)
    elif op == "beams":
        B, W, V = case["B"], case["W"], case["V"]
        x = torch.randn(B, W, case["ld"], device="cuda", generator=gen)
        x *= 1 + 2 * torch.rand(B, 1, 1, device="cuda", generator=gen)
        if case["banned"]:
            # tokens that may not come next, the same ones for a request's beams
            x.masked_fill_(torch.rand(B, 1, case["ld"], device="cuda", generator=gen) < 0.2, -math.inf)
        state["logits"] = x.view(B * W, case["ld"]).to(DTYPES[case["dtype"]])[:, :V]
        state["scores"] = -20 - 3 * torch.rand(B, W, device="cuda", generator=gen)
        state["finished"] = (torch.rand(B, W, device="cuda", generator=gen) < 0.3
                             if case["finished"] else None)
    else:
        B, W, dtype = case["B"], case["W"], DTYPES[case["dtype"]]
        shape = (B * W, case["heads"], case["capacity"], case["dim"])
        # keys and values of each layer, the tokens so far, and a small state of each beam
        state["states"] = [torch.randn(shape, device="cuda", generator=gen, dtype=dtype)[:, :, :case["length"]]
                           for _ in range(2 * case["layers"])]
        state["states"].append(torch.randint(0, 50000, (B * W, case["capacity"]), device="cuda",
                                             generator=gen)[:, :case["length"]])
        state["states"].append(torch.randn(B * W, 33, device="cuda", generator=gen).half())
        beams = torch.randint(0, W, (B, W), device="cuda", generator=gen)
        if case["place"]:
            # a beam that goes on keeps its place, the others' places take its copies
            goes_on = torch.zeros_like(beams).scatter_(1, beams, torch.ones_like(beams))
            beams = torch.where(goes_on > 0, torch.arange(W, device="cuda"), beams)
        state["beams"] = beams
    return state


# ---------------------------------------------------------------- the plain forms ---------

def _quantize(x):
    """(codes of 0 to 15, bytes of scales): a block's largest magnitude, its exponent less 2 as the
    scale's, and each value over the scale rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties
    to the even code."""
    M, K = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -K % 32)).view(M, -1, 32)
    exponent = blocks.abs().amax(2).view(torch.int32) >> 23
    scales = torch.where(exponent == 255, exponent, (exponent - 2).clamp_min(0))
    y = torch.ldexp(blocks, (127 - scales)[:, :, None])
    y = torch.where((scales == 255)[:, :, None], torch.zeros_like(y), y)
    size = y.abs()
    code = torch.where(size < 2, (2 * size).round(),
                       torch.where(size < 4, 2 + size.round(), 4 + (size / 2).round()).clamp_max(7))
    code = torch.where(torch.signbit(y), code + 8, code).to(torch.uint8)
    return code.view(M, -1)[:, :K], scales.to(torch.uint8)


def _values(codes, scales):
    M, K = codes.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    size = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    size = torch.where(scales == 255, torch.full_like(size, math.nan), size)
    return table[codes.int()] * size.repeat_interleave(32, 1)[:, :K]


def _unpack(q):
    return torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)


def _product(a, sa, b, sb, bias, dtype):
    c = _values(a, sa) @ _values(b, sb).t()
    return (c if bias is None else c + bias).to(dtype)


def _beams(logits, scores, top, finished, pad_token):
    """The best continuations of each request: of each beam its `top` largest logits, equal ones by their
    index, then of all beams' by score plus logarithm of probability, in 64 bits: which of two
    beams' tokens comes first may hang on a difference that 32 bits lose."""
    (B, W), V = scores.shape, logits.shape[1]
    n = min(top, V)
    x = logits.double()
    peak = x.amax(1, keepdim=True)
    offset = scores.double().view(-1) - peak[:, 0] - (x - peak).exp().sum(1).log()
    bits = logits.float().view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits - 1, bits)
    best = (order * 4294967296 + (4294967295 - torch.arange(V, device=x.device))).topk(n, dim=1).values
    tokens = 4294967295 - (best & 4294967295)
    keys = x.gather(1, tokens) + offset[:, None]
    if finished is not None:
        # a beam that has ended offers itself alone
        first = torch.arange(n, device=x.device) == 0
        alone = torch.where(first, scores.double().view(-1, 1), -math.inf)
        keys = torch.where(finished.view(-1, 1), alone, keys)
        tokens = torch.where(finished.view(-1, 1), torch.full_like(tokens, pad_token), tokens)
    keys = torch.where(keys > -math.inf, keys, -math.inf).view(B, W * n)
    keys, at = torch.nn.functional.pad(keys, (0, max(0, top - W * n)), value=-math.inf).sort(
        dim=1, descending=True, stable=True)
    keys, at = keys[:, :top], at[:, :top]
    some = keys > -math.inf
    tokens = tokens.view(B, W * n).gather(1, at.clamp_max(W * n - 1))
    return {"scores": keys.float(), "beams": torch.where(some, at // n, -1), "tokens": torch.where(some, tokens, -1)}


def _reorder(states, beams, place):
    B, W = beams.shape
    rows = (beams + W * torch.arange(B, device=beams.device)[:, None]).view(-1)
    moved = [t.index_select(0, rows) for t in states]
    return [t.copy_(m) for t, m in zip(states, moved)] if place else moved


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import fp32_gemm_f32_amd as g
        if op == "quantize":
            # what 4 bits hold comes back as the values it stands for
            q, scales = g.quantize_mx4(state["x"])
            return {"values": g.dequantize_mx4(q, scales, dtype=DTYPES[case["dtype"]], columns=case["K"]),
                    "scales": scales}
        if op == "product":
            return g.matmul_mx4(state["a"], state["sa"], state["b"], state["sb"],
                                bias=state["bias"], out_dtype=DTYPES[case["out"]])
        if op == "linear":
            return g.linear_mx4(state["x"], state["b"], state["sb"], bias=state["bias"])
        if op == "beams":
            r = g.beam_step(state["logits"], state["scores"], top=case["top"], finished=state["finished"],
                            pad_token=2)
            return {"scores": r.scores, "beams": r.beams, "tokens": r.tokens}
        return g.reorder_beams(state["states"], state["beams"], out=state["states"] if case["place"] else None)
    if op == "quantize":
        codes, scales = _quantize(state["x"])
        return {"values": _values(codes, scales).to(DTYPES[case["dtype"]]), "scales": scales}
    if op == "product":
        return _product(_unpack(state["a"]), state["sa"], _unpack(state["b"]), state["sb"], state["bias"],
                        DTYPES[case["out"]])
    if op == "linear":
        return _product(*_quantize(state["x"]), _unpack(state["b"]), state["sb"], state["bias"],
                        state["x"].dtype)
    if op == "beams":
        return _beams(state["logits"], state["scores"], case["top"], state["finished"], 2)
    return _reorder(state["states"], state["beams"], case["place"])


# ---------------------------------------------------------------- from the definitions ----

def _exact_quantized(x):
    """The values the 4-bit form of x stands for: among the 15 values of a block's scale the nearest one,
    of two as near the one whose magnitude's code is even."""
    M, K = x.shape
    x = torch.cat([x.double(), torch.zeros(M, -K % 32, device=x.device, dtype=torch.float64)], 1).view(M, -1, 32)
    peak = x.abs().max(dim=2, keepdim=True).values
    power = torch.floor(torch.log2(torch.where(peak > 0, peak, 1.0)))
    power = power - (torch.exp2(power) > peak).double() + (torch.exp2(power + 1) <= peak).double()
    unit = torch.exp2(torch.where(peak > 0, power - 2, -127.0).clamp_min(-127))
    y = (x / unit).abs()
    # a value lies above a border between two neighbours, or on it where the upper one's code is even
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    value = torch.zeros_like(y)
    for code in range(1, 8):
        border = (grid[code - 1] + grid[code]) / 2
        above = y >= border if code % 2 == 0 else y > border
        value = torch.where(above, grid[code], value)
    return (value * torch.sign(x) * unit).view(M, -1)[:, :K]


def _exact_values(q, scales):
    """Elements and scales by the bits' meaning."""
    b = torch.stack([q % 16, q // 16], dim=2).flatten(1).long()
    sign, exponent, mantissa = b // 8, b // 2 % 4, b % 2
    size = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * 2.0 ** (exponent - 1).double())
    unit = torch.exp2(scales.double() - 127).unsqueeze(2).expand(-1, -1, 32).flatten(1)[:, :b.shape[1]]
    return (1 - 2 * sign) * size * unit


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    op = case["op"]
    if op == "reorder":
        return None                      # copies
    s = prepare(case, seed)
    if op == "quantize":
        return {"values": _exact_quantized(s["x"]), "scales": None}
    if op in ("product", "linear"):
        a = _exact_values(s["a"], s["sa"]) if op == "product" else _exact_quantized(s["x"])
        c = torch.matmul(a, _exact_values(s["b"], s["sb"]).transpose(0, 1).contiguous())
        return c if s["bias"] is None else c + s["bias"].double().unsqueeze(0)
    B, W = s["scores"].shape
    best = []
    step = max(1, (1 << 27) // (W * case["V"]))          # requests at a time, 1 GiB in 64 bits
    for b in range(0, B, step):
        x = s["logits"][b * W:(b + step) * W].double()
        total = torch.log_softmax(x, dim=1).view(-1, W, case["V"]) + s["scores"][b:b + step].double().unsqueeze(2)
        if s["finished"] is not None:
            ended = s["finished"][b:b + step]
            total[ended] = -math.inf
            total[..., 2] = torch.where(ended, s["scores"][b:b + step].double(), total[..., 2])
        best.append(torch.topk(total.flatten(1), case["top"], dim=1).values)
    return {"scores": torch.cat(best), "beams": None, "tokens": None}


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + case["M"] * -(-case["K"] // 32), "flops": 4 * n}
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        row = K / 2 + -(-K // 32)
        first, size = (M * row, SIZE[case["out"]]) if op == "product" else (M * K * SIZE[case["dtype"]],
                                                                            SIZE[case["dtype"]])
        return {"bytes": first + N * row + M * N * size + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "beams":
        n = case["B"] * case["W"] * case["V"]
        live = 0.7 if case["finished"] else 1.0
        return {"bytes": live * n * SIZE[case["dtype"]] + case["B"] * (4 * case["W"] + 20 * case["top"]),
                "flops": 4 * live * n}
    W = case["W"]
    rows = case["B"] * W
    row = (2 * case["layers"] * case["heads"] * case["length"] * case["dim"] * SIZE[case["dtype"]]
           + 8 * case["length"] + 66)
    # of W draws from W, this share of the beams is drawn at all: out of place those are read and every
    # place is written; in place the other places are written, from no more rows than are drawn
    drawn = 1 - (1 - 1 / W) ** W
    moved = drawn + 1 if not case["place"] else (1 - drawn) + min(drawn, 1 - drawn)
    return {"bytes": rows * row * moved, "flops": 0}
