"""The operators next to the FP32 product, as they are measured: a product of 8-bit integers
with one scale for each token and channel, the quantiser that feeds it, and what scoring and
training read off the logits it writes (log-probabilities of given tokens with entropy and
top alternatives, and their gradient).

`own` chooses between the plain form (elementary torch operations) and the package's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a decode batch's activations on their way into a 8-bit product: latency counts
        {"name": "quantize 16x8192 bf16", "op": "quantize", "M": 16, "K": 8192, "ld": 8192,
         "dtype": "bf16"},
        # a prefill's activations, or a weight matrix laid out once
        {"name": "quantize 8192x8192 bf16", "op": "quantize", "M": 8192, "K": 8192, "ld": 8192,
         "dtype": "bf16"},
        # one new token through a square projection: every weight is read for one row
        {"name": "product 1x8192x8192 bf16", "op": "product", "M": 1, "N": 8192, "K": 8192,
         "lda": 8192, "ldb": 8192, "out": "bf16", "bias": False},
        # a decode batch through a wide projection with a bias
        {"name": "product 48x16384x4096 f16", "op": "product", "M": 48, "N": 16384, "K": 4096,
         "lda": 4096, "ldb": 4096, "out": "f16", "bias": True},
        # a short prompt through a small projection
        {"name": "product 1024x1024x1024 bf16", "op": "product", "M": 1024, "N": 1024, "K": 1024,
         "lda": 1024, "ldb": 1024, "out": "bf16", "bias": False},
        # ragged in every dimension: rows of odd length, so most rows start off alignment
        {"name": "product 1023x1025x1027 f32", "op": "product", "M": 1023, "N": 1025, "K": 1027,
         "lda": 1027, "ldb": 1027, "out": "f32", "bias": True},
        # a long prefill through a square projection: the matrix cores' bound
        {"name": "product 8192x8192x8192 bf16", "op": "product", "M": 8192, "N": 8192, "K": 8192,
         "lda": 8192, "ldb": 8192, "out": "bf16", "bias": False},
        # one new token's logits, with the alternatives a server returns beside it
        {"name": "logprobs 1x131072 f32 top 20", "op": "logprobs", "M": 1, "V": 131072,
         "ld": 131072, "dtype": "f32", "top": 20},
        # a prompt scored with alternatives, from logits with padded rows and an odd vocabulary
        {"name": "logprobs 600x50001 bf16 top 5", "op": "logprobs", "M": 600, "V": 50001,
         "ld": 50048, "dtype": "bf16", "top": 5},
        # the log-probabilities of a training batch
        {"name": "logprobs 4096x131072 bf16", "op": "logprobs", "M": 4096, "V": 131072,
         "ld": 131072, "dtype": "bf16", "top": 0},
        # their gradient with an entropy term, over the same logits
        {"name": "gradient 4096x131072 bf16", "op": "gradient", "M": 4096, "V": 131072,
         "ld": 131072, "dtype": "bf16", "entropy": True},
        # a small batch's gradient in 32 bits, no entropy term, an odd vocabulary
        {"name": "gradient 511x32001 f32", "op": "gradient", "M": 511, "V": 32001, "ld": 32001,
         "dtype": "f32", "entropy": False},
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
    op = rng.choice(["quantize", "product", "product", "logprobs", "logprobs", "gradient"])
    if op == "quantize":
        M, K = _size(rng, 1, 16384), _size(rng, 64, 16384)
        M = min(M, 8192 * 8192 // K)
        return {"op": op, "M": M, "K": K, "ld": K + rng.choice([0, 0, 0, 8, 13]),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "product":
        M, N, K = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
        M = max(1, min(M, 8192 ** 3 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "lda": K + rng.choice([0, 0, 0, 16, 5]),
                "ldb": K + rng.choice([0, 0, 0, 16, 3]),
                "out": rng.choice(["f32", "bf16", "f16"]), "bias": rng.random() < 0.5}
    M, V = _size(rng, 1, 4096), _size(rng, 1000, 131072)
    case = {"op": op, "M": M, "V": V, "ld": V + rng.choice([0, 0, 0, 64, 7]),
            "dtype": rng.choice(["f32", "bf16", "f16"])}
    if case["dtype"] == "f32":
        case["M"] = max(1, min(M, 2048 * 131072 // V))
    if op == "logprobs":
        case["top"] = rng.choice([0, 0, 1, 5, 20])
    else:
        case["entropy"] = rng.random() < 0.5
    return case


def _normal(rows, cols, ld, gen, scale=1.0):
    return (torch.randn(rows, ld, device="cuda", generator=gen) * scale)[:, :cols]


def _codes(rows, cols, ld, gen):
    """8-bit rows as a quantiser leaves them: a normal's values on a scale of 127 to about four
    of its deviations."""
    x = torch.randn(rows, ld, device="cuda", generator=gen) * 32
    return x.round_().clamp_(-127, 127).to(torch.int8)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "quantize":
        # activations: rows of different size, a few channels far larger than the others
        x = torch.randn(case["M"], case["ld"], device="cuda", generator=gen)
        x *= torch.exp(torch.randn(case["M"], 1, device="cuda", generator=gen))
        x[:, ::97] *= 8
        state["x"] = x.to(DTYPES[case["dtype"]])[:, :case["K"]]
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        state["a"] = _codes(M, K, case["lda"], gen)
        state["b"] = _codes(N, K, case["ldb"], gen)
        state["sa"] = torch.rand(M, device="cuda", generator=gen) * 0.05 + 0.005
        state["sb"] = torch.rand(N, device="cuda", generator=gen) * 0.002 + 0.0002
        state["bias"] = (torch.randn(N, device="cuda", generator=gen) * 0.1
                         if case["bias"] else None)
    else:
        M, V = case["M"], case["V"]
        x = torch.randn(M, case["ld"], device="cuda", generator=gen)
        x *= 1 + 2 * torch.rand(M, 1, device="cuda", generator=gen)
        state["logits"] = x.to(DTYPES[case["dtype"]])[:, :V]
        tokens = torch.randint(0, V, (M,), device="cuda", generator=gen)
        if M > 8:
            tokens[::9] = -100          # positions without a token, as a loss is padded
        state["tokens"] = tokens
        if case["op"] == "gradient":
            _, state["entropy"], state["lse"] = _stats(state["logits"], tokens)
            state["g_logprobs"] = torch.randn(M, device="cuda", generator=gen) / M
            state["g_entropy"] = (torch.randn(M, device="cuda", generator=gen) * (0.01 / M)
                                  if case["entropy"] else None)
    return state


# ---------------------------------------------------------------- the plain forms ---------

def _quantize(x):
    x = x.float()
    peak = x.abs().amax(1)
    wide, full = peak.double(), torch.full_like(peak, 127.0, dtype=torch.float64)
    scale, inverse = (wide / full).float(), (full / wide).float()
    dead = torch.isinf(inverse)
    scale = torch.where(dead, torch.zeros_like(scale), scale)
    q = (x * inverse[:, None]).round().clamp(-127, 127)
    return torch.where(dead[:, None] | torch.isnan(q), torch.zeros_like(q), q).to(torch.int8), scale


def _product(a, sa, b, sb, bias, dtype):
    c = (a.float() @ b.float().t()) * (sa[:, None] * sb[None, :])
    return (c if bias is None else c + bias).to(dtype)


def _stats(logits, tokens):
    x = logits.float()
    peak = x.amax(1, keepdim=True)
    shifted = x - peak
    e = shifted.exp()
    total = e.sum(1)
    entropy = total.log() - torch.where(e > 0, shifted * e, torch.zeros_like(e)).sum(1) / total
    lse = peak[:, 0] + total.log()
    at = shifted.gather(1, tokens.clamp_min(0)[:, None])[:, 0] - total.log()
    return torch.where(tokens < 0, torch.zeros_like(at), at), entropy, lse


def _top(logits, lse, top):
    """The `top` largest of each row, equal ones by their index: values in an order of whole
    numbers, and the index below them, so that no two are equal."""
    bits = logits.float().view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits - 1, bits)
    index = torch.arange(logits.shape[1], device=logits.device)
    best = (order * 4294967296 + (4294967295 - index)).topk(top, dim=1).values
    tokens = 4294967295 - (best & 4294967295)
    return logits.float().gather(1, tokens) - lse[:, None], tokens


def _gradient(logits, tokens, lse, entropy, g_logprobs, g_entropy):
    logp = logits.float() - lse[:, None]
    p = logp.exp()
    g = torch.where(tokens < 0, torch.zeros_like(g_logprobs), g_logprobs)
    d = -g[:, None] * p
    if g_entropy is not None:
        d -= g_entropy[:, None] * torch.where(p > 0, p * (logp + entropy[:, None]),
                                              torch.zeros_like(p))
    d.scatter_add_(1, tokens.clamp_min(0)[:, None], g[:, None])
    return d.to(logits.dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import fp32_gemm_f32_amd as g
        if op == "quantize":
            q, scales = g.quantize_rows(state["x"])
            return {"q": q, "scales": scales}
        if op == "product":
            return g.matmul_i8(state["a"], state["sa"], state["b"], state["sb"],
                               bias=state["bias"], out_dtype=DTYPES[case["out"]])
        if op == "logprobs":
            r = g.token_logprobs(state["logits"], state["tokens"], top=case["top"])
            out = {"logprobs": r.logprobs, "entropy": r.entropy, "lse": r.lse}
            if case["top"]:
                out["top_logprobs"], out["top_tokens"] = r.top_logprobs, r.top_tokens
            return out
        return g.token_logprobs_backward(state["logits"], state["tokens"], state["lse"],
                                         state["entropy"], state["g_logprobs"],
                                         state["g_entropy"])
    if op == "quantize":
        # the 8-bit numbers come back as the whole numbers they are, the scales beside them
        q, scales = _quantize(state["x"])
        return {"q": q, "scales": scales}
    if op == "product":
        return _product(state["a"], state["sa"], state["b"], state["sb"], state["bias"],
                        DTYPES[case["out"]])
    if op == "logprobs":
        logprobs, entropy, lse = _stats(state["logits"], state["tokens"])
        out = {"logprobs": logprobs, "entropy": entropy, "lse": lse}
        if case["top"]:
            out["top_logprobs"], out["top_tokens"] = _top(state["logits"], lse, case["top"])
        return out
    return _gradient(state["logits"], state["tokens"], state["lse"], state["entropy"],
                     state["g_logprobs"], state["g_entropy"])


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return {"q": None, "scales": s["x"].double().abs().max(dim=1).values.div(127.0)}
    if case["op"] == "product":
        c = torch.matmul(s["a"].double(), s["b"].double().transpose(0, 1).contiguous())
        c = c * s["sa"].double().unsqueeze(1) * s["sb"].double().unsqueeze(0)
        return c if s["bias"] is None else c + s["bias"].double().unsqueeze(0)
    parts = []
    rows = max(1, (1 << 28) // case["V"])          # in blocks of rows, 2 GiB each in 64 bits
    for r in range(0, case["M"], rows):
        x = s["logits"][r:r + rows].double()
        tokens = s["tokens"][r:r + rows]
        given = tokens >= 0
        hot = torch.zeros_like(x)
        hot[given, tokens[given]] = 1.0
        if case["op"] == "logprobs":
            logp = torch.log_softmax(x, dim=1)
            p = logp.exp()
            part = {"logprobs": torch.where(hot > 0, logp, 0.0).sum(dim=1),
                    "entropy": -(p * logp).sum(dim=1), "lse": torch.logsumexp(x, dim=1)}
            if case["top"]:
                part["top_logprobs"] = torch.sort(logp, dim=1, descending=True).values[:, :case["top"]]
        else:
            # the row's saved statistics are inputs here, as they are to run()
            logp = x - s["lse"][r:r + rows].double().unsqueeze(1)
            p = logp.exp()
            g = s["g_logprobs"][r:r + rows].double() * given
            part = g.unsqueeze(1) * (hot - p)
            if s["g_entropy"] is not None:
                part = part - s["g_entropy"][r:r + rows].double().unsqueeze(1) * (
                    p * (logp + s["entropy"][r:r + rows].double().unsqueeze(1)))
        parts.append(part)
    if case["op"] == "gradient":
        return torch.cat(parts)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["top"]:
        out["top_tokens"] = None
    return out


def work(case):
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * (SIZE[case["dtype"]] + 1) + 4 * case["M"], "flops": 4 * n}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + M * N * SIZE[case["out"]] + 4 * (M + N)
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    M, n = case["M"], case["M"] * case["V"]
    if case["op"] == "logprobs":
        return {"bytes": n * SIZE[case["dtype"]] + M * (20 + 12 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * SIZE[case["dtype"]] + M * (20 + (4 if case["entropy"] else 0)),
            "flops": (8 if case["entropy"] else 4) * n}
