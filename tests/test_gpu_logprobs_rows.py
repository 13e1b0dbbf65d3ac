"""Forward results of edge rows and edge tokens, and rows of large logits (read past the caches), of the
token log-probabilities and their gradient, against 64 bits."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    yield t
    t.cuda.empty_cache()


def log_sum_tolerance(V):
    """Terms of a row's log-sum are off by 64 U where they count (three roundings and the exponential's at
    |x - m| <= 20), and adding V / 256 + 32 of them one after another adds that many U."""
    return (64 + V / 256 + 32) * 2 * U


def same(got, want, tol, what):
    """Non-finite values equal (NaN to NaN); finite ones within tol of theirs and four roundings."""
    got, want = got.double().cpu().numpy(), np.asarray(want, dtype=np.float64)
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)
    finite = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), finite, err_msg=what)
    np.testing.assert_array_equal(got[~finite], want[~finite], err_msg=what)
    off = np.abs(got[finite] - want[finite]) - tol[finite] - 4 * U * np.abs(want[finite])
    assert off.size == 0 or off.max() <= 0, f"{what}: off by {off.max()} more than the roundings"


def edge_rows(V, low, rng):
    j = np.arange(V)
    return np.stack([
        np.full(V, -np.inf), np.zeros(V), np.linspace(-5, 5, V), np.where(j % 7 == 0, 1.0, -np.inf),
        np.full(V, 60000.0), np.full(V, -60000.0), np.where(j == V - 1, 3.0, -np.inf),
        np.where(j == V // 2, np.nan, rng.standard_normal(V)), np.where(j == 1, np.inf, rng.standard_normal(V)),
        np.full(V, np.nan), np.where(j % 2 == 0, 0.0, -0.0), np.where(j >= V - 2, np.nan, -np.inf),
        np.round(rng.standard_normal(V)), np.full(V, low), np.where(j % 5 == 0, rng.standard_normal(V), low)])


def definition(x, tokens, top):
    """lse, entropy, logprobs, alternatives of 64-bit rows, by token_logprobs.h."""
    M, V = x.shape
    lse, ent, lp = np.empty(M), np.empty(M), np.empty(M)
    tv, ti = np.empty((M, top)), np.empty((M, top), dtype=np.int64)
    for i, row in enumerate(x):
        undefined = np.isnan(row).any() or np.isposinf(row).any()
        empty = not undefined and np.isneginf(row).all()
        if undefined:
            lse[i] = ent[i] = np.nan
            logp = np.full(V, np.nan)
        elif empty:
            lse[i], ent[i] = -np.inf, 0.0
            logp = np.full(V, -np.inf)
        else:
            m = row.max()
            with np.errstate(under="ignore"):
                e = np.exp(row - m)
            s = e.sum()
            lse[i] = m + np.log(s)
            logp = (row - m) - np.log(s)               # (m + log s would drop digits at 60000 and beyond)
            live = e > 0
            ent[i] = -(e[live] / s * logp[live]).sum()
        t = int(tokens[i])
        lp[i] = 0.0 if t < 0 else np.nan if t >= V else logp[t]
        nan = np.isnan(row)
        order = np.lexsort((np.arange(V), -np.where(nan, -np.inf, row + 0.0), nan))[:top]
        ti[i] = order
        tv[i] = logp[order]
        tv[i][nan[order]] = np.nan
    return lse, ent, lp, tv, ti


@pytest.mark.parametrize("V", [3, 700, 9000, 40000, 300000])
@pytest.mark.parametrize("dt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("token_bits", [32, 64])
@pytest.mark.parametrize("repeat", [1, 20])
def test_edge_rows(torch, V, dt, token_bits, repeat):
    if repeat > 1 and V > 9000:
        repeat = 2
    rng = np.random.default_rng(V + token_bits)
    dtype, top = getattr(torch, dt), min(V, 20)
    host = edge_rows(V, torch.finfo(dtype).min, rng)
    x = torch.from_numpy(np.tile(host, (repeat, 1))).to(dtype).cuda()
    M = len(x)
    tokens = rng.integers(0, V, M)
    tokens[1::4] = rng.integers(0, min(V, 3), len(tokens[1::4]))
    # no token, and tokens past the vocabulary, in ordinary rows (1, 2, 3), an empty one (0) and one with a NaN (7)
    past = [V, V + 7, 2 ** 31 - 1] if token_bits == 32 else [V, 2 ** 31 + V, 2 ** 62]
    tokens[1], tokens[2], tokens[3] = past
    if repeat > 1:
        tokens[15], tokens[16], tokens[17], tokens[22] = V, -1, -2 ** 31 if token_bits == 32 else -2 ** 62, -5
    d = torch.from_numpy(tokens.astype(np.int32 if token_bits == 32 else np.int64)).cuda()
    print(f"[edge rows] {M}x{V} {dt} tokens of {token_bits} bits", flush=True)
    r = g.token_logprobs(x, d, top=top)
    lse, ent, lp, tv, ti = definition(x.double().cpu().numpy(), tokens, top)
    t = log_sum_tolerance(V)
    assert np.isnan(lp[1:4]).all() and np.isfinite(lse[1:4]).all()
    same(r.lse, lse, t, "lse")
    same(r.logprobs, lp, t, "logprobs")
    same(r.entropy, ent, t * (2 * np.log(V) + 2), "entropy")
    np.testing.assert_array_equal(r.top_tokens.cpu().numpy(), ti)
    same(r.top_logprobs, tv, t, "top")


# 128 MiB of logits and more
LARGE = [(600, 120001, "bfloat16", 120064, 5), (1100, 64003, "float16", 64003, 0), (300, 131072, "float32", 131072, 20),
         (2100, 17000, "float32", 17001, 3)]


@pytest.mark.parametrize("M,V,dt,ld,top", LARGE)
def test_large_logits(torch, M, V, dt, ld, top):
    dtype = getattr(torch, dt)
    assert M * V * (4 if dt == "float32" else 2) >= 128 << 20
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn(M, ld, device="cuda", generator=gen) * 3).to(dtype)[:, :V]
    tok = torch.randint(0, V, (M,), device="cuda", generator=gen)
    tok[3::5] = -1
    print(f"[large logits] {M}x{V} {dt} top {top}", flush=True)
    r = g.token_logprobs(x, tok, top=top)
    k, h, s = (torch.randn(M, device="cuda", generator=gen) for _ in range(3))
    grad = g.token_logprobs_backward(x, tok, r.lse, r.entropy, k, h, s)
    t = log_sum_tolerance(V)
    for i in range(0, M, 150):
        w = slice(i, min(M, i + 150))
        y = x[w].double()
        logp = y.log_softmax(1)
        lse = y.logsumexp(1)
        p = logp.exp()
        ent = -(p * logp).sum(1)
        given = tok[w] >= 0
        at = torch.where(given, logp.gather(1, tok[w].clamp_min(0)[:, None])[:, 0], 0.0)
        assert ((r.lse[w].double() - lse).abs() <= t + 4 * U * lse.abs()).all()
        assert ((r.logprobs[w].double() - at).abs() <= t + 4 * U * at.abs()).all()
        assert ((r.entropy[w].double() - ent).abs() <= t * (2 * np.log(V) + 2) + 4 * U * ent).all()
        if top:
            # equal logits by ascending index: a stable order of the descending values
            order = x[w].float().sort(dim=1, descending=True, stable=True)
            assert torch.equal(r.top_tokens[w], order.indices[:, :top])
            v = order.values[:, :top].double() - lse[:, None]
            assert ((r.top_logprobs[w].double() - v).abs() <= t + 4 * U * v.abs()).all()
        # the gradient from the statistics as they were given: p is off by (3 |log p| + 8) U relative
        l32, e32 = r.lse[w].double()[:, None], r.entropy[w].double()[:, None]
        lg = y - l32
        p = lg.exp()
        hot = torch.nn.functional.one_hot(tok[w].clamp_min(0), V) * given[:, None]
        kk, hh, ss = (v[w].double()[:, None] for v in (k, h, s))
        want = kk * (hot - given[:, None] * p) - hh * p * (lg + e32) + ss * p
        size = p * (kk.abs() + ss.abs()) + hh.abs() * p * (lg.abs() + e32)
        tol = size * (3 * lg.abs() + 8) * U + (kk * hot).abs() * U
        tol = tol + HALF[dt] * (want.abs() + tol) + {"float32": 2.0 ** -126, "bfloat16": 2.0 ** -126,
                                                     "float16": 2.0 ** -25}[dt]
        assert ((grad[w].double() - want).abs() <= tol).all()
    here = x.clone() if ld == V else None
    if here is not None:                               # in place
        assert g.token_logprobs_backward(here, tok, r.lse, r.entropy, k, h, s, out=here) is here
        assert torch.equal(here, grad)
