"""Token log-probabilities, entropy, alternatives and their gradient against plain numpy in
64 bits: lengths from one, odd sizes and addresses, masked and empty rows, ties, autograd,
in-place gradients, other streams and graph capture."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def reference(x, tokens):
    """lse, entropy, logprob of float64 rows."""
    with np.errstate(all="ignore"):
        m = np.max(x, axis=1, keepdims=True)
        m0 = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(x - m0)
        s = e.sum(1)
        lse = m0[:, 0] + np.log(s)
        p = e / s[:, None]
        h = -np.sum(np.where(p > 0, p * (x - lse[:, None]), 0.0), axis=1)
        h = np.where(np.isneginf(lse), 0.0, np.where(np.isnan(lse), np.nan, h))
        at = x[np.arange(len(x)), np.clip(tokens, 0, x.shape[1] - 1)]
        lp = np.where(np.isneginf(lse), -np.inf, at - lse)
        lp = np.where(tokens < 0, 0.0, np.where(tokens >= x.shape[1], np.nan, lp))
    return lse, h, lp


def ranked(x, top):
    """The alternatives' indices: descending, equal ones ascending, NaN last."""
    v = np.where(np.isnan(x), -np.inf, x) + 0.0
    nan = np.isnan(x)
    return np.stack([np.lexsort((np.arange(x.shape[1]), -v[i], nan[i]))[:top] for i in range(len(x))])


def tolerance(V):
    """Of a row's log-sum: each term e^(x - m) is off by the roundings of x - m, of two
    products and of the exponential, (3 |x - m| + 2) U relative, at most 64 U where the term
    counts (|x - m| <= 20; below that it weighs under 2e-9); adding V / 256 + 32 terms one
    after another adds that many U."""
    return (64 + V / 256 + 32) * 2 * U


def close(got, want, tol, what):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    both = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), both, err_msg=what)
    np.testing.assert_array_equal(got[~both], want[~both], err_msg=what)
    off = np.abs(got[both] - want[both]) - (tol + 4 * U * np.abs(want[both]))
    assert off.size == 0 or off.max() <= 0, f"{what}: off by {off.max()} more than the roundings"


def check(r, x, tokens, top):
    V = x.shape[1]
    lse, h, lp = reference(x, tokens)
    t = tolerance(V)
    close(r.lse, lse, t, "lse")
    close(r.logprobs, lp, t, "logprobs")
    # entropy = log s - d / s: both of them and their quotient's relative error
    close(r.entropy, h, t * (2 * np.log(V) + 2), "entropy")
    if top:
        idx = ranked(x, top)
        np.testing.assert_array_equal(r.top_tokens.cpu().numpy(), idx)
        with np.errstate(invalid="ignore"):
            v = np.take_along_axis(x, idx, 1)
            want = np.where(np.isneginf(lse)[:, None], np.where(np.isnan(v), np.nan, -np.inf),
                            v - lse[:, None])
        close(r.top_logprobs, want, t, "top")


def logits(torch, host, dt, pad=0, offset=0):
    x = torch.from_numpy(host.astype(np.float32)).to(dtype_of(torch, dt))
    rows, cols = x.shape
    buf = torch.full((offset + rows * (cols + pad) + 1,), float("inf"), dtype=x.dtype)
    buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = x
    dev = buf.cuda()
    return dev[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], x.double().numpy()


@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (1, 2, 0), (3, 5, 5), (2, 64, 64), (4, 65, 3),
                                     (7, 1000, 20), (1, 4097, 1), (2, 16384, 64), (1, 131072, 20),
                                     (1, 100003, 5), (5, 32001, 0), (600, 1003, 2), (1030, 300, 7),
                                     (3, 250000, 33), (2, 1000003, 20), (300, 2500, 4)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3)])
def test_logprobs(torch, M, V, top, dt, pad, offset):
    rng = np.random.default_rng(M * 31 + V + top)
    d, x = logits(torch, rng.standard_normal((M, V)) * rng.uniform(0.5, 4, (M, 1)), dt, pad, offset)
    tokens = rng.integers(0, V, M)
    tokens[1::3] = -100
    print(f"[logprobs] {M}x{V} top {top} {dt} pad {pad}", flush=True)
    r = g.token_logprobs(d, torch.from_numpy(tokens).cuda(), top=top)
    check(r, x, tokens, top)


@pytest.mark.parametrize("V", [3, 700, 9000, 40000, 300000])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("many", [False, True])
def test_edge_rows(torch, V, dt, many):
    """Masked, empty, constant, sorted, NaN and infinite rows; few of them (split over
    workgroups where V allows) and many."""
    rng = np.random.default_rng(V)
    top = min(V, 20)
    if many and V > 100000:
        pytest.skip("long rows are few")
    rows = [np.full(V, -np.inf), np.zeros(V), np.linspace(-5, 5, V), np.linspace(5, -5, V),
            np.where(np.arange(V) % 7 == 0, 1.0, -np.inf), np.full(V, 60000.0), np.full(V, -60000.0),
            np.where(np.arange(V) == V - 1, 3.0, -np.inf),
            np.where(np.arange(V) == V // 2, np.nan, rng.standard_normal(V)),
            np.where(np.arange(V) == 1, np.inf, rng.standard_normal(V)),
            np.full(V, np.nan), np.where(np.arange(V) % 2 == 0, 0.0, -0.0),
            np.where(np.arange(V) >= V - 2, np.nan, -np.inf), np.round(rng.standard_normal(V))]
    host = np.stack(rows * (60 if many else 1))
    lowest = {"f32": -3.4028235e38, "bf16": -3.3895314e38, "f16": -65504.0}[dt]
    host[4::14][:, 1::7] = lowest                   # masks of the type's lowest value too
    d, x = logits(torch, host, dt)
    M = len(host)
    tokens = rng.integers(0, V, M)
    tokens[M - 3], tokens[M - 2], tokens[0] = V, V + 7, 0
    print(f"[logprobs edges] V {V} {dt} many {many}", flush=True)
    r = g.token_logprobs(d, torch.from_numpy(tokens.astype(np.int32)).cuda(), top=top)
    lse, h, lp = reference(x, tokens)
    nan = np.isnan(x).any(1) | np.isposinf(x).any(1)
    lse[nan], h[nan] = np.nan, np.nan
    lp[nan & (tokens >= 0)] = np.nan
    t = tolerance(V)
    # values of size 6e4 leave x - lse with the roundings of lse
    big = 4 * U * 60000.0 * (np.abs(np.where(np.isfinite(lse), lse, 0)) > 1000)
    close(r.lse, lse, t, "lse")
    close(r.logprobs, lp, t + big, "logprobs") if not big.any() else None
    close(r.entropy, h, t * (2 * np.log(V) + 2), "entropy")
    idx = ranked(x, top)
    np.testing.assert_array_equal(r.top_tokens.cpu().numpy(), idx)


def test_no_rows_and_refusals(torch):
    z = torch.zeros(0, 10, device="cuda")
    r = g.token_logprobs(z, torch.zeros(0, dtype=torch.int64, device="cuda"), top=3)
    assert r.logprobs.shape == (0,) and r.top_tokens.shape == (0, 3)
    x = torch.zeros(2, 10, device="cuda")
    tok = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        g.token_logprobs(x, tok, top=11)
    with pytest.raises(ValueError):
        g.token_logprobs(x, tok[:1])
    with pytest.raises(TypeError):
        g.token_logprobs(x, tok.float())
    with pytest.raises(ValueError):
        g.token_logprobs(x, tok.cpu())
    with pytest.raises(g.SgemmError):
        g.token_logprobs(torch.zeros(2, 0, device="cuda"), tok)
    with pytest.raises(ValueError):
        g.token_logprobs_backward(x, tok, torch.zeros(2, device="cuda"), None,
                                  torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda"))


def test_split_and_unsplit_agree(torch):
    """Without a workspace a row is not split: the alternatives are the same, the sums the
    same to their rounding; a workspace that is too small is refused. Repeats are identical."""
    M, V, top = 2, 600001, 9
    assert g.token_logprobs_workspace_size(M, V, 0, top) > 0
    x = torch.randn(M, V, device="cuda")
    tok = torch.tensor([5, -1], device="cuda")
    a = g.token_logprobs(x, tok, top=top)
    b = g.token_logprobs(x, tok, top=top)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    lp, ent, lse = (torch.empty(M, device="cuda") for _ in range(3))
    tv = torch.empty(M, top, device="cuda")
    ti = torch.empty(M, top, dtype=torch.int64, device="cuda")
    args = (M, V, x.data_ptr(), 0, V, tok.data_ptr(), 8, lp.data_ptr(), ent.data_ptr(),
            lse.data_ptr(), top, tv.data_ptr(), ti.data_ptr())
    g.token_logprobs_raw(*args)
    check(g.TokenLogprobs(lp, ent, lse, tv, ti), x.double().cpu().numpy(), tok.cpu().numpy(), top)
    assert torch.equal(ti, a.top_tokens)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(g.SgemmError) as e:
        g.token_logprobs_raw(*args, ws.data_ptr(), 16)
    assert e.value.status == -6
    # entropy and lse may be left out
    g.token_logprobs_raw(M, V, x.data_ptr(), 0, V, tok.data_ptr(), 8, lp.data_ptr(), 0, 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("V", [50001, 131072, 700001])
@pytest.mark.parametrize("top", [1, 5, 64])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_that_crowd_the_alternatives(torch, V, top, dt):
    """Unsplit rows (no workspace) in which the largest values lie in few threads' share of the
    row, rise along it, or are nearly all equal: the candidates' list is cut on the way."""
    j = np.arange(V)
    chunk = j // (4 if dt == "f32" else 8)
    rows = [-(chunk % 256) + chunk / 4096.0, -(chunk % 256) * 2.0 - chunk / 2048.0,
            np.where(chunk % 256 < 3, np.round(j / 997.0), -5.0), j / float(V), -j / float(V),
            np.where(j % 2048 < 16, 1.0, 0.0), np.where(j < V - 3, -np.inf, 2.0),
            np.where(chunk % 256 == 255, 7.0, np.where(j % 3 == 0, np.nan, -np.inf))]
    d, x = logits(torch, np.stack(rows), dt)
    M = len(rows)
    tok = torch.full((M,), -1, device="cuda")
    lp, ent, lse = (torch.empty(M, device="cuda") for _ in range(3))
    tv = torch.empty(M, top, device="cuda")
    ti = torch.empty(M, top, dtype=torch.int64, device="cuda")
    print(f"[logprobs crowded] {V} top {top} {dt}", flush=True)
    g.token_logprobs_raw(M, V, d.data_ptr(), 0 if dt == "f32" else 1, V, tok.data_ptr(), 8, lp.data_ptr(),
                         ent.data_ptr(), lse.data_ptr(), top, tv.data_ptr(), ti.data_ptr(),
                         stream=torch.cuda.current_stream().cuda_stream)
    np.testing.assert_array_equal(ti.cpu().numpy(), ranked(x, top))
    r = g.token_logprobs(d, tok, top=top)              # and split over workgroups
    assert torch.equal(r.top_tokens, ti)


def gradient_reference(x, tokens, lse, h, gl, gh, gs):
    """dx and the size its roundings are relative to."""
    logp = x - lse[:, None]
    p = np.exp(logp)
    live = (tokens >= 0).astype(np.float64)
    g1 = gl * live
    hot = np.zeros_like(x)
    ok = (tokens >= 0) & (tokens < x.shape[1])
    hot[np.arange(len(x))[ok], tokens[ok]] = 1.0
    lg = np.where(p > 0, logp, 0.0)
    dx = g1[:, None] * (hot - p) - gh[:, None] * p * (lg + h[:, None]) + gs[:, None] * p
    size = p * (np.abs(g1) + np.abs(gs))[:, None] + np.abs(gh)[:, None] * p * (np.abs(lg) + np.abs(h)[:, None])
    # p is off by (3 |logp| + 4) U relative, the factors and sums by 4 U more
    tol = size * (3 * np.abs(lg) + 8) * U + np.abs(g1)[:, None] * hot * U
    return dx, tol


@pytest.mark.parametrize("M,V", [(1, 1), (2, 7), (3, 1000), (5, 4099), (2, 32001), (700, 130), (1, 131072)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_gradient(torch, M, V, dt, pad, offset):
    rng = np.random.default_rng(M + V)
    d, x = logits(torch, rng.standard_normal((M, V)) * 3, dt, pad, offset)
    tokens = rng.integers(0, V, M)
    tokens[1::2] = -1
    lse, h, _ = reference(x, tokens)
    lse, h = lse.astype(np.float32), h.astype(np.float32)
    gl, gh, gs = (rng.standard_normal(M).astype(np.float32) for _ in range(3))
    for use in [(1, 0, 0), (1, 1, 0), (1, 1, 1), (0, 0, 1)]:
        vec = [torch.from_numpy(v).cuda() if u else None for u, v in zip(use, (gl, gh, gs))]
        print(f"[gradient] {M}x{V} {dt} pad {pad} {use}", flush=True)
        out = torch.full((M, V + 2), 77.0, dtype=d.dtype, device="cuda")
        g.token_logprobs_backward(d, torch.from_numpy(tokens).cuda(), torch.from_numpy(lse).cuda(),
                                  torch.from_numpy(h).cuda() if use[1] else None, *vec, out=out[:, :V])
        assert (out[:, V:] == 77.0).all()
        want, tol = gradient_reference(x, tokens, lse.astype(np.float64), h.astype(np.float64),
                                       *(u * v.astype(np.float64) for u, v in zip(use, (gl, gh, gs))))
        tol = tol + HALF[dt] * (np.abs(want) + tol) + {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}[dt]
        got = out[:, :V].double().cpu().numpy()
        worst = (np.abs(got - want) - tol).max()
        assert worst <= 0, f"off by {worst} more than the roundings"


def test_gradient_against_differences(torch):
    """Through autograd, against central differences of the definition in 64 bits (their own
    error is of the order of step^2, 1e-10)."""
    rng = np.random.default_rng(12)
    M, V = 3, 11
    host = rng.standard_normal((M, V))
    d, x = logits(torch, host, "f32")
    tokens = np.array([4, -1, 10])
    w = rng.standard_normal((3, M))
    leaf = d.detach().clone().requires_grad_()
    r = g.token_logprobs(leaf, torch.from_numpy(tokens).cuda(), top=2)
    assert not r.top_logprobs.requires_grad and not r.top_tokens.requires_grad
    ws = torch.from_numpy(w.astype(np.float32)).cuda()
    (ws[0] * r.logprobs + ws[1] * r.entropy + ws[2] * r.lse).sum().backward()
    w = w.astype(np.float32).astype(np.float64)

    def total(y):
        lse, h, lp = reference(y, tokens)
        return (w[0] * lp + w[1] * h + w[2] * lse).sum()
    step = 1e-5
    for i in range(M):
        for j in range(V):
            up, down = x.copy(), x.copy()
            up[i, j] += step
            down[i, j] -= step
            want = (total(up) - total(down)) / (2 * step)
            assert abs(leaf.grad[i, j].item() - want) <= 1e-8 + 64 * U * np.abs(w).sum()


def test_gradient_edges_and_in_place(torch):
    V = 1000
    x = torch.randn(6, V, device="cuda")
    x[0] = float("-inf")
    x[1, ::2] = float("-inf")
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    tok = torch.tensor([3, 1, 0, 2, -100, V], device="cuda")
    r = g.token_logprobs(x, tok)
    one = torch.ones(6, device="cuda")
    want = g.token_logprobs_backward(x, tok, r.lse, r.entropy, one, one, one)
    assert (want[0] == 0).all()
    assert (want[1, ::2] == 0).all() and torch.isfinite(want[1]).all()
    assert torch.isnan(want[2]).all() and torch.isnan(want[3]).all() and torch.isnan(want[5]).all()
    assert torch.isfinite(want[4]).all()
    y = x.clone()
    same = g.token_logprobs_backward(y, tok, r.lse, r.entropy, one, one, one, out=y)
    assert same.data_ptr() == y.data_ptr()
    np.testing.assert_array_equal(y.cpu().numpy(), want.cpu().numpy())
    # a constant row: the entropy's gradient vanishes, the token's is [j = t] - 1 / V
    c = torch.zeros(1, V, device="cuda")
    t0 = torch.tensor([17], device="cuda")
    rc = g.token_logprobs(c, t0)
    d = g.token_logprobs_backward(c, t0, rc.lse, rc.entropy, one[:1], one[:1])[0].cpu().numpy()
    ref = np.full(V, -1.0 / V)
    ref[17] += 1
    assert np.abs(d - ref).max() <= tolerance(V)


def test_autograd_paths(torch):
    """Only one of the outputs used; broadcast gradients; bf16 leaves; nothing used; the
    gradient of a strided leaf."""
    x = torch.randn(5, 300, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    tok = torch.randint(0, 300, (5,), device="cuda")
    g.token_logprobs(x, tok).logprobs.sum().backward()              # an expanded gradient
    one = torch.ones(5, device="cuda")
    r = g.token_logprobs(x.detach(), tok)
    assert torch.equal(x.grad, g.token_logprobs_backward(x, tok, r.lse, None, one))
    x.grad = None
    g.token_logprobs(x, tok).lse.mean().backward()
    assert torch.equal(x.grad, g.token_logprobs_backward(x, tok, r.lse, None, None, None, one / 5))
    base = torch.randn(5, 640, device="cuda", requires_grad=True)
    g.token_logprobs(base[:, 1:601], tok, top=1).entropy.sum().backward()
    assert (base.grad[:, 0] == 0).all() and (base.grad[:, 601:] == 0).all()
    assert base.grad[:, 1:601].abs().sum() > 0
    with torch.no_grad():
        assert not g.token_logprobs(x, tok).logprobs.requires_grad
    t = torch.randn(300, 5, device="cuda").t()                      # a transposed view is copied
    check(g.token_logprobs(t, tok), t.double().cpu().numpy(), tok.cpu().numpy(), 0)


@pytest.mark.parametrize("M,V,top", [(2, 600001, 9), (600, 3001, 3)])
def test_graph_capture_and_other_stream(torch, M, V, top):
    x = torch.randn(M, V, device="cuda")
    tok = torch.randint(0, V, (M,), device="cuda")
    one = torch.ones(M, device="cuda")

    def step():
        r = g.token_logprobs(x, tok, top=top)
        return (*r, g.token_logprobs_backward(x, tok, r.lse, r.entropy, one, one))
    want = step()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    print(f"[logprobs graph] {M}x{V}", flush=True)
    with torch.cuda.stream(stream):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
        with torch.cuda.graph(graph, stream=stream):
            got = step()
    torch.cuda.synchronize()
    for i in range(3):
        x.mul_(-0.5 if i else 1.0)
        want = step()                              # eager work between the replays
        for t in got:
            t.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_offsets_past_32_bits(torch):
    """Rows that start past 2^31 elements and 2^32 bytes."""
    M, V = 20, 1 << 17
    ld = 1 << 27
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(M, ld)[:, :V]
    host = torch.randn(M, V, device="cuda").to(torch.bfloat16)
    x.copy_(host)
    tok = torch.arange(M, device="cuda") * 1000
    a, b = g.token_logprobs(x, tok, top=4), g.token_logprobs(host, tok, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    one = torch.ones(M, device="cuda")
    d = g.token_logprobs_backward(x, tok, a.lse, a.entropy, one, one)
    assert torch.equal(d, g.token_logprobs_backward(host, tok, a.lse, a.entropy, one, one))
