"""Beam search's step against its definition in 64 bits, and the reordering of states: ties, banned
tokens, beams that have ended, rows that hold no continuation, long and odd rows, strided and in place
states, other streams and graph capture."""
import numpy as np
import pytest

import fp32_gemm_f32_amd as g
from test_gpu_gemm_i8 import dtype_of, strided

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def reference(x, scores, top, finished=None, pad=0):
    """(scores, beams, tokens) of each request in 64 bits, and the totals and beams in order with one
    more: x (B W, V) and scores (B, W) as numpy arrays."""
    B, W = scores.shape
    x = x.astype(np.float64).reshape(B, W, -1)
    V = x.shape[2]
    out_s, out_b, out_t = np.full((B, top), -INF), np.full((B, top), -1), np.full((B, top), -1)
    edges, owners = np.full((B, top + 1), -INF), np.full((B, top + 1), -1)
    with np.errstate(all="ignore"):
        x = x - x.max(2, keepdims=True)                   # logits over the row's peak
        lse = np.log(np.exp(x).sum(2))
    for b in range(B):
        rows = []
        for w in range(W):
            s = float(scores[b, w])
            if finished is not None and finished[b, w]:
                if s > -INF:
                    rows.append((-s, w, 0.0, pad))
                continue
            if not np.isfinite(lse[b, w]):
                continue
            order = np.lexsort((np.arange(V), -x[b, w]))[:top + 1]
            for t in order:
                total = x[b, w, t] + (s - lse[b, w])
                if total > -INF:
                    rows.append((-total, w, -x[b, w, t], int(t)))
        rows.sort()
        for r, (total, w, _, t) in enumerate(rows[:top]):
            out_s[b, r], out_b[b, r], out_t[b, r] = -total, w, t
        edges[b, :min(len(rows), top + 1)] = [-r[0] for r in rows[:top + 1]]
        owners[b, :min(len(rows), top + 1)] = [r[1] for r in rows[:top + 1]]
    return out_s, out_b, out_t, edges, owners


def check(torch, r, want, V, ties=False):
    """Totals within their roundings: a thread adds at most V / 256 terms, half a step (2^-24) each; 64 more
    for the terms themselves (a unit of the exponential, half a step of an argument up to 30) and the
    joins of lanes, waves and parts; the score is rounded once. Beams and tokens wherever the totals'
    neighbours are further apart than that, or of one beam, whose order is its logits' (ties:
    everywhere)."""
    s, b, t, edges, owners = want
    n = V / 256 + 64
    got_s, got_b, got_t = (v.cpu().numpy() for v in r)
    fine = np.isfinite(s)
    assert np.array_equal(np.isfinite(got_s), fine)
    assert np.array_equal(got_s[~fine], s[~fine])
    tol = n * 2.0 ** -24 + 2.0 ** -24 * np.abs(s[fine])
    assert (np.abs(got_s[fine] - s[fine]) <= tol).all()
    with np.errstate(invalid="ignore"):
        gaps = edges[:, :-1] - edges[:, 1:]
    clear = np.isnan(gaps) | (gaps > 2 * n * 2.0 ** -24) | (owners[:, :-1] == owners[:, 1:])
    alone = clear & np.concatenate([np.ones((len(s), 1), dtype=bool), clear[:, :-1]], axis=1)
    if ties:
        alone[:] = True
    else:
        assert alone.mean() > 0.9
    assert np.array_equal(got_b[alone], b[alone]) and np.array_equal(got_t[alone], t[alone])


@pytest.mark.parametrize("B,W,V,top", [(1, 1, 1, 1), (1, 1, 7, 3), (3, 2, 5, 20), (1, 4, 1000, 4), (2, 3, 4097, 7),
                                       (1, 4, 40000, 8), (5, 5, 9001, 5), (1, 1, 131072, 64), (1, 64, 300, 64),
                                       (40, 8, 2000, 16), (3, 64, 5000, 64), (300, 2, 700, 4), (2, 2, 200001, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_step(torch, dtype, B, W, V, top):
    rng = np.random.default_rng(V + W)
    x = torch.from_numpy(rng.standard_normal((B * W, V)) * 2).to(dtype_of(torch, dtype))
    scores = (-5 * rng.random((B, W))).astype(np.float32)
    print(f"[beams] {dtype} {B}x{W}x{V} top {top}", flush=True)
    r = g.beam_step(x.cuda(), torch.from_numpy(scores).cuda(), top=top)
    assert r.scores.dtype == torch.float32 and r.beams.dtype == r.tokens.dtype == torch.int64
    assert r.scores.shape == r.beams.shape == r.tokens.shape == (B, top)
    check(torch, r, reference(x.double().numpy(), scores, top), V)


@pytest.mark.parametrize("pad,offset", [(1, 0), (7, 3), (64, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_rows(torch, dtype, pad, offset):
    B, W, V = 3, 4, 10001
    rng = np.random.default_rng(pad)
    x = torch.from_numpy(rng.standard_normal((B * W, V))).to(dtype_of(torch, dtype))
    scores = -rng.random((B, W)).astype(np.float32)
    _, dx = strided(torch, x, V + pad, offset, 100.0)
    r = g.beam_step(dx, torch.from_numpy(scores).cuda())
    check(torch, r, reference(x.double().numpy(), scores, W), V)


@pytest.mark.parametrize("B,W,V", [(2, 4, 50), (3, 5, 20000), (70, 6, 3000)])
def test_ended_beams_and_banned_tokens(torch, B, W, V):
    rng = np.random.default_rng(V)
    x = rng.standard_normal((B * W, V)).astype(np.float32)
    x[rng.random(x.shape) < 0.5] = -INF
    scores = -rng.random((B, W)).astype(np.float32)
    ended = rng.random((B, W)) < 0.4
    ended[0, :] = True                                   # a request that has ended: W continuations in all
    scores[0, 1] = -INF
    x[np.flatnonzero(ended.reshape(-1))] = np.nan        # their rows do not count
    top = W + 2
    r = g.beam_step(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda(), top=top,
                    finished=torch.from_numpy(ended).cuda(), pad_token=-7)
    check(torch, r, reference(x, scores, top, ended, -7), V)
    assert r.beams[0].tolist().count(-1) == 3 and (r.tokens[0, :W - 1] == -7).all() and (r.tokens[0, W - 1:] == -1).all()


def test_ties(torch):
    """Beams with the same row and score, constant rows, and many equal logits: lower beams, then lower
    tokens, also where more than a list's worth are equal."""
    row = np.random.default_rng(0).integers(-3, 4, size=(1, 3001)).astype(np.float32)
    for x, W in [(np.repeat(row, 4, axis=0), 4), (np.zeros((3, 100), np.float32), 3),
                 (np.full((2, 9000), 2.5, np.float32), 2), (np.repeat(row, 64, axis=0), 64),
                 (np.zeros((64, 70000), np.float32), 64), (np.full((4, 500), -3.0e38, np.float32), 4)]:
        for top in (1, W, 64):
            scores = np.zeros((1, W), np.float32)
            if x.shape[1] > 3001:                        # sums of equal terms: the same totals in both
                scores[:] = -2.0
            r = g.beam_step(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda(), top=top)
            check(torch, r, reference(x, scores, top), x.shape[1], ties=True)


@pytest.mark.parametrize("B,W,V,top", [(2, 64, 20001, 64), (1, 64, 33000, 32), (5, 48, 4000, 48), (1, 40, 66000, 63),
                                       (260, 1, 70001, 64), (130, 2, 65536, 33)])
@pytest.mark.parametrize("kind", ["spread", "alike", "steps"])
def test_many_beams(torch, kind, B, W, V, top):
    """More keys than the list of the choice holds: beams that differ, beams that are alike, and few
    distinct logits, whose best ones fill the list many times."""
    rng = np.random.default_rng(B + W + top)
    if kind == "steps":
        x = np.repeat(rng.integers(-2, 3, size=(B, V)), W, axis=0).astype(np.float32)
        scores = np.full((B, W), -2.0, np.float32)
    else:
        x = rng.standard_normal((B * W, V)).astype(np.float32)
        scores = (-rng.random((B, W)) * (2.0 if kind == "spread" else 0.0)).astype(np.float32)
    r = g.beam_step(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda(), top=top)
    want = reference(x, scores, top)
    if kind != "steps":
        check(torch, r, want, V)
        return
    # The beams of a request are the same, but rows of odd lengths lie differently in 16-byte chunks: their
    # sums of V terms go in other orders, each off by up to n 2^-24 (check's n), and so are the totals. Any
    # beam may come first, then; each beam's own continuations are the first ones of its order.
    n = V / 256 + 64
    assert np.abs(r.scores.cpu().numpy() - want[0]).max() <= n * 2.0 ** -24 + 2.0 ** -24 * np.abs(want[0]).max()
    beams, tokens = r.beams.cpu().numpy(), r.tokens.cpu().numpy()
    for b in range(B):
        order = np.lexsort((np.arange(V), -x[b * W]))[:top]
        for w in range(W):
            mine = tokens[b][beams[b] == w]
            assert np.array_equal(mine, order[:len(mine)])


def test_rows_without_a_continuation(torch):
    x = np.random.default_rng(1).standard_normal((12, 600)).astype(np.float32)
    x[0], x[1, 5], x[2, 7], x[3, 1:] = -INF, np.nan, INF, -INF
    x[4:8] = -INF                                        # a request with nothing
    x[8] = np.finfo(np.float32).min                      # a mask of the type's lowest value: all alike
    scores = -np.ones((3, 4), np.float32)
    scores[2, 1] = -INF
    scores[2, 2] = np.nan
    for top in (1, 4, 9):
        r = g.beam_step(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda(), top=top)
        check(torch, r, reference(x, np.where(np.isnan(scores), -INF, scores), top), 600, ties=True)
        assert (r.beams[1] == -1).all() and (r.tokens[1] == -1).all() and torch.isinf(r.scores[1]).all()
    assert r.beams[0].tolist() == [3] + [-1] * 8 and r.tokens[0, 0] == 0 and float(r.scores[0, 0]) == -1.0


def test_first_step(torch):
    """All of a request's beams are the same prompt: only the first one's score counts."""
    x = np.repeat(np.random.default_rng(2).standard_normal((2, 5000)), 4, axis=0).astype(np.float32)
    scores = np.full((2, 4), -INF, np.float32)
    scores[:, 0] = 0
    r = g.beam_step(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda())
    check(torch, r, reference(x, scores, 4), 5000)
    assert (r.beams == 0).all()


def test_step_refusals(torch):
    x, s = torch.zeros(6, 10, device="cuda"), torch.zeros(2, 3, device="cuda")
    with pytest.raises(ValueError):
        g.beam_step(x, torch.zeros(2, 4, device="cuda"))
    with pytest.raises(ValueError):
        g.beam_step(x, s, top=0)
    with pytest.raises(ValueError):
        g.beam_step(x, s, top=-1)
    with pytest.raises(ValueError):
        g.beam_step(x, s, top=65)
    with pytest.raises(ValueError):
        g.beam_step(torch.zeros(65, 10, device="cuda"), torch.zeros(1, 65, device="cuda"))
    with pytest.raises(TypeError):
        g.beam_step(x, s.double())
    with pytest.raises(TypeError):
        g.beam_step(x.double(), s)
    with pytest.raises(TypeError):
        g.beam_step(x, s, finished=torch.zeros(2, 3, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g.beam_step(x, s, finished=torch.zeros(3, 2, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        g.beam_step(x, s.cpu())
    with pytest.raises(g.SgemmError) as e:
        g.beam_step(torch.zeros(6, 0, device="cuda"), s)
    assert e.value.status == -1
    r = g.beam_step(torch.zeros(0, 10, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert r.scores.shape == (0, 3)


# ------------------------------------------------------------------ the states ----------

def chosen(rng, B, W):
    b = rng.integers(0, W, size=(B, W))
    b[0, 0] = W - 1
    return b


def moved(torch, t, beams):
    """The reordered tensor, by indexing on the host."""
    B, W = beams.shape
    ok = (beams >= 0) & (beams < W)
    rows = np.where(ok, beams, np.arange(W)) + W * np.arange(B)[:, None]
    return t.cpu()[torch.from_numpy(rows.reshape(-1))]


def states_of(torch, n):
    """Tensors of n rows: caches whole and as views of their first positions, odd sizes, other types."""
    kv = torch.randn(n, 3, 20, 16, device="cuda", dtype=torch.bfloat16)
    both = torch.randn(n, 2, 5, 7, device="cuda", dtype=torch.float16)
    return [kv, torch.randn(n, 3, 20, 16, device="cuda")[:, :, :11], torch.randn(n, 33, device="cuda").half(),
            torch.randint(0, 99, (n, 50), device="cuda")[:, :13], torch.randint(0, 2, (n, 5), device="cuda").bool(),
            torch.randn(n, device="cuda"), torch.randn(n, 4, 6, 31, device="cuda")[:, 1:3, :, 2:9],
            torch.randint(0, 255, (n, 3), device="cuda").to(torch.uint8), both[:, 0], both[:, 1],
            torch.randn(n, 6, 4, device="cuda").transpose(1, 2), torch.randn(n, 0, 4, device="cuda"),
            torch.randn(n, 2, 3, device="cuda", dtype=torch.complex64)]


@pytest.mark.parametrize("B,W", [(1, 1), (1, 4), (3, 5), (2, 8), (5, 16), (2, 17), (1, 33), (2, 64), (40, 3)])
@pytest.mark.parametrize("index", ["int64", "int32"])
def test_reorder(torch, B, W, index):
    rng = np.random.default_rng(W)
    beams = chosen(rng, B, W)
    dev = torch.from_numpy(beams).to(getattr(torch, index)).cuda()
    states = states_of(torch, B * W)
    want = [moved(torch, t, beams) for t in states]
    before = [t.clone() for t in states]
    print(f"[reorder] {B}x{W}", flush=True)
    got = g.reorder_beams(states, dev)
    for a, b, c, d in zip(got, want, states, before):
        assert a.dtype == b.dtype and torch.equal(a.cpu(), b) and torch.equal(c, d)
    back = g.reorder_beams(states, dev, out=states)
    assert all(a is b for a, b in zip(back, states))
    for a, b in zip(states, want):
        assert torch.equal(a.cpu(), b)


def test_reorder_leaves_the_rest(torch):
    """Positions behind the live ones keep what they held, indices out of range leave their rows."""
    cache = torch.randn(8, 2, 10, 4, device="cuda")
    before = cache.clone()
    beams = np.array([[1, -1, 0, 7], [3, 3, 4, 2 ** 40]])
    g.reorder_beams([cache[:, :, :6]], torch.from_numpy(beams).cuda(), out=[cache[:, :, :6]])
    assert torch.equal(cache[:, :, 6:], before[:, :, 6:])
    assert torch.equal(cache[:, :, :6].cpu(), moved(torch, before, beams)[:, :, :6])


def test_reorder_single_and_many_states(torch):
    beams = torch.tensor([[2, 0, 0]], device="cuda")
    t = torch.randn(3, 1000, device="cuda")
    assert torch.equal(g.reorder_beams(t, beams), t[beams[0]])
    assert torch.equal(g.reorder_beams(torch.nn.Parameter(t), beams), t[beams[0]])
    many = [torch.randn(3, i, device="cuda") for i in range(100)]
    for a, b in zip(g.reorder_beams(tuple(many), beams), many):
        assert torch.equal(a, b[beams[0]])
    assert g.reorder_beams([], beams) == []
    assert g.reorder_beams([torch.zeros(0, 5, device="cuda")], beams[:0])[0].shape == (0, 5)
    # a view that takes more than two strides is copied first, and refused in place
    odd = torch.randn(3, 4, 6, 8, 10, device="cuda")[:, ::2, ::2, ::2, ::2]
    assert torch.equal(g.reorder_beams([odd], beams)[0], odd[beams[0]])
    with pytest.raises(ValueError):
        g.reorder_beams([odd], beams, out=[odd])


def test_reordered_tensors_are_ordinary_ones(torch):
    """Results that share an allocation: of every type, apart, and good for a graph of gradients."""
    beams = torch.tensor([[1, 1, 0], [2, 0, 1]], device="cuda", dtype=torch.int32)
    rows = torch.tensor([1, 1, 0, 5, 3, 4], device="cuda")
    kinds = [torch.float32, torch.bool, torch.int64, torch.complex64, torch.float8_e4m3fn, torch.float64, torch.int8]
    states = [torch.randint(0, 2, (6, 3, 5), device="cuda").to(kind) for kind in kinds]
    moved = g.reorder_beams(states, beams)
    for kind, s, m in zip(kinds, states, moved):
        assert m.dtype == kind and m.is_contiguous()
        assert torch.equal(m.view(6, -1).view(torch.uint8), s[rows].view(6, -1).view(torch.uint8))
    moved[0].zero_()
    assert torch.equal(moved[2], states[2][rows])
    x = moved[5].requires_grad_()
    (x * x).sum().backward()
    assert torch.equal(x.grad, 2 * states[5][rows])
    with torch.inference_mode():
        assert all(t.is_inference() for t in g.reorder_beams(states, beams))
    # the first columns of more continuations than beams
    r = g.beam_step(torch.randn(6, 50, device="cuda"), torch.zeros(2, 3, device="cuda"), top=7)
    got = g.reorder_beams(states[:1], r.beams[:, :3])[0]
    assert torch.equal(got, states[0][(r.beams[:, :3] + 3 * torch.arange(2, device="cuda")[:, None]).view(-1)])


def test_reorder_into_other_tensors(torch):
    beams = torch.tensor([[1, 1, 2], [0, 2, 1]], device="cuda")
    src, dst = torch.randn(6, 4, 9, device="cuda"), torch.zeros(6, 4, 20, device="cuda")
    rows = (beams + 3 * torch.arange(2, device="cuda")[:, None]).view(-1)
    g.reorder_beams([src], beams, out=[dst[:, :, 5:14]])
    assert torch.equal(dst[:, :, 5:14], src[rows]) and (dst[:, :, :5] == 0).all() and (dst[:, :, 14:] == 0).all()


def test_reorder_refusals(torch):
    beams, t = torch.zeros(2, 3, dtype=torch.int64, device="cuda"), torch.zeros(6, 8, device="cuda")
    with pytest.raises(TypeError):
        g.reorder_beams([t], beams.float())
    with pytest.raises(ValueError):
        g.reorder_beams([t], beams.view(-1))
    with pytest.raises(ValueError):
        g.reorder_beams([t[:5]], beams)
    with pytest.raises(ValueError):
        g.reorder_beams([t.cpu()], beams)
    with pytest.raises(ValueError):
        g.reorder_beams([t], beams, out=[t, t])
    with pytest.raises(ValueError):
        g.reorder_beams([t], beams, out=[torch.zeros(6, 9, device="cuda")])
    with pytest.raises(ValueError):
        g.reorder_beams([torch.zeros(65, 2, device="cuda")], torch.zeros(1, 65, dtype=torch.int64, device="cuda"))
    for states, out in [([t, t], [t, t]),                              # written twice
                        ([t[:, :5]], [t[:, 1:6]]),                     # shifted onto itself
                        ([t[:, :4], t[:, 4:]], [t[:, 4:], torch.zeros(6, 4, device="cuda")]),
                        ([t], [torch.zeros(6, 1, device="cuda").expand(6, 8)])]:
        with pytest.raises(g.SgemmError):
            g.reorder_beams(states, beams, out=out)


def test_graph_of_a_decoding_step(torch):
    """Logits of a 4-bit head, the step and the reordering in place, captured and replayed: the same as
    the calls one after another."""
    B, W, K, V = 3, 4, 256, 5003
    torch.manual_seed(0)
    w, ws = g.quantize_mx4(torch.randn(V, K, device="cuda"))
    hidden = torch.randn(B * W, K, device="cuda", dtype=torch.bfloat16)
    scores = -torch.rand(B, W, device="cuda")
    start = [torch.randn(B * W, 2, 40, 8, device="cuda", dtype=torch.bfloat16), torch.randint(0, V, (B * W, 40), device="cuda")]

    def step(states):
        r = g.beam_step(g.linear_mx4(hidden, w, ws), scores)
        g.reorder_beams(states, r.beams, out=states)
        return r

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    caught, eager = [t.clone() for t in start], [t.clone() for t in start]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step([t.clone() for t in start])
        with torch.cuda.graph(graph, stream=stream):
            r = step(caught)
    torch.cuda.synchronize()
    for a, b in zip(caught, start):
        a.copy_(b)
    for i in range(3):
        hidden.mul_(-1.3)
        scores.add_(torch.rand(B, W, device="cuda"))
        want = step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want)), i
        assert all(torch.equal(a, b) for a, b in zip(caught, eager)), i


def test_two_streams_at_once(torch):
    """Calls on two streams, each with its own workspace, do not meet."""
    xs = [torch.randn(8, 60000, device="cuda") for _ in range(2)]
    scores = torch.zeros(2, 4, device="cuda")
    want = [g.beam_step(x, scores, top=16) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(g.beam_step(xs[k], scores, top=16))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[k]))
