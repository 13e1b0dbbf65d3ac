"""Outputs that a caller gives to the decoding operators, and autograd: what a backward pass saved is not
changed unseen."""
import pytest

import fp32_gemm_f32_amd as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    g.library()
    return t


def test_saved_states_are_not_changed_unseen(torch):
    """x * h saves h for x's gradient; a reordering of h in place, whole or of a view, stops the backward
    pass, and one of something else does not."""
    beams = torch.tensor([[1, 1, 0]], device="cuda")
    for way in ("list", "single", "view", "other"):
        h = torch.randn(3, 4, 8, device="cuda")
        x = torch.ones(3, 4, 8, device="cuda", requires_grad=True)
        y = (x * h).sum()
        if way == "list":
            g.reorder_beams([h, torch.zeros(3, device="cuda")], beams, out=[h, torch.zeros(3, device="cuda")])
        elif way == "single":
            g.reorder_beams(h, beams, out=h)
        elif way == "view":
            g.reorder_beams([h[:, :2]], beams, out=[h[:, :2]])
        else:
            g.reorder_beams([h], beams)
            g.reorder_beams([h], beams, out=[torch.zeros_like(h)])
        if way == "other":
            y.backward()
            assert torch.equal(x.grad, h)
        else:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()


def test_versions_of_other_outputs(torch):
    x = torch.randn(4, 64, device="cuda")
    q, s = g.quantize_mx4(x)
    y, c = torch.empty(4, 64, device="cuda"), torch.empty(4, 4, device="cuda")
    before = [t._version for t in (q, s, y, c)]
    g.quantize_mx4(x, out=q, scales=s)
    g.dequantize_mx4(q, s, out=y)
    g.matmul_mx4(q, s, q, s, out=c)
    assert all(t._version > v for t, v in zip((q, s, y, c), before))
    assert x._version == 0
    # new tensors, also by the longer way in
    assert all(t._version == 0 for t in g.quantize_mx4(x.t().contiguous().t()))
    assert g.reorder_beams(x, torch.zeros(2, 2, dtype=torch.int64, device="cuda"))._version == 0


def test_outputs_that_require_grad(torch):
    """Refused where gradients are recorded, written where not; inference tensors have no versions."""
    beams = torch.tensor([[1, 1, 0]], device="cuda")
    p = torch.nn.Parameter(torch.arange(6, device="cuda", dtype=torch.float32).view(3, 2))
    hidden = p * 1
    for t in (p, hidden):
        with pytest.raises(RuntimeError, match="requires grad"):
            g.reorder_beams([t], beams, out=[t])
    with torch.no_grad():
        g.reorder_beams([p], beams, out=[p])
    assert p.tolist() == [[2, 3], [2, 3], [0, 1]] and p.requires_grad
    with torch.inference_mode():
        t = torch.arange(3, device="cuda")
        g.reorder_beams([t], beams, out=[t])
    assert t.tolist() == [1, 1, 0]
    g.reorder_beams([t], beams, out=[t])
    g.reorder_beams(t, beams, out=t)
    assert t.tolist() == [1, 1, 1]


def test_tangents_are_refused(torch):
    """Also on the shorter way in, which takes ordinary tensors on a GPU; others are served in a dual level as
    outside of it."""
    fa = torch.autograd.forward_ad
    x, bias, scores = torch.randn(4, 64, device="cuda"), torch.randn(8, device="cuda"), torch.zeros(2, 2, device="cuda")
    w, ws = g.quantize_mx4(torch.randn(8, 64, device="cuda"))
    beams = torch.tensor([[1, 0], [0, 0]], device="cuda")
    q, s = g.quantize_mx4(x)

    with fa.dual_level():
        dx, dbias, dscores = (fa.make_dual(t, torch.ones_like(t)) for t in (x, bias, scores))
        for call in (lambda: g.quantize_mx4(dx), lambda: g.linear_mx4(dx, w, ws), lambda: g.linear_mx4(x, w, ws, bias=dbias),
                     lambda: g.matmul_mx4(q, s, w, ws, bias=dbias), lambda: g.beam_step(dx, scores),
                     lambda: g.beam_step(x, dscores), lambda: g.reorder_beams([beams.view(-1), dx], beams),
                     lambda: g.reorder_beams([torch.zeros_like(x)], beams, out=[dx])):
            with pytest.raises(NotImplementedError):
                call()
        inside = g.linear_mx4(x, w, ws, bias=bias)
    assert torch.equal(inside, g.linear_mx4(x, w, ws, bias=bias))


def test_a_list_that_changes_meanwhile(torch):
    """Another thread empties and fills the caller's list while calls run: each call takes it as it was when
    it began, or refuses one that it found in between."""
    import threading

    beams = torch.tensor([[1, 0]], device="cuda")
    states = [torch.zeros(2, i + 1, device="cuda") for i in range(12)]
    outs, over = list(states), threading.Event()

    def churn():
        while not over.is_set():
            del outs[3:]
            outs.extend(states[3:])

    t = threading.Thread(target=churn)
    t.start()
    try:
        done = 0
        for _ in range(300):
            try:
                r = g.reorder_beams(states, beams, out=outs)
            except ValueError:                                   # the list was short
                continue
            done += 1
            assert len(r) == 12 and all(a is b for a, b in zip(r, states))
    finally:
        over.set()
        t.join()
    assert done > 0
