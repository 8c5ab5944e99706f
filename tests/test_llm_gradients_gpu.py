"""Gradients through the language-model operators as a training program meets
them: dispatch and combine are differentiable where they are called, and what
has no derivative says so when one is asked for.  No gradient is lost without
an error."""
import pytest

pytestmark = pytest.mark.gpu

V = 2.0 ** -24


def _layer(t=50, k=2, experts=4, hidden=24, seed=3):
    """A route with dropped entries, and leaves x, w and the experts' matrices in 32 and in 64 bits."""
    import torch
    import load_balanced_csr_gb300 as lb
    torch.manual_seed(seed)
    ids = torch.randint(-1, experts, (t, k), device="cuda")
    leaves = torch.randn(t, hidden), torch.rand(t, k), torch.randn(experts, hidden, hidden) / hidden ** 0.5
    narrow = [v.cuda().requires_grad_() for v in leaves]
    wide = [v.double().cuda().requires_grad_() for v in leaves]
    return lb.ExpertRoute(t, k, experts).build(ids), ids, narrow, wide


def _through(route, x, w, m, **kw):
    import torch
    rows = route.dispatch(x, **kw)
    begin = route.expert_ptr.tolist()
    parts = [rows[begin[e]:begin[e + 1]] @ m[e] for e in range(m.shape[0])] + [rows[begin[-1]:]]
    return route.combine(torch.cat(parts), w, **kw)


def _definition(ids, x, w, m):
    import torch
    kept = (ids >= 0).double()
    return (torch.einsum("th,tkhf->tkf", x, m[ids.clamp(min=0)]) * (w * kept)[:, :, None]).sum(1)


def _agree(pairs):
    # sums of at most a few hundred products of values of a few units, in 32 bits
    for a, b in pairs:
        assert float((a.double() - b).abs().max()) <= 512 * V * float(b.abs().max())


@pytest.mark.parametrize("loss", ["squares", "sum"])  # the gradient of a sum is one number, expanded
def test_a_layer_trains(loss):
    route, ids, narrow, wide = _layer()
    y, y64 = _through(route, *narrow), _definition(ids, *wide)
    for v in (y, y64):
        (v.square().sum() / 2 if loss == "squares" else v.sum()).backward()
    _agree([(y.detach(), y64.detach())] + [(a.grad, b.grad) for a, b in zip(narrow, wide)])


def test_only_what_requires_a_gradient_gets_one():
    import torch
    route, ids, narrow, wide = _layer(seed=5)
    narrow[0].requires_grad_(False), wide[0].requires_grad_(False)
    for v in (_through(route, *narrow), _definition(ids, *wide)):
        v.square().sum().backward()
    assert narrow[0].grad is None
    _agree([(a.grad, b.grad) for a, b in zip(narrow[1:], wide[1:])])
    with torch.no_grad():
        assert _through(route, *narrow).grad_fn is None
    xs = route.dispatch(narrow[0])
    assert xs.grad_fn is None and not xs.requires_grad
    # without weights
    ys = torch.randn(100, 24, device="cuda", requires_grad=True)
    route.combine(ys).backward(narrow[0])
    assert torch.equal(ys.grad, route.dispatch(narrow[0]))


def test_on_another_stream():
    """The gradient's kernels go where the forward's went, behind what they need."""
    import torch
    route, ids, narrow, wide = _layer(t=3000, hidden=64, seed=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rows = route.dispatch(narrow[0])
    torch.cuda.current_stream().wait_stream(s)
    twice = rows * 2
    s.wait_stream(torch.cuda.current_stream())
    y = route.combine(twice, narrow[1], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    (y.square().sum() / 2).backward()
    torch.cuda.synchronize()
    kept = (ids >= 0).double()
    y64 = 2 * (wide[1] * kept).sum(1, keepdim=True) * wide[0]
    (y64.square().sum() / 2).backward()
    _agree([(y.detach(), y64.detach())] + [(a.grad, b.grad) for a, b in zip(narrow[:2], wide[:2])])


def test_a_route_rebuilt_before_its_backward_pass():
    """As for micro-batches, or a forward pass that is run again."""
    route, ids, narrow, wide = _layer()
    y = _through(route, *narrow)
    route.build(ids[:7].flip(0).contiguous())
    (y.square().sum() / 2).backward()
    (_definition(ids, *wide).square().sum() / 2).backward()
    _agree([(a.grad, b.grad) for a, b in zip(narrow, wide)])


def test_gradients_of_gradients():
    """dispatch is linear: the gradient's gradient is dispatch again.  combine's gradient has none."""
    import torch
    route, _, (x, w, _), _ = _layer()
    dxs = torch.randn(100, 24, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(route.dispatch(x), x, dxs, create_graph=True)
    again, = torch.autograd.grad(dx, dxs, x.detach())
    assert torch.equal(again, route.dispatch(x.detach()))
    ys = torch.randn(100, 24, device="cuda", requires_grad=True)
    dys, = torch.autograd.grad(route.combine(ys, w), ys, torch.ones(50, 24, device="cuda", requires_grad=True), create_graph=True)
    with pytest.raises(RuntimeError):
        dys.sum().backward()


def test_what_cannot_be_differentiated_says_so():
    import torch
    import load_balanced_csr_gb300 as lb
    route, _, (x, w, _), _ = _layer()
    ys, out = torch.randn(100, 24, device="cuda"), torch.empty(50, 24, device="cuda")
    # an output of the caller's, as torch's own operators have it
    for call in (lambda: route.dispatch(x, out=torch.empty(100, 24, device="cuda")), lambda: route.combine(ys, w, out=out),
                 lambda: route.combine_backward(x, ys, w, out=torch.empty_like(ys))):
        with pytest.raises(RuntimeError, match="out="):
            call()
    with torch.no_grad():
        route.combine(ys, w, out=out)
    # the gradient's own result
    dys, dw = route.combine_backward(x, ys, w)
    for v in (dys, dw):
        with pytest.raises(RuntimeError, match="no derivative"):
            v.sum().backward(retain_graph=True)
    # attention of one token, for serving
    attend = lb.PagedAttention(1, 2, 1, 16, torch.float32)
    cache = torch.randn(2, 4, 1, 16, device="cuda")
    table, lens = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([7], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, 16, device="cuda", requires_grad=True)
    got, lse = attend(q, cache, cache, table, lens)
    with torch.no_grad():
        want, want_lse = attend(q, cache, cache, table, lens)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and want.grad_fn is None
    for v in (got, lse):
        with pytest.raises(RuntimeError, match="no derivative"):
            v.sum().backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="out="):
        attend(q, cache, cache, table, lens, out=torch.empty_like(want))


def test_forward_mode_is_refused():
    import torch
    import torch.autograd.forward_ad as forward
    route, _, (x, w, _), _ = _layer()
    x, ys, w = x.detach(), torch.randn(100, 24, device="cuda"), w.detach()
    with forward.dual_level():
        assert torch.equal(route.dispatch(x)[:1], route.dispatch(x)[:1])  # no tangent: as ever
        with pytest.raises(Exception, match="jvp|forward"):
            route.dispatch(forward.make_dual(x, x))
        with pytest.raises(Exception, match="jvp|forward"):
            route.combine(ys, forward.make_dual(w, w))
