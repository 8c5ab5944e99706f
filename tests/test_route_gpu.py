"""Routing to experts against its definition in 64 bits: the sorted order bit
for bit, the rows' passes within bounds derived from the roundings they make.

With u = 2^-24 (f32), 2^-8 (bf16), 2^-11 (f16) the half-unit of the element
type and v = 2^-24 that of the sums: combine adds k products in 32 bits and
rounds once, |y - y64| <= (k + 1) v sum|w ys| + u |y64| (+ the smallest
subnormal); dys is one product rounded once; dw is a sum of `hidden` products,
whatever the order: |dw - dw64| <= (hidden + 1) v sum|dy ys|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
V = 2.0 ** -24


def _torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def sorted_entries(ids, experts):
    """(expert_ptr, entry, slot) of the definition, entry by entry in numpy."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    entry = np.argsort(key, kind="stable").astype(np.int32)
    ptr = np.searchsorted(key[entry], np.arange(experts + 1)).astype(np.int32)
    pos = np.empty(flat.size, np.int32)
    pos[entry] = np.arange(flat.size, dtype=np.int32)
    return ptr, entry, np.where(key < experts, pos, -1 - pos).reshape(ids.shape)


def random_ids(rng, t, k, experts, drop, skew=False):
    ids = rng.integers(0, experts, (t, k))
    if skew:  # most entries on one expert
        ids = np.where(rng.random((t, k)) < 0.8, experts // 3, ids)
    wild = rng.choice([-1, -7, experts, experts + 5, -2 ** 31, 2 ** 31 - 1], (t, k))
    return np.where(rng.random((t, k)) < drop, wild, ids)


def build(ids, experts, wide, max_tokens=None, stride=None):
    import torch
    import load_balanced_csr_gb300 as lb
    t, k = ids.shape
    dev = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    if stride:
        held = torch.full((t, stride), experts - 1, dtype=dev.dtype, device="cuda")
        held[:, :k] = dev
        dev = held[:, :k]
    return lb.ExpertRoute(max_tokens or t, k, experts).build(dev)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("t,k,experts,drop", [
    (0, 4, 8, 0.0), (1, 1, 1, 0.0), (1, 8, 128, 0.0), (3, 2, 2048, 0.2), (33, 7, 5, 0.3), (512, 8, 128, 0.0),
    (513, 8, 127, 1.0), (2048, 2, 16, 0.1), (2049, 2, 16, 0.1), (4097, 3, 300, 0.05), (20000, 8, 256, 0.0),
    (100003, 8, 61, 0.01), (5000, 5, 2048, 0.5),
    (16384, 8, 33, 0.0), (16385, 8, 33, 0.0), (200003, 8, 61, 0.01)])  # a cluster's last size, two launches, several rounds
def test_sorted_by_expert(t, k, experts, drop, wide):
    rng = np.random.default_rng(t + experts)
    ids = random_ids(rng, t, k, experts, drop, skew=t % 2 == 1)
    ptr, entry, slot = sorted_entries(ids, experts)
    r = build(ids, experts, wide)
    np.testing.assert_array_equal(r.expert_ptr.cpu().numpy(), ptr)
    np.testing.assert_array_equal(r.entry.cpu().numpy(), entry)
    np.testing.assert_array_equal(r.slot.cpu().numpy(), slot)


def test_ids_of_64_bits_do_not_wrap():
    """An id of 2^32 is outside [0, experts), not expert 0."""
    ids = np.array([[0, 2 ** 32], [-2 ** 32, 1], [2 ** 62, 1]], np.int64)
    ptr, entry, slot = sorted_entries(ids, 2)
    r = build(ids, 2, True)
    np.testing.assert_array_equal(r.expert_ptr.cpu().numpy(), ptr)
    np.testing.assert_array_equal(r.slot.cpu().numpy(), slot)


def test_strided_ids_fewer_tokens_and_rebuilds():
    rng = np.random.default_rng(5)
    import torch
    import load_balanced_csr_gb300 as lb
    route = lb.ExpertRoute(5000, 3, 40)
    for t in (5000, 17, 0, 4999):
        ids = random_ids(rng, t, 3, 40, 0.1)
        held = torch.zeros(t, 11, dtype=torch.int64, device="cuda")
        held[:, 4:7] = torch.from_numpy(ids).cuda()
        route.build(held[:, 4:7])
        ptr, entry, slot = sorted_entries(ids, 40)
        np.testing.assert_array_equal(route.expert_ptr.cpu().numpy(), ptr)
        np.testing.assert_array_equal(route.entry.cpu().numpy(), entry)
        np.testing.assert_array_equal(route.slot.cpu().numpy(), slot)


def _matrix(rng, rows, cols, dtype, pad=0, offset=0):
    """A (rows, cols) CUDA matrix, its rows `pad` elements apart and `offset` elements into its memory."""
    import torch
    data = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(_torch_dtype(dtype)).cuda()
    held = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=data.dtype, device="cuda")
    view = held[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(data)
    return view


def _f64(t):
    return t.double().cpu().numpy()


def _within(got, want, bound, label):
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{label}: {err.max()} off, {(err - bound).max()} over the bound"


ROWS = [
    # tokens, k, experts, hidden, drop, pad, offset
    (1, 1, 4, 1, 0.0, 0, 0), (1, 8, 8, 2048, 0.0, 0, 0), (37, 3, 5, 8, 0.0, 0, 0), (64, 8, 128, 2048, 0.0, 0, 0),
    (50, 2, 7, 1001, 0.2, 0, 0), (50, 5, 7, 512, 0.2, 8, 0), (50, 4, 7, 512, 0.2, 1, 0), (33, 4, 9, 264, 0.5, 0, 1),
    (9, 13, 20, 4104, 0.3, 0, 0), (20, 2, 3, 40, 1.0, 0, 0), (700, 6, 60, 96, 0.1, 0, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t,k,experts,hidden,drop,pad,offset", ROWS)
def test_rows_forward_and_backward(t, k, experts, hidden, drop, pad, offset, dtype):
    import torch
    rng = np.random.default_rng(t * hidden + k)
    ids = random_ids(rng, t, k, experts, drop)
    _, entry, slot = sorted_entries(ids, experts)
    r = build(ids, experts, True)
    x = _matrix(rng, t, hidden, dtype, pad, offset)
    dy = _matrix(rng, t, hidden, dtype, pad, offset)
    ys = _matrix(rng, t * k, hidden, dtype, pad, offset)
    w = torch.from_numpy(rng.random((t, k + 2)).astype(np.float32)).cuda()[:, 1:k + 1]
    kept = slot >= 0
    # what dropped entries hold must not matter
    pos = np.where(kept, slot, -1 - slot)
    if (~kept).any():
        ys[torch.from_numpy(pos[~kept]).long().cuda()] = float("nan")
        w[torch.from_numpy(~kept).cuda()] = float("inf")
    w64 = np.where(kept, _f64(w), 0.0)
    ys64 = np.where(kept[:, :, None], _f64(ys)[pos], 0.0)
    dy64 = _f64(dy)

    out = _matrix(rng, t * k, hidden, dtype, pad, offset)
    xs = r.dispatch(x, out=out)
    want = np.where(kept.reshape(-1)[entry][:, None], _f64(x)[entry // k], 0.0)
    np.testing.assert_array_equal(_f64(xs), want)

    u, tiny = U[dtype], TINY[dtype]
    for weights, wt in ((w, w64), (None, kept.astype(np.float64))):
        y64 = (wt[:, :, None] * ys64).sum(1)
        mag = (np.abs(wt)[:, :, None] * np.abs(ys64)).sum(1)
        bound = (k + 1) * V * mag + u * np.abs(y64) + tiny
        _within(_f64(r.combine(ys, weights)), y64, bound, "combine")

    dys, dw = r.combine_backward(dy, ys, w)
    want = np.zeros((t * k, hidden))
    want[pos[kept]] = (w64[:, :, None] * dy64[:, None, :])[kept]
    _within(_f64(dys), want, (u + V) * np.abs(want) + tiny, "dys")
    np.testing.assert_array_equal(_f64(dys)[pos[~kept]], 0.0)
    dw64 = (dy64[:, None, :] * ys64).sum(2)
    mag = (np.abs(dy64)[:, None, :] * np.abs(ys64)).sum(2)
    _within(_f64(dw), dw64, (hidden + 1) * V * mag, "dw")
    assert (_f64(dw)[~kept] == 0).all()

    # the gradient may take the place of ys
    again, dw2 = r.combine_backward(dy, ys, w, out=ys)
    assert again.data_ptr() == ys.data_ptr()
    assert torch.equal(again, dys) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """combine is linear in ys and in the weights, dispatch in x: the central
    difference over a step of any size is the derivative, up to the roundings of
    the two 32-bit evaluations (bounded as in the module's docstring)."""
    import torch
    rng = np.random.default_rng(3)
    t, k, experts, hidden = 40, 3, 6, 130
    r = build(random_ids(rng, t, k, experts, 0.2), experts, False)
    m = lambda rows, cols: _matrix(rng, rows, cols, "f32")
    ys, dy, x, dxs, d = m(t * k, hidden), m(t, hidden), m(t, hidden), m(t * k, hidden), m(t * k, hidden)
    w, dwt, dx_ = m(t, k), m(t, k), m(t, hidden)
    dys, dw = r.combine_backward(dy, ys, w)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    size = lambda a, b: float((a.double().abs() * b.double().abs()).sum())

    def check(f, at, along, cot, grad):
        plus, minus = f(at + along), f(at - along)
        diff = (dot(cot, plus) - dot(cot, minus)) / 2
        # each value of f carries (k + 2) roundings, the argument's own sum one more; grad hidden + 1
        bound = (k + 3) * V * (size(cot, f(at.abs() + along.abs())) * 4 + size(cot, plus) + size(cot, minus))
        bound += (hidden + 2) * V * size(grad.abs(), along) * hidden
        assert abs(diff - dot(grad, along)) <= bound, (diff, dot(grad, along), bound)

    wa = w.abs()
    check(lambda v: r.combine(v, wa), ys, d, dy, r.combine_backward(dy, ys, wa)[0])
    check(lambda v: r.combine(ys.abs(), v), w, dwt, dy, r.combine_backward(dy, ys.abs(), w)[1])
    check(lambda v: r.dispatch(v), x, dx_, dxs, r.dispatch_backward(dxs))
    assert dys.shape == ys.shape and dw.shape == w.shape


def test_through_autograd():
    """A layer's training step: dispatch and combine as autograd functions
    around a product per expert, against the same layer written token by token
    in 64 bits."""
    import torch
    import load_balanced_csr_gb300 as lb
    t, k, experts, hidden = 50, 2, 4, 24

    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, route):
            ctx.route = route
            return route.dispatch(x)

        @staticmethod
        def backward(ctx, dxs):
            return ctx.route.dispatch_backward(dxs.contiguous()), None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ys, w, route):
            ctx.route = route
            ctx.save_for_backward(ys, w)
            return route.combine(ys, w)

        @staticmethod
        def backward(ctx, dy):
            return *ctx.route.combine_backward(dy.contiguous(), *ctx.saved_tensors), None

    torch.manual_seed(3)
    ids = torch.randint(-1, experts, (t, k), device="cuda")
    x, w, m = torch.randn(t, hidden), torch.rand(t, k), torch.randn(experts, hidden, hidden) / hidden ** 0.5
    got = [v.cuda().requires_grad_() for v in (x, w, m)]
    route = lb.ExpertRoute(t, k, experts).build(ids)
    rows = Dispatch.apply(got[0], route)
    begin = route.expert_ptr.tolist()
    parts = [rows[begin[e]:begin[e + 1]] @ got[2][e] for e in range(experts)] + [rows[begin[-1]:]]
    y = Combine.apply(torch.cat(parts), got[1], route)
    want = [v.double().cuda().requires_grad_() for v in (x, w, m)]
    kept = (ids >= 0).double()
    each = torch.einsum("th,tkhf->tkf", want[0], want[2][ids.clamp(min=0)])
    y64 = (each * (want[1] * kept)[:, :, None]).sum(1)
    (y.square().sum() / 2).backward()
    (y64.square().sum() / 2).backward()
    # sums of at most a few hundred products of values of a few units, in 32 bits
    for a, b in ((y, y64), *((g.grad, h.grad) for g, h in zip(got, want))):
        a, b = a.detach().double(), b.detach()
        assert float((a - b).abs().max()) <= 512 * V * float(b.abs().max())


def test_dispatch_keeps_bits_and_another_stream():
    """NaN payloads and signed zeros pass through; a call on its own stream
    uses that stream's memory."""
    import torch
    import load_balanced_csr_gb300 as lb
    t, k, h = 300, 4, 72
    bits = torch.randint(-2 ** 15, 2 ** 15, (t, h), dtype=torch.int16, device="cuda")
    x = bits.view(torch.bfloat16)
    ids = torch.randint(0, 9, (t, k), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = lb.ExpertRoute(t, k, 9)
    r.build(ids, stream=s)
    xs = r.dispatch(x, stream=s.cuda_stream)
    s.synchronize()
    want = bits[(r.entry // k).long()]
    assert torch.equal(xs.view(torch.int16), want)


def test_rows_past_32_bit_offsets():
    """(tokens * top_k) x hidden past 2^31 elements."""
    import torch
    import load_balanced_csr_gb300 as lb
    t, k, h = 70000, 2, 16384
    ids = torch.randint(0, 4, (t, k), device="cuda", dtype=torch.int32)
    r = lb.ExpertRoute(t, k, 4).build(ids)
    x = torch.randn(t, h, device="cuda", dtype=torch.bfloat16)
    xs = r.dispatch(x)
    at = torch.tensor([0, 1, t * k // 2, t * k - 2, t * k - 1], device="cuda")
    assert torch.equal(xs[at], x[(r.entry[at] // k).long()])
    y = r.combine(xs, torch.full((t, k), 0.5, device="cuda"))
    assert torch.equal(y, x)  # 0.5 x + 0.5 x is exact
    dys, dw = r.combine_backward(y, xs, torch.full((t, k), 0.5, device="cuda"))
    assert torch.equal(dys[at], (0.5 * x[(r.entry[at] // k).long()].float()).bfloat16())
    assert bool((dw > 0).all())


def test_refusals():
    import torch
    import load_balanced_csr_gb300 as lb
    with pytest.raises(lb.SpmvError):
        lb.ExpertRoute(4, 2, 2049)
    with pytest.raises(lb.SpmvError):
        lb.ExpertRoute(4, 2, 0)
    with pytest.raises(lb.SpmvError):
        lb.ExpertRoute(2 ** 30, 2, 4)
    r = lb.ExpertRoute(4, 2, 3)
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(RuntimeError):
        r.dispatch(x)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        r.build(ids.float())
    with pytest.raises(TypeError):
        r.build(ids.cpu())
    with pytest.raises(ValueError):
        r.build(torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        r.build(torch.zeros(4, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        r.build(torch.zeros(2, 4, dtype=torch.int32, device="cuda").t())
    r.build(ids)
    with pytest.raises(TypeError):
        r.dispatch(x.double())
    with pytest.raises(TypeError):
        r.dispatch(x.cpu())
    with pytest.raises(ValueError):
        r.dispatch(x[:3])
    with pytest.raises(ValueError):
        r.dispatch(torch.zeros(8, 4, device="cuda").t())
    ys = torch.zeros(8, 8, device="cuda")
    with pytest.raises(TypeError):
        r.combine(ys, torch.zeros(4, 2, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        r.combine(ys, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(TypeError):
        r.combine(ys, out=torch.zeros(4, 8, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        r.combine_backward(x, ys.half())


@pytest.mark.parametrize("made_for,built", [(160000, 150000), (320000, 311296)])
def test_fewer_tokens_than_the_route_was_made_for(made_for, built):
    """The workspace of more tokens serves fewer, also where these are cut into more tiles."""
    rng = np.random.default_rng(built)
    ids = random_ids(rng, built, 8, 24, 0.01)
    ptr, entry, slot = sorted_entries(ids, 24)
    r = build(ids, 24, False, max_tokens=made_for)
    np.testing.assert_array_equal(r.expert_ptr.cpu().numpy(), ptr)
    np.testing.assert_array_equal(r.entry.cpu().numpy(), entry)
    np.testing.assert_array_equal(r.slot.cpu().numpy(), slot)
