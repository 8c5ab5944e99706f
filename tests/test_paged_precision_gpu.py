"""Attention of one token with 16-bit elements: what the weights' second half
is for, and infinities in V.

With v = 2^-24 and u the half-unit of the element type (2^-8, 2^-11): a weight
goes into the product as two elements, so it is off by at most u^2 of itself
(f16 also by half of 2^-39 of the row's largest), beside the factor 1 + e of
its score, e = 2 (head_dim + 8) v scale max|q||k| + 2^-20 (1 + max|s - lse|),
and n v of the sums over n positions.  Hence |out - out64| <= (2 e + 2 n v +
u^2) sum p|v| + n 2^-40 max|v| + u |out64| + the smallest subnormal."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
V = 2.0 ** -24


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _inputs(batch, n, q_heads, kv_heads, dim, dtype, page=16, seed=0, spread=0.5):
    """Requests of n positions each over one cache whose pages lie in order, last page first."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-n // page)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(_dtype(dtype))
    table = torch.arange(batch * per - 1, -1, -1, dtype=torch.int32, device="cuda").view(batch, per)
    k, v = (normal(batch * per, page, kv_heads, dim) for _ in range(2))
    return (spread * normal(batch, q_heads, dim)).to(_dtype(dtype)), k, v, table, torch.full((batch,), n, dtype=torch.int32, device="cuda")


def _definition(q, k, v, table, n, scale):
    """(scores, weights, values) in 64 bits: (batch, kv head, group, n) twice, (batch, kv head, n, dim)."""
    import torch
    b, hq, d = q.shape
    hk = k.shape[2]
    kk, vv = (c[table.long()].reshape(b, -1, hk, d)[:, :n].double().transpose(1, 2) for c in (k, v))
    s = torch.einsum("bhgd,bhnd->bhgn", q.double().view(b, hk, hq // hk, d), kk) * scale
    return s, torch.softmax(s, -1), kk, vv


def _bound(q, kk, vv, s, p, want, dtype, scale):
    import torch
    b, hk, n, d = kk.shape
    size = abs(scale) * torch.einsum("bhgd,bhnd->bhgn", q.double().abs().view(b, hk, -1, d), kk.abs()).amax(-1, keepdim=True)
    e = 2 * (d + 8) * V * size + 2.0 ** -20 * (1 + (s - torch.logsumexp(s, -1, keepdim=True)).abs().amax(-1, keepdim=True))
    u = U[dtype]
    return (2 * e + 2 * n * V + u * u) * (p @ vv.abs()) + n * 2.0 ** -40 * float(vv.abs().max()) + u * want.abs() + TINY[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_heads", [4, 32])
def test_weights_carry_two_elements(q_heads, dtype):
    """Values of either sign, whose averages are now and then next to zero:
    the output's own rounding is then small and the weights' shows.  Weights
    of one element each would not pass."""
    import torch
    import load_balanced_csr_gb300 as lb
    n, hk, d, scale = 16, 2, 16, 0.25
    q, k, v, table, lens = _inputs(64, n, q_heads, hk, d, dtype, seed=q_heads)
    v = torch.where(v >= 0, 1.0, -1.0).to(v.dtype)
    attend = lb.PagedAttention(64, q_heads, hk, d, _dtype(dtype))
    out, _ = attend(q, k, v, table, lens, scale=scale)
    s, p, kk, vv = _definition(q, k, v, table, n, scale)
    want = p @ vv
    bound = _bound(q, kk, vv, s, p, want, dtype, scale)
    err = (out.double().view(want.shape) - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    w = torch.exp(s - s.amax(-1, keepdim=True))
    one = (w.to(_dtype(dtype)).double() @ vv) / w.sum(-1, keepdim=True)
    assert bool(((one - want).abs() > bound).any()), "the bound does not see a weight's second half"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("q_heads,dim", [(4, 64), (14, 72), (32, 128), (24, 256)])
@pytest.mark.parametrize("n", [40, 20000], ids=["short", "cut"])
def test_infinities_in_values(n, q_heads, dim, dtype):
    """An infinite value whose weight is not lost makes its element infinite,
    two of either sign make it NaN, and the other elements stay as they are."""
    import torch
    import load_balanced_csr_gb300 as lb
    hk, batch, scale = 2, 3, dim ** -0.5
    q, k, v, table, lens = _inputs(batch, n, q_heads, hk, dim, dtype, seed=dim)
    at = lambda b, t: (int(table[b, t // 16]), t % 16)
    inf = float("inf")
    for t in (0, 1, 7, n // 2, n - 1):  # several, so that some weight's second half is negative, some zero
        v[at(0, t)][:, 3] = inf
        v[at(0, t)][:, 5] = -inf
    v[at(1, 2)][0, 0], v[at(1, n - 2)][0, 0] = inf, -inf
    v[at(2, n - 3)][1, dim - 1] = inf
    attend = lb.PagedAttention(batch, q_heads, hk, dim, _dtype(dtype))
    out, lse = attend(q, k, v, table, lens, scale=scale)
    assert attend.device_status() == 0 and bool(torch.isfinite(lse).all())
    s, p, kk, vv = _definition(q, k, v, table, n, scale)
    want, got = p @ vv, out.double().view(batch, hk, -1, dim)
    assert bool(torch.isinf(want[0, :, :, 3]).all()) and bool(torch.isnan(want[1, 0, :, 0]).all())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    infinite = torch.isinf(want)
    assert torch.equal(got[infinite], want[infinite])
    finite = torch.isfinite(want)
    bound = _bound(q, kk, torch.where(torch.isfinite(vv), vv, 0), s, p, torch.where(finite, want, 0), dtype, scale)
    assert bool(((got - want).abs()[finite] <= bound[finite]).all())
    assert math.isfinite(float(bound.max()))
