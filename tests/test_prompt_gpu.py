"""Attention of packed prompts against its definition in 64 bits.

The bound.  With v = 2^-24 and u the half-unit of the element type (2^-8,
2^-11): a score carries a dot product of head_dim terms, its scaling and the
exponential's own error (a few units of its argument), so each weight is off by
a factor of at most 1 + e, e = 2 (head_dim + 8) v scale max|q||k| + 2^-20 (1 +
max|s - lse|); sums over n keys add n v, and a weight is rounded to the element
type once (u; an f16 weight below its normal range by 2^-36 of the row's
largest, which is at most 1).  Hence
|out - out64| <= (2 e + 2 n v + u) sum p|v| + [f16] n 2^-36 max|v| + u |out64| + smallest subnormal,
|lse - lse64| <= e + n v + 4 v |lse64|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}
LOST = {"bf16": 0.0, "f16": 2.0 ** -36}
V = 2.0 ** -24


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


class Prompts:
    """Packed prompts, NaN and infinities in every row that belongs to no request."""

    def __init__(self, nq, nk, q_heads, kv_heads, dim, dtype, layout="dense", seed=0, before=0, behind=3, size=1.0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.nq, self.nk, self.dtype, self.shape = list(nq), list(nk or nq), dtype, (q_heads, kv_heads, dim)
        self.before = before
        q_ptr = before + np.concatenate([[0], np.cumsum(self.nq)])
        kv_ptr = before + np.concatenate([[0], np.cumsum(self.nk)])
        tokens, keys = int(q_ptr[-1]) + behind, int(kv_ptr[-1]) + behind
        dt = _dtype(dtype)
        if layout == "fused" and nk is None:
            self.q, self.k, self.v = torch.randn(tokens, q_heads + 2 * kv_heads, dim, generator=g, device="cuda").to(dt).split(
                [q_heads, kv_heads, kv_heads], 1)
        elif layout == "heads":
            self.q, self.k, self.v = (torch.randn(h, n, dim, generator=g, device="cuda").to(dt).transpose(0, 1)
                                      for h, n in ((q_heads, tokens), (kv_heads, keys), (kv_heads, keys)))
        elif layout == "padded":
            self.q, self.k, self.v = (torch.randn(n, h + 1, dim + 24, generator=g, device="cuda").to(dt)[:, 1:, 8:dim + 8]
                                      for h, n in ((q_heads, tokens), (kv_heads, keys), (kv_heads, keys)))
        else:
            self.q, self.k, self.v = (torch.randn(n, h, dim, generator=g, device="cuda").to(dt)
                                      for h, n in ((q_heads, tokens), (kv_heads, keys), (kv_heads, keys)))
        self.q *= size
        for x, ptr in ((self.q, q_ptr), (self.k, kv_ptr), (self.v, kv_ptr)):
            x[:before], x[int(ptr[-1]):] = float("nan"), float("inf")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.q_ptr, self.kv_ptr = torch.tensor(q_ptr, **i32), None if nk is None else torch.tensor(kv_ptr, **i32)

    def attention(self):
        import load_balanced_csr_gb300 as lb
        return lb.PromptAttention(len(self.nq), *self.shape, _dtype(self.dtype))

    def run(self, **kw):
        attend = self.attention()
        out, lse = attend(self.q, self.k, self.v, self.q_ptr, self.kv_ptr, **kw)
        assert attend.device_status() == 0
        return out, lse

    def check(self, out, lse, causal=True, scale=None):
        """Every request against the definition, a head at a time."""
        import torch
        hq, hk, dim = self.shape
        scale = dim ** -0.5 if scale is None else scale
        u, at_q, at_k = U[self.dtype], self.before, self.before
        for r, (nq, nk) in enumerate(zip(self.nq, self.nk)):
            rows, keys = slice(at_q, at_q + nq), slice(at_k, at_k + nk)
            at_q, at_k = at_q + nq, at_k + nk
            if nq == 0:
                continue
            i, j = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
            seen = (j[None, :] <= i[:, None] + nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool, device="cuda")
            for h in range(hq):
                o, got_lse = out[rows, h], lse[rows, h]
                none = ~seen.any(1)
                assert bool((o[none] == 0).all()) and bool((got_lse[none] == -np.inf).all()), f"request {r}: rows without keys"
                if bool(none.all()):
                    continue
                k, v = (x[keys, h // (hq // hk)].double() for x in (self.k, self.v))
                q = self.q[rows, h].double()
                s = (q @ k.T * scale).masked_fill(~seen, -np.inf)
                want_lse = torch.logsumexp(s, 1)
                p = torch.exp(s - want_lse[:, None]).nan_to_num()
                want, spread = p @ v, p @ v.abs()
                size = float((q.abs().amax(0) @ k.abs().amax(0))) * abs(scale)
                gap = (s - want_lse[:, None]).masked_fill(~seen, 0).abs().amax(1)
                e = 2 * (dim + 8) * V * size + 2.0 ** -20 * (1 + gap)
                bound = (2 * e + 2 * nk * V + u)[:, None] * spread + LOST[self.dtype] * nk * float(v.abs().max()) + u * want.abs() + TINY[self.dtype]
                off = (o.double() - want).abs()
                ok = (off <= bound)[~none]
                assert bool(ok.all()), f"request {r} of {nq} over {nk}, head {h}: {float((off / bound)[~none].max())} of the bound"
                off = (got_lse.double() - want_lse).abs()
                assert bool((off <= e + nk * V + 4 * V * want_lse.abs())[~none].all()), f"request {r}, head {h}: lse off by {float(off[~none].max())}"


LENS = [1, 0, 127, 128, 129, 2, 300, 0, 16, 17, 15, 513]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_heads,kv_heads,dim,layout", [
    (8, 1, 128, "fused"), (4, 4, 64, "dense"), (6, 2, 80, "padded"), (7, 1, 72, "heads"), (16, 1, 256, "dense"), (2, 2, 8, "dense"),
    (20, 1, 96, "fused"), (3, 3, 192, "heads"), (5, 1, 136, "padded"), (71, 1, 64, "dense"), (128, 1, 40, "dense"), (2, 1, 248, "fused"),
    (4, 2, 16, "heads"), (16, 8, 128, "padded")])
def test_prompts(q_heads, kv_heads, dim, layout, dtype):
    p = Prompts(LENS, None, q_heads, kv_heads, dim, dtype, layout, seed=dim)
    p.check(*p.run())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 1, 128), (4, 4, 64), (7, 1, 72), (4, 1, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(q_heads, kv_heads, dim, causal, dtype):
    """Chunks behind a past, fewer keys than queries (rows that see none), no keys at all, single queries over many keys."""
    nq, nk = [1, 64, 130, 5, 40, 0, 300, 1, 200], [1000, 64, 777, 0, 20, 9, 1300, 1, 129]
    p = Prompts(nq, nk, q_heads, kv_heads, dim, dtype, seed=dim, before=5)
    p.check(*p.run(causal=causal), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_long_prompt(dtype, causal):
    p = Prompts([5000], None, 8, 1, 128, dtype, seed=1)
    p.check(*p.run(causal=causal), causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,q_heads,kv_heads", [(128, 8, 2), (64, 1, 1), (256, 4, 1), (80, 7, 1)])
def test_few_queries_over_a_long_past(dim, q_heads, kv_heads, dtype):
    """Their keys are cut into shares: more shares than some have keys for, rows that see none, rows of no request."""
    p = Prompts([1, 3, 0, 40, 5], [70001, 33000, 7, 900, 0], q_heads, kv_heads, dim, dtype, seed=2, before=3)
    attend = p.attention()
    given, lse = p.q.new_full(p.q.shape, 3.0), p.q.new_full(p.q.shape[:2], 3.0).float()
    attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr, out=given, lse=lse)
    assert attend.device_status() == 0
    p.check(given, lse)
    assert bool((given[:3] == 3).all()) and bool((given[52:] == 3).all()) and bool((lse[:3] == 3).all()) and bool((lse[52:] == 3).all())
    again, _ = attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr, causal=False)
    whole, _ = attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr, causal=False)
    assert again[3:52].equal(whole[3:52])
    out, lse = p.run(causal=False)
    p.check(out, lse, causal=False)


def test_infinities_in_shares():
    """Values and scores that are not finite in one share of the keys alone."""
    import torch
    p = Prompts([2], [9000], 2, 1, 64, "bf16", seed=3)
    clean, _ = p.run()
    p.v[4000, 0, 3], p.v[8999, 0, 5], p.v[8998, 0, 6] = float("inf"), float("-inf"), float("nan")
    out, _ = p.run()
    want = clean.clone()
    want[:2, :, 3], want[1, :, 5], want[:2, :, 6] = float("inf"), float("-inf"), float("nan")
    assert torch.equal(out[:2].nan_to_num(7, 8, 9), want[:2].nan_to_num(7, 8, 9))
    p.k[:9000, 0, 0] = float("-inf")
    p.q[:, :, 0] = 1
    out, lse = p.run()
    assert bool((lse[:2] == -np.inf).all()) and bool((out[:2, :, 8:] == 0).all())
    p.k[5000, 0, 0] = 0
    out, lse = p.run()
    assert torch.equal(out[:2, :, 8:], p.v[5000, 0, 8:].expand(2, 2, -1)) and bool(torch.isfinite(lse[:2]).all())
    p.k[6000, 0, 0] = float("inf")
    out, lse = p.run()
    assert bool(torch.isnan(out[:2]).all()) and bool(torch.isnan(lse[:2]).all())


def test_many_short_prompts():
    rng = np.random.default_rng(0)
    p = Prompts(rng.integers(0, 12, 3000).tolist(), None, 2, 1, 64, "bf16", seed=3)
    p.check(*p.run())


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales(scale, dtype):
    """Scores from all alike to far apart: the maximum keeps rising along the keys."""
    import torch
    p = Prompts([400, 30], None, 4, 2, 64, dtype, seed=4)
    p.check(*p.run(scale=scale), scale=scale)
    p.k *= (torch.arange(p.k.shape[0], device="cuda") / 60).to(p.k.dtype)[:, None, None]
    p.check(*p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_past_2_24(dtype):
    """The highest score's weight is 1 however large the scores."""
    import torch
    p = Prompts([200], None, 2, 1, 64, dtype, seed=5)
    big = 2.0 ** 60 if dtype == "bf16" else 2.0 ** 14
    p.q.zero_(), p.k.zero_()
    p.q[:200, :, 0] = big
    order = torch.randperm(200, generator=torch.Generator().manual_seed(0)).cuda()
    p.k[:200, 0, 0] = (order.float() + 1).to(p.k.dtype)
    out, lse = p.run(scale=2.0)
    best = torch.stack([order[:i + 1].argmax() for i in range(200)])
    assert torch.equal(out[:200, 0], p.v[best, 0]) and torch.equal(out[:200, 1], p.v[best, 0])


def test_a_falling_and_a_rising_maximum():
    """One key far above all others, first, last or in between: what lies behind it keeps its sum."""
    import torch
    for dtype in ("bf16", "f16"):
        for at in (0, 200, 399):
            p = Prompts([1], [400], 1, 1, 64, dtype, seed=6)
            p.q[0] = 1
            p.k[:400] = 0
            p.k[at] = 0.25
            p.check(*p.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,dim", [(1, 64), (8, 128), (4, 256)])
def test_nothing_masked_is_seen(dtype, group, dim):
    """NaN and infinities in the keys and values of later positions change no earlier row."""
    import torch
    nq, nk = [300, 200, 1], [300, 450, 129]
    p = Prompts(nq, nk, group, 1, dim, dtype, seed=7)
    clean, clean_lse = p.run()
    starts_q, starts_k = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    for bad in (float("nan"), float("inf"), float("-inf")):
        for back in (1, 50, 140):
            k, v = p.k.clone(), p.v.clone()
            for r in range(2):
                first = int(starts_k[r + 1]) - back
                k[first:int(starts_k[r + 1])] = bad
                v[first:int(starts_k[r + 1])] = bad
            attend = p.attention()
            out, lse = attend(p.q, k, v, p.q_ptr, p.kv_ptr)
            for r in range(3):
                rows = slice(int(starts_q[r]), int(starts_q[r + 1]) - (back if r < 2 else 0))
                assert torch.equal(out[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows]), (bad, back, r)
                if r < 2:  # and every later row does see them
                    assert not bool(torch.isfinite(out[rows.stop:int(starts_q[r + 1])]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_in_values(dtype):
    """An infinity is its element's alone and reaches the rows that see it; two of both signs are NaN."""
    import torch
    p = Prompts([300], None, 2, 1, 64, dtype, seed=8)
    clean, _ = p.run()
    p.v[100, 0, 3] = float("inf")
    p.v[200, 0, 5] = float("-inf")
    p.v[130, 0, 9] = float("inf")
    p.v[131, 0, 9] = float("-inf")
    p.v[290, 0, 11] = float("nan")
    out, _ = p.run()
    want = clean.clone()
    want[100:300, :, 3] = float("inf")
    want[200:300, :, 5] = float("-inf")
    want[130, :, 9] = float("inf")
    want[131:300, :, 9] = float("nan")
    want[290:300, :, 11] = float("nan")
    assert torch.equal(out[:300].nan_to_num(7, 8, 9), want[:300].nan_to_num(7, 8, 9))


def test_infinite_scores():
    """A score of minus infinity weighs nothing, one of plus infinity or NaN makes its row NaN, rows before are whole."""
    import torch
    p = Prompts([100], None, 1, 1, 64, "bf16", seed=9)
    p.q[:, :, 0] = 1
    q = p.k.clone()
    p.k[50, 0, 0] = float("-inf")
    out, lse = p.run()
    assert bool(torch.isfinite(out[:100]).all()) and bool(torch.isfinite(lse[:100]).all())
    p.k = q.clone()
    p.k[:60, 0, 0] = float("-inf")
    out, lse = p.run()
    assert bool((out[:60] == 0).all()) and bool((lse[:60] == -np.inf).all()) and bool(torch.isfinite(out[60:100]).all())
    p.k = q.clone()
    p.k[50, 0, 0] = float("inf")
    out, lse = p.run()
    assert bool(torch.isfinite(out[:50]).all()) and bool(torch.isnan(out[50:100]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_outputs_given(dtype):
    """Strided outputs, their other elements untouched; rows of no request stay."""
    import torch
    p = Prompts([40, 0, 130], None, 6, 2, 72, dtype, seed=10, before=4, behind=9)
    want, want_lse = p.run()
    n = p.q.shape[0]
    held = torch.full((n, 8, 80), 3.0, dtype=_dtype(dtype), device="cuda")
    out, lse = held[:, 1:7, :72], torch.full((n, 6), 3.0, device="cuda")
    got = p.attention()(p.q, p.k, p.v, p.q_ptr, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    rows = slice(4, 174)
    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])
    for t in (held[:4], held[174:], lse[:4], lse[174:], held[:, 0], held[:, 7], held[:, :, 72:]):
        assert bool((t == 3).all())


def test_dimensions_of_one():
    """Strides of dimensions with one element are of no matter."""
    import torch
    import load_balanced_csr_gb300 as lb
    ptr = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 64, device="cuda").half()
    q, k, v = (x[i].as_strided((1, 1, 64), (3, 5, 1)) for i in range(3))
    out, lse = lb.PromptAttention(1, 1, 1, 64, torch.float16)(q, k, v, ptr)
    assert torch.equal(out, v) and abs(float(lse) - float(q.double().flatten() @ k.double().flatten()) / 8) < 1e-4
    many = torch.randn(40, 1, 64, device="cuda").half()
    odd = many.as_strided((40, 1, 64), (64, 3, 1))
    ptr = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    attend = lb.PromptAttention(1, 1, 1, 64, torch.float16)
    assert torch.equal(attend(many, many, many, ptr)[0], attend(odd, odd, odd, ptr)[0])


def test_bad_pointers():
    """Queries or keys that are not rows of the tensors: the request is left out and flagged."""
    import torch
    import load_balanced_csr_gb300 as lb
    p = Prompts([30, 30, 30], [40, 40, 40], 2, 1, 64, "bf16", seed=11, behind=0)
    want, _ = p.run()
    i32 = dict(dtype=torch.int32, device="cuda")
    for q_ptr, kv_ptr, flag, left in (([0, 30, 60, 91], [0, 40, 80, 120], 1, [2]), ([0, 30, 60, 90], [0, 40, 80, 121], 2, [2]),
                                      ([0, 30, 60, 90], [-1, 40, 80, 120], 2, [0]), ([-5, 30, 60, 90], [0, 40, 80, 120], 1, [0]),
                                      ([0, 30, 60, 90], [0, 40, 39, 120], 2, [1, 2])):
        attend = p.attention()
        out = torch.full_like(p.q, 3.0)
        attend(p.q, p.k, p.v, torch.tensor(q_ptr, **i32), torch.tensor(kv_ptr, **i32), out=out)
        assert attend.device_status() == flag
        for r in range(3):
            rows = slice(30 * r, 30 * r + 30)
            if r not in left:
                assert torch.equal(out[rows], want[rows]), (q_ptr, kv_ptr, r)
            elif kv_ptr[2] != 39 or r == 1:
                assert bool((out[rows] == 3).all()), (q_ptr, kv_ptr, r)
    # pointers that fall: no fault, a flag
    attend = p.attention()
    attend(p.q, p.k, p.v, torch.tensor([0, 60, 30, 90], **i32), torch.tensor([0, 40, 80, 120], **i32))
    assert attend.device_status() & 1
    assert lb.PromptAttention(1, 2, 1, 64, torch.bfloat16).device_status() == 0


def test_repeated_calls_and_streams():
    """The same bits from every call, on another stream, and out of a graph."""
    import torch
    p = Prompts([700, 3, 0, 260], [900, 3, 0, 260], 8, 2, 128, "bf16", seed=12)
    attend = p.attention()
    want, want_lse = attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr)
    n = 963
    for _ in range(5):
        out, lse = attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr)
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    out, lse = attend(p.q, p.k, p.v, p.q_ptr, p.kv_ptr, stream=stream)
    stream.synchronize()
    assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])
    # on two streams at once, each with its object
    other, second = torch.cuda.Stream(), p.attention()
    outs = []
    for i in range(20):
        outs.append((attend, second)[i % 2](p.q, p.k, p.v, p.q_ptr, p.kv_ptr, stream=(stream, other)[i % 2]))
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])
    graph = torch.cuda.CUDAGraph()
    q = torch.zeros_like(p.q)
    with torch.cuda.graph(graph):
        out, lse = attend(q, p.k, p.v, p.q_ptr, p.kv_ptr)
    q.copy_(p.q)
    for _ in range(2):
        graph.replay()
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])


def test_offsets_past_32_bits():
    import torch
    import load_balanced_csr_gb300 as lb
    rows, dim = 70000, 256
    held = torch.zeros(rows, 130, dim, dtype=torch.bfloat16, device="cuda")  # 2.3e9 elements, one head of each tensor used
    q, k, v = held[:, 0:1], held[:, 64:65], held[:, 129:130]
    q[-300:], k[-300:], v[-300:] = (torch.randn(300, 1, dim, device="cuda").bfloat16() for _ in range(3))
    ptr = torch.tensor([0, 0, rows - 300, rows], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(held)[:, 129:130]
    lb.PromptAttention(3, 1, 1, dim, torch.bfloat16)(q, k, v, ptr, out=out)
    few = [t[-300:].contiguous() for t in (q, k, v)]
    want, _ = lb.PromptAttention(1, 1, 1, dim, torch.bfloat16)(*few, torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    assert torch.equal(out[-300:], want) and bool((out[:-300] == 0).all())


def test_a_step_of_chunks_over_an_8_bit_cache():
    """Chunks appended, stored, read back and attended to: as one pass over the whole prompts with the codes' values."""
    import torch
    import load_balanced_csr_gb300 as lb
    i32 = dict(dtype=torch.int32, device="cuda")
    hq, hk, d, page, pages_n = 8, 2, 128, 16, 100
    lens = [200, 33, 0, 470]
    torch.manual_seed(1)
    cache = [torch.zeros(pages_n, page, hk, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(pages_n, 1, hk, device="cuda") for _ in range(2)]
    tables = lb.PageTable(torch.full((4, 32), -1, **i32), page, pages_n, max_tokens=400)
    free = torch.randperm(pages_n).to(**i32)
    x = [torch.randn(n, hq + 2 * hk, d, device="cuda").bfloat16() for n in lens]
    attend = lb.PromptAttention(4, hq, hk, d, torch.bfloat16)
    past, outs = [0] * 4, [[] for _ in lens]
    while past != lens:
        fresh = [min(n - p, c) for n, p, c in zip(lens, past, (70, 33, 5, 160))]
        step = torch.cat([t[p:p + f] for t, p, f in zip(x, past, fresh)])
        q, k, v = step.split([hq, hk, hk], 1)
        pages = tables.append(torch.tensor(past, **i32), torch.tensor(fresh, **i32), free)
        free = free[int(pages.taken):]
        lb.paged_store_e4m3(k, v, *cache, *scales, pages.slots)
        past = [p + f for p, f in zip(past, fresh)]
        kv_ptr = torch.tensor(np.concatenate([[0], np.cumsum(past)]), **i32)
        ks, vs = lb.paged_load(*cache, pages.table, kv_ptr, sum(past), *scales, dtype=torch.bfloat16)
        out, _ = attend(q, ks, vs, pages.token_ptr, kv_ptr)
        for r, (o, f) in enumerate(zip(out.split(fresh), fresh)):
            outs[r].append(o)
    assert attend.device_status() == 0
    # a chunk's keys are read with the scales of that step; those of the last step differ by a rounding where a scale grew since
    kv_ptr = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **i32)
    ks, vs = lb.paged_load(*cache, tables.table, kv_ptr, sum(lens), *scales, dtype=torch.bfloat16)
    want, _ = attend(torch.cat(x)[:, :hq], ks, vs, kv_ptr)
    got = torch.cat([torch.cat(o) for o in outs])
    assert float((got.float() - want.float()).norm() / want.float().norm()) < 2.0 ** -7
    # and the 8-bit attention of each request's last token gives its last row
    last = kv_ptr[1:].long()[torch.tensor([0, 1, 3])] - 1
    one = lb.PagedAttentionE4M3(4, hq, hk, d, torch.bfloat16)
    q = torch.zeros(4, hq, d, device="cuda").bfloat16()
    q[[0, 1, 3]] = torch.cat(x)[last, :hq]
    out, _ = one(q, *cache, *scales, tables.table, torch.tensor(lens, **i32))
    assert bool((out[2] == 0).all())
    assert float((out[[0, 1, 3]].float() - want[last].float()).norm() / want[last].float().norm()) < 2.0 ** -7


def test_steps_one_behind_the_other():
    """Store, load, prompts and single tokens on one stream without a wait, each step's inputs written over the last one's:
    the same bits as with a wait behind every call."""
    import torch
    import load_balanced_csr_gb300 as lb
    i32 = dict(dtype=torch.int32, device="cuda")
    hq, hk, d, page, n = 16, 4, 128, 16, 600
    lens = [200, 399, 1]
    held = [-(-x // page) for x in lens]
    order = torch.randperm(sum(held)).to(**i32)
    table = torch.zeros(3, max(held), **i32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = order[at:at + h]
        at += h
    ptr = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **i32)
    pos = torch.cat([torch.arange(x) for x in lens]).cuda()
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).cuda()
    slots = (table[req, pos // page] * page + pos % page).to(torch.int32)
    codes = [torch.zeros(sum(held), page, hk, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(sum(held), 2, hk, device="cuda") for _ in range(2)]
    k, v = (torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, lse = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hq, device="cuda")
    prompts, one = lb.PromptAttention(3, hq, hk, d, torch.bfloat16), lb.PagedAttentionE4M3(3, hq, hk, d, torch.bfloat16)
    inputs = [torch.randn(n, hq + 2 * hk, d, device="cuda").bfloat16() * (1 + i) for i in range(12)]
    dev_lens, last = torch.tensor(lens, **i32), ptr[1:].long() - 1

    def run(wait):
        kept = []
        for x in inputs:
            q, kx, vx = x.split([hq, hk, hk], 1)
            for step in (lambda: lb.paged_store_e4m3(kx, vx, *codes, *scales, slots),
                         lambda: lb.paged_load(*codes, table, ptr, n, *scales, dtype=torch.bfloat16, k=k, v=v),
                         lambda: prompts(q, k, v, ptr, out=out, lse=lse),
                         lambda: kept.append(one(q[last], *codes, *scales, table, dev_lens)[0]),
                         lambda: kept.append(out.clone())):
                step()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return kept

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


def test_refusals():
    import torch
    import load_balanced_csr_gb300 as lb
    bad = (TypeError, ValueError, lb.SpmvError)
    for args in ((1, 4, 3, 64, torch.bfloat16), (1, 4, 2, 60, torch.bfloat16), (1, 4, 2, 264, torch.bfloat16), (1, 4, 2, 64, torch.float32),
                 (1, 129, 1, 64, torch.bfloat16), (1, 4, 0, 64, torch.bfloat16), (1, 4, 2, 64, torch.float8_e4m3fn)):
        with pytest.raises(bad):
            lb.PromptAttention(*args)
    p = Prompts([5, 6], None, 4, 2, 64, "bf16")
    attend = p.attention()
    q, k, v, ptr = p.q, p.k, p.v, p.q_ptr
    odd = torch.zeros(q.shape[0], 4, 68, dtype=torch.bfloat16, device="cuda")[:, :, 4:]
    for args in ((q.half(), k, v, ptr), (q, k.cpu(), v, ptr), (q, k, v[:-1], ptr), (q[:, :2], k, v, ptr), (q, k, v, ptr.long()),
                 (q, k, v, torch.cat([ptr, ptr[-1:]])), (q, k, v, ptr[:0]), (q, k, v, ptr, ptr[:2]), (q, k, v, ptr[::2]),
                 (odd, k, v, ptr), (q.mT.contiguous().mT, k, v, ptr)):
        with pytest.raises(bad):
            attend(*args)
    with pytest.raises(bad):
        attend(q, k, v, ptr, out=torch.empty_like(q)[:3])
    with pytest.raises(bad):
        attend(q, k, v, ptr, lse=torch.empty(q.shape[0], 4, device="cuda").half())
    w = q.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="no derivative"):
        attend(w, k, v, ptr)[0].float().sum().backward()
    with pytest.raises(RuntimeError):
        attend(w, k, v, ptr, out=torch.empty_like(q))


def test_nothing_to_do():
    import torch
    import load_balanced_csr_gb300 as lb
    i32 = dict(dtype=torch.int32, device="cuda")
    attend = lb.PromptAttention(3, 4, 2, 64, torch.bfloat16)
    x = torch.ones(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    none = x[:0, :2]
    out, lse = attend(x[:0], none, none, torch.zeros(3, **i32))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = attend(x, none, none, torch.tensor([0, 2, 5], **i32), torch.zeros(3, **i32))
    assert bool((out == 0).all()) and bool((lse == -np.inf).all()) and attend.device_status() == 0
    given = torch.full_like(x, 3.0)
    attend(x, x[:, :2], x[:, :2], torch.zeros(1, **i32), out=given)
    attend(x, x[:, :2], x[:, :2], torch.zeros(3, **i32), out=given)
    assert bool((given == 3).all()) and attend.device_status() == 0


@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 115])
@pytest.mark.parametrize("dim", [64, 192, 256])
def test_large_values_under_rising_scores(dim, size):
    """Outputs are no larger than the largest value, and so are the sums before the division but for the number of keys:
    512 times 2^115 is 2^124.  Scores rise by 0.5 to 60 powers of two from a step's keys to the next one's."""
    import torch
    for rise in (0.5, 7.0, 20.0, 39.0, 60.0):
        p = Prompts([300, 3], [512, 300], 4, 2, dim, "bf16", seed=13)
        p.q.zero_(), p.k.zero_()
        p.q[:, :, 0] = 1
        keys = torch.arange(p.k.shape[0], device="cuda")
        p.k[:, :, 0] = (keys // 64 * rise).to(p.k.dtype)[:, None]
        p.v *= size
        for scale in (np.log(2), -np.log(2)):
            out, lse = p.run(scale=float(scale))
            assert bool(torch.isfinite(out[:303]).all())
            p.check(out, lse, scale=float(scale))
    # one key 39 powers of two above all before it
    p = Prompts([1], [129], 1, 1, dim, "bf16", seed=14)
    p.q.zero_(), p.k.zero_(), p.v.fill_(1)
    p.q[0, 0, 0], p.k[128, 0, 0], p.v[128] = 1, 39, size
    out, _ = p.run(scale=float(np.log(2)))
    assert bool((out[0] == size).all())


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -105, 2.0 ** -118])
@pytest.mark.parametrize("scale", [0.1, 1.5])
def test_small_values(size, scale):
    """Values near the bottom of bf16's range keep their bits."""
    p = Prompts([300, 3], [512, 300], 4, 2, 128, "bf16", seed=15)
    p.v *= size
    p.check(*p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 192, 256])
@pytest.mark.parametrize("requests,nq,nk", [(1, 2, 9000), (30, 260, 700)])
def test_infinities_whose_weight_vanishes(requests, nq, nk, dim, dtype):
    """Wherever a key stands, and whatever it weighs: an infinity it brings is its element's, one of the other sign or a NaN
    makes that NaN, and nothing else changes.  Rows whose scores are all minus infinity stay zero."""
    import torch
    hk = 4 if requests > 1 else 1
    p = Prompts([nq] * requests, [nk] * requests, hk, hk, dim, dtype, seed=16, behind=0)
    p.q.zero_(), p.k.zero_()
    p.q[:, :, 0] = 1
    k, v = p.k.view(requests, nk, hk, dim), p.v.view(requests, nk, hk, dim)
    for key in (10, 11, 12, 14, 15, nk - 2):
        k[:, key, :, 0] = -300
    scale = float(np.log(2))  # 300 powers of two below the others
    clean, clean_lse = p.run(scale=scale)
    inf, nan = float("inf"), float("nan")
    v[:, 10, :, 3], v[:, 11, :, 4], v[:, 12, :, 5], v[:, 13, :, 5], v[:, 14, :, 6] = inf, -inf, inf, -inf, nan
    v[:, 15, :, 7], v[:, nk - 1, :, 7], v[:, nk - 2, :, 40] = inf, -inf, -inf
    out, lse = p.run(scale=scale)
    want = clean.clone().view(requests, nq, hk, dim)
    want[..., 3], want[..., 4], want[..., 5], want[..., 6], want[..., 7] = inf, -inf, nan, nan, inf
    want[:, -1, :, 7], want[:, -2:, :, 40] = nan, -inf
    assert torch.equal(out.nan_to_num(7, 8, 9), want.view(out.shape).nan_to_num(7, 8, 9)) and torch.equal(lse, clean_lse)
    k[..., 0] = -inf
    out, lse = p.run(scale=scale)
    assert bool((out == 0).all()) and bool((lse == -inf).all())


def test_infinities_in_shares_whose_weight_vanishes():
    """All of a share's keys weigh nothing next to another's: its infinities count, its finite values do not."""
    import torch
    p = Prompts([2], [20000], 2, 1, 64, "bf16", seed=18, behind=0)
    p.q.zero_(), p.k.zero_()
    p.q[:, :, 0] = 1
    p.k[:15000, 0, 0] = -300
    clean, lse = p.run(scale=float(np.log(2)))
    p.check(clean, lse, scale=float(np.log(2)))
    p.v[5, 0, 3], p.v[9999, 0, 4], p.v[2, 0, 5], p.v[12000, 0, 5], p.v[7000, 0, 6] = np.inf, -np.inf, np.inf, -np.inf, np.nan
    out, lse2 = p.run(scale=float(np.log(2)))
    want = clean.clone()
    want[:, :, 3], want[:, :, 4], want[:, :, 5], want[:, :, 6] = np.inf, -np.inf, np.nan, np.nan
    assert torch.equal(out.nan_to_num(7, 8, 9), want.nan_to_num(7, 8, 9)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [64, 128])
def test_values_of_nan_alone(dim):
    """All rows are NaN, and the call ends."""
    import torch
    p = Prompts([700, 1], [3000, 20000], 4, 2, dim, "bf16", seed=17, behind=0)
    p.v.fill_(float("nan"))
    out, lse = p.run()
    assert bool(torch.isnan(out).all()) and bool(torch.isfinite(lse).all())
