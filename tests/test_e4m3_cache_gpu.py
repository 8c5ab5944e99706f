"""The paged cache in 8 bits: stores and loads bit for bit against plain loops,
attention of one new token against its definition in 64 bits.

Attention's bound.  With v = 2^-24 and u the half-unit of the output's type
(2^-8, 2^-11): a score carries a dot product of head_dim terms, its three
factors and the exponential's own error (a few units of its argument), and q
loses at most 2^-39 of its largest element (below the rest), so each weight is
off by a factor of at most 1 + e, e = 2 (head_dim + 12) v scale max|q||k| +
2^-20 (1 + max|s - lse|); the sum over len positions adds len v; a weight times
its scale carries 22 bits (2^-21 with its two factors' roundings) or, small as
it is, half a step of 2^-38 of the largest times the largest scale.  Hence
|out - out64| <= (2 e + 2 len v + 2^-20) sum p|v| + len 2^-38 448 max(vs) + u |out64| + smallest subnormal,
|lse - lse64| <= e + len v + 4 v |lse64|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}
V = 2.0 ** -24


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


# ------------------------------------------------------------------ codes


def _code_values():
    """What the 256 codes stand for."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


VALUES = _code_values()


def encode(x):
    """The nearest codes, ties to even, of values of at most 448; NaN what is not finite."""
    grid = VALUES[:127]
    a = np.abs(np.where(np.isfinite(x), x, 0))
    assert (a <= 448).all()
    up = np.clip(np.searchsorted(grid, a), 1, 126)
    low, high = a - grid[up - 1], grid[up] - a
    code = np.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)
    code = np.where(a == grid[up], up, code)
    return np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 127).astype(np.uint8)


def scale_for(x):
    """The least power of two p >= 2^-126 with every finite |x| <= 448 p, per head of (tokens, heads, dim)."""
    top = np.where(np.isfinite(x), np.abs(x), 0).max((0, 2)) / 448
    out = np.full(top.shape, 2.0 ** -126)
    for h, t in enumerate(top):
        while out[h] < t:
            out[h] *= 2
    return out


def store_loop(x, codes, scales, slots, block):
    """The definition, block by block; codes (pages, page, heads, dim) uint8 and scales (pages, blocks, heads) in place."""
    pages, page = codes.shape[:2]
    of = {}
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            of.setdefault(s // block, []).append(i)
    for b, tokens in of.items():
        at, first = b * block // page, b * block % page
        rows = codes[at, first:first + block]
        inside = [int(slots[i]) - b * block for i in tokens]
        need = scale_for(x[tokens])
        old = scales[at, first // block].astype(np.float64)
        if 0 not in inside:
            new = np.maximum(old, need)
            for h in np.nonzero(new > old)[0]:
                keep = [r for r in range(block) if r not in inside]
                rows[keep, h] = encode(VALUES[rows[keep, h]] * (old[h] / new[h]))
        else:
            new = need
        rows[inside] = encode(x[tokens] / new[:, None])
        scales[at, first // block] = new


def _same_codes(got, want):
    nan = (want & 127) == 127
    assert (((got & 127) == 127) == nan).all()
    np.testing.assert_array_equal(got[~nan], want[~nan])


def _cache(pages, page, heads, dim, layout, torch, dtype=None):
    """An uninitialised cache of one of the layouts."""
    dt = dtype or torch.uint8
    if layout == "heads":
        t = torch.zeros(pages, heads, page, dim, dtype=dt, device="cuda").transpose(1, 2)
    elif layout == "padded":
        t = torch.zeros(pages, page + 1, heads + 1, dim + 32, dtype=dt, device="cuda")[:, :page, :heads, 16:dim + 16]
    elif layout == "odd":
        t = torch.zeros(pages, page, heads, dim + 3, dtype=dt, device="cuda")[..., 1:dim + 1]
    else:
        t = torch.zeros(pages, page, heads, dim, dtype=dt, device="cuda")
    return t


def _scales(pages, blocks, heads, layout, torch):
    if layout == "heads":
        return torch.zeros(heads, pages, blocks, device="cuda").permute(1, 2, 0)
    if layout in ("padded", "odd"):
        return torch.zeros(pages, blocks + 1, heads + 2, device="cuda")[:, :blocks, 1:heads + 1]
    return torch.zeros(pages, blocks, heads, device="cuda")


class Cache8:
    """Codes and scales with anything in them, on the device and for the loops."""

    def __init__(self, pages, page, heads, dim, block, layout="tokens", seed=0, low=-9, high=4):
        import torch
        rng = np.random.default_rng(seed)
        self.block = block
        self.codes = [rng.integers(0, 256, (pages, page, heads, dim)).astype(np.uint8) for _ in range(2)]
        self.scales = [(2.0 ** rng.integers(low, high, (pages, page // block, heads))).astype(np.float32) for _ in range(2)]
        self.kc, self.vc = (_cache(pages, page, heads, dim, layout, torch) for _ in range(2))
        self.ks, self.vs = (_scales(pages, page // block, heads, layout, torch) for _ in range(2))
        for dev, host in zip((self.kc, self.vc, self.ks, self.vs), (*self.codes, *self.scales)):
            dev.copy_(torch.from_numpy(host))

    def args(self):
        import torch
        return self.kc.view(torch.float8_e4m3fn), self.vc.view(torch.float8_e4m3fn), self.ks, self.vs

    def store(self, k, v, slots):
        import torch
        import load_balanced_csr_gb300 as lb
        lb.paged_store_e4m3(k, v, *self.args(), torch.as_tensor(slots, dtype=torch.int32).cuda())
        for x, codes, scales in zip((k, v), self.codes, self.scales):
            store_loop(x.double().cpu().numpy(), codes, scales, np.asarray(slots), self.block)

    def check(self):
        for codes, scales, dc, ds in zip(self.codes, self.scales, (self.kc, self.vc), (self.ks, self.vs)):
            np.testing.assert_array_equal(ds.cpu().numpy(), scales)
            _same_codes(dc.cpu().numpy(), codes)


def _tokens(n, heads, dim, dtype, seed, torch):
    """Keys and values as views of one projection, tokens of very different sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp2(torch.randint(-12, 12, (n, 2 * heads + 1, 1), generator=g, device="cuda").float())
    x = (torch.randn(n, 2 * heads + 1, dim, generator=g, device="cuda") * size).to(_dtype(dtype))
    return x[:, :heads], x[:, heads:2 * heads]


def _append_slots(rng, requests, page, longest, pages):
    """Slots of requests' new tokens as a page table gives them, some requests not served, a tail of padding."""
    order, slots = rng.permutation(pages).tolist(), []
    for _ in range(requests):
        past, fresh = int(rng.integers(0, 3 * page)), int(rng.integers(0, longest + 1))
        mine = [order.pop() for _ in range(-(-(past + fresh) // page))]
        if rng.random() < 0.1:
            slots += [-1] * fresh
        else:
            slots += [mine[t // page] * page + t % page for t in range(past, past + fresh)]
    return np.array(slots + [-1] * int(rng.integers(0, 200)), np.int32)


CASES = [(1, 1, 8, 1, 1, "tokens"), (3, 8, 128, 16, 16, "tokens"), (9, 8, 128, 64, 16, "heads"), (5, 3, 72, 7, 7, "padded"),
         (5, 3, 72, 7, 1, "padded"), (4, 5, 33, 6, 3, "odd"), (2, 1, 256, 128, 64, "tokens"), (3, 2, 320, 32, 32, "tokens"),
         (40, 2, 64, 16, 4, "heads"), (6, 4, 192, 16, 1, "tokens"), (2, 3, 40, 9, 1, "odd")]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("requests,heads,dim,page,block,layout", CASES)
def test_store(requests, heads, dim, page, block, layout, dtype):
    """Two steps, each a few chunks: bit for bit."""
    import torch
    rng = np.random.default_rng(dim + block)
    pages = requests * (3 + 90 // page + 2) + 2
    cache = Cache8(pages, page, heads, dim, block, layout, seed=dim)
    for step in range(2):
        slots = _append_slots(rng, requests, page, 90, pages)
        cache.store(*_tokens(len(slots), heads, dim, dtype, step, torch), slots)
        cache.check()


@pytest.mark.parametrize("block", [2, 16, 64])
def test_store_token_by_token(block):
    """Every token a call of its own: a block's scale grows with its tokens."""
    import torch
    cache = Cache8(3, 64, 2, 64, block, seed=1)
    k, v = _tokens(150, 2, 64, "bf16", 3, torch)
    for i in range(150):
        cache.store(k[i:i + 1], v[i:i + 1], [i])
    cache.check()
    # what is held is within the sum of its roundings: half a step of 2^-3 relative, or of the least code, doubled by the scale's growth
    for x, codes, scales in zip((k, v), cache.codes, cache.scales):
        rows = VALUES[codes.reshape(-1, 2, 64)[:150]]
        scale = scales.reshape(-1, 2)[np.arange(150) // block].astype(np.float64)[..., None]
        want = x.double().cpu().numpy()
        assert (np.abs(rows * scale - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * scale).all()


def test_store_skipped_tokens_inside_runs():
    """Up to 63 skipped slots between two tokens of a block, over tiles' ends; slots in any order within a block."""
    import torch
    rng = np.random.default_rng(3)
    cache = Cache8(40, 16, 3, 64, 16, seed=2)
    slots = []
    for page in rng.permutation(40).tolist():
        inside = rng.permutation(16)[:rng.integers(1, 17)]
        for s in inside.tolist():
            slots += [page * 16 + s] + rng.choice([-1, 40 * 16, 2 ** 31 - 1, -2 ** 31]).repeat(rng.choice([0, 0, 1, 5, 63])).tolist()
        slots += [-1] * int(rng.integers(0, 300))
    cache.store(*_tokens(len(slots), 3, 64, "bf16", 4, torch), np.array(slots, np.int64).astype(np.int32))
    cache.check()


def test_store_values_at_the_edges():
    """Zeros, subnormals, the largest values, 448 times a power of two and its neighbours, ties, infinities and NaN."""
    import torch
    edge = [0.0, -0.0, 448.0, -448.0, 449.0, 464.0, 480.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -149, 2.0 ** -126, 3.4e38,
            -3.4e38, 1e-38, 17.0, 19.0, 25.5, float("inf"), float("-inf"), float("nan")]
    rng = np.random.default_rng(5)
    n = 400
    x = torch.tensor(rng.choice(edge, (n, 4, 64)), dtype=torch.float32, device="cuda")
    x[:40] = 0
    x[40:60] = 2.0 ** -140
    x[60:70] = float("nan")
    x[70:120, :, 1:] *= 2.0 ** -20  # a few large ones beside small ones
    x = torch.where(torch.rand(n, 4, 64, device="cuda") < 0.5, x, torch.randn(n, 4, 64, device="cuda"))
    for block in (1, 16):
        cache = Cache8(30, 16, 4, 64, block, seed=7)
        slots = rng.permutation(30)[:25].repeat(16) * 16 + np.tile(np.arange(16), 25)
        cache.store(x, x.flip(0), slots)
        cache.check()


def test_store_many_tokens_and_heads():
    """Tiles, slices and rounds of every launch shape."""
    import torch
    for tokens, heads, page, block, dim in ((5000, 1, 16, 16, 64), (1300, 40, 16, 8, 64), (20000, 2, 128, 64, 128), (9, 300, 16, 16, 64)):
        pages = -(-tokens // page) + 1
        cache = Cache8(pages, page, heads, dim, block, seed=tokens)
        cache.store(*_tokens(tokens, heads, dim, "f16", tokens, torch), np.arange(tokens) + page // 2)
        cache.check()


def test_store_offsets_past_32_bits():
    import torch
    import load_balanced_csr_gb300 as lb
    pages, page, heads, dim = 1200, 256, 64, 128  # 2.5e9 codes
    kc, vc = (torch.zeros(pages, page, heads, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(pages, page // 16, heads, device="cuda") for _ in range(2))
    k, v = _tokens(40, heads, dim, "bf16", 1, torch)
    slots = torch.arange(pages * page - 40, pages * page, dtype=torch.int32, device="cuda")
    lb.paged_store_e4m3(k, v, kc, vc, ks, vs, slots)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, page], dtype=torch.int32, device="cuda")
    got, _ = lb.paged_load(kc, vc, table, ptr, page, ks, vs, dtype=torch.float32)
    scale = ks[-1, -3:].repeat_interleave(16, 0)[8:, :, None]
    assert bool(((got[-40:] - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * scale).all())
    assert bool((got[:-48] == 0).all())


# ------------------------------------------------------------------ load


def load_loop(cache, table, ptr, values, out):
    """values(page, position) are a cache's rows; rows that no request has stay."""
    pages, page = cache.shape[:2]
    for r in range(len(ptr) - 1):
        for i in range(ptr[r], min(ptr[r + 1], len(out))):
            t = i - ptr[r]
            p = table[r, t // page] if t // page < table.shape[1] else -1
            out[i] = values(p, t % page) if 0 <= p < pages else 0
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("lens,heads,dim,page,block,layout", [
    ([1], 1, 8, 1, 1, "tokens"), ([0, 17, 0, 0, 200, 16, 0], 8, 128, 16, 16, "tokens"), ([33, 5, 64], 2, 64, 16, 4, "heads"),
    ([20, 7, 8], 3, 72, 7, 7, "padded"), ([20, 7, 8], 3, 33, 6, 3, "odd"), ([300], 5, 256, 128, 64, "tokens"), ([0, 0], 2, 64, 16, 16, "tokens"),
    ([2, 0, 1] * 700, 1, 64, 1, 1, "tokens"), ([3000, 1], 16, 192, 32, 8, "heads")])
def test_load(lens, heads, dim, page, block, layout, codes, dtype):
    import torch
    import load_balanced_csr_gb300 as lb
    rng = np.random.default_rng(sum(lens) + dim)
    held = [-(-n // page) for n in lens]
    pages, dt = sum(held) + 2, _dtype(dtype)
    table = np.full((len(lens) + 1, max(held) + 1), 2 ** 30, np.int32)
    order, at = rng.permutation(pages), 0
    for r, n in enumerate(held):
        table[r, :n] = order[at:at + n]
        at += n
    ptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = int(ptr[-1]) + 3
    if codes:
        cache = Cache8(pages, page, heads, dim, block, layout, seed=dim, low=-20)
        # any scales will do here
        cache.ks.mul_(1.37), cache.vs.mul_(0.9)
        k_cache, v_cache, ks, vs = cache.args()
        whole = [c.float() * s.repeat_interleave(block, 1)[..., None] for c, s in ((k_cache, ks), (v_cache, vs))]
    else:
        k_cache, v_cache = (_cache(pages, page, heads, dim, layout, torch, dt) for _ in range(2))
        for c in (k_cache, v_cache):
            c.copy_(torch.randn(c.shape, device="cuda"))
        ks = vs = None
        whole = [k_cache, v_cache]
    outs = [torch.full((tokens, heads + 1, dim + 1), 7.0, device="cuda").to(dt)[:, 1:, :dim] for _ in range(2)]
    dense = [torch.full((tokens, heads, dim), 7.0, device="cuda").to(dt) for _ in range(2)]
    dev_table, dev_ptr = torch.from_numpy(table).cuda(), torch.from_numpy(ptr).cuda()
    for given in (outs, dense):
        got = lb.paged_load(k_cache, v_cache, dev_table, dev_ptr, tokens, ks, vs, dtype=dt, k=given[0], v=given[1])
        assert got[0] is given[0] and got[1] is given[1]
        for x, w in zip(given, whole):
            w = w.to(dt).float().cpu().numpy()
            want = load_loop(w, table, ptr, lambda p, s: w[p, s], np.full((tokens, heads, dim), 7.0, np.float32))
            np.testing.assert_array_equal(x.float().cpu().numpy(), want)
    assert bool((outs[0]._base[:, 0] == 7).all())
    k, v = lb.paged_load(k_cache, v_cache, dev_table, dev_ptr, tokens, ks, vs, dtype=dt)
    n = int(ptr[-1])
    assert k.is_contiguous() and torch.equal(k[:n].nan_to_num(5), dense[0][:n].nan_to_num(5))
    assert torch.equal(v[:n].nan_to_num(5), dense[1][:n].nan_to_num(5))


def test_load_bad_pages_and_pointers():
    """Pages outside the cache, positions past the row, pointers that fall: zeros or nothing, never a read outside."""
    import torch
    import load_balanced_csr_gb300 as lb
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.ones(4, 16, 2, 64, device="cuda")
    table = torch.tensor([[0, -1], [9, 2], [3, 2 ** 31 - 1]], **i32)

    def load(ptr, tokens):
        k, v = (torch.full((tokens, 2, 64), 7.0, device="cuda") for _ in range(2))
        lb.paged_load(cache, cache, table, torch.tensor(ptr, **i32), tokens, k=k, v=v)
        assert torch.equal(k, v) and bool((k == k[:, :1, :1]).all())
        return k[:, 0, 0].tolist()

    assert load([0, 20, 40, 60], 70) == [1] * 16 + [0] * 4 + [0] * 16 + [1] * 4 + [1] * 16 + [0] * 4 + [7] * 10
    assert load([0, 50, 50, 50], 50) == [1] * 16 + [0] * 34           # past the table's row
    assert load([0, 20, 40, 60], 10) == [1] * 10                      # fewer rows than there are
    assert set(load([0, 60, 3, 60], 64)) <= {0.0, 1.0, 7.0}
    assert set(load([5, 2 ** 31 - 1, -2 ** 31, 40], 64)) <= {0.0, 1.0, 7.0}
    assert load([2, 4, 4, 6], 8) == [7, 7, 1, 1, 1, 1, 7, 7]


# ------------------------------------------------------------------ attention


class Requests:
    """Codes and scales that are NaN wherever no request's position (block) is, tables far outside wherever no request reaches."""

    def __init__(self, lens, q_heads, kv_heads, dim, page, block, dtype, layout="tokens", seed=0, low=-12, high=-4, powers=True):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_host, self.dtype, self.block = list(lens), dtype, block
        held = [-(-n // page) for n in lens]
        pages, width = sum(held) + 3, max(held + [1]) + 2
        order, table, at = rng.permutation(pages), np.full((len(lens), width), 2 ** 30, np.int32), 0
        self.kc, self.vc = (_cache(pages, page, kv_heads, dim, layout, torch) for _ in range(2))
        self.ks, self.vs = (_scales(pages, page // block, kv_heads, layout, torch) for _ in range(2))
        for t in (self.kc, self.vc):
            t.fill_(0x7f)
        for t in (self.ks, self.vs):
            t.fill_(float("nan"))
        where = []
        for b, n in enumerate(lens):
            table[b, :held[b]] = order[at:at + held[b]]
            pos = np.arange(n)
            where.append(table[b, pos // page].astype(np.int64) * page + pos % page)
            at += held[b]
        where = torch.from_numpy(np.concatenate(where) if where else np.zeros(0, np.int64)).cuda()
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            codes = (100 * torch.randn(where.numel(), kv_heads, dim, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
            c[where // page, where % page] = codes.view(torch.uint8)
            size = torch.exp2(torch.randint(low, high + 1, s.shape, generator=g, device="cuda").float())
            if not powers:
                size = size * (1 + torch.rand(s.shape, generator=g, device="cuda"))
            used = torch.zeros(s.shape, dtype=torch.bool, device="cuda")
            used[where // page, where % page // block] = True
            s.copy_(torch.where(used, size, torch.nan))
        self.q = torch.randn(len(lens), q_heads, dim, generator=g, device="cuda").to(_dtype(dtype))
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32, device="cuda")
        self.shape = (q_heads, kv_heads, dim, page)

    def caches(self):
        import torch
        return self.kc.view(torch.float8_e4m3fn), self.vc.view(torch.float8_e4m3fn), self.ks, self.vs

    def attention(self, max_batch=None):
        import load_balanced_csr_gb300 as lb
        hq, hk, dim, _ = self.shape
        return lb.PagedAttentionE4M3(max_batch or len(self.lens_host), hq, hk, dim, _dtype(self.dtype))

    def check(self, out, lse, scale):
        """Every request and head against the definition in 64 bits."""
        import torch
        hq, hk, dim, page = self.shape
        u = U[self.dtype]
        kc, vc, ks, vs = self.caches()
        for b, n in enumerate(self.lens_host):
            if n == 0:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all(), f"request {b} of length 0"
                continue
            pos = torch.arange(n, device="cuda")
            at, inside = self.table[b].long()[pos // page], pos % page
            bl = inside // self.block
            k, v = (c[at, inside].double() * s[at, bl].double()[..., None] for c, s in ((kc, ks), (vc, vs)))
            k, v = (x.repeat_interleave(hq // hk, 1) for x in (k, v))
            q = self.q[b].double()
            s = torch.einsum("hd,nhd->hn", q, k) * scale
            want_lse = torch.logsumexp(s, 1)
            p = torch.exp(s - want_lse[:, None])
            want = torch.einsum("hn,nhd->hd", p, v)
            spread = torch.einsum("hn,nhd->hd", p, v.abs())
            size = torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1) * abs(scale)
            e = 2 * (dim + 12) * V * size + 2.0 ** -20 * (1 + (s - want_lse[:, None]).abs().amax(1))
            lost = n * 2.0 ** -38 * 448 * float(vs[at, bl].max())
            bound = (2 * e + 2 * n * V + 2.0 ** -20)[:, None] * spread + lost + u * want.abs() + TINY[self.dtype]
            off = (out[b].double() - want).abs()
            assert bool((off <= bound).all()), f"request {b} of {n}: {float((off / bound).max())} of the bound"
            off = (lse[b].double() - want_lse).abs()
            assert bool((off <= e + n * V + 4 * V * want_lse.abs()).all()), f"request {b} of {n}: lse off by {float(off.max())}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_heads,kv_heads,dim,page,block,layout", [
    (64, 8, 128, 16, 16, "tokens"), (8, 8, 64, 16, 1, "heads"), (6, 2, 80, 7, 7, "padded"), (32, 2, 128, 64, 16, "heads"),
    (20, 1, 96, 128, 32, "tokens"), (4, 1, 192, 1, 1, "tokens"), (16, 1, 192, 16, 8, "padded"), (12, 2, 256, 32, 4, "tokens"),
    (16, 1, 256, 16, 16, "heads"), (9, 3, 16, 48, 48, "tokens"), (16, 1, 64, 16, 16, "tokens"), (7, 7, 112, 7, 1, "tokens"),
    (32, 2, 96, 16, 2, "tokens")])
def test_attention(q_heads, kv_heads, dim, page, block, layout, dtype):
    r = Requests([0, 1, 15, 16, 17, 31, 33, 500, 0, 1023, 4097, 64], q_heads, kv_heads, dim, page, block, dtype, layout, seed=dim)
    attend = r.attention()
    out, lse = attend(r.q, *r.caches(), r.table, r.lens)
    r.check(out, lse, dim ** -0.5)
    assert attend.device_status() == 0
    again, lse2 = attend(r.q, *r.caches(), r.table, r.lens)
    assert out.equal(again) and lse.equal(lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_one_long_request(dtype):
    r = Requests([70001], 16, 2, 128, 16, 16, dtype, seed=3)
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    r.check(out, lse, 128 ** -0.5)


def test_attention_many_requests():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 60, 1300).tolist()
    r = Requests(lens, 8, 2, 64, 16, 4, "bf16", seed=4)
    out, lse = r.attention(1400)(r.q, *r.caches(), r.table, r.lens)
    r.check(out, lse, 64 ** -0.5)


@pytest.mark.parametrize("scale", [0.3, -0.05, 0.0, 4.0])
def test_attention_scales_of_scores(scale):
    r = Requests([5, 700, 64], 8, 2, 128, 16, 16, "bf16", seed=5)
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens, scale=scale)
    r.check(out, lse, scale)


@pytest.mark.parametrize("low,high,powers", [(-40, -8, True), (-100, -90, True), (-12, -4, False), (20, 30, True), (-126, -120, False)])
@pytest.mark.parametrize("heads", [(8, 1), (32, 2)])
def test_attention_scales_of_blocks(low, high, powers, heads):
    """Scales that differ widely, very small and very large ones, none a power of two."""
    r = Requests([1, 300, 2000, 17], *heads, 128, 16, 4, "bf16", seed=6, low=low, high=high, powers=powers)
    import torch
    if high > 0:
        r.ks.mul_(2.0 ** -32)
    if high < -20:
        r.ks.mul_(2.0 ** (-6 - high))
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    assert bool(torch.isfinite(out).all())
    r.check(out, lse, 128 ** -0.5)


def test_attention_of_queries_of_any_size():
    """bf16 queries past what f16 holds, and elements far below a head's largest."""
    import torch
    r = Requests([40, 333], 8, 2, 64, 16, 16, "bf16", seed=7)
    r.q[:, 0] *= 2.0 ** 60
    r.q[:, 1] *= 2.0 ** -60
    r.q[:, 2, ::3] *= 2.0 ** -20
    r.q[:, 3] = 0
    r.q[:, 4] *= 2.0 ** -120
    scale = torch.tensor(64 ** -0.5)
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens, scale=float(scale) * 2.0 ** -58)
    r.check(out, lse, float(scale) * 2.0 ** -58)
    r.q[:, 0] = 1
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    r.check(out, lse, 64 ** -0.5)


def test_attention_nan_codes():
    """A NaN in a value is its element's alone, one in a key its request's and kv head's."""
    import torch
    r = Requests([100, 100], 8, 2, 64, 16, 16, "bf16", seed=8)
    clean, _ = r.attention()(r.q, *r.caches(), r.table, r.lens)
    page = int(r.table[0, 2])
    r.vc[page, 5, 1, 7] = 0x7f
    r.kc[int(r.table[1, 0]), 3, 0, 2] = 0xff
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[0, 4:, 7] = True
    want[1, :4] = True
    assert torch.equal(bad, want) and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_attention_scales_that_are_not_finite(scale):
    """They spoil their request's and kv head's outputs, and no other's."""
    import torch
    r = Requests([64, 64], 8, 2, 64, 16, 16, "bf16", seed=11)
    clean, _ = r.attention()(r.q, *r.caches(), r.table, r.lens)
    r.vs[int(r.table[0, 1]), 0, 0] = scale
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    assert not bool(torch.isfinite(out[0, :4]).any()) and bool(torch.isfinite(lse).all())
    assert torch.equal(out[0, 4:], clean[0, 4:]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("heads", [(8, 2), (16, 1)])
def test_attention_of_the_largest_scale(heads):
    """2^127, whose reciprocal is subnormal: as with 2^100, times 2^27."""
    import torch
    r = Requests([17, 5], *heads, 64, 16, 16, "bf16", seed=12)
    for lens, page in ((17, 0), (17, 1), (5, 0)):
        at = int(r.table[0 if lens == 17 else 1, page])
        r.vc[at].remainder_(9)  # codes of 0 to 2^-6
        r.vs[at] = 2.0 ** 100
    small, _ = r.attention()(r.q, *r.caches(), r.table, r.lens)
    r.vs.mul_(2.0 ** 27)
    out, _ = r.attention()(r.q, *r.caches(), r.table, r.lens)
    assert bool((small > 2.0 ** 80).any()) and torch.equal(out.float(), small.float() * 2.0 ** 27)


def test_attention_bad_pages_and_lengths():
    import torch
    r = Requests([64, 64, 64], 4, 1, 64, 16, 16, "bf16", seed=9)
    r.table[0, 1] = -1
    r.lens[1] = -5
    attend = r.attention()
    out, lse = attend(r.q, *r.caches(), r.table, r.lens)
    assert attend.device_status() == 3
    assert bool((out[1] == 0).all()) and bool(torch.isfinite(out).all())
    r.lens_host = [0, 0, 64]
    r.check(torch.cat([torch.zeros_like(out[:2]), out[2:]]), torch.cat([torch.full_like(lse[:2], -np.inf), lse[2:]]), 0.125)


def test_a_chain_in_a_graph():
    """Tokens appended, stored and attended to step by step, captured once, replayed with other tokens: as eager calls give."""
    import torch
    import load_balanced_csr_gb300 as lb
    i32 = dict(dtype=torch.int32, device="cuda")
    n, hq, hk, d, page, block, pages_n = 5, 8, 2, 64, 16, 16, 64

    def make():
        torch.manual_seed(0)
        s = {"table": lb.PageTable(torch.full((n, 8), -1, **i32), page, pages_n, max_tokens=n), "past": torch.zeros(n, **i32),
             "free": torch.randperm(pages_n).to(**i32), "attend": lb.PagedAttentionE4M3(n, hq, hk, d, torch.bfloat16),
             "x": torch.zeros(n, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")}
        s["cache"] = [torch.zeros(pages_n, page, hk, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)] + \
                     [torch.zeros(pages_n, page // block, hk, device="cuda") for _ in range(2)]
        return s

    def step(s):
        one = torch.ones_like(s["past"])
        p = s["table"].append(s["past"], one, s["free"])
        q, k, v = s["x"].split([hq, hk, hk], 1)
        lb.paged_store_e4m3(k, v, *s["cache"], p.slots)
        out, lse = s["attend"](q, *s["cache"], p.table, p.lens)
        s["past"].copy_(p.lens)
        return out, lse

    tokens = torch.randn(12, n, hq + 2 * hk, d, device="cuda").bfloat16()
    eager = make()
    want = []
    # with a fresh list of free pages per step, since taken pages are the host's to drop
    for t in range(12):
        eager["x"].copy_(tokens[t])
        eager["free"].copy_(torch.arange(t * n, t * n + pages_n, **i32) % pages_n)
        want.append([y.clone() for y in step(eager)])
    graphed = make()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(graphed)
    torch.cuda.current_stream().wait_stream(stream)
    graphed = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(graphed)
    for t in range(12):
        graphed["x"].copy_(tokens[t])
        graphed["free"].copy_(torch.arange(t * n, t * n + pages_n, **i32) % pages_n)
        graph.replay()
        assert torch.equal(got[0], want[t][0]) and torch.equal(got[1], want[t][1]), t


def test_refusals():
    import torch
    import load_balanced_csr_gb300 as lb
    c = Cache8(4, 16, 2, 64, 16)
    kc, vc, ks, vs = c.args()
    k, v = _tokens(3, 2, 64, "bf16", 0, torch)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    table, ptr = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    bad = (TypeError, ValueError, lb.SpmvError)
    for args in ((k.cpu(), v, kc, vc, ks, vs, slots), (k, v.float(), kc, vc, ks, vs, slots), (k, v, kc.float(), vc, ks, vs, slots),
                 (k, v, kc, vc[:2], ks, vs, slots), (k, v, kc, vc, ks.double(), vs, slots), (k, v, kc, vc, ks[:, :0], vs, slots),
                 (k, v, kc, vc, ks, vs[:3], slots), (k, v, kc, vc, torch.ones(4, 3, 2, device="cuda"), vs, slots),
                 (k, v, kc, vc, ks, vs, slots[:2]), (k, v, kc, vc, ks, vs, slots.long()), (k.mT, v.mT, kc, vc, ks, vs, slots),
                 (k[:, :1], v[:, :1], kc, vc, ks, vs, slots)):
        with pytest.raises(bad):
            lb.paged_store_e4m3(*args)
    big = [torch.zeros(2, 128, 2, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    with pytest.raises(lb.SpmvError, match="block"):
        lb.paged_store_e4m3(k, v, *big, *(torch.ones(2, 1, 2, device="cuda") for _ in range(2)), slots)
    for args, kw in (((kc, vc, table, ptr, 3, ks, vs), {}), ((kc, vc, table, ptr, -1, ks, vs), dict(dtype=torch.bfloat16)),
                     ((kc, vc, table, ptr, 3), dict(dtype=torch.bfloat16)), ((kc, vc, table, ptr.long(), 3, ks, vs), dict(dtype=torch.bfloat16)),
                     ((kc, vc, table[:0], ptr, 3, ks, vs), dict(dtype=torch.bfloat16)),
                     ((kc.float(), vc.float(), table, ptr, 3), dict(dtype=torch.bfloat16)),
                     ((kc.float(), vc.float(), table, ptr, 3, ks, vs), {}), ((kc.double(), vc.double(), table, ptr, 3), {}),
                     ((kc, vc, table, ptr, 3, ks, vs), dict(dtype=torch.bfloat16, k=torch.zeros(2, 2, 64, device="cuda").bfloat16())),
                     ((kc, vc, table, ptr, 3, ks, vs), dict(dtype=torch.bfloat16, v=torch.zeros(3, 2, 64, device="cuda")))):
        with pytest.raises(bad):
            lb.paged_load(*args, **kw)
    with pytest.raises(bad):
        lb.PagedAttentionE4M3(1, 2, 2, 64, torch.float32)
    with pytest.raises(bad):
        lb.PagedAttentionE4M3(1, 2, 2, 72, torch.bfloat16)
    attend = lb.PagedAttentionE4M3(1, 4, 2, 64, torch.bfloat16)
    q, lens = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for args in ((q.half(), kc, vc, ks, vs, table, lens), (q, kc.bfloat16(), vc, ks, vs, table, lens), (q, kc, vc, ks, None, table, lens),
                 (q, kc, vc, ks, vs[:, :, :1], table, lens), (q, kc, vc, ks.half(), vs, table, lens), (q, kc, vc, ks, vs, table, lens.long())):
        with pytest.raises(bad):
            attend(*args)
    w = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    out, _ = attend(w, kc, vc, ks, vs, table, lens)
    with pytest.raises(RuntimeError, match="no derivative"):
        out.float().sum().backward()
    rows = torch.zeros(4, 16, 2, 64, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        lb.paged_load(rows, rows, table, ptr, 3)[0].sum().backward()


def test_nothing_to_do():
    import torch
    import load_balanced_csr_gb300 as lb
    c = Cache8(4, 16, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    lb.paged_store_e4m3(none, none, *c.args(), torch.zeros(0, **i32))
    c.check()
    kc, vc, ks, vs = c.args()
    for table, ptr, tokens in ((torch.zeros(0, 4, **i32), torch.zeros(1, **i32), 0), (torch.zeros(2, 4, **i32), torch.zeros(3, **i32), 0),
                               (torch.zeros(2, 0, **i32), torch.tensor([0, 3, 4], **i32), 4)):
        k, v = lb.paged_load(kc, vc, table, ptr, tokens, ks, vs, dtype=torch.float16)
        assert k.shape == v.shape == (tokens, 2, 64) and bool((k == 0).all())
    none = [t[:0] for t in (kc, vc, ks, vs)]
    k, v = _tokens(3, 2, 64, "bf16", 0, torch)
    lb.paged_store_e4m3(k, v, *none, torch.arange(3, **i32))
    k, v = lb.paged_load(*none[:2], torch.zeros(1, 4, **i32), torch.tensor([0, 3], **i32), 3, *none[2:], dtype=torch.float16)
    assert bool((k == 0).all())
    attend = lb.PagedAttentionE4M3(2, 4, 2, 64, torch.bfloat16)
    out, lse = attend(torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda"), *none, torch.zeros(2, 0, **i32), torch.zeros(2, **i32))
    assert bool((out == 0).all()) and bool((lse == -np.inf).all())


def test_streams():
    """On a stream of the caller's: outputs taken from it, ordered with it."""
    import torch
    r = Requests([100, 5], 8, 2, 64, 16, 16, "bf16", seed=10)
    attend, stream = r.attention(), torch.cuda.Stream()
    want = attend(r.q, *r.caches(), r.table, r.lens)
    torch.cuda.synchronize()
    out, lse = attend(r.q, *r.caches(), r.table, r.lens, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("heads", [(8, 1), (32, 2)])
@pytest.mark.parametrize("power,low,high", [(-112, 100, 110), (-122, 112, 121), (100, -114, -104)])
def test_attention_of_large_key_scales_and_small_queries(power, low, high, heads):
    """Scores are of the usual size: neither factor's range is the product's."""
    r = Requests([1, 300, 2000, 17], *heads, 128, 16, 4, "bf16", seed=13, low=low, high=high)
    r.vs.mul_(2.0 ** (-8 - high))
    r.q.mul_(2.0 ** power)
    out, lse = r.attention()(r.q, *r.caches(), r.table, r.lens)
    r.check(out, lse, 128 ** -0.5)


def test_load_of_more_than_2_30_requests():
    """Nearly all of them empty: the search for a row's request goes up to the last."""
    import torch
    import load_balanced_csr_gb300 as lb
    requests = 2 ** 30 + 9
    ptr = torch.zeros(requests + 1, dtype=torch.int32, device="cuda")  # 4 GiB
    ptr[requests - 4:] = 2
    ptr[requests:] = 5
    cache = torch.randn(3, 4, 1, 8, device="cuda")
    table = torch.tensor([[2, 1]], dtype=torch.int32, device="cuda").expand(requests, 2)
    k, v = lb.paged_load(cache, cache + 1, table, ptr, 5)
    # two rows of request 2^30 + 4, three of the last
    want = cache[2, [0, 1, 0, 1, 2]]
    assert torch.equal(k, want) and torch.equal(v, want + 1)


def test_load_keeps_no_gradient_of_scales_without_a_word():
    """The rows are codes times scales: a scale that requires a gradient is told that there is none."""
    import torch
    import load_balanced_csr_gb300 as lb
    kc, vc, ks, vs = Cache8(4, 16, 2, 64, 16).args()
    table, ptr = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want = lb.paged_load(kc, vc, table, ptr, 3, ks, vs, dtype=torch.float32)
    for which in (0, 1):
        scales = [ks.clone(), vs.clone()]
        scales[which].requires_grad_()
        got = lb.paged_load(kc, vc, table, ptr, 3, *scales, dtype=torch.float32)
        assert got[0].requires_grad and all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(got, want))
        with pytest.raises(RuntimeError, match="no derivative"):
            got[which].sum().backward()
        with pytest.raises(RuntimeError, match="outputs given"):
            lb.paged_load(kc, vc, table, ptr, 3, *scales, dtype=torch.float32, k=torch.empty_like(want[0]))
        with torch.no_grad():
            assert not lb.paged_load(kc, vc, table, ptr, 3, *scales, dtype=torch.float32)[0].requires_grad


def test_sizes_past_32_bits_are_refused():
    """ctypes drops the bits above: 2^32 + 3 rows would be taken as 3."""
    import torch
    import load_balanced_csr_gb300 as lb
    many, i32 = 2 ** 32 + 3, dict(dtype=torch.int32, device="cuda")
    c = Cache8(4, 16, 2, 64, 16).args()
    big = [t[:1].expand(many, *t.shape[1:]) for t in c]
    table, ptr, lens = torch.zeros(1, 4, **i32), torch.tensor([0, 3], **i32), torch.ones(1, **i32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    rows, wide = x.expand(many, 2, 64), torch.empty(1, many, **i32)  # 16 GiB: its rows have to be contiguous
    attend8, attend = (kind(1, 2, 2, 64, torch.bfloat16) for kind in (lb.PagedAttentionE4M3, lb.PagedAttention))
    whole = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    prompts = lb.PromptAttention(1, 2, 2, 64, torch.bfloat16)
    load = dict(dtype=torch.bfloat16, k=rows, v=rows)
    for call in (lambda: lb.paged_load(*c[:2], table, ptr, many, *c[2:], **load),
                 lambda: lb.paged_load(*big[:2], table, ptr, 3, *big[2:], dtype=torch.bfloat16),
                 lambda: lb.paged_load(*c[:2], wide, ptr, 3, *c[2:], dtype=torch.bfloat16),
                 lambda: lb.paged_store_e4m3(rows, rows, *c, lens),
                 lambda: lb.paged_store_e4m3(x, x, *big, lens),
                 lambda: lb.paged_store(x, x, whole.expand(many, 16, 2, 64), whole.expand(many, 16, 2, 64), lens),
                 lambda: attend8(x, *big, table, lens),
                 lambda: attend8(x, *c, wide, lens),
                 lambda: attend(x, whole.expand(many, 16, 2, 64), whole.expand(many, 16, 2, 64), table, lens),
                 lambda: prompts(rows, x, x, ptr),
                 lambda: prompts(x, rows, rows, ptr),
                 lambda: lb.PromptAttention(1, many + 1, 2, 64, torch.bfloat16),
                 lambda: lb.PagedAttentionE4M3(1, 2 ** 32 + 2, 2, 64, torch.bfloat16),
                 lambda: lb.PagedAttention(2 ** 32 + 2, 2, 2, 64, torch.bfloat16)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
