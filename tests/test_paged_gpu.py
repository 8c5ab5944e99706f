"""The paged cache: page tables and slots against a plain loop, bit for bit;
stores bit for bit; attention of one new token against its definition in 64
bits.

Attention's bound.  With v = 2^-24 and u the half-unit of the element type
(2^-24, 2^-8, 2^-11): a score carries a dot product of head_dim terms, its
scaling and the exponential's own error (a few units of its argument), so each
weight is off by a factor of at most 1 + e, e = 2 (head_dim + 8) v scale
max|q||k| + 2^-20 (1 + max|s - lse|); sums over len positions add len v, and a
weight may be rounded to the element type once (u).  Hence
|out - out64| <= (2 e + 2 len v + u) sum p|v| + u |out64| + smallest subnormal,
|lse - lse64| <= e + len v + 4 v |lse64|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
V = 2.0 ** -24


def _torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


# ------------------------------------------------------------------ page tables


def append_loop(past, fresh, page, num_pages, free, table, max_tokens):
    """The definition, request by request and token by token."""
    table = table.copy()
    max_pages = table.shape[1]
    slots = np.full(max_tokens, -1, np.int32)
    positions = np.full(max_tokens, -1, np.int32)
    ptr, lens, used, first, flags = [0], [], 0, 0, 0
    for r, (p, f) in enumerate(zip(past.tolist(), fresh.tolist())):
        if p < 0 or f < 0:
            flags |= 8
            p, f = max(p, 0), max(f, 0)
        held, want = -(-p // page), -(-(p + f) // page)
        need, served = want - held, True
        if held > max_pages:
            flags, need, served = flags | 8, 0, False
        elif want > max_pages:
            flags, need, served = flags | 2, 0, False
        if need and first + need > len(free):
            flags, served = flags | 1, False
        if f and ptr[-1] + f > max_tokens:
            flags, served = flags | 4, False
        if served and need:
            used = max(used, first + need)
            table[r, held:want] = free[first:first + need]
        for j in range(f):
            i, at = ptr[-1] + j, p + j
            if i >= max_tokens:
                continue
            positions[i] = at
            if served:
                entry = table[r, at // page]
                if 0 <= entry < num_pages:
                    slots[i] = entry * page + at % page
                else:
                    flags |= 16
        ptr.append(ptr[-1] + f)
        lens.append(p + f if served else p)
        first += need
    return table, np.array(ptr, np.int32), np.array(lens, np.int32), slots, positions, used, flags


def _tables(rng, past, page, max_pages, pool):
    table = np.full((len(past), max_pages), -5, np.int32)
    order = rng.permutation(pool).astype(np.int32)
    at = 0
    for r, p in enumerate(past):
        n = min(-(-max(p, 0) // page), max_pages)
        table[r, :n] = order[at:at + n]
        at += n
    return table, order[at:]


def check_append(past, fresh, page, max_pages, short=0, slack=5, num_pages=None, pitch=None, seed=0, width=None):
    import torch
    import load_balanced_csr_gb300 as lb
    rng = np.random.default_rng(seed)
    past, fresh = np.asarray(past, np.int32), np.asarray(fresh, np.int32)
    held = int(sum(-(-max(p, 0) // page) for p in past.tolist()))
    new = int(sum(-(-(max(p, 0) + max(f, 0)) // page) - -(-max(p, 0) // page) for p, f in zip(past.tolist(), fresh.tolist())))
    pool = held + new + 3
    table, free = _tables(rng, past.tolist(), page, max_pages, pool)
    if short:
        free = free[:max(0, new - short)]
    tokens = int(np.maximum(fresh, 0).sum())
    max_tokens = max(0, tokens + slack)
    num_pages = pool if num_pages is None else num_pages
    want = append_loop(past, fresh, page, num_pages, free, table, max_tokens)
    rows = len(past) + 2  # the table may have more rows than the step has requests
    held_table = torch.full((rows, (pitch or max_pages)), -9, dtype=torch.int32, device="cuda")
    dev = held_table[:, :max_pages]
    dev[:len(past)] = torch.from_numpy(table).cuda()
    pages = lb.PageTable(dev, page, num_pages, max_tokens)
    for _ in range(2):  # the same step again changes nothing
        pages.append(torch.from_numpy(past).cuda(), torch.from_numpy(fresh).cuda(), torch.from_numpy(free.copy()).cuda())
        # what a row holds past its pages is not the definition's
        got = pages.table[:len(past)].cpu().numpy()
        np.testing.assert_array_equal(got, want[0])
        assert (held_table[len(past):] == -9).all() and (held_table[:, max_pages:] == -9).all()
        np.testing.assert_array_equal(pages.token_ptr.cpu().numpy(), want[1])
        np.testing.assert_array_equal(pages.lens.cpu().numpy(), want[2])
        np.testing.assert_array_equal(pages.slots.cpu().numpy(), want[3])
        np.testing.assert_array_equal(pages.positions.cpu().numpy(), want[4])
        assert int(pages.taken) == want[5] and int(pages.status) == want[6]
    return want


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("requests", [1, 2, 31, 256, 1025, 5000])
def test_append(requests, page):
    rng = np.random.default_rng(requests * page)
    past = rng.integers(0, 200, requests)
    fresh = np.where(rng.random(requests) < 0.5, 1, rng.integers(0, 40, requests))
    want = check_append(past, fresh, page, -(-240 // page), seed=requests)
    assert want[6] == 0
    want = check_append(past, fresh, page, -(-240 // page), short=1 + requests // 3, seed=requests, pitch=300)
    assert want[6] == 1 or int(want[5]) == 0


def test_append_page_edges():
    """Lengths at, before and past a page's end; nothing held; nothing new."""
    past = [0, 0, 0, 15, 16, 17, 31, 32, 15, 16, 0, 48]
    fresh = [0, 1, 16, 1, 1, 15, 2, 0, 17, 16, 49, 0]
    assert check_append(past, fresh, 16, 4)[6] == 0


def test_append_nothing():
    import torch
    import load_balanced_csr_gb300 as lb
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    pages = lb.PageTable(torch.zeros(4, 3, dtype=torch.int32, device="cuda"), 16, 10, 7)
    pages.append(e, e, e)
    assert pages.token_ptr.tolist() == [0] and int(pages.taken) == 0 and int(pages.status) == 0
    assert pages.slots.tolist() == [-1] * 7 and pages.positions.tolist() == [-1] * 7
    pages = lb.PageTable(torch.zeros(4, 3, dtype=torch.int32, device="cuda"), 16, 10, 0)
    pages.append(torch.full((2,), 16, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), e)
    assert pages.lens.tolist() == [16, 16] and int(pages.status) == 0


def test_append_refused_requests():
    # a row too short, at its very end, a past beyond the row, a negative length
    want = check_append([10, 30, 64, 100, -3, 5, 63], [60, 34, 0, 1, 4, -2, 1], 16, 4)
    assert want[6] == 2 | 8
    # fewer slots than tokens
    want = check_append([0, 5, 9], [10, 10, 10], 8, 4, slack=-7)
    assert want[6] == 4
    # pages outside the cache
    want = check_append([3, 5, 40], [10, 10, 10], 8, 8, num_pages=4)
    assert want[6] & 16


def test_append_long_prefill():
    """Many tokens for few requests, over many blocks."""
    check_append([1000, 0, 77], [70000, 0, 131071], 16, 9000, seed=4)


# ------------------------------------------------------------------ stores


def _cache(pages, page, heads, dim, dtype, layout, fill=float("nan")):
    """A cache of one of the layouts: token by token, head by head, padded, or with odd strides."""
    import torch
    dt = _torch_dtype(dtype)
    if layout == "heads":
        return torch.full((pages, heads, page, dim), fill, dtype=dt, device="cuda").transpose(1, 2)
    if layout == "padded":
        return torch.full((pages, page + 1, heads + 1, dim + 16), fill, dtype=dt, device="cuda")[:, :page, :heads, 8:dim + 8]
    if layout == "odd":
        return torch.full((pages, page, heads, dim + 1), fill, dtype=dt, device="cuda")[:, :, :, :dim]
    return torch.full((pages, page, heads, dim), fill, dtype=dt, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,page,layout", [
    (1, 1, 8, 1, "tokens"), (300, 8, 128, 16, "tokens"), (300, 8, 128, 16, "heads"), (97, 3, 72, 7, "padded"),
    (97, 3, 40, 7, "odd"), (50, 5, 33, 5, "tokens"), (1000, 1, 256, 64, "heads")])
def test_store(tokens, heads, dim, page, layout, dtype):
    import torch
    import load_balanced_csr_gb300 as lb
    rng = np.random.default_rng(tokens)
    pages = -(-tokens // page) + 2
    fused = torch.randn(tokens, 2 * heads + 1, dim, device="cuda").to(_torch_dtype(dtype))
    k, v = fused[:, :heads], fused[:, heads:2 * heads]
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    skipped = rng.random(tokens) < 0.2
    slots[skipped] = rng.choice([-1, -100, pages * page, 2 ** 31 - 1], int(skipped.sum()))
    kc, vc = (_cache(pages, page, heads, dim, dtype, layout, 3.0) for _ in range(2))
    wk, wv = kc.clone(), vc.clone()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            wk[s // page, s % page], wv[s // page, s % page] = k[i], v[i]
    lb.paged_store(k, v, kc, vc, torch.from_numpy(slots).cuda())
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


# ------------------------------------------------------------------ attention


class Requests:
    """Caches holding NaN wherever no request's position is, tables holding
    pages far outside wherever no request reaches, and queries."""

    def __init__(self, lens, q_heads, kv_heads, dim, page, dtype, layout="tokens", seed=0, extra_pages=3):
        import torch
        rng = np.random.default_rng(seed)
        dt = _torch_dtype(dtype)
        self.lens_host, self.dtype = list(lens), dtype
        held = [-(-n // page) for n in lens]
        pages = sum(held) + extra_pages
        width = max(held + [1]) + 2
        order = rng.permutation(pages)
        table = np.full((len(lens), width), 2 ** 30, np.int32)
        self.k, self.v = (_cache(pages, page, kv_heads, dim, dtype, layout) for _ in range(2))
        at, where = 0, []
        for b, n in enumerate(lens):
            table[b, :held[b]] = order[at:at + held[b]]
            pos = np.arange(n)
            where.append(table[b, pos // page].astype(np.int64) * page + pos % page)
            at += held[b]
        where = torch.from_numpy(np.concatenate(where) if where else np.zeros(0, np.int64)).cuda()
        for c in (self.k, self.v):
            c[where // page, where % page] = torch.randn(where.numel(), kv_heads, dim, device="cuda").to(dt)
        self.q = (1.5 * torch.randn(len(lens), q_heads, dim, device="cuda")).to(dt)
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32, device="cuda")
        self.shape = (q_heads, kv_heads, dim, page)

    def attention(self, max_batch=None):
        import load_balanced_csr_gb300 as lb
        hq, hk, dim, _ = self.shape
        return lb.PagedAttention(max_batch or len(self.lens_host), hq, hk, dim, _torch_dtype(self.dtype))

    def check(self, out, lse, scale):
        """Every request and head against the definition in 64 bits."""
        import torch
        hq, hk, dim, page = self.shape
        u = U[self.dtype]
        for b, n in enumerate(self.lens_host):
            if n == 0:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all(), f"request {b} of length 0"
                continue
            pos = torch.arange(n, device="cuda")
            at, inside = self.table[b].long()[pos // page], pos % page
            k = self.k[at, inside].double().repeat_interleave(hq // hk, 1)  # (n, hq, dim)
            v = self.v[at, inside].double().repeat_interleave(hq // hk, 1)
            q = self.q[b].double()
            s = torch.einsum("hd,nhd->hn", q, k) * scale
            want_lse = torch.logsumexp(s, 1)
            p = torch.exp(s - want_lse[:, None])
            want = torch.einsum("hn,nhd->hd", p, v)
            spread = torch.einsum("hn,nhd->hd", p, v.abs())
            size = abs(scale) * torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1)
            e = 2 * (dim + 8) * V * size + 2.0 ** -20 * (1 + (s - want_lse[:, None]).abs().amax(1))
            bound = (2 * e + 2 * n * V + u)[:, None] * spread + u * want.abs() + TINY[self.dtype]
            err = (out[b].double() - want).abs()
            assert bool((err <= bound).all()), f"request {b} (length {n}): out {float((err - bound).max())} over its bound"
            err = (lse[b].double() - want_lse).abs()
            assert bool((err <= e + n * V + 4 * V * want_lse.abs()).all()), f"request {b} (length {n}): lse off by {float(err.max())}"


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 0, 255, 257, 1000, 3]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("q_heads,kv_heads,dim,page,layout", [
    (8, 8, 64, 16, "tokens"), (8, 2, 128, 16, "tokens"), (32, 4, 128, 64, "heads"), (16, 1, 128, 1, "tokens"),
    (7, 1, 72, 7, "padded"), (6, 3, 8, 5, "tokens"), (20, 1, 96, 16, "heads"), (48, 1, 64, 33, "tokens"),
    (4, 2, 256, 16, "tokens"), (12, 4, 192, 128, "padded"), (10, 2, 136, 3, "tokens"), (2, 1, 16, 17, "heads")])
def test_attention(q_heads, kv_heads, dim, page, layout, dtype):
    r = Requests(LENS, q_heads, kv_heads, dim, page, dtype, layout, seed=dim + page)
    attend = r.attention()
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens)
    assert attend.device_status() == 0
    r.check(out, lse, dim ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[20011], [70000, 1, 0, 40000], [1] * 700, [0] * 5 + [5000] + [0] * 5, [0, 0, 0],
                                  [9] * 3000 + [4000], [64 * i for i in range(64)]],
                         ids=["one", "two long", "many of one", "one among empty", "empty", "thousands", "steps"])
def test_attention_lengths(lens, dtype):
    """Requests cut between many warps and blocks, and many requests in one."""
    r = Requests(lens, 8, 2, 64, 16, dtype, seed=len(lens))
    attend = r.attention()
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens, scale=0.2)
    assert attend.device_status() == 0
    r.check(out, lse, 0.2)
    for _ in range(3):  # the same call again gives the same bits
        again, lse2 = attend(r.q, r.k, r.v, r.table, r.lens, scale=0.2)
        import torch
        assert torch.equal(again, out) and torch.equal(lse2, lse)


def test_attention_one_object_many_shapes():
    """One workspace through batches of all sizes, in any order."""
    whole = Requests([300, 0, 5000, 17, 64, 900, 1, 2500], 4, 2, 64, 16, "bf16", seed=9)
    attend = whole.attention(max_batch=20)
    for n in (8, 1, 5, 0, 8, 3):
        out, lse = attend(whole.q[:n], whole.k, whole.v, whole.table, whole.lens)
        part = Requests.__new__(Requests)
        part.__dict__.update(whole.__dict__, lens_host=whole.lens_host[:n])
        part.check(out, lse, 64 ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_views_and_streams(dtype):
    """Queries out of a fused projection, outputs into a wider buffer, on another stream."""
    import torch
    r = Requests([500, 3, 0, 129], 6, 2, 64, 16, dtype, seed=2)
    fused = torch.full((4, 9, 65), float("nan"), dtype=r.q.dtype, device="cuda")  # rows at odd offsets
    fused[:, 1:7, 1:] = r.q
    wide = torch.full((4, 8, 80), 7.0, dtype=r.q.dtype, device="cuda")
    attend = r.attention()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = attend(fused[:, 1:7, 1:], r.k, r.v, r.table, r.lens, out=wide[:, 1:7, 3:67], stream=s)
    s.synchronize()
    r.check(out, lse, 64 ** -0.5)
    assert (wide[:, 0] == 7).all() and (wide[:, 7] == 7).all() and (wide[:, :, :3] == 7).all() and (wide[:, :, 67:] == 7).all()


def test_objects_made_on_a_busy_stream():
    """Made while the current stream is still at work, used on another at once."""
    import torch
    import load_balanced_csr_gb300 as lb
    r = Requests([60000, 3], 4, 2, 64, 16, "bf16", seed=4)
    attend = r.attention()
    attend(r.q, r.k, r.v, r.table, r.lens)  # a kernel's first call may wait for the device
    attend._workspace.fill_(0x7f)  # what the memory that the next object takes may hold
    attend._status.fill_(64)
    del attend
    past, fresh = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([3, 20], [1, 30]))
    free = torch.arange(4, 40, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, -1, -1, -1], [1, 2, -1, -1]], dtype=torch.int32, device="cuda")
    lb.PageTable(table.clone(), 16, 64, 40).append(past, fresh, free)
    s = torch.cuda.Stream()
    out, lse = torch.empty_like(r.q), torch.empty(2, 4, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    attend = r.attention()
    attend(r.q, r.k, r.v, r.table, r.lens, out=out, lse=lse, stream=s)
    torch.cuda._sleep(100_000_000)
    pages = lb.PageTable(table, 16, 64, 40)
    pages.append(past, fresh, free, stream=s)
    s.synchronize()
    flags, taken = attend.device_status(), int(pages.taken)
    r.check(out, lse, 64 ** -0.5)
    assert flags == 0 and taken == 2 and int(pages.status) == 0 and pages.lens.tolist() == [4, 50]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 7), (128, 64), (128, 5), (96, 16)])
def test_attention_caches_of_two_layouts(dim, page, dtype):
    """Keys kept token by token, values head by head."""
    r = Requests([77, 0, 300, 5, 1024], 6, 2, dim, page, dtype, seed=dim)
    held = r.v
    r.v = _cache(held.shape[0], page, 2, dim, dtype, "heads")
    r.v.copy_(held)
    assert r.v.stride() != r.k.stride()
    attend = r.attention()
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens)
    assert attend.device_status() == 0
    r.check(out, lse, dim ** -0.5)
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens, scale=-0.11)  # a negative scale turns the scores around
    r.check(out, lse, -0.11)
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens, scale=0.0)    # no scale: the values' mean
    r.check(out, lse, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens", [[33, 900], [40000]], ids=["short", "cut"])
@pytest.mark.parametrize("q_heads", [4, 32])
def test_attention_scores_past_24_bits(q_heads, lens, dtype):
    """Scores so large that rounding them moves them by many units: the
    highest one still has weight 1.  All products but one are zero and the
    highest score is far above the others, so the output is that position's
    value (the weight's own error, the sum and the division: 8 V), and the
    log-sum the score (its scale and units: 8 V)."""
    import torch
    r = Requests(lens, q_heads, 2, 64, 16, dtype, seed=5)
    big = {"f32": 1e15, "bf16": 1e15, "f16": 2.0 ** 15}[dtype]
    r.q.zero_()
    r.q[:, :, 0] = big * (1 + torch.rand(len(lens), q_heads, device="cuda") / 2).to(r.q.dtype)
    top = []
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        at = r.table[b].long()[pos // 16]
        r.k[at, pos % 16, :, 0] = big / 2
        top.append((int(r.table[b, (n // 3) // 16]), n // 3 % 16))
        r.k[top[b]][:, 0] = big
    attend = r.attention()
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens, scale=0.3)
    assert attend.device_status() == 0
    for b in range(len(lens)):
        v = r.v[top[b]].double().repeat_interleave(q_heads // 2, 0)
        assert bool(((out[b].double() - v).abs() <= (U[dtype] + 8 * V) * v.abs() + TINY[dtype]).all())
        score = 0.3 * r.q[b, :, 0].double() * r.k[top[b]][:, 0].double().repeat_interleave(q_heads // 2)
        assert bool(((lse[b].double() - score).abs() <= 8 * V * score).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("q_heads,dim", [(4, 64), (32, 128)])
@pytest.mark.parametrize("above", [17.0, 19.0])
def test_attention_one_score_far_above(above, q_heads, dim, dtype):
    """One position with most of the weight and a value of zero: the output is
    what the others, of weights around 2^-24 and 2^-27, add up to."""
    import torch
    lens = [3000, 700, 20000]
    r = Requests(lens, q_heads, 2, dim, 16, dtype, seed=6)
    r.q[:, :, 0] = 16.0
    scale = dim ** -0.5
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        at = r.table[b].long()[pos // 16]
        r.k[at, pos % 16] = (r.k[at, pos % 16].float() / 4).to(r.k.dtype)
        r.k[at, pos % 16, :, 0] = 0.0
        r.v[at, pos % 16] = (r.v[at, pos % 16].float() + 3).to(r.v.dtype)
        first = int(r.table[b, 0])
        r.k[first, 0, :, 0] = above / (16 * scale)
        r.v[first, 0] = 0.0
    out, lse = r.attention()(r.q, r.k, r.v, r.table, r.lens)
    r.check(out, lse, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_extreme_scores(dtype):
    """Scores hundreds apart: the running maximum moves late, early and never;
    a score of minus infinity weighs nothing; NaN and infinity in V show up
    where they are weighed, and only there."""
    import torch
    for order in (1, -1):
        r = Requests([400, 400], 4, 2, 64, 16, dtype, seed=1)
        n = torch.arange(400, device="cuda")
        ramp = (n if order > 0 else 399 - n).to(r.k.dtype) / 8
        for b in range(2):
            at = r.table[b].long()[n // 16]
            r.k[at, n % 16, :, 0] = ramp[:, None]
        r.q[:, :, 0] = 40.0
        out, lse = r.attention()(r.q, r.k, r.v, r.table, r.lens)
        r.check(out, lse, 64 ** -0.5)
    r = Requests([40, 40], 4, 2, 64, 16, dtype, seed=1)
    r.q[:, :, 0] = 1.0
    page, inside = int(r.table[0, 1]), 5  # position 21 of request 0
    r.k[page, inside, :, 0] = -float("inf")
    r.k[page, inside, :, 1:] = 0.0
    out, lse = r.attention()(r.q, r.k, r.v, r.table, r.lens)
    keep = [i for i in range(40) if i != 21]
    pos = torch.tensor(keep, device="cuda")
    at = r.table[0].long()[pos // 16]
    k = r.k[at, pos % 16].double().repeat_interleave(2, 1)
    v = r.v[at, pos % 16].double().repeat_interleave(2, 1)
    s = torch.einsum("hd,nhd->hn", r.q[0].double(), k) / 8
    want = torch.einsum("hn,nhd->hd", torch.softmax(s, 1), v)
    assert bool(((out[0].double() - want).abs() <= 4 * U[dtype] * v.abs().amax() + 1e-4).all())
    r.v[int(r.table[1, 0]), 0, 0, 3] = float("nan")
    out, _ = r.attention()(r.q, r.k, r.v, r.table, r.lens)
    bad = torch.isnan(out)
    assert bool(bad[1, :2, 3].all()) and int(bad.sum()) == 2


def test_attention_flags():
    """A page outside the cache is left out, a length past its row is cut."""
    import torch
    r = Requests([64, 40], 2, 1, 64, 16, "bf16", seed=3)
    r.table[0, 2] = 2 ** 30
    attend = r.attention()
    out, lse = attend(r.q, r.k, r.v, r.table, r.lens)
    assert attend.device_status() == 1
    assert bool(torch.isfinite(out).all())
    r2 = Requests([64, 40], 2, 1, 64, 16, "bf16", seed=3)
    attend = r2.attention()
    lens = torch.tensor([1000, -4], dtype=torch.int32, device="cuda")
    out, lse = attend(r2.q, r2.k, r2.v, r2.table[:, :4].contiguous(), lens)
    assert attend.device_status() == 2
    r2.lens_host = [64, 0]
    r2.check(out, lse, 64 ** -0.5)


def test_cache_past_32_bit_offsets():
    """Pages past 2^31 elements of the cache: stored to and read from."""
    import torch
    import load_balanced_csr_gb300 as lb
    heads, dim, page = 8, 128, 64
    pages = 2 ** 31 // (heads * dim * page) + 40
    kc, vc = (torch.empty(pages, page, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 150
    table = torch.tensor([[pages - 1, 0, pages - 3, -1]], dtype=torch.int32, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).int()
    k, v = (torch.randn(n, heads, dim, device="cuda").bfloat16() for _ in range(2))
    lb.paged_store(k, v, kc, vc, slots)
    assert torch.equal(kc[pages - 1], k[:64]) and torch.equal(vc[pages - 3][:22], v[128:])
    r = Requests.__new__(Requests)
    r.lens_host, r.dtype, r.shape = [n], "bf16", (16, heads, dim, page)
    r.k, r.v, r.table = kc, vc, table
    r.q = torch.randn(1, 16, dim, device="cuda").bfloat16()
    out, lse = lb.PagedAttention(1, 16, heads, dim, torch.bfloat16)(r.q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    r.check(out, lse, dim ** -0.5)


def test_refusals():
    import torch
    import load_balanced_csr_gb300 as lb
    for heads in ((6, 4, 64), (4, 0, 64), (4, 2, 60), (4, 2, 264), (4, 2, 0)):
        with pytest.raises(lb.SpmvError):
            lb.PagedAttention(2, *heads, torch.bfloat16)
    with pytest.raises(TypeError):
        lb.PagedAttention(2, 4, 2, 64, torch.float64)
    r = Requests([5, 9], 4, 2, 64, 16, "bf16")
    attend = r.attention()
    with pytest.raises(TypeError):
        attend(r.q.float(), r.k, r.v, r.table, r.lens)
    with pytest.raises(TypeError):
        attend(r.q, r.k.float(), r.v, r.table, r.lens)
    with pytest.raises(ValueError):
        attend(r.q[:, :2], r.k, r.v, r.table, r.lens)
    with pytest.raises(ValueError):
        attend(torch.cat([r.q, r.q]), r.k, r.v, r.table, r.lens)
    with pytest.raises(ValueError):
        attend(r.q, r.k, r.v[:-1], r.table, r.lens)
    with pytest.raises(ValueError):
        attend(r.q, r.k, r.v, r.table[:1], r.lens)
    with pytest.raises(TypeError):
        attend(r.q, r.k, r.v, r.table.long(), r.lens)
    with pytest.raises(ValueError):
        attend(r.q, r.k, r.v, r.table, r.lens[:1])
    odd = _cache(8, 16, 2, 64, "bf16", "odd")
    with pytest.raises(lb.SpmvError):
        attend(r.q, odd, odd, r.table, r.lens)
    with pytest.raises(TypeError):
        lb.PageTable(r.table.long(), 16, 8, 4)
    pages = lb.PageTable(r.table, 16, 8, 4)
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pages.append(one, one, one)
    with pytest.raises(ValueError):
        pages.append(one[:2], one[:1], one)
    with pytest.raises(TypeError):
        pages.append(one[:2].long(), one[:2], one)
    with pytest.raises(lb.SpmvError):
        lb.PageTable(r.table, 0, 8, 4).append(one[:2], one[:2], one)
    with pytest.raises(lb.SpmvError):
        lb.PageTable(r.table, 2 ** 16, 2 ** 15, 4).append(one[:2], one[:2], one)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lb.paged_store(k, k[:2], r.k, r.v, one)
    with pytest.raises(TypeError):
        lb.paged_store(k, k, r.k.float(), r.v, one)
    with pytest.raises(TypeError):
        lb.paged_store(k, k, r.k, r.v, one.long())
    with pytest.raises(ValueError):
        lb.paged_store(k, k, r.k, r.v, one[:2])
