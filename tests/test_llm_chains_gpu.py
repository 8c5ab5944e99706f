"""Steps of the operators one behind the other with no wait between them, each
kernel launched while the one before it runs: what a step reads was written
by the kernels just before, over many blocks.  Against the definitions in 64
bits, with 32-bit elements: an attention output is an average of values with
weights off by at most 2 e + 2 n v (v = 2^-24, e = 2 (dim + 8) v max|q||k|
scale + 2^-20 (1 + max|s - lse|)), plus its own rounding."""
import pytest

pytestmark = pytest.mark.gpu

V = 2.0 ** -24


@pytest.mark.parametrize("page", [1, 16])
def test_append_store_attend(page):
    """Prompts of thousands of tokens (an append of several blocks, each
    reading table rows that others extend), stored and attended to at once."""
    import torch
    import load_balanced_csr_gb300 as lb
    torch.manual_seed(page)
    steps, b, hq, hk, d, room = 6, 7, 4, 2, 32, 20000
    i32 = dict(dtype=torch.int32, device="cuda")
    fresh = [torch.tensor([(977 * (s + 1) * (r + 3)) % 3001 if (s + r) % 4 else r % 2 for r in range(b)], **i32) for s in range(steps)]
    lens = torch.stack(fresh).cumsum(0)
    past = [torch.zeros(b, **i32)] + [lens[s].int() for s in range(steps - 1)]
    width = -(-int(lens.max()) // page) + 1
    num_pages = b * width
    order = torch.randperm(num_pages).to(**i32)
    table = torch.full((b, width), -1, **i32)
    # what the free list holds when each step begins: the steps before took a prefix
    held = [int(((x.long() + page - 1) // page).sum()) for x in past]
    free = [order[n:] for n in held]
    k, v = (torch.randn(steps, room, hk, d, device="cuda") for _ in range(2))
    q = torch.randn(steps, b, hq, d, device="cuda")
    assert all(int(f.sum()) <= room for f in fresh) and max(int(f.sum()) for f in fresh) > 2 * 4096
    kc, vc = (torch.full((num_pages, page, hk, d), float("nan"), device="cuda") for _ in range(2))
    pages, attend = lb.PageTable(table, page, num_pages, room), lb.PagedAttention(b, hq, hk, d, torch.float32)
    outs = [(torch.empty(b, hq, d, device="cuda"), torch.empty(b, hq, device="cuda")) for _ in range(steps)]
    torch.cuda.synchronize()
    for s in range(steps):
        pages.append(past[s], fresh[s], free[s])
        lb.paged_store(k[s], v[s], kc, vc, pages.slots)
        attend(q[s], kc, vc, table, pages.lens, out=outs[s][0], lse=outs[s][1])
    assert attend.device_status() == 0 and int(pages.status) == 0
    assert torch.equal(pages.lens.long(), lens[-1])
    starts = [torch.cat([f.new_zeros(1), f.cumsum(0)]).tolist() for f in fresh]
    for r in range(b):
        kk, vv = (torch.cat([x[s, starts[s][r]:starts[s][r + 1]] for s in range(steps)]).double().repeat_interleave(hq // hk, 1)
                  for x in (k, v))
        for s in range(steps):
            n, (out, lse) = int(lens[s, r]), outs[s]
            if n == 0:
                assert (out[r] == 0).all() and (lse[r] == -float("inf")).all()
                continue
            scores = torch.einsum("hd,nhd->hn", q[s, r].double(), kk[:n]) * d ** -0.5
            want_lse = torch.logsumexp(scores, 1)
            p = torch.exp(scores - want_lse[:, None])
            want, spread = torch.einsum("hn,nhd->hd", p, vv[:n]), torch.einsum("hn,nhd->hd", p, vv[:n].abs())
            size = d ** -0.5 * torch.einsum("hd,nhd->hn", q[s, r].double().abs(), kk[:n].abs()).amax(1)
            e = 2 * (d + 8) * V * size + 2.0 ** -20 * (1 + (scores - want_lse[:, None]).abs().amax(1))
            bound = (2 * e + 2 * n * V)[:, None] * spread + V * want.abs() + 2.0 ** -149
            assert bool(((out[r].double() - want).abs() <= bound).all()), (s, r, n)
            assert bool(((lse[r].double() - want_lse).abs() <= e + n * V + 4 * V * want_lse.abs()).all()), (s, r, n)


@pytest.mark.parametrize("tokens,k", [(700, 3), (50000, 4)])  # one launch of a cluster; a counting launch before it
def test_build_dispatch_combine(tokens, k):
    """One route rebuilt for new ids again and again.  Weights are powers of
    two that add up to 1 and every token keeps all choices, so combine of
    dispatch gives the token's row, up to the sum's roundings."""
    import torch
    import load_balanced_csr_gb300 as lb
    torch.manual_seed(k)
    steps, experts, hidden = 8, 37, 24
    ids = [torch.randint(0, experts, (tokens, k), device="cuda") for _ in range(steps)]
    x = torch.randn(steps, tokens, hidden, device="cuda")
    w = torch.tensor([0.5 ** (j + 1) for j in range(k - 1)] + [0.5 ** (k - 1)], device="cuda").expand(tokens, k).contiguous()
    route = lb.ExpertRoute(tokens, k, experts)
    xs, y = torch.empty(steps, tokens * k, hidden, device="cuda"), torch.empty(steps, tokens, hidden, device="cuda")
    torch.cuda.synchronize()
    for s in range(steps):
        route.build(ids[s])
        route.dispatch(x[s], out=xs[s])
        route.combine(xs[s], w, out=y[s])
    torch.cuda.synchronize()
    assert bool(((y - x).abs() <= (k + 1) * V * x.abs()).all())
    for s in range(steps):
        entry = torch.argsort(ids[s].reshape(-1), stable=True)
        assert torch.equal(xs[s], x[s][entry // k])


def _from_two_threads(*calls, times=4000):
    """Each call made `times` times by a host thread of its own; the statuses other than 0."""
    import threading
    start, failed = threading.Barrier(len(calls)), []

    def work(call):
        start.wait()
        for _ in range(times):
            status = call()
            if status:
                failed.append(status)
                return

    threads = [threading.Thread(target=work, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


def test_builds_from_two_host_threads():
    """Routes of 2,048 and of 700 experts, whose kernels need different
    amounts of shared memory, built on streams of their own."""
    import torch
    import load_balanced_csr_gb300 as lb
    L, n = lb.lib(), 64
    calls, routes = [], []
    for experts in (2048, 700):
        ids = torch.randint(0, experts, (n, 1), device="cuda", dtype=torch.int32)
        route, stream = lb.ExpertRoute(n, 1, experts).build(ids), torch.cuda.Stream()
        routes.append((route, ids, stream))
        ptr, entry, slot = (x.data_ptr() for x in (route.expert_ptr, route.entry, route.slot))
        args = (n, 1, experts, ids.data_ptr(), 4, 1, ptr, entry, slot, None, 0, stream.cuda_stream)
        calls.append(lambda args=args: L.spmv_route_build(*args))
    torch.cuda.synchronize()
    failed = _from_two_threads(*calls)
    torch.cuda.synchronize()
    assert not failed, lb.lib().spmv_last_error()
    for route, ids, _ in routes:
        assert torch.equal(route.entry.long(), torch.argsort(ids[:, 0], stable=True))


def test_appends_from_two_host_threads():
    """Steps of 4,096 and of 4,020 requests, as above."""
    import torch
    import load_balanced_csr_gb300 as lb
    L = lb.lib()
    calls, tables = [], []
    for requests in (4096, 4020):
        i32 = dict(dtype=torch.int32, device="cuda")
        past, fresh, free = torch.zeros(requests, **i32), torch.ones(requests, **i32), torch.arange(requests, **i32)
        pages, stream = lb.PageTable(torch.full((requests, 1), -1, **i32), 16, requests, requests), torch.cuda.Stream()
        tables.append((pages, past, fresh, free, stream))
        args = (requests, past.data_ptr(), fresh.data_ptr(), 16, requests, free.data_ptr(), requests, pages.table.data_ptr(),
                1, 1, requests, *pages._outputs, stream.cuda_stream)
        calls.append(lambda args=args: L.spmv_pages_append(*args))
    torch.cuda.synchronize()
    failed = _from_two_threads(*calls)
    torch.cuda.synchronize()
    assert not failed
    for pages, _, fresh, free, _ in tables:
        assert int(pages.status) == 0 and torch.equal(pages.table[:, 0], free) and torch.equal(pages.slots, free * 16)


def test_graph_with_copies_and_a_side_stream_between():
    """Captured with copies, memsets and another stream's work before the
    kernels: an edge to what is not a kernel, or is on another stream, is a
    whole dependency."""
    import torch
    import load_balanced_csr_gb300 as lb
    torch.manual_seed(4)
    tokens, k, experts, hidden = 900, 2, 11, 64
    source = [torch.randint(0, experts, (tokens, k), device="cuda") for _ in range(4)]
    x, w = torch.randn(tokens, hidden, device="cuda"), torch.full((tokens, k), 0.5, device="cuda")
    now, ids, row = source[0].clone(), torch.zeros_like(source[0]), torch.zeros_like(x)
    route, side = lb.ExpertRoute(tokens, k, experts), torch.cuda.Stream()
    xs, y = torch.empty(tokens * k, hidden, device="cuda"), torch.empty(tokens, hidden, device="cuda")

    def step():
        ids.zero_()
        ids.copy_(now)
        route.build(ids)
        row.copy_(x)
        route.dispatch(row, out=xs)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y.zero_()
            route.combine(xs, w, out=y)
        torch.cuda.current_stream().wait_stream(side)
        route.dispatch(y, out=xs)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in source:
        now.copy_(s)
        x.normal_()
        graph.replay()
        entry = torch.argsort(s.reshape(-1), stable=True)
        assert torch.equal(y, x)  # x / 2 + x / 2 is exact
        assert torch.equal(xs, x[entry // k]) and torch.equal(route.entry.long(), entry)
