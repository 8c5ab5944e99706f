"""The operators together: the example's decoding steps against the same layer
in plain 64-bit torch over contiguous caches, and a chain of them captured in a
CUDA graph and replayed on new inputs."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_decode_step", os.path.join(ROOT, "examples", "moe_decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_match_a_plain_layer():
    """32-bit weights and caches, so that the router's choices agree; each
    output carries a few thousand 32-bit roundings of values near 1."""
    import torch
    requests = 9
    layer = _example().Layer(requests=requests, hidden=96, q_heads=6, kv_heads=2, head_dim=32, experts=7, top_k=3,
                             expert_hidden=40, page_size=4, num_pages=64, max_pages=8, dtype=torch.float32)
    wide = {name: getattr(layer, name).double() for name in ("qkv", "out", "router", "up", "down")}
    keys, values = [], []
    for s in range(14):
        x = torch.randn(requests, 96, device="cuda")
        got = layer.step(x)
        xw = x.double()
        heads = (xw @ wide["qkv"]).view(requests, 10, 32)
        q = heads[:, :6].reshape(requests, 2, 3, 32)
        keys.append(heads[:, 6:8]), values.append(heads[:, 8:])
        k, v = torch.stack(keys, 1), torch.stack(values, 1)  # (request, position, head, element)
        p = torch.softmax(torch.einsum("bhgd,bthd->bhgt", q, k) * 32 ** -0.5, -1)
        xw = xw + torch.einsum("bhgt,bthd->bhgd", p, v).reshape(requests, -1) @ wide["out"]
        top, ids = torch.topk(xw @ wide["router"], 3, dim=1)
        up = torch.relu(torch.einsum("bh,bkhf->bkf", xw, wide["up"][ids]))
        y = xw + (torch.einsum("bkf,bkfh->bkh", up, wide["down"][ids]) * torch.softmax(top, 1)[:, :, None]).sum(1)
        assert layer.lens.tolist() == [s + 1] * requests
        assert float((got.double() - y).abs().max()) <= 4096 * 2.0 ** -24 * float(y.abs().max())
    assert int(layer.pages.status) == 0 and layer.attend.device_status() == 0


def test_chain_in_a_cuda_graph():
    """append, store, attention, build, dispatch, combine: captured once,
    replayed for other lengths, pages, tokens and experts."""
    import torch
    import load_balanced_csr_gb300 as lb
    b, hq, hk, d, page, pages = 6, 8, 2, 64, 16, 40
    i32 = dict(dtype=torch.int32, device="cuda")
    table, free = torch.full((b, 16), -1, **i32), torch.arange(pages, **i32)
    past, fresh = torch.zeros(b, **i32), torch.ones(b, **i32)
    kc, vc = (torch.zeros(pages, page, hk, d, device="cuda") for _ in range(2))
    q, k, v = torch.zeros(b, hq, d, device="cuda"), torch.zeros(64, hk, d, device="cuda"), torch.zeros(64, hk, d, device="cuda")
    ids, w, x = torch.zeros(b, 2, **i32), torch.zeros(b, 2, device="cuda"), torch.zeros(b, 40, device="cuda")
    tables = lb.PageTable(table, page, pages, max_tokens=64)
    attend, route = lb.PagedAttention(b, hq, hk, d, torch.float32), lb.ExpertRoute(b, 2, 5)

    def chain():
        tables.append(past, fresh, free)
        lb.paged_store(k, v, kc, vc, tables.slots)
        out, lse = attend(q, kc, vc, table, tables.lens)
        route.build(ids)
        return out, lse, route.combine(route.dispatch(x), w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outputs = chain()
    for seed in range(3):
        torch.manual_seed(seed)
        past.zero_(), table.fill_(-1), kc.fill_(float("nan")), vc.fill_(float("nan"))
        fresh.copy_(torch.randint(0, 11, (b,)))
        free.copy_(torch.randperm(pages))
        for t in (q, k, v, w, x):
            t.normal_()
        ids.copy_(torch.randint(-1, 5, (b, 2)))
        graph.replay()
        out, lse, y = (o.clone() for o in outputs)
        n = fresh.tolist()
        at = 0
        for r in range(b):
            if n[r]:
                kk, vv = (t[at:at + n[r]].double().repeat_interleave(hq // hk, 1) for t in (k, v))
                p = torch.softmax(torch.einsum("hd,nhd->hn", q[r].double(), kk) / 8, 1)
                want = torch.einsum("hn,nhd->hd", p, vv)
                assert float((out[r].double() - want).abs().max()) <= 2048 * 2.0 ** -24 * float(vv.abs().max())
            else:
                assert (out[r] == 0).all()
            at += n[r]
        want = ((ids >= 0) * w).sum(1, keepdim=True) * x
        mag = (w.abs().sum(1, keepdim=True) * x.abs())
        assert bool(((y - want).abs() <= 6 * 2.0 ** -24 * mag + 1e-37).all())
    assert attend.device_status() == 0 and int(tables.status) == 0
