"""Cases that time the language-model operators: routing to experts, page tables, the paged cache and its attention.

Five kinds of case, each one pass through one operator as a program calls it:

  route   tokens sorted by expert, their rows gathered, and the experts' rows combined back with the routers' weights (serving)
  train   the same and its gradients: of the tokens, the experts' rows and the weights
  pages   block tables and slot maps of a step, from the requests' lengths
  store   a step's keys and values written into the paged cache by slot
  attend  attention of one new token per request over the paged cache

`own` chooses the framework's kernels; otherwise the plain forms below, in elementary torch operations, run.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a small decode batch, 8 experts a token: latency counts
        {"name": "route decode 64x2048", "op": "route", "tokens": 64, "k": 8, "experts": 128, "hidden": 2048, "dtype": "bf16", "ids": "i64", "drop": 0.0},
        # a prefill of 8,192 tokens, 8 of 128 experts
        {"name": "route prefill 8192x4096", "op": "route", "tokens": 8192, "k": 8, "experts": 128, "hidden": 4096, "dtype": "bf16", "ids": "i64", "drop": 0.0},
        # a training micro-batch, 2 of 16 experts
        {"name": "train 16384x4096 top 2", "op": "train", "tokens": 16384, "k": 2, "experts": 16, "hidden": 4096, "dtype": "bf16", "ids": "i32", "drop": 0.0},
        # 32-bit training, rows of an odd length, a tenth of the choices dropped (a capacity, or experts held elsewhere)
        {"name": "train odd 2999x1001 f32", "op": "train", "tokens": 2999, "k": 6, "experts": 60, "hidden": 1001, "dtype": "f32", "ids": "i32", "drop": 0.1},
        # a decode step of 256 requests: one token each, a page taken now and then
        {"name": "pages decode 256", "op": "pages", "requests": 256, "past": 32768, "fresh": 1, "page": 16, "short": 0},
        # a large step of chunked prefills beside decodes: about a million tokens
        {"name": "pages prefill 2048", "op": "pages", "requests": 2048, "past": 8192, "fresh": 1024, "page": 64, "short": 0},
        # the new keys and values of that decode step
        {"name": "store decode 256", "op": "store", "tokens": 256, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "bf16", "pad": 0.0},
        # the keys and values of a prefill of 65,535 tokens, views of one fused projection, some of the map padding
        {"name": "store prefill 65535", "op": "store", "tokens": 65535, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "f16", "pad": 0.05},
        # one request with a long context
        {"name": "attend one long 131071", "op": "attend", "batch": 1, "longest": 131071, "spread": "one", "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # a serving batch of very uneven lengths, empty ones among them
        {"name": "attend ragged 128", "op": "attend", "batch": 128, "longest": 16384, "spread": "log", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "bf16"},
        # a few short requests, a key head for each query head: latency counts
        {"name": "attend short 4 f16", "op": "attend", "batch": 4, "longest": 300, "spread": "log", "q_heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "dtype": "f16"},
        # 32 bits, a head and a page of odd sizes
        {"name": "attend f32 16 odd", "op": "attend", "batch": 16, "longest": 5000, "spread": "even", "q_heads": 12, "kv_heads": 4, "dim": 72, "page": 7, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["route", "train", "pages", "store", "attend", "attend"])
    if op in ("route", "train"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        k, experts = rng.randint(1, 8), _log_int(rng, 8, 256)
        hidden = _log_int(rng, 32, 512) * 8 if rng.random() < 0.8 else _log_int(rng, 257, 4096)
        room = (1 << 26 if op == "train" else 1 << 27) // (hidden * (k + 1))
        return {"op": op, "tokens": _log_int(rng, 1, min(16384, room)), "k": k, "experts": experts, "hidden": hidden, "dtype": dtype,
                "ids": rng.choice(["i32", "i64"]), "drop": rng.choice([0.0, 0.0, 0.05, 0.5])}
    if op == "pages":
        requests = _log_int(rng, 1, 4096)
        return {"op": op, "requests": requests, "past": _log_int(rng, 16, 32768), "fresh": rng.choice([1, _log_int(rng, 2, max(2, min(2048, (1 << 20) // requests)))]),
                "page": rng.choice([1, 7, 16, 32, 64, 128]), "short": rng.choice([0, 0, _log_int(rng, 1, 200)])}
    if op == "store":
        heads, dim = rng.choice([1, 2, 5, 8, 16]), rng.choice([64, 72, 128, 192, 256])
        return {"op": op, "tokens": _log_int(rng, 1, min(65535, (1 << 26) // (heads * dim))), "kv_heads": heads, "dim": dim, "page": rng.choice([1, 7, 16, 64]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "pad": rng.choice([0.0, 0.05, 0.5])}
    batch, heads, dim = _log_int(rng, 1, 256), rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 80, 128, 128, 128, 192, 256])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    longest = min(131071, max(16, (1 << (26 if dtype == "f32" else 27)) // (batch * heads * dim)))
    return {"op": op, "batch": batch, "longest": _log_int(rng, 16, longest), "spread": rng.choice(["log", "even", "one"]),
            "q_heads": heads * rng.choice([1, 2, 4, 7, 8, 16]), "kv_heads": heads, "dim": dim, "page": rng.choice([1, 7, 16, 16, 64, 128]),
            "dtype": dtype}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _lengths(case, g):
    """Cache lengths of the requests of an attend case: all near the longest, spread evenly, or over the logarithm with some empty."""
    u = torch.rand(case["batch"], generator=g, device="cuda", dtype=torch.float64)
    top = case["longest"]
    if case["spread"] == "one":
        lens = torch.full_like(u, top) - (u * min(8, top - 1)).floor()
    elif case["spread"] == "even":
        lens = (u * (top + 1)).floor()
    else:
        lens = torch.exp(u * math.log(top + 1)).floor()
        lens[u < 0.03] = 0
    lens[0] = top
    return lens.to(torch.int32)


def prepare(case, seed):
    """What a program has in hand before the call."""
    return _PREPARE[case["op"]](case, _generator(seed))


def _prepare_route(case, g):
    t, k, e, h, dt = case["tokens"], case["k"], case["experts"], case["hidden"], DTYPES[case["dtype"]]
    # experts differ in how often they are chosen, as trained routers' do
    logits = _normal(g, t, e) + 0.7 * _normal(g, e)
    top, ids = torch.topk(logits, min(k, e), dim=1)
    weights = torch.softmax(top, dim=1)
    if case["drop"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < case["drop"], -1, ids)
    s = {"case": case, "ids": ids if case["ids"] == "i64" else ids.to(torch.int32), "weights": weights,
         "x": _normal(g, t, h, dtype=dt), "ys": _normal(g, t * k, h, dtype=dt)}
    if case["op"] == "train":
        s["dy"], s["dxs"] = _normal(g, t, h, dtype=dt), _normal(g, t * k, h, dtype=dt)
    return s


def _prepare_pages(case, g):
    r, p = case["requests"], case["page"]
    past = torch.exp(torch.rand(r, generator=g, device="cuda", dtype=torch.float64) * math.log(case["past"] + 1)).floor() - 1
    fresh = torch.ones(r, dtype=torch.float64, device="cuda")
    if case["fresh"] > 1:  # a tenth of the requests rest, a tenth decode, the others prefill a chunk, in any order
        u = (torch.arange(r, device="cuda", dtype=torch.float64) + 0.5) / r
        fresh = torch.where(u < 0.1, 0.0, torch.where(u < 0.2, 1.0, ((u - 0.2) / 0.8 * case["fresh"]).floor() + 1))
        fresh = fresh[torch.randperm(r, generator=g, device="cuda")]
    past, fresh = past.to(torch.int32), fresh.to(torch.int32)
    width = -(-(case["past"] + case["fresh"]) // p)
    held = (past + p - 1) // p
    need = (past + fresh + p - 1) // p - held
    pool = int(held.sum()) + int(need.sum()) + 16
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((r, width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None, :] < held[:, None]
    table[at] = order[: int(held.sum())]
    free = order[int(held.sum()):]
    free = free[: max(0, int(need.sum()) + 16 - (16 + case["short"] if case["short"] else 0))].contiguous()
    return {"case": case, "past": past, "fresh": fresh, "table": table, "free": free, "num_pages": pool, "tokens": int(fresh.sum())}


def _prepare_store(case, g):
    n, h, d, p, dt = case["tokens"], case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    fused = _normal(g, n, 2 * h, d, dtype=dt)
    pages = -(-n // p) + 3
    slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * p + torch.arange(p, device="cuda")[None, :]
    slots = slots.reshape(-1)[:n].to(torch.int32)
    if case["pad"]:
        slots = torch.where(torch.rand(n, generator=g, device="cuda") < case["pad"], -1, slots)
    return {"case": case, "k": fused[:, :h], "v": fused[:, h:], "slots": slots,
            "k_cache": torch.zeros(pages, p, h, d, dtype=dt, device="cuda"), "v_cache": torch.zeros(pages, p, h, d, dtype=dt, device="cuda")}


def _prepare_attend(case, g):
    b, hq, hk, d, p, dt = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    lens = _lengths(case, g)
    held = (lens.long() + p - 1) // p
    width = int(held.max())
    pages = int(held.sum()) + 2
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < held[:, None]] = torch.randperm(pages, generator=g, device="cuda")[: pages - 2].to(torch.int32)
    return {"case": case, "q": 2 * _normal(g, b, hq, d, dtype=dt), "lens": lens, "table": table, "scale": d ** -0.5,
            "k_cache": _normal(g, pages, p, hk, d, dtype=dt), "v_cache": _normal(g, pages, p, hk, d, dtype=dt)}


_PREPARE = {"route": _prepare_route, "train": _prepare_route, "pages": _prepare_pages, "store": _prepare_store, "attend": _prepare_attend}


def run(state):
    """One pass."""
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ the framework's operators


def _own_route(s):
    import load_balanced_csr_gb300 as lb

    c = s["case"]
    if "route" not in s:
        s["route"] = lb.ExpertRoute(c["tokens"], s["ids"].shape[1], c["experts"])
    r = s["route"].build(s["ids"])
    out = {"expert_ptr": r.expert_ptr, "entry": r.entry, "slot": r.slot, "xs": r.dispatch(s["x"]), "y": r.combine(s["ys"], s["weights"])}
    if c["op"] == "train":
        out["dys"], out["dw"] = r.combine_backward(s["dy"], s["ys"], s["weights"])
        out["dx"] = r.dispatch_backward(s["dxs"])
    return out


def _own_pages(s):
    import load_balanced_csr_gb300 as lb

    if "pages" not in s:
        s["pages"] = lb.PageTable(s["table"], s["case"]["page"], s["num_pages"], max_tokens=s["tokens"])
    p = s["pages"].append(s["past"], s["fresh"], s["free"])
    return {"table": p.table, "token_ptr": p.token_ptr, "lens": p.lens, "slots": p.slots, "positions": p.positions, "taken": p.taken}


def _own_store(s):
    import load_balanced_csr_gb300 as lb

    lb.paged_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import load_balanced_csr_gb300 as lb

    if "attention" not in s:
        c = s["case"]
        s["attention"] = lb.PagedAttention(c["batch"], c["q_heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]])
    out, lse = s["attention"](s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=s["scale"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ their plain forms


def _plain_route(s):
    c, x, ids, w = s["case"], s["x"], s["ids"], s["weights"]
    (t, k), e, h = ids.shape, c["experts"], c["hidden"]
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(t * k, device="cuda")
    kept = key < e
    ptr = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    ptr[1:] = torch.cumsum((key[:, None] == torch.arange(e, device="cuda")).sum(0), 0)
    slot = torch.where(kept, place, -1 - place)
    live = kept[order][:, None]
    xs = torch.where(live, x[order // k], 0)
    keep = kept.reshape(t, k, 1)
    rows = torch.where(keep, s["ys"][place].reshape(t, k, h).float(), 0)
    y = (rows * w[:, :, None]).sum(1).to(x.dtype)
    out = {"expert_ptr": ptr, "entry": order.to(torch.int32), "slot": slot.to(torch.int32).reshape(t, k), "xs": xs, "y": y}
    if c["op"] == "train":
        dy = s["dy"].float()
        out["dys"] = torch.where(live, w.reshape(-1)[order][:, None] * dy[order // k], 0).to(x.dtype)
        out["dw"] = (rows * dy[:, None, :]).sum(2)
        out["dx"] = torch.where(keep, s["dxs"][place].reshape(t, k, h).float(), 0).sum(1).to(x.dtype)
    return out


def _plain_pages(s):
    p, table, past, fresh, free = s["case"]["page"], s["table"], s["past"].long(), s["fresh"].long(), s["free"]
    held = (past + p - 1) // p
    need = (past + fresh + p - 1) // p - held
    first = torch.cumsum(need, 0) - need
    served = (need == 0) | (first + need <= free.numel())  # a request whose pages do not all fit gets none of them
    end = torch.cumsum(fresh, 0)
    ptr = torch.zeros(past.numel() + 1, dtype=torch.int32, device="cuda")
    ptr[1:] = end
    i = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(end, i, right=True)
    position = past[r] + i - (end[r] - fresh[r])
    page = position // p
    new = page - held[r]
    ok = served[r]
    fetched = torch.cat([free, free.new_zeros(1)])[torch.where(ok & (new >= 0), first[r] + new, free.numel())]
    there = torch.where(new >= 0, fetched, table[r, page])
    table[r, page] = torch.where(ok, there, table[r, page])
    slots = torch.where(ok, there.long() * p + position % p, -1)
    taken = torch.where(served & (need > 0), first + need, 0).max().reshape(1)
    return {"table": table, "token_ptr": ptr, "lens": torch.where(served, past + fresh, past).to(torch.int32), "slots": slots.to(torch.int32),
            "positions": position.to(torch.int32), "taken": taken.to(torch.int32)}


def _plain_store(s):
    h, d = s["case"]["kv_heads"], s["case"]["dim"]
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    s["k_cache"].view(-1, h, d)[at] = s["k"][live]
    s["v_cache"].view(-1, h, d)[at] = s["v"][live]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c, q, table, lens = s["case"], s["q"], s["table"].long(), s["lens"].long()
    b, hq, hk, d, p = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    t = torch.arange(table.shape[1] * p, device="cuda")
    at = torch.where(t[None, :] < lens[:, None], table[:, t // p] * p + t % p, 0)  # (b, t): the slot of each position
    seen = (t[None, :] < lens[:, None])[:, None, None, :]
    k = s["k_cache"].view(-1, hk, d)[at].float()
    scores = torch.einsum("bhgd,bthd->bhgt", q.float().view(b, hk, hq // hk, d), k) * s["scale"]
    del k
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    weight = torch.exp(scores - torch.where(top > -math.inf, top, 0))
    total = weight.sum(-1, keepdim=True)
    v = s["v_cache"].view(-1, hk, d)[at].float()
    y = torch.einsum("bhgt,bthd->bhgd", weight, v) / torch.where(total > 0, total, 1)
    return {"out": y.reshape(b, hq, d).to(q.dtype), "lse": (top + torch.log(total)).reshape(b, hq)}


_OWN = {"route": _own_route, "train": _own_route, "pages": _own_pages, "store": _own_store, "attend": _own_attend}
_PLAIN = {"route": _plain_route, "train": _plain_route, "pages": _plain_pages, "store": _plain_store, "attend": _plain_attend}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    op = case["op"]
    if op in ("route", "train"):
        t, n = case["tokens"], case["tokens"] * case["k"]
        row = case["hidden"] * size
        index = n * (8 if case["ids"] == "i64" else 4) + 8 * n + 4 * (case["experts"] + 1) + 4 * n
        live = n * (1 - case["drop"])
        moved, flops = t + n + live + t, 2 * live * case["hidden"]
        if op == "train":
            moved += t + n + live + t  # dy, dys, dxs, dx; the experts' rows are read for combine already
            index += 4 * n
            flops += 4 * live * case["hidden"]
        return {"bytes": moved * row + index, "flops": flops}
    if op == "pages":
        r, p = case["requests"], case["page"]
        tokens = r * (1 if case["fresh"] == 1 else 0.1 + 0.8 * (case["fresh"] + 1) / 2)
        return {"bytes": 16 * r + 8 * tokens + 8 * tokens / p + 4 * r, "flops": 0}
    if op == "store":
        return {"bytes": 4 * case["tokens"] * (1 - case["pad"]) * case["kv_heads"] * case["dim"] * size + 4 * case["tokens"], "flops": 0}
    top = case["longest"]
    share = {"one": top, "even": top / 2, "log": 0.97 * top / math.log(top + 1)}[case["spread"]]
    tokens = top + (case["batch"] - 1) * share
    return {"bytes": 2 * tokens * case["kv_heads"] * case["dim"] * size + 2 * case["batch"] * case["q_heads"] * case["dim"] * size + 4 * tokens / case["page"],
            "flops": 4 * tokens * case["q_heads"] * case["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    """The outputs from the definitions in 64 bits; None for whole numbers and for rows that are copied."""
    s = prepare(case, seed)
    return {"route": _exact_route, "train": _exact_route, "attend": _exact_attend}.get(case["op"], lambda s: None)(s)


def _exact_route(s):
    case, ids, w = s["case"], s["ids"].cpu(), s["weights"].double()
    (t, k), h = ids.shape, case["hidden"]
    out = {"expert_ptr": None, "entry": None, "slot": None, "xs": None, "y": torch.zeros(t, h, dtype=torch.float64, device="cuda")}
    if case["op"] == "train":
        out["dys"] = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        out["dw"] = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        out["dx"] = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    begin = 0
    for e in range(case["experts"]):  # expert by expert: its tokens in their order
        rows, cols = torch.nonzero(ids == e, as_tuple=True)
        rows, cols = rows.cuda(), cols.cuda()
        here = slice(begin, begin + rows.numel())
        begin += rows.numel()
        ys = s["ys"][here].double()
        out["y"].index_add_(0, rows, ys * w[rows, cols][:, None])
        if case["op"] == "train":
            dy = s["dy"][rows].double()
            out["dys"][here] = dy * w[rows, cols][:, None]
            out["dw"][rows, cols] = (dy * ys).sum(1)
            out["dx"].index_add_(0, rows, s["dxs"][here].double())
    return out


def _exact_attend(s):
    case, q, lens, table = s["case"], s["q"].double(), s["lens"].tolist(), s["table"].long()
    b, hq, hk, d, p = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[i, : -(-n // p)]
        for h in range(hk):
            group = slice(h * (hq // hk), (h + 1) * (hq // hk))
            k = s["k_cache"][pages, :, h].reshape(-1, d)[:n].double()
            v = s["v_cache"][pages, :, h].reshape(-1, d)[:n].double()
            scores = q[i, group] @ k.T * s["scale"]
            lse[i, group] = torch.logsumexp(scores, 1)
            out[i, group] = torch.softmax(scores, 1) @ v
    return {"out": out, "lse": lse}
