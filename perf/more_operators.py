"""Cases that time the operators of an 8-bit paged cache and the attention of whole prompts.

Four kinds of case, each one pass through one operator as a program calls it:

  store   a step's keys and values quantised as they are written into the paged cache: e4m3 codes, a power-of-two scale per
          block of tokens and head, which grows with the tokens that come
  load    requests' keys and values read back from the paged cache into packed rows
  attend  attention of one new token per request over the 8-bit cache
  prompt  attention of packed prompts, or of chunks of them behind what their requests hold already

`own` chooses the framework's kernels; otherwise the plain forms below, in elementary torch operations, run.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # the new keys and values of a decode step of 256 requests, each behind what its block holds
        {"name": "store decode 256", "op": "store", "requests": 256, "fresh": 1, "kv_heads": 8, "dim": 128, "page": 16, "block": 16, "dtype": "bf16", "pad": 0.0},
        # a prefill of about 65,000 tokens, views of one fused projection, a request in twenty not served
        {"name": "store prefill 32x2047", "op": "store", "requests": 32, "fresh": 2047, "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "dtype": "f16", "pad": 0.05},
        # 32-bit keys, a head and a page of odd sizes, a scale for each token
        {"name": "store f32 odd", "op": "store", "requests": 40, "fresh": 75, "kv_heads": 5, "dim": 72, "page": 7, "block": 1, "dtype": "f32", "pad": 0.0},
        # the past of sixteen requests' chunks, about 130,000 positions in all
        {"name": "load 16 of 16384", "op": "load", "batch": 16, "longest": 16384, "spread": "even", "kv_heads": 8, "dim": 128, "page": 16, "block": 16, "dtype": "bf16", "codes": True},
        # a few short requests of a cache that holds its elements whole
        {"name": "load 4 of 300 f16", "op": "load", "batch": 4, "longest": 300, "spread": "log", "kv_heads": 4, "dim": 72, "page": 7, "block": 1, "dtype": "f16", "codes": False},
        # one request with a long context
        {"name": "attend one long 131071", "op": "attend", "batch": 1, "longest": 131071, "spread": "one", "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "dtype": "bf16"},
        # a serving batch of very uneven lengths, empty ones among them
        {"name": "attend ragged 128", "op": "attend", "batch": 128, "longest": 16384, "spread": "log", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "block": 16, "dtype": "bf16"},
        # a few short requests, a key head for each query head: latency counts
        {"name": "attend short 4 f16", "op": "attend", "batch": 4, "longest": 300, "spread": "log", "q_heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "block": 1, "dtype": "f16"},
        # one long prompt
        {"name": "prompt 8192", "op": "prompt", "batch": 1, "longest": 8192, "spread": "one", "past": 0, "q_heads": 64, "kv_heads": 8, "dim": 128, "causal": True, "dtype": "bf16"},
        # sixteen prompts of very uneven lengths, empty ones among them, small heads
        {"name": "prompt packed 16 f16", "op": "prompt", "batch": 16, "longest": 2048, "spread": "log", "past": 0, "q_heads": 32, "kv_heads": 8, "dim": 64, "causal": True, "dtype": "f16"},
        # a step's chunks of eight requests, behind what they hold already
        {"name": "prompt chunks 8x512", "op": "prompt", "batch": 8, "longest": 512, "spread": "one", "past": 7000, "q_heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "dtype": "bf16"},
        # a few short prompts, a key head for each query head: latency counts
        {"name": "prompt short 4", "op": "prompt", "batch": 4, "longest": 300, "spread": "log", "past": 0, "q_heads": 16, "kv_heads": 16, "dim": 80, "causal": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["store", "load", "attend", "attend", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "f16"] + (["f32"] if op in ("store", "load") else []))
    page = rng.choice([1, 7, 16, 16, 32, 64, 128])
    block = rng.choice([b for b in (1, 4, 7, 16, 32, 64) if page % b == 0])
    heads = rng.choice([1, 2, 4, 5, 8])
    if op == "store":
        dim, requests = rng.choice([64, 72, 128, 128, 192, 256]), _log_int(rng, 1, 512)
        most = (1 << 26) // (heads * dim * requests)
        return {"op": op, "requests": requests, "fresh": rng.choice([1, _log_int(rng, 2, max(2, min(2047, most)))]), "kv_heads": heads, "dim": dim, "page": page,
                "block": block, "dtype": dtype, "pad": rng.choice([0.0, 0.0, 0.05, 0.5])}
    if op == "load":
        dim, batch = rng.choice([64, 72, 128, 128, 192, 256]), _log_int(rng, 1, 128)
        longest = min(16384, max(16, (1 << 26) // (batch * heads * dim)))
        return {"op": op, "batch": batch, "longest": _log_int(rng, 16, longest), "spread": rng.choice(["log", "even", "one"]), "kv_heads": heads, "dim": dim,
                "page": page, "block": block, "dtype": dtype, "codes": rng.random() < 0.7}
    group, spread = rng.choice([1, 2, 4, 7, 8, 16]), rng.choice(["log", "even", "one"])
    if op == "attend":
        batch, dim = _log_int(rng, 1, 256), rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        longest = min(131071, max(16, (1 << 27) // (batch * heads * dim)))
        return {"op": op, "batch": batch, "longest": _log_int(rng, 16, longest), "spread": spread, "q_heads": heads * group, "kv_heads": heads, "dim": dim,
                "page": page, "block": block, "dtype": dtype}
    dim, batch, past = rng.choice([64, 72, 80, 96, 128, 128, 128, 192, 256]), _log_int(rng, 1, 32), rng.choice([0, 0, _log_int(rng, 16, 8192)])
    room = (1 << 31) / (batch * heads * group * max(1, dim / 128))  # pairs of queries and keys of a request
    longest = min(8192, int(room / (past + math.sqrt(room))))
    return {"op": op, "batch": batch, "longest": _log_int(rng, 1, max(1, longest)), "spread": spread, "past": past, "q_heads": heads * group, "kv_heads": heads,
            "dim": dim, "causal": rng.random() < 0.8, "dtype": dtype}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _spread(n, g):
    """n numbers over (0, 1), evenly, in any order: the seed changes their order alone, so that sums do not depend on it."""
    return ((torch.arange(n, device="cuda", dtype=torch.float64) + 0.5) / n)[torch.randperm(n, generator=g, device="cuda")]


def _lengths(batch, top, spread, g):
    """Lengths of requests: all near the longest, spread evenly, or over the logarithm with some empty."""
    u = _spread(batch, g)
    if spread == "one":
        lens = top - (u * min(8, top - 1)).floor()
    elif spread == "even":
        lens = (u * (top + 1)).floor()
    else:
        lens = torch.where(u < 0.04, 0, torch.exp(u * math.log(top + 1)).floor())
    lens[u.argmin() if spread == "one" else u.argmax()] = top
    return lens.to(torch.int32)


def _prefix(lens):
    ptr = torch.zeros(lens.numel() + 1, dtype=torch.int32, device=lens.device)
    ptr[1:] = torch.cumsum(lens, 0)
    return ptr


def _codes(g, pages, page, heads, dim, block):
    """A cache in 8 bits as earlier steps left it: codes up to 448, power-of-two scales that differ from block to block."""
    codes = (100 * _normal(g, pages, page, heads, dim, dtype=torch.bfloat16)).clamp_(-448, 448).to(E4M3)
    return codes, torch.exp2(torch.randint(-8, -4, (pages, page // block, heads), generator=g, device="cuda").float())


def _tables(lens, page, g, extra=2):
    """Tables of requests' pages in any order, and how many pages there are."""
    held = (lens.long() + page - 1) // page
    width, pages = max(1, int(held.max())), int(held.sum()) + extra
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < held[:, None]] = torch.randperm(pages, generator=g, device="cuda")[: pages - extra].to(torch.int32)
    return table, pages


def prepare(case, seed):
    """What a program has in hand before the call."""
    return _PREPARE[case["op"]](case, _generator(seed))


def _prepare_store(case, g):
    h, d, p, dt = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    past = (_spread(case["requests"], g) * 2 * max(p, 16)).long()
    table, pages = _tables(past + case["fresh"], p, g)
    position = past[:, None] + torch.arange(case["fresh"], device="cuda")
    slots = torch.gather(table.long(), 1, position // p) * p + position % p
    if case["pad"]:
        slots[torch.rand(case["requests"], generator=g, device="cuda") < case["pad"]] = -1
    n = case["requests"] * case["fresh"]
    # tokens differ in size, as keys do
    fused = (_normal(g, n, 2 * h, d) * torch.exp(0.7 * _normal(g, n, 2 * h, 1))).to(dt)
    k_cache, k_scales = _codes(g, pages, p, h, d, case["block"])
    v_cache, v_scales = _codes(g, pages, p, h, d, case["block"])
    return {"case": case, "k": fused[:, :h], "v": fused[:, h:], "slots": slots.reshape(-1).to(torch.int32), "k_cache": k_cache, "v_cache": v_cache,
            "k_scales": k_scales, "v_scales": v_scales}


def _prepare_load(case, g):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case["batch"], case["longest"], case["spread"], g)
    table, pages = _tables(lens, p, g)
    ptr = _prefix(lens)
    s = {"case": case, "table": table, "ptr": ptr, "tokens": int(ptr[-1]), "k_scales": None, "v_scales": None}
    if case["codes"]:
        s["k_cache"], s["k_scales"] = _codes(g, pages, p, h, d, case["block"])
        s["v_cache"], s["v_scales"] = _codes(g, pages, p, h, d, case["block"])
    else:
        s["k_cache"], s["v_cache"] = (_normal(g, pages, p, h, d, dtype=DTYPES[case["dtype"]]) for _ in range(2))
    return s


def _prepare_attend(case, g):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case["batch"], case["longest"], case["spread"], g)
    table, pages = _tables(lens, p, g)
    k_cache, k_scales = _codes(g, pages, p, h, d, case["block"])
    v_cache, v_scales = _codes(g, pages, p, h, d, case["block"])
    return {"case": case, "q": _normal(g, case["batch"], case["q_heads"], d, dtype=DTYPES[case["dtype"]]), "lens": lens, "table": table, "scale": d ** -0.5,
            "k_cache": k_cache, "v_cache": v_cache, "k_scales": k_scales, "v_scales": v_scales}


def _prepare_prompt(case, g):
    dt, d, hq, hk = DTYPES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"]
    nq = _lengths(case["batch"], case["longest"], case["spread"], g)
    nk = nq + (case["past"] * (0.5 + 0.5 * _spread(case["batch"], g))).to(torch.int32) if case["past"] else nq
    q_ptr, kv_ptr = _prefix(nq), _prefix(nk)
    if case["past"]:  # keys and values of a past and the chunk behind it were read back from the cache
        q, k, v = (_normal(g, n, heads, d, dtype=dt) for n, heads in ((int(q_ptr[-1]), hq), (int(kv_ptr[-1]), hk), (int(kv_ptr[-1]), hk)))
    else:  # views of one fused projection
        q, k, v = _normal(g, int(q_ptr[-1]), hq + 2 * hk, d, dtype=dt).split([hq, hk, hk], 1)
    return {"case": case, "q": q, "k": k, "v": v, "q_ptr": q_ptr, "kv_ptr": kv_ptr if case["past"] else None, "scale": d ** -0.5,
            "most_q": int(nq.max()), "most_k": int(nk.max())}


_PREPARE = {"store": _prepare_store, "load": _prepare_load, "attend": _prepare_attend, "prompt": _prepare_prompt}


def run(state):
    """One pass."""
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ the framework's operators


def _own_store(s):
    import load_balanced_csr_gb300 as lb

    lb.paged_store_e4m3(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["slots"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _own_load(s):
    import load_balanced_csr_gb300 as lb

    k, v = lb.paged_load(s["k_cache"], s["v_cache"], s["table"], s["ptr"], s["tokens"], s["k_scales"], s["v_scales"], dtype=DTYPES[s["case"]["dtype"]])
    return {"k": k, "v": v}


def _own_attend(s):
    import load_balanced_csr_gb300 as lb

    if "attention" not in s:
        c = s["case"]
        s["attention"] = lb.PagedAttentionE4M3(c["batch"], c["q_heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]])
    out, lse = s["attention"](s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["lens"], scale=s["scale"])
    return {"out": out, "lse": lse}


def _own_prompt(s):
    import load_balanced_csr_gb300 as lb

    c = s["case"]
    if "attention" not in s:
        s["attention"] = lb.PromptAttention(c["batch"], c["q_heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]])
    out, lse = s["attention"](s["q"], s["k"], s["v"], s["q_ptr"], s["kv_ptr"], causal=c["causal"], scale=s["scale"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ their plain forms


def _plain_quantise(x, cache, scales, slots, block):
    h, d = x.shape[1:]
    x = x.float()
    size = torch.where(torch.isfinite(x), x.abs(), 0).amax(-1).clamp(min=448 * 2.0 ** -126)
    f = torch.frexp(size)[0]
    need = size / f * torch.where(f > 0.875, 2.0 ** -8, 2.0 ** -9)  # the least power of two p with size <= 448 p; 448 = 0.875 * 2^9
    blocks, of = torch.unique(slots // block, return_inverse=True)
    top = torch.zeros(blocks.numel(), h, device="cuda").index_reduce_(0, of, need, "amax")
    begun = torch.zeros(blocks.numel(), device="cuda").index_reduce_(0, of, (slots % block == 0).float(), "amax")[:, None] > 0
    held = scales.view(-1, h)
    old = held[blocks]
    new = torch.where(begun, top, torch.maximum(old, top))
    held[blocks] = new
    codes = cache.view(torch.uint8).view(-1, block, h, d)
    kept = codes[blocks].view(E4M3).float() * torch.where(begun, 1, old / new)[:, None, :, None]
    codes[blocks] = kept.to(E4M3).view(torch.uint8)
    codes.view(-1, h, d)[slots] = (x / new[of][:, :, None]).to(E4M3).view(torch.uint8)


def _plain_store(s):
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    _plain_quantise(s["k"][live], s["k_cache"], s["k_scales"], slots, s["case"]["block"])
    _plain_quantise(s["v"][live], s["v_cache"], s["v_scales"], slots, s["case"]["block"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_rows(cache, scales, at):
    """The rows of slots `at` in 32 bits."""
    pages, page, h, d = cache.shape
    if scales is None:
        return cache.view(-1, h, d)[at].float()
    block = page // scales.shape[1]
    return cache.view(torch.uint8).view(-1, h, d)[at].view(E4M3).float() * scales.view(-1, h)[at // block][..., None]


def _plain_load(s):
    p, dt = s["case"]["page"], DTYPES[s["case"]["dtype"]]
    i = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(s["ptr"][1:], i, right=True)
    t = i - s["ptr"][r]
    at = s["table"][r, t // p].long() * p + t % p
    return {"k": _plain_rows(s["k_cache"], s["k_scales"], at).to(dt), "v": _plain_rows(s["v_cache"], s["v_scales"], at).to(dt)}


def _plain_weights(scores):
    """The weights of the last dimension's scores, unnormalised, their sums (1 where nothing is seen) and the logarithm of the scores' sum."""
    top = scores.amax(-1, keepdim=True)
    weight = torch.exp(scores - torch.where(top > -math.inf, top, 0))
    total = weight.sum(-1)
    return weight, torch.where(total > 0, total, 1), top.squeeze(-1) + torch.log(total)


def _plain_attend(s):
    c, q, table, lens = s["case"], s["q"], s["table"].long(), s["lens"].long()
    b, hq, hk, d, p = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    t = torch.arange(table.shape[1] * p, device="cuda")
    seen = t[None, :] < lens[:, None]
    at = torch.where(seen, table[:, t // p] * p + t % p, 0)  # (b, t): the slot of each position
    k = _plain_rows(s["k_cache"], s["k_scales"], at)
    scores = torch.einsum("bhgd,bthd->bhgt", q.float().view(b, hk, hq // hk, d), k) * s["scale"]
    del k
    scores = torch.where(seen[:, None, None, :], scores, -math.inf)
    weight, total, lse = _plain_weights(scores)
    y = torch.einsum("bhgt,bthd->bhgd", weight, _plain_rows(s["v_cache"], s["v_scales"], at)) / total[..., None]
    return {"out": y.reshape(b, hq, d).to(q.dtype), "lse": lse.reshape(b, hq)}


def _plain_padded(x, ptr, most):
    """(requests, most, heads, dim) in 32 bits, zeros past each request's rows."""
    j = torch.arange(most, device="cuda")
    n = (ptr[1:] - ptr[:-1]).long()
    there = j[None, :] < n[:, None]
    return torch.where(there[:, :, None, None], x[torch.where(there, ptr[:-1, None] + j, 0)].float(), 0), there, n


def _plain_prompt(s):
    c = s["case"]
    hq, hk, d, q_ptr = c["q_heads"], c["kv_heads"], c["dim"], s["q_ptr"].long()
    kv_ptr = q_ptr if s["kv_ptr"] is None else s["kv_ptr"].long()
    q, _, nq = _plain_padded(s["q"], q_ptr, s["most_q"])
    k, seen, nk = _plain_padded(s["k"], kv_ptr, s["most_k"])
    v, _, _ = _plain_padded(s["v"], kv_ptr, s["most_k"])
    scores = torch.einsum("bihgd,bjhd->bhgij", q.view(c["batch"], -1, hk, hq // hk, d), k) * s["scale"]
    i, j = torch.arange(s["most_q"], device="cuda"), torch.arange(s["most_k"], device="cuda")
    seen = seen[:, None, :]
    if c["causal"]:
        seen = seen & (j[None, None, :] <= i[None, :, None] + (nk - nq)[:, None, None])
    scores = torch.where(seen[:, None, None, :, :], scores, -math.inf)
    weight, total, lse = _plain_weights(scores)
    y = torch.einsum("bhgij,bjhd->bihgd", weight, v) / total.permute(0, 3, 1, 2)[..., None]
    lse = lse.permute(0, 3, 1, 2)
    n = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(q_ptr[1:], n, right=True)
    t = n - q_ptr[r]
    return {"out": y[r, t].reshape(-1, hq, d).to(s["q"].dtype), "lse": lse[r, t].reshape(-1, hq)}


_OWN = {"store": _own_store, "load": _own_load, "attend": _own_attend, "prompt": _own_prompt}
_PLAIN = {"store": _plain_store, "load": _plain_load, "attend": _plain_attend, "prompt": _plain_prompt}


# ------------------------------------------------------------------ what a pass cannot do without


def _mean_tokens(case):
    """How many positions a case's requests have, on average over the seeds."""
    top = case["longest"]
    share = {"one": top, "even": top / 2, "log": 0.97 * top / math.log(top + 1)}[case["spread"]]
    return top + (case["batch"] - 1) * share


def work(case):
    size, op = 4 if case["dtype"] == "f32" else 2, case["op"]
    row = case["kv_heads"] * case["dim"]
    if op == "store":
        n = case["requests"] * case["fresh"] * (1 - case["pad"])
        return {"bytes": 2 * n * row * (size + 1) + 4 * n + 8 * n * case["kv_heads"] / min(case["block"], case["fresh"]), "flops": 0}
    tokens = _mean_tokens(case)
    if op == "load":
        held = 1 + 4 / (case["block"] * case["dim"]) if case["codes"] else size
        return {"bytes": 2 * tokens * row * (held + size) + 4 * tokens / case["page"], "flops": 0}
    if op == "attend":
        return {"bytes": 2 * tokens * row * (1 + 4 / (case["block"] * case["dim"])) + 2 * case["batch"] * case["q_heads"] * case["dim"] * size + 4 * tokens / case["page"],
                "flops": 4 * tokens * case["q_heads"] * case["dim"]}
    top, past = case["longest"], 0.75 * case["past"]
    square = {"one": top * top, "even": top * top / 3, "log": 0.97 * top * top / (2 * math.log(top + 1))}[case["spread"]]
    square = top * top + (case["batch"] - 1) * square  # of the queries' own lengths
    pairs = square * (0.5 if case["causal"] else 1) + tokens * past
    return {"bytes": (2 * tokens * case["q_heads"] * case["dim"] + 2 * (tokens + case["batch"] * past) * row) * size,
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"store": _exact_store, "load": _exact_load, "attend": _exact_attend, "prompt": _exact_prompt}[case["op"]](s)


def _exact_e4m3(x):
    """The nearest values of four exponent and three mantissa bits, ties to even mantissas."""
    size = x.abs().clamp(min=2.0 ** -6)
    step = size / torch.frexp(size)[0] / 16  # frexp's mantissas are in [1/2, 1); the quotient is a power of two, exactly
    return torch.round(x / step) * step


def _exact_store(s):
    block, out = s["case"]["block"], {}
    slots = s["slots"].tolist()
    of_block = {}
    for i, slot in enumerate(slots):
        if slot >= 0:
            of_block.setdefault(slot // block, []).append(i)
    if len(of_block) > 20000:
        return None
    for name in ("k", "v"):
        codes = s[name + "_cache"].double().view(-1, block, s["case"]["kv_heads"], s["case"]["dim"])
        scales = s[name + "_scales"].double().reshape(-1, s["case"]["kv_heads"])
        for b, tokens in of_block.items():
            x = s[name][tokens].double()
            need = (x.abs().amax((0, 2)) / 448).clamp(min=2.0 ** -126)
            f = torch.frexp(need)[0]
            need = torch.where(f == 0.5, need, need / f)
            inside = [slots[i] - b * block for i in tokens]
            if 0 not in inside:
                need = torch.maximum(need, scales[b])
                codes[b] = _exact_e4m3(codes[b] * (scales[b] / need)[:, None])
            codes[b, inside] = _exact_e4m3(x / need[:, None])
            scales[b] = need
        out[name + "_cache"], out[name + "_scales"] = codes.view(s[name + "_cache"].shape), scales.view(s[name + "_scales"].shape)
    return out


def _exact_values(s, name):
    """A cache's values in 64 bits."""
    cache, scales = s[name + "_cache"].double(), s[name + "_scales"]
    return cache if scales is None else cache * scales.double().repeat_interleave(cache.shape[1] // scales.shape[1], 1)[..., None]


def _exact_load(s):
    ptr, p, out = s["ptr"].tolist(), s["case"]["page"], {}
    for name in ("k", "v"):
        values = _exact_values(s, name)
        rows = [values[s["table"][r, : -(-(b - a) // p)].long()].flatten(0, 1)[: b - a] for r, (a, b) in enumerate(zip(ptr, ptr[1:]))]
        out[name] = torch.cat(rows)
    return out


def _exact_attend(s):
    case, q, lens, table = s["case"], s["q"].double(), s["lens"].tolist(), s["table"].long()
    b, hq, hk, d, p = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    k_all, v_all = _exact_values(s, "k"), _exact_values(s, "v")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[i, : -(-n // p)]
        for h in range(hk):
            group = slice(h * (hq // hk), (h + 1) * (hq // hk))
            k = k_all[pages, :, h].reshape(-1, d)[:n]
            v = v_all[pages, :, h].reshape(-1, d)[:n]
            scores = q[i, group] @ k.T * s["scale"]
            lse[i, group] = torch.logsumexp(scores, 1)
            out[i, group] = torch.softmax(scores, 1) @ v
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    case, q_ptr = s["case"], s["q_ptr"].tolist()
    kv_ptr = q_ptr if s["kv_ptr"] is None else s["kv_ptr"].tolist()
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(q_ptr[-1], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((q_ptr[-1], hq), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(case["batch"]):
        nq, nk = q_ptr[r + 1] - q_ptr[r], kv_ptr[r + 1] - kv_ptr[r]
        for h in range(hq):
            for at in range(0, nq, 2048):  # so many queries at once, and no more keys than they see
                some = slice(q_ptr[r] + at, q_ptr[r] + min(nq, at + 2048))
                first = nk - nq + at  # the last key of the first of them
                keys = min(nk, nk - nq + at + 2048) if case["causal"] else nk
                if keys <= 0:
                    continue
                k, v = (s[x][kv_ptr[r] : kv_ptr[r] + keys, h // (hq // hk)].double() for x in ("k", "v"))
                scores = s["q"][some, h].double() @ k.T * s["scale"]
                if case["causal"]:
                    rows = torch.arange(scores.shape[0], device="cuda")
                    scores.masked_fill_(torch.arange(keys, device="cuda")[None, :] > first + rows[:, None], -math.inf)
                lse[some, h] = torch.logsumexp(scores, 1)
                out[some, h] = torch.nan_to_num(torch.softmax(scores, 1)) @ v
    return {"out": out, "lse": lse}
