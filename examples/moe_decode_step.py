"""One decoding step of a decoder layer with a mixture of experts, on the
library's language-model operators:

    page tables and slots for the step's tokens   PageTable.append
    keys and values into the paged cache          paged_store
    attention over the cache                      PagedAttention
    tokens sorted by expert, and their rows       ExpertRoute.build, dispatch
    (the experts' products, plain torch)
    the experts' rows back, weighted              ExpertRoute.combine

    python examples/moe_decode_step.py            # a few steps of random weights, with the time of one
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import load_balanced_csr_gb300 as lb  # noqa: E402


class Layer:
    """A decoder layer's weights, cache and handles for up to `requests` requests."""

    def __init__(self, requests=32, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, experts=16, top_k=4, expert_hidden=512,
                 page_size=16, num_pages=1024, max_pages=64, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.top_k = q_heads, kv_heads, head_dim, top_k

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-2] ** -0.5).to(dtype)

        self.qkv = weight(hidden, (q_heads + 2 * kv_heads) * head_dim)
        self.out = weight(q_heads * head_dim, hidden)
        self.router = weight(hidden, experts)
        self.up, self.down = weight(experts, hidden, expert_hidden), weight(experts, expert_hidden, hidden)
        self.k_cache, self.v_cache = (torch.zeros(num_pages, page_size, kv_heads, head_dim, dtype=dtype, device="cuda")
                                      for _ in range(2))
        table = torch.full((requests, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
        self.pages = lb.PageTable(table, page_size, num_pages, max_tokens=requests)
        self.attend = lb.PagedAttention(requests, q_heads, kv_heads, head_dim, dtype)
        self.route = lb.ExpertRoute(requests, top_k, experts)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step(self, x):
        """x (requests, hidden): the new token of each request; returns the layer's output."""
        n = x.shape[0]
        heads = (x @ self.qkv).view(n, -1, self.head_dim)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        pages = self.pages.append(self.lens, torch.ones_like(self.lens), self.free)
        self.free = self.free[int(pages.taken):]  # the host's bookkeeping; a server does it a step behind
        self.lens = pages.lens.clone()            # the next append overwrites pages.lens
        lb.paged_store(k, v, self.k_cache, self.v_cache, pages.slots)
        attended, _ = self.attend(q, self.k_cache, self.v_cache, pages.table, self.lens)
        x = x + attended.view(n, -1) @ self.out
        weights, experts = torch.topk((x @ self.router).float(), self.top_k, dim=1)
        route = self.route.build(experts)
        rows = route.dispatch(x)
        begin = route.expert_ptr.tolist()
        for e in range(len(begin) - 1):
            mine = rows[begin[e]:begin[e + 1]]
            mine.copy_(torch.relu(mine @ self.up[e]) @ self.down[e])
        return x + route.combine(rows, torch.softmax(weights, dim=1))


def main():
    layer = Layer()
    x = torch.randn(32, 1024, device="cuda").bfloat16()
    for _ in range(40):
        y = layer.step(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        y = layer.step(x)
    end.record()
    torch.cuda.synchronize()
    assert int(layer.pages.status) == 0 and layer.attend.device_status() == 0 and bool(torch.isfinite(y).all())
    print(f"{layer.lens.tolist()[0]} tokens a request, {start.elapsed_time(end) / 20 * 1000:.0f} us a step")


if __name__ == "__main__":
    main()
