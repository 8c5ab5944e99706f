"""The prompts' kernel when a wait inside it runs out.  The debug build takes
the limit from SPMV_PROMPT_CLOCKS: with a short one the planning warp's wait for
a long piece of work (all shapes) and the wait of a tile without rows for the
next piece (two tiles) run out while copies and products are under way.  The
kernel ends by itself: every wait has a limit, copies and products in flight
are waited for, tensor memory is given back.  The call returns, the status has
bit 2, and the next call is as if nothing had been."""
import os

import pytest

pytestmark = pytest.mark.gpu

KEYS = 1 << 20  # about 20 clocks each: a piece of work takes some 10 ms, the longest of the limits 2


@pytest.fixture
def clocks():
    def limit(n):
        os.environ["SPMV_PROMPT_CLOCKS"] = str(n)
    yield limit
    os.environ.pop("SPMV_PROMPT_CLOCKS", None)


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_waits_that_run_out(dim, dtype, cut, clocks):
    import torch
    import load_balanced_csr_gb300 as lb
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    keys, heads, kv_heads = (4 * KEYS, 2, 1) if cut else (KEYS, 6, 3)
    g = torch.Generator(device="cuda").manual_seed(dim)
    q = torch.randn(10, heads, dim, generator=g, device="cuda").to(dt)
    k, v = (torch.randn(keys, kv_heads, dim, generator=g, device="cuda").to(dt) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    q_ptr, kv_ptr = torch.tensor([0, 10], **i32), torch.tensor([0, keys], **i32)

    def attention(L):
        attend = lb.PromptAttention(1, heads, kv_heads, dim, dt)
        attend._L = L
        if not cut:  # without a workspace the keys of a piece stay together
            attend._args.workspace, attend._args.workspace_bytes = None, 0
        return attend

    want, want_lse = attention(lb.lib())(q, k, v, q_ptr, kv_ptr)
    torch.cuda.synchronize()
    for n in (0, 1 << 12, 1 << 16, 1 << 22) if not cut else (0, 1 << 12):
        clocks(n)
        attend = attention(lb.debug_lib())
        out, lse = attend(q, k, v, q_ptr, kv_ptr)
        assert attend.device_status() == 4, n
        os.environ.pop("SPMV_PROMPT_CLOCKS")
        again = attention(lb.debug_lib())  # the same code, nothing left behind
        out, lse = again(q, k, v, q_ptr, kv_ptr)
        assert again.device_status() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_many_blocks_give_up(clocks):
    """Several rounds of blocks on every SM, some taken over, each of which gives up."""
    import torch
    import load_balanced_csr_gb300 as lb
    heads, keys, dim = 640, 1 << 18, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(10, heads, dim, generator=g, device="cuda").bfloat16()
    row = dim + 8 * heads  # neighbouring heads' keys overlap
    k, v = (torch.randn(keys * row, generator=g, device="cuda").bfloat16().as_strided((keys, heads, dim), (row, 8, 1)) for _ in range(2))
    q_ptr, kv_ptr = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (10, keys))
    attend = lb.PromptAttention(1, heads, heads, dim, torch.bfloat16)
    want, want_lse = attend(q, k, v, q_ptr, kv_ptr)
    assert attend.device_status() == 0
    attend._L = lb.debug_lib()
    for n in (0, 1 << 10, 1 << 14):
        clocks(n)
        attend(q, k, v, q_ptr, kv_ptr)
        assert attend.device_status() == 4, n
        os.environ.pop("SPMV_PROMPT_CLOCKS")
        attend._status.zero_()
        out, lse = attend(q, k, v, q_ptr, kv_ptr)
        assert attend.device_status() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
