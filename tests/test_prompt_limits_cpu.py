"""Sizes that the C entry points of prompts' attention and of loads refuse, or take."""
import load_balanced_csr_gb300 as lb
from test_e4m3_abi_cpu import BAD, prompt


def test_requests_are_counted_up_to_the_end_of_their_last_128():
    """The planning warp goes through the requests 128 at a time: with nearly 2^31 of them the next batch's first would pass
    32 bits and be read from before the pointers."""
    L = lb.lib()
    for requests in (2 ** 31 - 512, 2 ** 31 - 1):
        assert L.spmv_prompt_attention(prompt(requests=requests), None) == BAD
        assert b"requests" in L.spmv_last_error()
    assert L.spmv_prompt_attention(prompt(requests=2 ** 31 - 513, tokens=0, q=None, out=None), None) == 0
