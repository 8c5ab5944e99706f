"""How the kernels of prompts' and of single tokens' attention read: what no run would show."""
import os
import re

from load_balanced_csr_gb300 import _build


def code(name="prompt_attention.cu"):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_lanes_meet_before_instructions_of_a_whole_warp():
    """Loads and stores of tensor memory are .aligned: all lanes of the warp execute the same one.  Behind code that sends
    lanes different ways they have to be brought together; nothing promises that they meet at the end of a loop's body."""
    text = code()
    outputs, = re.findall(r"for \(int c = 0; c < p\.a\.head_dim && [^{]*\{(.*?)tc::load32\(", text, re.S)
    assert "__syncwarp();" in outputs  # rows without a place, and values that are not finite, go their own way
    masks, = re.findall(r"if \(c \+ i >= left\) s\[i\] = -INFINITY;(.*?)tc::store32\(", text, re.S)
    assert "__syncwarp();" in masks
    raised, = re.findall(r"if \(raise\) m = high;(.*?)tc::bar_wait\(", text, re.S)
    assert "__syncwarp();" in raised


def test_lanes_meet_behind_the_queries_of_single_tokens():
    """Lanes whose head a group does not have read no queries; ldmatrix and mma, of the whole warp, come next."""
    begun, = re.findall(r"tile\.begin\((.*?)tile\.chunk\(", code("paged_attention.cuh"), re.S)
    assert "__syncwarp();" in begun
