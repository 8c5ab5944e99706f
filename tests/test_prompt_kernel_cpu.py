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
    raised, = re.findall(r"if \(raise\) m = high;(.*?)\bwait\(", text, re.S)
    assert "__syncwarp();" in raised


def test_lanes_meet_behind_the_queries_of_single_tokens():
    """Lanes whose head a group does not have read no queries; ldmatrix and mma, of the whole warp, come next."""
    begun, = re.findall(r"tile\.begin\((.*?)tile\.chunk\(", code("paged_attention.cuh"), re.S)
    assert "__syncwarp();" in begun


def kernel_code():
    text = code()
    return text[text.index("prompt_attention_kernel(const __grid_constant__"):text.index("prompt_join_kernel(")]


def test_what_is_under_way_is_waited_for_when_all_warps_have_stopped():
    """A warp can come to its end before another one gives up: only behind a barrier of them all is it known that copies and
    products are to be waited for, and do all lanes read the same."""
    kernel = kernel_code()
    assert "if (*gave_up)" not in kernel  # read lane by lane, and too early
    stopped, = re.findall(r"auto stopped = \[&\] \{(.*?)\};", kernel, re.S)
    assert re.sub(r"\s+", " ", stopped).strip() == "tc::fence_before(); tc::block_barrier(1, S::THREADS); return sh.gave_up != 0;"
    # each of the five kinds of warp comes to it once, as its last step but for these waits
    ends = re.split(r"\bstopped\(\)", kernel)[1:]
    assert len(ends) == 5
    loader, issuer = ends[0][:ends[0].index("else if")], ends[1][:ends[1].index("else if")]
    assert re.findall(r"bar_wait\(&sh\.(\w+)[^;]*nullptr\);", loader) == ["q_full", "full"] and len(re.findall("bar_wait", loader)) == 2
    assert "tc::commit(&sh.last)" in issuer and re.findall(r"bar_wait\(&sh\.(\w+), 0, nullptr\);.*?tc::(dealloc)", issuer, re.S) == [("last", "dealloc")]
    assert kernel.count("tc::dealloc") == 1
    for other in ends[2:]:
        assert not re.findall(r"\bwait\(|bar_wait|load32|store32", other.split("else")[0])


def test_waits_for_whole_pieces_of_work_last_as_long_as_these():
    """A tile without rows waits for the next piece while the other tile goes through all keys of this one, an announcement
    waits behind a row's end, and so on: no wait on another warp is for a step alone.  A step of 128 keys takes about 2,550
    clocks; 2^31 of them are the most a piece can have."""
    kernel = kernel_code()
    assert re.findall(r"auto wait = \[&\]\(uint64_t \*bar, uint32_t parity\) \{ return tc::bar_wait\(bar, parity, gave_up, p\.clocks\); \};", kernel)
    # by their own time alone: the answer about another block, which must not come behind this one's end, and a block's end
    assert sorted(re.findall(r"bar_wait\(([^,]*),", kernel)) == ["&sh.answered", "&sh.full[i % S::STAGES]", "&sh.last", "&sh.q_full", "bar"]
    assert len(re.findall(r"\bwait\(", kernel)) >= 15
    each, = map(int, re.findall(r"kEachClocks = (\d+);", code()))
    assert re.findall(r"p\.clocks = \(1ll << 31\) \+ kEachClocks \* \(\(int64_t\)a\.keys \+ a\.requests\);", code())
    assert each >= 4 * 2550 / 128
