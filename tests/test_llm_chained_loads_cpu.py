"""The language-model operators' kernels are launched while the kernel before
them still runs.  What that one writes is visible after the wait to ordinary
loads only; the read-only path (__ldg, or what a compiler makes of a const
__restrict__ pointer) is defined for data that nobody writes while the kernel
lives.  Read from the source: a stale load would show up only now and then."""
import os
import re

import pytest

from load_balanced_csr_gb300 import _build

SOURCES = ["llm.cuh", "route.cu", "pages.cu", "paged_attention.cuh", "paged_attention.cu", "paged_attention_bf16.cu",
           "paged_attention_f16.cu"]


def code(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_through_the_read_only_path(name):
    found = re.findall(r"__ldg\w*|__restrict__|ld\.global\.nc", code(name))
    assert not found, f"{name}: {sorted(set(found))}"


@pytest.mark.parametrize("name", ["route.cu", "pages.cu", "paged_attention.cuh"])
def test_every_kernel_waits_for_the_one_before_it(name):
    """and does so before it names an argument's memory: only declarations come first."""
    text = code(name)
    kernels = list(re.finditer(r"__global__[^{;]*\{", text))
    assert kernels
    for k in kernels:
        body = text[k.end():]
        before = body[:body.index("after_previous();")]
        assert len(before) < 1500 and "__global__" not in before, k.group()[:200]
        for statement in before.split(";")[:-1]:
            declares = re.match(r"\s*(using |constexpr |enum |extern __shared__|__shared__|const int lane|char \*mine|char \*qs|"
                                r"const Request \*req)", statement)
            assert declares, f"{k.group()[-80:]}: {statement.strip()}"
