"""The C entry points of the 8-bit cache and of prompts' attention refuse bad
arguments before touching the device and lay out their structures as the
header does; how their kernels read."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import load_balanced_csr_gb300 as lb
from load_balanced_csr_gb300 import _build

FAKE, ODD, BAD = 0x1000, 0x1001, 1
S2, S3 = (ctypes.c_int64 * 2), (ctypes.c_int64 * 3)


def cache(**kw):
    from load_balanced_csr_gb300.paged_e4m3 import PagedCacheArgs
    a = PagedCacheArgs()
    base = dict(num_pages=4, page_size=16, block=8, k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), k_scale_stride=(4, 2, 1),
                v_scale_stride=(4, 2, 1), k_cache=FAKE, v_cache=FAKE, k_scales=FAKE, v_scales=FAKE)
    for name, value in {**base, **kw}.items():
        if isinstance(value, tuple):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return ctypes.byref(a)


def test_the_operators_are_exported():
    names = set(lb.header_functions())
    assert {"spmv_paged_store_e4m3", "spmv_paged_load", "spmv_paged_attention_e4m3", "spmv_paged_attention_e4m3_workspace",
            "spmv_prompt_attention", "spmv_prompt_attention_workspace"} <= names
    for L in (lb.lib(), lb.debug_lib()):
        for name in names:
            assert hasattr(L, name), name


def test_store_refusals():
    L = lb.lib()

    def store(tokens=1, heads=2, dim=64, elem=0, slots=FAKE, c=None, k=FAKE, ks=S2(128, 64), v=FAKE, vs=S2(128, 64), **kw):
        return L.spmv_paged_store_e4m3(tokens, heads, dim, elem, slots, cache(**kw) if c is None else c, k, ks, v, vs, None)

    for bad in (dict(tokens=-1), dict(heads=-1), dict(dim=-1), dict(elem=3), dict(elem=-1), dict(slots=None), dict(slots=ODD), dict(k=None),
                dict(k=ODD), dict(v=None), dict(ks=None), dict(vs=None), dict(num_pages=-1), dict(page_size=0), dict(num_pages=2 ** 27),
                dict(block=0), dict(block=-1), dict(block=5), dict(block=128, page_size=128), dict(k_cache=None), dict(v_cache=None),
                dict(k_scales=None), dict(v_scales=ODD), dict(heads=2 ** 20, dim=2 ** 11), dict(heads=2 ** 24, dim=1), dict(tokens=2 ** 30, heads=2 ** 4)):
        assert store(**bad) == BAD, bad
        assert L.spmv_last_error()
    assert L.spmv_paged_store_e4m3(1, 2, 64, 0, FAKE, None, FAKE, S2(128, 64), FAKE, S2(128, 64), None) == BAD
    for nothing in (dict(tokens=0, slots=None, k=None), dict(heads=0), dict(dim=0), dict(num_pages=0, k_cache=None, k_scales=None)):
        assert store(**nothing) == 0, nothing


def test_load_refusals():
    L = lb.lib()

    def load(requests=1, tokens=5, heads=2, dim=64, elem=1, table=FAKE, stride=4, max_pages=4, ptr=FAKE, k=FAKE, ks=S2(128, 64), v=FAKE,
             vs=S2(128, 64), **kw):
        return L.spmv_paged_load(requests, tokens, heads, dim, elem, table, stride, max_pages, ptr, cache(**kw), k, ks, v, vs, None)

    for bad in (dict(requests=-1), dict(tokens=-1), dict(heads=-1), dict(dim=-1), dict(elem=3), dict(table=None), dict(table=ODD),
                dict(max_pages=-1), dict(ptr=None), dict(ptr=ODD), dict(k=None), dict(v=ODD), dict(ks=None), dict(page_size=0), dict(block=3),
                dict(block=-1), dict(k_cache=None), dict(k_scales=None), dict(v_scales=ODD), dict(num_pages=2 ** 27),
                dict(tokens=2 ** 30, heads=2 ** 5, dim=2 ** 6), dict(block=0, k_cache=ODD)):
        assert load(**bad) == BAD, bad
        assert L.spmv_last_error()
    for nothing in (dict(requests=0, ptr=None), dict(tokens=0, k=None), dict(heads=0), dict(dim=0)):
        assert load(**nothing) == 0, nothing


def attention(**kw):
    from load_balanced_csr_gb300.paged import PagedAttentionArgs
    a = PagedAttentionArgs()
    base = dict(batch=1, q_heads=4, kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages=4, elem=1, scale=0.1, table_stride=4,
                q=FAKE, k_cache=FAKE, v_cache=FAKE, table=FAKE, lens=FAKE, out=FAKE, workspace=FAKE, workspace_bytes=1 << 40, status=FAKE,
                q_stride=(256, 64), k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), out_stride=(256, 64))
    for name, value in {**base, **kw}.items():
        if isinstance(value, tuple):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return ctypes.byref(a)


def test_attention_refusals():
    L = lb.lib()

    def call(block=8, ks=FAKE, kst=S3(4, 2, 1), vs=FAKE, vst=S3(4, 2, 1), **kw):
        return L.spmv_paged_attention_e4m3(attention(**kw), block, ks, kst, vs, vst, None)

    for bad in (dict(elem=0), dict(elem=3), dict(head_dim=72), dict(head_dim=272), dict(block=0), dict(block=5), dict(ks=None), dict(vs=ODD),
                dict(kst=None), dict(vst=None), dict(k_stride=(2048, 128, 72)), dict(v_stride=(2040, 128, 64)), dict(k_cache=0x1008),
                dict(q=None), dict(q=ODD), dict(out=None), dict(lens=None), dict(status=None), dict(table=None), dict(batch=-1),
                dict(q_heads=3), dict(page_size=0), dict(num_pages=2 ** 27), dict(max_pages=2 ** 27)):
        assert call(**bad) == BAD, bad
        assert L.spmv_last_error()
    assert L.spmv_paged_attention_e4m3(None, 8, FAKE, S3(4, 2, 1), FAKE, S3(4, 2, 1), None) == BAD
    assert call(batch=0, q=None, lens=None) == 0
    size = ctypes.c_size_t(77)
    work = L.spmv_paged_attention_e4m3_workspace
    assert work(1, 4, 2, 64, 1, None) == BAD
    for args in ((1, 4, 2, 64, 0), (1, 4, 2, 72, 1), (-1, 4, 2, 64, 1), (1, 3, 2, 64, 1), (2 ** 30, 4, 2, 64, 1)):
        assert work(*args, ctypes.byref(size)) == BAD and size.value == 0


def prompt(**kw):
    from load_balanced_csr_gb300.prompt import PromptAttentionArgs
    a = PromptAttentionArgs()
    base = dict(requests=1, tokens=8, keys=8, q_heads=4, kv_heads=2, head_dim=64, elem=1, causal=1, scale=0.1, q_stride=(256, 64),
                k_stride=(128, 64), v_stride=(128, 64), out_stride=(256, 64), q=FAKE, k=FAKE, v=FAKE, q_ptr=FAKE, kv_ptr=None, out=FAKE,
                lse=None, status=FAKE, workspace=None, workspace_bytes=0)
    for name, value in {**base, **kw}.items():
        if isinstance(value, tuple):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return ctypes.byref(a)


def test_prompt_refusals():
    L = lb.lib()
    for bad in (dict(requests=-1), dict(tokens=-1), dict(keys=-1), dict(q_heads=-1), dict(kv_heads=0), dict(q_heads=3), dict(elem=0), dict(elem=3),
                dict(head_dim=0), dict(head_dim=60), dict(head_dim=264), dict(q_heads=258, kv_heads=2), dict(tokens=2 ** 29, q_heads=4),
                dict(q=None), dict(k=None), dict(v=None), dict(q_ptr=None), dict(out=None), dict(status=None), dict(q=0x1008), dict(k=0x1002),
                dict(v=ODD), dict(out=0x1004), dict(q_ptr=ODD), dict(kv_ptr=ODD), dict(lse=ODD), dict(status=ODD), dict(workspace=0x1008),
                dict(q_stride=(260, 64)), dict(k_stride=(128, 68)), dict(v_stride=(4, 64)), dict(out_stride=(256, 60)), dict(q_stride=(0, 64)),
                dict(k_stride=(-128, 64)), dict(v_stride=(128, 0)), dict(q_stride=(2 ** 38, 64)), dict(keys=2 ** 31 - 512), dict(tokens=2 ** 31 - 512, q_heads=1, kv_heads=1)):
        assert L.spmv_prompt_attention(prompt(**bad), None) == BAD, bad
        assert L.spmv_last_error()
    assert L.spmv_prompt_attention(None, None) == BAD
    for nothing in (dict(requests=0, q_ptr=None), dict(tokens=0, q=None, out=None), dict(q_heads=0, q=None)):
        assert L.spmv_prompt_attention(prompt(**nothing), None) == 0, nothing
    size = ctypes.c_size_t(77)
    assert L.spmv_prompt_attention_workspace(4, 2, 64, 1, None) == BAD
    for args in ((3, 2, 64, 1), (4, 2, 60, 1), (4, 2, 64, 0), (4, 0, 64, 1)):
        assert L.spmv_prompt_attention_workspace(*args, ctypes.byref(size)) == BAD and size.value == 0


@pytest.mark.parametrize("struct,module,name", [("spmv_paged_cache_t", "paged_e4m3", "PagedCacheArgs"),
                                                 ("spmv_prompt_attention_t", "prompt", "PromptAttentionArgs")])
def test_structures_match_the_header(struct, module, name, tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    import importlib
    cls = getattr(importlib.import_module(f"load_balanced_csr_gb300.{module}"), name)
    fields = [f[0] for f in cls._fields_]
    source = tmp_path / "layout.c"
    source.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spmv.h"\nint main(void) {\n    printf("%zu\\n", sizeof(' + struct + "));\n" +
                      "".join(f'    printf("%zu\\n", offsetof({struct}, {f}));\n' for f in fields) + "    return 0;\n}\n")
    binary = tmp_path / "layout"
    subprocess.run([gcc, "-I", os.path.join(_build.ROOT, "include"), str(source), "-o", str(binary)], check=True)
    said = [int(x) for x in subprocess.run([str(binary)], check=True, capture_output=True, text=True).stdout.split()]
    assert said == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


SOURCES = ["e4m3.cuh", "tcgen05.cuh", "pages_e4m3.cu", "paged_attention_e4m3.cu", "prompt_attention.cu"]


def code(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_through_the_read_only_path(name):
    """A kernel begins before the one in front of it has ended: what that one writes is there for ordinary loads (and the
    tensor copies issued after the wait) only."""
    assert not re.findall(r"__ldg\w*|__restrict__|ld\.global\.nc", code(name)), name


@pytest.mark.parametrize("name", ["pages_e4m3.cu", "prompt_attention.cu"])
def test_every_kernel_waits_for_the_one_before_it(name):
    text = code(name)
    kernels = list(re.finditer(r"__global__[^{;]*\{", text))
    assert kernels
    for k in kernels:
        body = text[k.end():]
        before = body[:body.index("after_previous();")]
        assert len(before) < 1500 and "__global__" not in before, k.group()[:200]
        for statement in before.split(";")[:-1]:
            assert re.match(r"\s*(using |constexpr |enum |extern __shared__|__shared__|const int lane)", statement), statement.strip()


def test_waits_inside_kernels_end():
    """Every wait on a barrier goes through the bounded one."""
    text = code("prompt_attention.cu") + code("tcgen05.cuh")
    assert "while (!tma::mbar_try_wait" not in text
    assert len(re.findall(r"mbar_try_wait", text)) == 2 and "1ll << 31" in text


def test_registers_handed_over_are_the_launch_s():
    """setmaxnreg.inc waits for registers that others gave back: the shares have to fit what the block was launched with."""
    text = code("prompt_attention.cu")
    down, = map(int, re.findall(r"setmaxnreg\.dec\.sync\.aligned\.u32 (\d+)", text))
    up, = map(int, re.findall(r"setmaxnreg\.inc\.sync\.aligned\.u32 (\d+)", text))
    launched = 65536 // 384 // 8 * 8
    assert 128 * down + 256 * up <= 384 * launched
