"""The language-model operators' C entry points refuse bad arguments before
touching the device, size their workspaces, and lay out their argument
structure as the header does."""
import ctypes
import shutil
import subprocess

import pytest

import load_balanced_csr_gb300 as lb
from load_balanced_csr_gb300 import _build

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
OTHER = ctypes.c_void_p(0x2000)
BAD = 1


def test_the_operators_are_exported():
    names = set(lb.header_functions())
    assert {"spmv_route_build", "spmv_route_dispatch", "spmv_route_combine", "spmv_route_combine_backward",
            "spmv_pages_append", "spmv_paged_store", "spmv_paged_attention"} <= names
    for L in (lb.lib(), lb.debug_lib()):
        for name in names:
            assert hasattr(L, name), name


def test_route_refusals():
    L = lb.lib()
    size = ctypes.c_size_t(77)
    assert L.spmv_route_workspace(10, 2, 4, None) == BAD
    for args in ((-1, 2, 4), (1, -2, 4), (1, 2, 0), (1, 2, 2049), (2 ** 30, 2, 4)):
        assert L.spmv_route_workspace(*args, ctypes.byref(size)) == BAD and size.value == 0
        assert lb.lib().spmv_last_error()
    assert L.spmv_route_workspace(100000, 8, 256, ctypes.byref(size)) == 0 and size.value % (257 * 4) == 0
    need = size.value
    build = lambda *a: L.spmv_route_build(*a, None)
    assert build(1, 2, 4, FAKE, 2, 2, FAKE, FAKE, FAKE, None, 0) == BAD          # ids of 2 bytes
    assert build(1, 2, 4, None, 4, 2, FAKE, FAKE, FAKE, None, 0) == BAD          # no ids
    assert build(1, 2, 4, FAKE, 4, 2, None, FAKE, FAKE, None, 0) == BAD
    assert build(1, 2, 4, FAKE, 4, 2, FAKE, None, FAKE, None, 0) == BAD
    assert build(1, 2, 4, ODD, 4, 2, FAKE, FAKE, FAKE, None, 0) == BAD           # misaligned
    assert build(100000, 8, 256, FAKE, 8, 8, FAKE, FAKE, FAKE, None, need) == BAD
    assert build(100000, 8, 256, FAKE, 8, 8, FAKE, FAKE, FAKE, FAKE, need - 1) == BAD
    assert build(100000, 8, 256, FAKE, 8, 8, FAKE, FAKE, FAKE, ctypes.c_void_p(0x1004), need) == BAD
    assert L.spmv_route_dispatch(1, 2, 8, 3, FAKE, FAKE, 8, FAKE, 8, None) == BAD   # element type
    assert L.spmv_route_dispatch(1, 2, -8, 0, FAKE, FAKE, 8, FAKE, 8, None) == BAD
    assert L.spmv_route_dispatch(1, 2, 8, 0, FAKE, FAKE, 8, FAKE, 7, None) == BAD   # rows overlap
    assert L.spmv_route_dispatch(1, 2, 8, 0, None, FAKE, 8, FAKE, 8, None) == BAD
    assert L.spmv_route_dispatch(1, 2, 8, 0, FAKE, ODD, 8, FAKE, 8, None) == BAD
    assert L.spmv_route_dispatch(0, 2, 8, 0, None, None, 8, None, 8, None) == 0     # nothing to do
    assert L.spmv_route_combine(1, 2, 8, 0, FAKE, None, 0, FAKE, 8, None, 8, None) == BAD
    assert L.spmv_route_combine(1, 2, 8, 0, FAKE, None, 0, FAKE, 8, FAKE, 4, None) == BAD
    assert L.spmv_route_combine(2 ** 20, 2 ** 11, 8, 0, FAKE, None, 0, FAKE, 8, FAKE, 8, None) == BAD
    back = L.spmv_route_combine_backward
    assert back(1, 2, 8, 1, FAKE, None, 0, FAKE, 8, FAKE, 8, None, 8, FAKE, 2, None) == BAD
    assert back(1, 2, 8, 1, FAKE, None, 0, FAKE, 8, None, 8, FAKE, 8, FAKE, 2, None) == BAD   # dweights need ys
    assert back(1, 2, 8, 1, FAKE, None, 0, FAKE, 8, FAKE, 8, FAKE, 8, FAKE, 1, None) == BAD
    assert back(1, 2, 8, 1, FAKE, None, 0, FAKE, 8, FAKE, 8, FAKE, 16, FAKE, 2, None) == BAD  # in place, other stride


def test_pages_refusals():
    L = lb.lib()
    size = ctypes.c_size_t()
    assert L.spmv_pages_workspace(-1, ctypes.byref(size)) == BAD and L.spmv_pages_workspace(1, None) == BAD
    assert L.spmv_pages_workspace(100, ctypes.byref(size)) == 0

    def append(requests=2, past=FAKE, fresh=FAKE, page=16, num_pages=10, free=FAKE, num_free=4, table=FAKE, ld=8,
               max_pages=8, max_tokens=5, ptr=FAKE, lens=OTHER, slots=FAKE, positions=FAKE, taken=FAKE, status=FAKE,
               work=FAKE, room=1 << 20):
        return L.spmv_pages_append(requests, past, fresh, page, num_pages, free, num_free, table, ld, max_pages,
                                   max_tokens, ptr, lens, slots, positions, taken, status, work, room, None)

    for bad in (dict(requests=-1), dict(page=0), dict(num_pages=-1), dict(num_free=-1), dict(max_pages=-1, ld=0),
                dict(max_tokens=-1), dict(num_pages=2 ** 27), dict(past=None), dict(fresh=None), dict(lens=None),
                dict(ptr=None), dict(taken=None), dict(status=None), dict(table=None), dict(ld=7), dict(free=None),
                dict(slots=None), dict(positions=None), dict(lens=FAKE)):
        assert append(**bad) == BAD, bad
    if size.value:
        assert append(work=None) == BAD and append(room=0) == BAD

    s2, s3 = (ctypes.c_int64 * 2)(64, 8), (ctypes.c_int64 * 3)(512, 64, 8)

    def store(tokens=1, heads=8, dim=8, elem=0, slots=FAKE, pages=4, page=8, k=FAKE, ks=s2, kc=FAKE, kcs=s3):
        return L.spmv_paged_store(tokens, heads, dim, elem, slots, pages, page, k, ks, FAKE, s2, kc, kcs, FAKE, s3, None)

    for bad in (dict(tokens=-1), dict(heads=-1), dict(dim=-1), dict(elem=5), dict(slots=None), dict(pages=-1),
                dict(page=0), dict(pages=2 ** 28), dict(k=None), dict(ks=None), dict(kc=None), dict(kcs=None),
                dict(k=ODD), dict(heads=2 ** 20, dim=2 ** 11)):
        assert store(**bad) == BAD, bad
    assert store(tokens=0, slots=None) == 0


def args(**kw):
    from load_balanced_csr_gb300.paged import PagedAttentionArgs
    a = PagedAttentionArgs()
    base = dict(batch=1, q_heads=4, kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages=4, elem=1, scale=0.1,
                table_stride=4, q=0x1000, k_cache=0x1000, v_cache=0x1000, table=0x1000, lens=0x1000, out=0x1000,
                workspace=0x1000, workspace_bytes=1 << 40, status=0x1000)
    strides = dict(q_stride=(256, 64), k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), out_stride=(256, 64))
    for name, value in {**base, **strides, **kw}.items():
        if isinstance(value, tuple):
            getattr(a, name)[:] = value
        else:
            setattr(a, name, value)
    return ctypes.byref(a)


def test_attention_refusals():
    L = lb.lib()
    assert L.spmv_paged_attention(None, None) == BAD
    for bad in (dict(batch=-1), dict(kv_heads=3), dict(kv_heads=0), dict(q_heads=-4), dict(head_dim=60),
                dict(head_dim=264), dict(head_dim=0), dict(elem=3), dict(page_size=0), dict(num_pages=-1),
                dict(num_pages=2 ** 27), dict(max_pages=-1), dict(q=None), dict(out=None), dict(lens=None),
                dict(status=None), dict(table=None), dict(k_cache=None), dict(v_cache=None), dict(q=0x1001),
                dict(k_cache=0x1008), dict(v_cache=0x1002), dict(k_stride=(2048, 132, 64)),
                dict(v_stride=(2052, 128, 64)), dict(v_stride=(2048, 128, 65))):
        assert L.spmv_paged_attention(args(**bad), None) == BAD, bad
    assert L.spmv_paged_attention(args(batch=0), None) == 0


def test_attention_refuses_rows_past_32_bits():
    """A request's elements are counted in 32 bits."""
    L = lb.lib()
    size = ctypes.c_size_t(77)
    assert L.spmv_paged_attention_workspace(1, 2 ** 23, 1, 256, 1, ctypes.byref(size)) == BAD and size.value == 0
    assert L.spmv_paged_attention(args(q_heads=2 ** 23, kv_heads=1, head_dim=256, max_pages=1), None) == BAD


def test_attention_arguments_match_the_header(tmp_path):
    from load_balanced_csr_gb300.paged import PagedAttentionArgs
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in PagedAttentionArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spmv.h"\nint main(void) {\n'
                   + '    printf("%zu\\n", sizeof(spmv_paged_attention_t));\n'
                   + "".join(f'    printf("%zu\\n", offsetof(spmv_paged_attention_t, {n}));\n' for n in names)
                   + "    return 0;\n}\n")
    subprocess.run([cc, "-I", _build.INCLUDE, str(src), "-o", str(tmp_path / "layout")], check=True, capture_output=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()]
    assert got[0] == ctypes.sizeof(PagedAttentionArgs)
    assert got[1:] == [getattr(PagedAttentionArgs, n).offset for n in names]
