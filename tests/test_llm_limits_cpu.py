"""Sizes and limits of the language-model operators' C entry points."""
import ctypes

import load_balanced_csr_gb300 as lb


def test_route_workspace_never_shrinks():
    """A workspace sized for more tokens serves fewer."""
    L, size, last = lb.lib(), ctypes.c_size_t(), 0
    edges = [0, 1, 131072, 131073, 1245184, 1245185, 2490368, 2490369, 3735552, 3735553, 2 ** 30, 2 ** 31 - 1]
    for n in sorted(set(edges + [8192 * i + d for i in range(1, 700) for d in (0, 1)])):
        assert L.spmv_route_workspace(n, 1, 2048, ctypes.byref(size)) == 0
        assert size.value >= last, n
        last = size.value


def test_rows_of_nearly_2_31_elements_are_refused():
    """A lane's place in a row is counted in 32 bits, up to 1,024 elements past its end."""
    L, fake, bad = lb.lib(), ctypes.c_void_p(0x1000), 1
    for hidden in (2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 1024):
        assert L.spmv_route_dispatch(1, 1, hidden, 1, fake, fake, hidden, fake, hidden, None) == bad
        assert L.spmv_route_combine(1, 1, hidden, 1, fake, None, 0, fake, hidden, fake, hidden, None) == bad
        assert L.spmv_route_combine_backward(1, 1, hidden, 1, fake, None, 0, fake, hidden, fake, hidden, fake, hidden, fake, 1,
                                             None) == bad
    assert L.spmv_route_dispatch(0, 1, 2 ** 31 - 1025, 1, None, None, 2 ** 31, None, 2 ** 31, None) == 0


def append(L, requests=100, work=0x900000, room=1 << 20, **at):
    """spmv_pages_append with arguments that do not overlap, but for those given."""
    p = dict(past=0x100000, fresh=0x200000, table=0x300000, free=0x400000, ptr=0x500000, lens=0x600000, slots=0x700000,
             positions=0x800000, taken=0xa00000, status=0xb00000)
    p.update(at)
    return L.spmv_pages_append(requests, p["past"], p["fresh"], 16, 100, p["free"], 50, p["table"], 8, 8, 300, p["ptr"], p["lens"],
                               p["slots"], p["positions"], p["taken"], p["status"], work, room, None)


def test_outputs_of_an_append_may_not_overlap_the_lengths():
    """Every block reads past and fresh while others write."""
    L = lb.lib()
    for name in ("past", "fresh"):
        base = 0x100000
        for out, length in (("lens", 100), ("ptr", 101), ("slots", 300), ("positions", 300)):
            for off in (-4 * (length - 1), -4, 0, 4, 4 * 99):
                assert append(L, **{name: base, out: base + off, "fresh" if name == "past" else "past": 0x200000}) == 1, (name, out, off)
                assert b"overlap" in L.spmv_last_error()


def test_workspace_of_an_append():
    """Needed above 4,096 requests only, and then whole and aligned."""
    L, size = lb.lib(), ctypes.c_size_t(77)
    assert L.spmv_pages_workspace(4096, ctypes.byref(size)) == 0 and size.value == 0
    assert L.spmv_pages_workspace(5000, ctypes.byref(size)) == 0 and size.value > 0
    for work, room in ((None, size.value), (0x900000, size.value - 1), (0x900000, 0), (0x900008, size.value)):
        assert append(L, requests=5000, work=work, room=room) == 1
        assert b"workspace" in L.spmv_last_error()
