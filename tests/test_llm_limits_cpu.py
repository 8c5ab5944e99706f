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
