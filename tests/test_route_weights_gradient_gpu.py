"""The weights' gradient is one dot product per entry, summed in parts so that
no part is long: with 32 lanes and 8 partial sums a lane, a sum of h products
of one value x makes partial sums of at most n = ceil(h / 256) + 8 terms (the
last turn of a lane may be uneven).  The i-th addition is off by at most v i x
(v = 2^-24), n / 2 + 1 units of the whole in all, and joining the parts adds 3
+ 5 more: |dw - dw64| <= (n / 2 + 9) v |dw64|."""
import pytest

pytestmark = pytest.mark.gpu

V = 2.0 ** -24


@pytest.mark.parametrize("hidden", [1 << 16, (1 << 16) + 1, 1 << 18, (1 << 18) + 1])  # in vectors, and element by element
@pytest.mark.parametrize("below", [12, 13, 14, 15, 16, 17])
def test_equal_products(below, hidden):
    """Just below half of a step of some partial sums, where each addition rounds the same way."""
    import torch
    import load_balanced_csr_gb300 as lb
    x = 1 + 0.49 * 2.0 ** -below
    route = lb.ExpertRoute(2, 1, 1).build(torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    ys = torch.full((2, hidden), x, device="cuda")
    _, dw = route.combine_backward(torch.ones(2, hidden, device="cuda"), ys, torch.ones(2, 1, device="cuda"))
    want = hidden * float(ys[0, 0].double())
    n = -(-hidden // 256) + 8
    assert float((dw.double() - want).abs().max()) <= (n / 2 + 9) * V * want
