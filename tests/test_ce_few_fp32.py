"""The linear cross entropy of 16 to 33 fp32 rows in split arithmetic, on either side of the
widths at which the kernel changes; the bounds are those of test_linear_ce.py."""
import pytest

from test_linear_ce import both, check_grads, check_loss, make, on_gpu, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [16, 17, 25, 32, 33])
@pytest.mark.parametrize("D,pad", [(1536, 0), (1537, 0), (1600, 3), (4100, 1)])
def test_split_rows_on_either_kernel(T, D, pad):
    h, w, y, up = make(T, 1031, D, "f32", T + D, spread=2.0)
    y[1::5] = -100
    r = reference(h, w, y, up)
    h[1::5] = float("nan")
    loss, lse, dh, dw = both(on_gpu(h, pad), on_gpu(w, pad), y.cuda(), up.cuda(), "f32", "3xtf32")
    check_loss(loss, lse, r)
    check_grads(dh, dw, r, "f32")
    assert not dh[1::5].any()
