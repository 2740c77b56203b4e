"""flashhead_rmsnorm over the whole range of its types: rows whose squares
leave the range of fp32 (tolerances: tests/around_ref.py)."""
import numpy as np
import pytest

from . import around_ref as ref
from .test_gpu_norm import check, fh, rand, run  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 256, 1152, 2056, 8192])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6])
def test_norm_of_rows_at_the_ends_of_the_range(fh, dtype, d, eps):
    sizes = [1e-36, 1e-30, 1e-25, 1e-22, 1e-19, 1e-16, 1e-10, 1.0, 1e10, 1e17, 3e18, 1e20, 1e30,
             1e37]
    x = rand((len(sizes), d), torch.float32, d).clamp(-8, 8)
    x = (x.double() * torch.tensor(sizes, dtype=torch.float64, device="cuda")[:, None]).to(dtype)
    w = rand((d,), dtype, 5, 0.3)
    o = run(fh, x, None, w, 1.0, "both", eps=eps)
    # the scale of a row or block: never below 2^-126, so that codes of values
    # far below it are zero (check_codes counts that)
    check(o, x, None, w, 1.0, float(np.float32(eps)))
    assert torch.all(torch.isfinite(o["y"].float()))


def test_norm_of_rows_that_differ_in_size_do_not_meet(fh):
    # small, ordinary and large rows beside each other, in one workgroup (a
    # wave a row) and in several: each as it is alone
    for d in (256, 2048):
        x = rand((9, d), torch.float32, 3)
        x[1] *= 1e-28
        x[4] *= 1e25
        x[5] = 0.0
        x[5, 7] = 1e-40
        a = run(fh, x, None, None, 0.0, "y", eps=0.0)["y"]
        check(dict(residual_out=None, y=a, y8=None), x, None, None, 0.0, 0.0)
        for i in range(9):
            b = run(fh, x[i:i + 1].contiguous(), None, None, 0.0, "y", eps=0.0)["y"]
            assert torch.equal(a[i], b[0])


def test_norm_rows_without_a_norm(fh):
    # by the definition: 0 / 0 in a row of zeros with eps = 0; a NaN takes its
    # row; an infinity is NaN itself and leaves the row's other values zero
    x = torch.ones(3, 256, device="cuda")
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    y = run(fh, x, None, None, 0.0, "y", eps=0.0)["y"]
    assert torch.all(torch.isnan(y[0])) and torch.all(torch.isnan(y[1]))
    assert torch.isnan(y[2, 3]) and torch.all(y[2, :3] == 0) and torch.all(y[2, 4:] == 0)


def test_norm_residual_sum_of_small_rows(fh):
    for dtype in (torch.bfloat16, torch.float32):
        x = rand((5, 1152), dtype, 1, 1e-24)
        r = rand((5, 1152), dtype, 2, 3e-24)
        check(run(fh, x, r, None, 0.0, "both", eps=0.0), x, r, None, 0.0, 0.0)
