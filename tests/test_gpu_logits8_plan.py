"""Every kernel of dense_logits_fp8, in both output types, against the float64
definition, at the shapes of tests/logits8_shapes.py."""
import numpy as np
import pytest

from . import around_ref as ref
from .logits8_shapes import FAR, SHAPES, ldo
from .test_gpu_logits8 import fh, inputs  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check(fh, rows, v, d, dtype, ld, seed):
    h8, hs, E8, es = inputs(rows, v, d, seed)
    base = torch.full((rows, ld), 5.0, dtype=dtype, device="cuda")
    out = base[:, :v]
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    torch.cuda.synchronize()
    assert torch.all(base[:, v:v + 512] == 5.0)
    z, mag = ref.logits(h8, hs, E8, es)
    # products exact, sums in fp32: the bound of check_logits without the term
    # for products that are cut short
    e = (128 * 2 + 2 + -(-d // 128)) * ref.U32 * 1.001
    got = ref.f64(out)
    assert np.all(np.abs(got - z) <= e * mag + ref.half_step(dtype) * (1.001 * np.abs(z) + e * mag)
                  + 2.0 ** -133)
    # and over all outputs: the rounding to the type (uniform in half a step of
    # at most eps / 2 of the value: eps / 2 / sqrt(3)) and 160 roundings of
    # 2^-24 that add up like a random walk, of partial sums about twice the
    # result
    rms = np.sqrt(np.mean((got - z) ** 2)) / np.sqrt(np.mean(z ** 2))
    assert rms <= ref.half_step(dtype) / 3 ** 0.5 + 2 * 160 ** 0.5 * ref.U32
    again = torch.empty_like(base)[:, :v]
    fh.dense_logits_fp8(h8, hs, E8, es, again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kernel,rows,v,d", SHAPES)
def test_every_kernel(fh, dtype, kernel, rows, v, d):
    size = torch.finfo(dtype).bits // 8
    check(fh, rows, v, d, dtype, ldo(v, size) + 16, rows + d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_out_far_apart(fh, dtype):
    _, rows, v, d, far = FAR
    check(fh, rows, v, d, dtype, far[torch.finfo(dtype).bits // 8], 9)
