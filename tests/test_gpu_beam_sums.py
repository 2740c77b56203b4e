"""The sums behind beam search's scores, to their last digits: a beam's score near
the logarithm of its row's sum leaves their difference, with fp32's relative step."""
from __future__ import annotations

from decimal import Decimal, localcontext

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from .test_gpu_beam import BF16, F32, gen, padded, select  # noqa: E402

pytestmark = pytest.mark.gpu

# Of the sum: the weights' polynomial 4e-14; some 60 roundings of 2^-53 on the way
# (a weight's own, a lane's 16 values, the wave, the chunks).  The logarithm, up to 10,
# and its difference from the score: two roundings of 2^-50.
BOUND = 4e-14 + 60 * 2.0 ** -53 + 2 * 2.0 ** -50


def logs(rows):
    """log(sum exp(x)) of each row with 40 digits."""
    with localcontext() as c:
        c.prec = 40
        out = []
        for row in rows:
            values, counts = torch.unique(row.double().cpu(), return_counts=True)
            out.append(sum(Decimal(float(x)).exp() * int(n)
                           for x, n in zip(values, counts)).ln())
    return out


def check_sums(logits, first):
    want = logs(logits)
    scores = torch.tensor([[float(x)] for x in want], dtype=F32)   # (rounded)
    out = select(logits, scores.cuda(), 1)
    assert bool((out[2][:, 0].cpu() == first).all())
    for got, score, x in zip(out[0][:, 0].cpu(), scores[:, 0], want):
        left = Decimal(float(score)) - x
        assert abs(Decimal(float(got)) - left) <= abs(left) * Decimal(2.0 ** -24) + \
            Decimal(BOUND), (float(got), float(left))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [2, 511, 4097])
def test_one_value_beside_the_largest(v, dtype):
    """Every fraction that the exponential is made of, alone in its row."""
    logits = padded(64, v, dtype)
    logits.copy_(-torch.linspace(0.01, 7.0, 64, device="cuda")[:, None])
    logits[:, v // 2] = 0.0
    check_sums(logits, v // 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_values_over_many_chunks(dtype):
    v = 20011
    logits = padded(8, v, dtype)
    logits.copy_(-torch.randint(1, 90, (8, v), generator=gen(6), device="cuda") * 0.09375)
    logits[:, 17000] = 0.0
    check_sums(logits, 17000)
