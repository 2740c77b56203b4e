"""dense_logits_fp8 takes the products of two codes in full, whatever the
number of rows and the type of the output (tolerances: tests/around_ref.py and
beside each check)."""
import numpy as np
import pytest

from . import around_ref as ref
from .test_gpu_logits8 import F8, fh, inputs  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROWS = [1, 16, 17, 40, 130, 333]


def bits_apart(rows, v, d, seed):
    """Whole-number codes whose products in a group of 8 columns are one of
    448^2 and seven of at most 4; the large ones cancel over a block of 128."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randint(-2, 3, (rows, d), generator=g).float()
    E = torch.randint(-2, 3, (v, d), generator=g).float()
    for c in range(0, d, 8):
        at = c + int(torch.randint(0, 8, (1,), generator=g))
        h[:, at] = 448.0
        E[:, at] = 448.0 if (c // 8) % 2 else -448.0
    return h.to(F8).cuda(), E.to(F8).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("v,d", [(300, 128), (1000, 512), (20000, 384)])
def test_logits_keep_every_bit_of_a_product(fh, dtype, rows, v, d):
    # Every partial sum is a multiple of 1/2 below 2^23 (16 groups of 448^2
    # times a scale of 2 are 2^22.7), so fp32 holds it in any order of
    # summation, and the result is the definition's, rounded once.
    h8, E8 = bits_apart(rows, v, d, rows + d)
    g = torch.Generator().manual_seed(7)
    hs = 2.0 ** torch.randint(0, 2, (rows, d // 128), generator=g).float().cuda()
    es = 2.0 ** torch.randint(-1, 1, (-(-v // 128), d // 128), generator=g).float().cuda()
    out = torch.empty(rows, -(-v // 8) * 8, dtype=dtype, device="cuda")[:, :v]
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    z, _ = ref.logits(h8, hs, E8, es)
    assert np.abs(z).max() < 2.0 ** 24
    assert torch.equal(out.cpu(), torch.from_numpy(z).to(dtype))


@pytest.mark.parametrize("rows,v,d", [(16, 4000, 1104), (17, 4000, 1104), (300, 9000, 1104),
                                      (64, 40000, 512), (600, 12000, 2048)])
def test_logits_to_bf16_are_the_rounded_sums(fh, rows, v, d):
    # A sum of d + d / 128 terms in fp32 is off by about sqrt(d) / 2 roundings
    # of 2^-24 of its size, 1.4e-6 at d = 2048; it then rounds to another bf16
    # value where it is that near to a midpoint: those lie 2^-8 or more of the
    # value apart, so in at most 1.4e-6 / 2^-9 = 7e-4 of the outputs (smaller
    # sums, which cancel, have the midpoints closer: five times as many).
    h8, hs, E8, es = inputs(rows, v, d, 3)
    out = torch.empty(rows, v, dtype=torch.bfloat16, device="cuda")
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    z, mag = ref.logits(h8, hs, E8, es)
    want = torch.from_numpy(z).to(torch.bfloat16)
    assert (out.cpu() != want).double().mean().item() < 4e-3
    # and each within the sum's own error of it (the bound of check_logits for fp32)
    e = (128 * 2 + 2 + -(-d // 128)) * ref.U32 * 1.001
    assert np.all(np.abs(ref.f64(out) - z) <= e * mag + ref.half_step(torch.bfloat16)
                  * (1.001 * np.abs(z) + e * mag))
