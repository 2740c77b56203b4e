"""What flashhead_quantize_fp8 makes of values that are not finite."""
import pytest

from .test_gpu_norm import F8, fh, rand  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity(fh, dtype):
    v, d = 300, 384

    def codes(E):
        E8 = torch.empty(v, d, dtype=F8, device="cuda")
        es = torch.empty(3, 3, device="cuda")
        fh.flashhead_quantize_fp8(E, E8, es)
        return E8.float(), es

    E = rand((v, d), dtype, 4, 0.02)
    a, sa = codes(E)
    bad = E.clone()
    bad[5, 130] = float("nan")
    bad[140, 3] = float("inf")
    bad[141, 260] = float("-inf")
    b, sb = codes(bad)
    # a NaN has the NaN code and takes no part in its block's maximum
    assert torch.isnan(b[5, 130])
    E[5, 130] = 0.0
    a, sa = codes(E)
    keep = torch.ones(v, d, dtype=torch.bool, device="cuda")
    keep[5, 130] = False
    keep[128:256, 0:128] = False
    keep[128:256, 256:384] = False
    assert torch.equal(a[keep], b[keep])
    # an infinity makes its block's scale infinite: its code is NaN, the others
    # 0, and none of the block's values can be read back
    inf = torch.zeros(3, 3, dtype=torch.bool, device="cuda")
    inf[1, 0] = inf[1, 2] = True
    assert torch.all(torch.isinf(sb[inf])) and torch.equal(sa[~inf], sb[~inf])
    for r, c in ((140, 3), (141, 260)):
        j = c // 128 * 128
        block = b[128:256, j:j + 128].clone()
        assert torch.isnan(block[r - 128, c - j])
        block[r - 128, c - j] = 0
        assert torch.all(block == 0)
