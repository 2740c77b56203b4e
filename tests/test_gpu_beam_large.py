"""Beam search's selection for logits of any finite size."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from .test_gpu_beam import BF16, F32, check, gen, padded, select  # noqa: E402

pytestmark = pytest.mark.gpu

LARGE = [2.0 ** 31, 3e9, 1e10, 1.8e10, 1e12, 1e15, 3e19, 9e19, 1e20, 4e20, 5e20, 8e24, 2e25, 1e30,
         1.6e38]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", LARGE)
def test_large_logits(size, dtype):
    """One large logit among ordinary ones, masks of that size for a whole chunk of
    a row, for most of it and for all of it."""
    v, n = 5003, 8
    g = gen(5)
    plain = padded(2, v, dtype)
    plain.copy_(torch.randn(2, v, generator=g, device="cuda") * 2.5)

    def best(rows, scores):
        logits = padded(len(rows), v, dtype)
        for r, row in enumerate(rows):
            logits[r] = row
        scores = torch.tensor([scores], device="cuda")
        out = select(logits, scores, n)
        check(out, logits, scores, n)
        return [x.cpu().numpy()[0] for x in out]

    one = plain[0].clone()
    one[2500] = size
    for scores in ([-0.25, -1.5], [-7.0, -0.125]):
        s, p, t, _ = best([one, plain[1]], scores)
        # its probability is 1, so a beam with the better score comes first with it
        assert scores[0] < scores[1] or (p[0], t[0]) == (0, 2500)
    s, p, t, _ = best([one], [-0.5])
    assert t[0] == 2500 and np.all(s[1:] < -0.99 * float(one[2500]))
    one[2500] = -size
    best([plain[1], one], [-1.0, 0.0])
    chunk, most = plain[0].clone(), plain[1].clone()
    chunk[2048:4096] = -size
    most[torch.rand(v, generator=g, device="cuda") < 0.97] = -size
    best([chunk, most], [-0.75, 0.0])
    for s0 in (-size, size):
        s, p, t, _ = best([torch.full_like(one, s0)], [-2.5])
        assert list(t) == list(range(n)) and not p.any()
