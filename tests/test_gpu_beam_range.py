"""Beam search's selection for logits of any finite size: scores that a large
logit must not absorb."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from . import int4_ref as ref  # noqa: E402
from .test_gpu_beam import BF16, F32, check, gen, padded, select  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [1, 20, 5003])
def test_a_beam_masked_by_the_lowest_value_beside_live_ones(v, dtype):
    """All of a beam's tokens are alike: each has the probability 1 / v, so its
    candidates come with the beam's score - log(v), tokens in order."""
    B, K, n = 3, 4, 64
    logits = padded(B * K, v, dtype)
    logits.copy_(torch.randn(B * K, v, generator=gen(v), device="cuda") * 2.5)
    lowest = torch.finfo(dtype).min
    logits[2] = lowest                  # the third beam of four
    logits[4:8] = lowest                # every beam
    logits[8] = -lowest                 # and the largest value
    scores = torch.tensor([[-1.0, -2.0, -20.0, -3.0], [-4.0, -3.0, -12.5, -3.5],
                           [-30.0, -0.5, -1.5, -0.25]], device="cuda")
    out = select(logits, scores, n)
    check(out, logits, scores, n)
    got, parent, token = (x.cpu().numpy() for x in out[:3])

    def near(x, want):   # a few roundings in fp64, then one to fp32
        return np.all(np.abs(x.astype(np.float64) - want) <= abs(want) * (2.0 ** -24 + 2.0 ** -48))

    # every beam alike: by their scores, and within one by the token
    order = np.argsort(-scores[1].cpu().numpy(), kind="stable")
    want = [(k, t) for k in order for t in range(v)][:n]
    there = len(want)
    assert [tuple(x) for x in zip(parent[1][:there], token[1][:there])] == want
    for k in range(K):
        assert near(got[1][parent[1] == k], float(scores[1, k]) - math.log(v))
    # beside live beams: no candidate of theirs comes behind it for its size alone
    if v == 1:
        assert list(parent[0][:K]) == [0, 1, 3, 2] and list(parent[2][:K]) == [3, 1, 2, 0]
    if v == 5003:
        assert not (parent[0] == 2).any() and not (parent[2] == 0).any()
    for s, k in ((0, 2), (2, 0)):
        assert near(got[s][parent[s] == k], float(scores[s, k]) - math.log(v))


@pytest.mark.parametrize("size", [0.0, 1.0, 2.0 ** 20, -2.0 ** 20, -2.0 ** 29])
def test_scores_do_not_change_with_a_number_added_to_a_row(size):
    """A logit more or less for all of a row's tokens (all of them fp32 numbers)
    changes nothing, however large it is."""
    v, K, n = 5003, 4, 16
    logits = padded(K, v, F32)
    step = max(2.0 ** -20, abs(size) * 2.0 ** -23)
    whole = torch.randint(-4, 5, (K, v), generator=gen(3), device="cuda").float()
    whole = torch.where(whole == 4, whole * (1 + (torch.arange(v, device="cuda") % 9 == 0)), whole)
    scores = torch.tensor([[-1.0, -0.5, -2.0, -0.25]], device="cuda")
    logits.copy_(whole * step)
    plain = select(logits, scores, n)
    logits.copy_(whole * step + size)
    check(plain, whole * step, scores, n)
    moved = select(logits, scores, n)
    assert all(torch.equal(a, b) for a, b in zip(plain, moved))


@pytest.mark.parametrize("K,v,dtype", [(32, 524288, BF16), (1, 1 << 24, F32), (31, 540671, F32)])
def test_the_largest_sequences(K, v, dtype):
    """K * ceil(v / 2048) of 8192 and just below it, the most candidates that there
    can be, the best ones in the last beam's last tokens."""
    n = 64
    logits = padded(K, v, dtype)
    logits.normal_(generator=gen(K))
    logits[K - 1, v - 40:] += 9.0
    scores = torch.linspace(-0.5, 0.0, K, device="cuda")[None].contiguous()
    out = select(logits, scores, n)
    key = scores[0].cpu().double()[:, None] + torch.log_softmax(logits.cpu().double(), 1)
    order = torch.sort(key.view(-1), descending=True, stable=True)[1][:n]
    assert torch.equal(out[1][0].cpu().long(), order // v)
    assert torch.equal(out[2][0].cpu().long(), order % v)
    best = key.view(-1)[order]
    assert bool(((out[0][0].cpu().double() - best).abs() <= best.abs() * 2.0 ** -24 + 1e-11).all())
