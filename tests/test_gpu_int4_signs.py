"""The 4-bit logits for an h of one sign, where sums with 24 + code are large beside
the logits, and zeros that are no whole numbers."""
from __future__ import annotations

import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from two_stage_retrieval_amd import binding as fh  # noqa: E402

from . import int4_ref as ref  # noqa: E402
from .logits4_shapes import SHAPES  # noqa: E402
from .test_gpu_int4 import BF16, F32, gen, random_copy, room  # noqa: E402

pytestmark = pytest.mark.gpu


def in_the_mean(h, scale, zero, group):
    """The size that errors of fp32 sums have in the mean, for each logit.  A group's
    sum of -h takes 128 additions whose roundings count 24 + |z| times, and 128 of
    products follow (three parts of h each, of which the lower two are 2^-8 of the
    first); 24 + z, its product with the sum and the product with the scale are one
    more each.  No sum is over (31 + |z|) sum |h| = A, so a rounding is at most 2^-24 A
    and in the mean 2^-24 A / sqrt(3); 3 * 128 + 8 that are independent add up to
    sqrt(392 / 3) < 11.5 times 2^-24 A, and groups by their squares.  The sum over
    groups adds a rounding of the logit itself a group."""
    a = np.abs(ref.f64(h))
    s, G = ref.f64(scale), scale.shape[0]
    z = np.abs(ref.f64(zero)) if zero is not None else np.zeros_like(s)
    total = np.zeros((a.shape[0], s.shape[1]))
    for g in range(G):
        total += np.outer(a[:, g * group:(g + 1) * group].sum(1), s[g] * (31 + z[g])) ** 2
    return 11.5 * 2.0 ** -24 * np.sqrt(total)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("group,zero", itertools.product((32, 64, 128), (False, True)))
@pytest.mark.parametrize("kind,name,rows,v,d",
                         [(h, *s) for h in ("bf16", "f32") for s in SHAPES[h]])
def test_one_sign(kind, name, rows, v, d, group, zero, sign):
    E4, scale, z = random_copy(v, d, group, zero, rows + v + d)
    if zero:
        z.clamp_(-15, 15)
    h, _ = room(rows, d, BF16 if kind == "bf16" else F32)
    h.copy_((torch.rand(rows, d, generator=gen(d), device="cuda") + 0.5) * sign)
    out, _ = room(rows, v, F32)
    fh.dense_logits_int4(h, E4, scale, out, E_zero=z, group=group)
    want = ref.f64(h) @ ref.values(E4, scale, z, group).T
    off = np.abs(ref.f64(out) - want)
    assert np.all(off <= ref.logits_bound(h, E4, scale, z, group))
    G = scale.shape[0]
    mean = in_the_mean(h, scale, z, group)
    assert np.linalg.norm(off) <= np.linalg.norm(mean) + \
        G ** 0.5 * 2.0 ** -24 * np.linalg.norm(want)
