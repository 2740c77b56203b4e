"""The 4-bit copy of an E that holds NaNs of either kind: they get the code 0 and
take no part in the scales."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from two_stage_retrieval_amd import binding as fh  # noqa: E402

from . import int4_ref as ref  # noqa: E402
from .test_gpu_int4 import BF16, F32, copy_room, gen  # noqa: E402

pytestmark = pytest.mark.gpu

# quiet and signalling ones, of either sign
BITS = {BF16: (torch.int16, [0x7FC0, 0x7F81, 0x7FC0 - 0x8000, 0x7F81 - 0x8000]),
        F32: (torch.int32, [0x7FC00000, 0x7F800001, 0x7FC00000 - 2 ** 31, 0x7F800001 - 2 ** 31])}


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_nan_anywhere_beside_the_largest_value(dtype, zero, group):
    """In each row the group's largest (and, with zeros, smallest) value and a NaN in
    the same eight columns, the one before the other in every pair of places."""
    kind, nans = BITS[dtype]
    places = [(a, b, n) for n in nans for a in range(8) for b in range(8) if a != b]
    v, d = len(places), 144
    plain = torch.randn(v, d, generator=gen(group), device="cuda").to(dtype)
    for r, (big, nan, _) in enumerate(places):
        plain[r, 40 + big] = 50.0 if r % 2 else -50.0
        plain[r, 40 + nan] = 0.0
    bits = plain.view(kind).clone()
    for r, (_, nan, n) in enumerate(places):
        bits[r, 40 + nan] = n
    E = bits.view(dtype)
    assert int(torch.isnan(E).sum()) == v
    (E4, scale, z), _ = copy_room(v, d, group, zero)
    fh.flashhead_quantize_int4(E, E4, scale, z, group=group)
    q, s64, z64 = ref.quantize(plain, group, zero)
    for r, (_, nan, _) in enumerate(places):
        q[r, 40 + nan] = 0
    assert np.array_equal(ref.f64(scale), s64) and np.array_equal(ref.unpack(E4), q)
    assert z is None or np.array_equal(ref.f64(z), z64)
