"""The dense heads behind their norm refuse what they could never project, before
they make anything, without a GPU."""
from __future__ import annotations

import pytest

from .test_around_host import LIB, fh  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("head", ["DenseHeadFP8", "DenseHeadInt4"])
def test_widths_that_the_norm_does_not_take(fh, head):
    make = getattr(fh, head)
    with pytest.raises(ValueError, match="8192 at most"):
        make(torch.zeros(16, fh.FH_MAX_NORM_D + 16))
    with pytest.raises(ValueError, match="multiple of 16"):
        make(torch.zeros(16, 40))
