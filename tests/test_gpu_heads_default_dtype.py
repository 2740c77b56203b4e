"""The dense heads under another default dtype than fp32, as programs set it that
build their models in bf16."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from two_stage_retrieval_amd import binding as fh  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[torch.bfloat16, torch.float64])
def default(request):
    was = torch.get_default_dtype()
    yield request.param
    torch.set_default_dtype(was)


@pytest.mark.parametrize("head", ["DenseHeadFP8", "DenseHeadInt4"])
def test_calls(head, default):
    g = torch.Generator(device="cuda").manual_seed(1)
    v, d, B, K = 1003, 272, 2, 3
    E = (torch.randn(v, d, generator=g, device="cuda") * 0.05).bfloat16()
    x = torch.randn(B * K, d, generator=g, device="cuda").bfloat16()
    scores = -torch.rand(B, K, generator=g, device="cuda")
    starts = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    drafts = torch.randint(0, v, (4,), generator=g, device="cuda", dtype=torch.int32)

    def run():
        h = getattr(fh, head)(E, max_rows=B * K, max_sequences=B)
        out = [h.logits(x), *h.verify(x, starts, drafts, 3, mode=fh.FH_MODE_GREEDY),
               *h.beam_select(x, scores, 2 * K)]
        if head == "DenseHeadInt4":
            out.append(h.rows(drafts))
        return out

    want = run()
    torch.set_default_dtype(default)
    got = run()
    assert all(torch.equal(a, b) and a.dtype == b.dtype for a, b in zip(got, want))
