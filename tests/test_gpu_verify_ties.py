"""Draws whose uniform number falls exactly on a border between two tokens:
equal logits have equal weights, so that the running sums of a row of equal
logits are exact multiples of one weight."""
import pytest

from .test_gpu_verify import fh  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
INF = float("inf")


def draw(fh, logits, u, tau=1.0):
    """One plain draw (no drafts) per row."""
    B, v = logits.shape
    out = torch.empty(B, 1, dtype=torch.int32, device="cuda")
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(fh.flashhead_verify_workspace_bytes(B, B, v), dtype=torch.uint8,
                     device="cuda")
    fh.flashhead_verify(logits, torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                        torch.empty(0, dtype=torch.int32, device="cuda"), out, acc, ws, tau=tau,
                        u_accept=torch.empty(0, device="cuda"), u_sample=u)
    return out[:, 0].cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [1, 4, 10, 12, 15, 17])
def test_uniform_row_at_the_borders(fh, dtype, bits):
    # v = 2^bits equal logits and u = k / v: the smallest t with t + 1 > k is k
    v = 1 << bits
    B = min(v, 2048)
    k = torch.arange(B) * (v // B) + (torch.arange(B) % (v // B) if v > B else 0)
    u = (k.double() / v).float().cuda()
    z = torch.full((B, max(v, 8)), -1.5, dtype=dtype, device="cuda")[:, :v]  # 16-byte rows
    assert torch.equal(draw(fh, z, u, 0.7), k.int())


def test_equal_tokens_among_masked_ones(fh):
    # 2^9 equal tokens left by a mask, anywhere in the row
    v, left = 9000, 512
    g = torch.Generator().manual_seed(3)
    at = torch.randperm(v, generator=g)[:left].sort().values
    z = torch.full((left, v), -INF)
    z[:, at] = 4.25
    u = (torch.arange(left).double() / left).float().cuda()
    assert torch.equal(draw(fh, z.cuda(), u, 1.3), at.int())


def test_equal_masked_at_the_lowest_value(fh):
    # every token at the type's lowest value: a uniform row
    for dtype in (torch.float32, torch.bfloat16):
        v = 4096
        z = torch.full((1024, v), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        k = torch.arange(1024) * 4 + 1
        assert torch.equal(draw(fh, z, (k.double() / v).float().cuda()), k.int())
