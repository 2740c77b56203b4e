"""DenseHeadFP8 on streams: given as a raw handle, the default stream's among
them."""
import pytest

from .test_gpu_around_head import fh, rand  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_the_default_streams_handle(fh):
    # the default stream's handle is 0: tensors for it are its own, also when
    # another stream is current
    assert torch.cuda.default_stream().cuda_stream == 0
    with fh._made_on(0):
        assert torch.cuda.current_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with fh._made_on(0):
            assert torch.cuda.current_stream().cuda_stream == 0
        assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
        with fh._made_on(side.cuda_stream):
            assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
        with fh._made_on(None):
            assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
    with fh._made_on(side.cuda_stream):
        assert torch.cuda.current_stream().cuda_stream == side.cuda_stream


def test_calls_on_the_default_stream_by_its_handle(fh):
    v, d, rows = 5000, 256, 9
    head = fh.DenseHeadFP8(rand((v, d), 1, 0.05), max_rows=rows, max_sequences=3, stream=0)
    x = rand((rows, d), 2)
    want = head.logits(x)
    got = [head.logits(x, stream=0) for _ in range(3)]
    torch.cuda.synchronize()
    for z in got:
        assert torch.equal(z, want)
