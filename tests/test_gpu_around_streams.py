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


def test_an_object_dropped_while_a_call_is_queued(fh):
    # its memory is not handed on before the call on the other stream is done
    v, d, rows = 20000, 512, 12
    E, w, x = rand((v, d), 3, 0.05), rand((d,), 4, 0.1), rand((rows, d), 5)
    head = fh.DenseHeadFP8(E, w, max_rows=rows, max_sequences=4)
    want = head.logits(x).clone()
    st = torch.arange(0, rows + 1, 3, dtype=torch.int32, device="cuda")
    drafts = torch.arange(8, dtype=torch.int32, device="cuda")
    tokens, accepted = head.verify(x, st, drafts, 2, mode=fh.FH_MODE_GREEDY)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for made in (None, torch.cuda.Stream()):
        on = None if made is None else made.cuda_stream
        head = fh.DenseHeadFP8(rand((v, d), 3, 0.05), rand((d,), 4, 0.1), max_rows=rows,
                               max_sequences=4, stream=on)
        own = (head.E8, head.E_scale, head.h8, head.h_scale, head.workspace, head.norm_weight)
        sizes = [t.numel() * t.element_size() for t in own]
        old = [t.data_ptr() for t in own]
        del own
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(300_000_000)      # 0.1 s and more, then the calls
        z = head.logits(x, stream=side.cuda_stream)
        got = head.verify(x, st, drafts, 2, mode=fh.FH_MODE_GREEDY, stream=side.cuda_stream)
        del head
        junk = []
        for s in [torch.cuda.current_stream()] + ([made] if made else []):
            with torch.cuda.stream(s):
                junk += [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes]
        assert not side.query()                 # the calls are still to come
        assert not {t.data_ptr() for t in junk} & set(old)
        torch.cuda.synchronize()
        assert torch.equal(z, want)
        assert torch.equal(got[0], tokens) and torch.equal(got[1], accepted)
