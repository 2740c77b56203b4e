"""dense_logits_fp8 on the GPU against the float64 definition (tolerances:
tests/around_ref.py)."""
import numpy as np
import pytest

from . import around_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def fh():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from two_stage_retrieval_amd import binding
    return binding


def codes(shape, seed):
    """Codes over the whole format, with zeros and both signs."""
    g = torch.Generator().manual_seed(seed)
    c = (torch.randn(*shape, generator=g) * torch.exp(torch.randn(*shape, generator=g)) * 30)
    return c.clamp(-448, 448).to(F8).cuda()


def scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp(torch.randn(*shape, generator=g)).cuda() * 2e-3


def inputs(rows, v, d, seed=0):
    g = -(-d // 128)
    return (codes((rows, d), seed + 1), scales((rows, g), seed + 2), codes((v, d), seed + 3),
            scales((-(-v // 128), g), seed + 4))


def out_of(rows, v, dtype, extra=0):
    per = 16 if dtype == torch.bfloat16 else 8
    ld = -(-v // per) * per + extra
    base = torch.full((rows, ld), 5.0, dtype=dtype, device="cuda")
    return base, base[:, :v]


def check(fh, rows, v, d, dtype, extra=0, seed=0):
    h8, hs, E8, es = inputs(rows, v, d, seed)
    base, out = out_of(rows, v, dtype, extra)
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    torch.cuda.synchronize()
    assert torch.all(base[:, v:] == 5.0)
    z, mag = ref.logits(h8, hs, E8, es)
    ref.check_logits(out, z, mag, d)
    return h8, hs, E8, es, out


ROWS = [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 130, 257, 515]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("v,d", [(1000, 256), (515, 1104)])
def test_logits_rows(fh, rows, v, d):
    check(fh, rows, v, d, torch.float32 if rows % 2 else torch.bfloat16)


@pytest.mark.parametrize("v", [1, 3, 15, 16, 17, 127, 128, 129, 255, 257, 5003])
@pytest.mark.parametrize("rows", [1, 20, 150])
def test_logits_vocabulary_sizes(fh, v, rows):
    check(fh, rows, v, 384, torch.bfloat16 if v % 2 else torch.float32, extra=16)


@pytest.mark.parametrize("d", [16, 64, 80, 112, 128, 144, 192, 256, 1152, 2048, 2064, 4096, 8192])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_logits_widths(fh, d, rows):
    check(fh, rows, 333, d, torch.float32)


def test_logits_strided_inputs(fh):
    rows, v, d = 70, 400, 304
    h8, hs, E8, es = inputs(rows, v, d)
    out = torch.empty(rows, v, device="cuda")
    fh.dense_logits_fp8(h8, hs, E8, es, out)

    def wide(t, extra):
        w = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=torch.float32, device="cuda")
        w[:] = float("nan")
        w = w.to(t.dtype)
        w[:, :t.shape[1]] = t
        return w[:, :t.shape[1]]

    # NaN codes and scales beside the rows are never used
    out2 = torch.empty(rows, v, device="cuda")
    fh.dense_logits_fp8(wide(h8, 48), wide(hs, 3), wide(E8, 208), wide(es, 5), out2)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("rows", [1, 20, 33, 70, 300])
def test_logits_rows_do_not_depend_on_each_other(fh, rows):
    # a row alone, within a batch of its size class and beside NaN rows
    h8, hs, E8, es, out = check(fh, rows, 700, 512, torch.float32)
    bad = h8.clone()
    bad[0] = float("nan")
    out2 = torch.empty_like(out)
    fh.dense_logits_fp8(bad, hs, E8, es, out2)
    assert torch.equal(out[1:], out2[1:])
    assert torch.all(torch.isnan(out2[0]))
    again = torch.empty_like(out)
    fh.dense_logits_fp8(h8, hs, E8, es, again)
    assert torch.equal(out, again)


def test_logits_one_nan_code_of_E(fh):
    for rows in (1, 40, 300):
        h8, hs, E8, es = inputs(rows, 300, 256)
        out, out2 = (torch.empty(rows, 300, device="cuda") for _ in range(2))
        fh.dense_logits_fp8(h8, hs, E8, es, out)
        E8[77, 200] = float("nan")
        fh.dense_logits_fp8(h8, hs, E8, es, out2)
        keep = [t for t in range(300) if t != 77]
        assert torch.equal(out[:, keep], out2[:, keep])
        assert torch.all(torch.isnan(out2[:, 77]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,v,d", [(65, 65600, 144), (130, 65537, 256), (300, 40000, 1104),
                                      (513, 33001, 384), (257, 65536, 16), (2100, 9000, 400),
                                      (20, 30000, 272), (300, 4000, 1040), (90, 20000, 640),
                                      (1030, 2100, 528), (700, 12000, 160)])
def test_logits_many_tiles(fh, dtype, rows, v, d):
    # enough tiles for the tiled kernels, cut in every direction
    check(fh, rows, v, d, dtype, extra=16)


def test_logits_no_rows(fh):
    h8, hs, E8, es = inputs(1, 64, 128)
    fh.dense_logits_fp8(h8[:0], hs[:0], E8, es, torch.empty(0, 64, device="cuda"))


def test_logits_offsets_past_32_bits(fh):
    # E of more than 2^31 codes: the last rows against the definition
    v, d = 1100000, 2048
    h8, hs, E8s, _ = inputs(3, 512, d)
    E8 = torch.zeros(v, d, dtype=torch.uint8, device="cuda").view(F8)
    E8[-512:] = E8s
    es = scales((-(-v // 128), d // 128), 8)
    out = torch.empty(3, v, device="cuda")
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    torch.cuda.synchronize()
    assert v * d > 2 ** 31
    assert torch.all(out[:, :-512] == 0)
    # rows of the tail and their blocks (v - 512 is not a multiple of 128)
    at = v - 512
    b = np.arange(at, v) // 128
    E = ref.f64(E8s) * np.repeat(ref.f64(es), 128, 1)[b]
    h = ref.dequant(h8, hs, 1)
    ref.check_logits(out[:, at:], h @ E.T, np.abs(h) @ np.abs(E).T, d)


def test_logits_outputs_past_32_bits(fh):
    # rows x v past 2^31 outputs: the last rows and columns against the definition
    rows, v, d = 4100, 524288 + 128, 128
    h8, hs, E8, es = inputs(rows, v, d)
    out = torch.empty(rows, v, dtype=torch.bfloat16, device="cuda")
    fh.dense_logits_fp8(h8, hs, E8, es, out)
    torch.cuda.synchronize()
    assert rows * v > 2 ** 31
    z, mag = ref.logits(h8[-70:], hs[-70:], E8[-1280:], es[-10:])
    ref.check_logits(out[-70:, -1280:], z, mag, d)
    z, mag = ref.logits(h8[:70], hs[:70], E8[:1280], es[:10])
    ref.check_logits(out[:70, :1280], z, mag, d)
