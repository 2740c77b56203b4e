"""flashhead_rmsnorm and flashhead_quantize_fp8 on the GPU against the
float64 definitions (tolerances: tests/around_ref.py)."""
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


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def padded(rows, cols, dtype, extra, fill):
    """A rows x cols view whose rows are `extra` elements apart, filled around."""
    base = torch.full((rows + 1, cols + extra), fill, device="cuda").to(dtype)
    return base, base[:rows, :cols]


def run(fh, x, r, w, offset, outputs, eps=1e-6, pad=0):
    rows, d = x.shape
    o = dict(residual_out=None, y=None, y8=None, y_scale=None)
    if r is not None:
        o["residual_out"] = torch.empty_like(x)
    if outputs in ("y", "both"):
        o["y"] = torch.empty_like(x)
    if outputs in ("fp8", "both"):
        o["y8"] = torch.empty(rows, d + pad, dtype=F8, device="cuda")[:, :d]
        o["y_scale"] = torch.empty(rows, -(-d // 128) + pad, device="cuda")[:, :-(-d // 128)]
    fh.flashhead_rmsnorm(x, w, residual=r, eps=eps, weight_offset=offset, **o)
    torch.cuda.synchronize()
    return o


def check(o, x, r, w, offset, eps=1e-6):
    t, y = ref.norm(x, r, w, eps, offset)
    if o["residual_out"] is not None:
        got = o["residual_out"]
        e = (ref.U32 + ref.half_step(got.dtype)) * 1.001
        assert np.all(np.abs(ref.f64(got) - t) <= e * np.abs(t))
    if o["y"] is not None:
        ref.check_norm(o["y"], y)
    if o["y8"] is not None:
        ref.check_codes(o["y8"], o["y_scale"], y, 1, ref.NORM_STEPS)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 2048), (3, 128), (5, 136), (37, 1152), (2, 1000),
                                    (64, 2056), (9, 4096), (7, 4104), (3, 8192), (300, 64)])
@pytest.mark.parametrize("outputs", ["y", "fp8", "both"])
def test_norm_matches_float64(fh, dtype, rows, d, outputs):
    x = rand((rows, d), dtype, 10 * rows + d)
    r = rand((rows, d), dtype, 11 * rows + d, 3.0) if d % 3 else None
    offset = 1.0 if rows % 2 else 0.0
    w = rand((d,), dtype, 5, 0.3)
    check(run(fh, x, r, w, offset, outputs, pad=16 if rows > 4 else 0), x, r, w, offset)


def test_norm_fp32_rows_of_four_columns(fh):
    for d in (4, 12, 132, 1028):
        x = rand((6, d), torch.float32, d)
        check(run(fh, x, None, None, 0.0, "both"), x, None, None, 0.0)


def test_norm_in_place_and_strided(fh):
    # residual_out over the residual and y over x, rows inside a wider buffer
    for dtype in (torch.bfloat16, torch.float32):
        bx, x = padded(11, 264, dtype, 24, 7.0)
        br, r = padded(11, 264, dtype, 8, -3.0)
        x.copy_(rand((11, 264), dtype, 1))
        r.copy_(rand((11, 264), dtype, 2))
        x0, r0, w = x.clone(), r.clone(), rand((264,), dtype, 3)
        fh.flashhead_rmsnorm(x, w, residual=r, residual_out=r, y=x)
        torch.cuda.synchronize()
        check(dict(residual_out=r, y=x, y8=None), x0, r0, w, 0.0)
        # nothing outside the views changed
        assert torch.all(bx[:11, 264:] == 7.0) and torch.all(bx[11] == 7.0)
        assert torch.all(br[:11, 264:] == -3.0) and torch.all(br[11] == -3.0)


def test_norm_zero_rows_tiny_and_large_values(fh):
    w = torch.ones(256, device="cuda")
    x = torch.zeros(6, 256, device="cuda")
    x[1] = 1e-30
    x[2, 5] = 1e15
    x[3] = -3e-20
    x[4, :128] = 1.0          # the second block is all zero
    x[5] = 2.0 ** 40
    o = run(fh, x, None, w, 0.0, "both")
    check(o, x, None, w, 0.0)
    assert torch.all(o["y8"][0].float() == 0)
    assert torch.all(o["y_scale"][0] == 2.0 ** -126)
    assert float(o["y_scale"][4, 1]) == 2.0 ** -126
    # eps = 0 on a nonzero row: scale free
    o = run(fh, x[5:], None, w, 0.0, "y", eps=0.0)
    assert torch.all(o["y"] == 1.0)


def test_norm_rows_are_independent_and_non_finite_rows_stay_alone(fh):
    x = rand((40, 512), torch.bfloat16, 4)
    a = run(fh, x, None, None, 0.0, "both")
    x2 = x.clone()
    x2[7, 3] = float("nan")
    x2[20, 500] = float("inf")
    b = run(fh, x2, None, None, 0.0, "both")
    keep = [i for i in range(40) if i not in (7, 20)]
    for n in ("y", "y8", "y_scale"):
        assert torch.equal(a[n][keep].float(), b[n][keep].float())
    assert torch.all(torch.isnan(b["y"][7]))


def test_norm_no_rows(fh):
    x = torch.empty(0, 256, device="cuda")
    fh.flashhead_rmsnorm(x, y=torch.empty_like(x))


def test_norm_offsets_past_32_bits(fh):
    # rows 2^17 + 8 elements apart, so that the last ones start past 2^31 elements
    rows, ld, d = 16400, (1 << 17) + 8, 64
    base = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = base.view(rows, ld)[:, :d]
    x.copy_(rand((rows, d), torch.bfloat16, 9))
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    fh.flashhead_rmsnorm(x, y=y)
    torch.cuda.synchronize()
    assert (rows - 1) * ld > 2 ** 31
    ref.check_norm(y, ref.norm(x, None, None, 1e-6, 0.0)[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v,d", [(1, 8), (128, 128), (127, 136), (129, 120), (300, 1000),
                                 (1003, 384), (5, 2048)])
def test_quantize_matches_float64(fh, dtype, v, d):
    E = rand((v, d), dtype, v + d, 0.02)
    E[v // 2] *= 50
    pad = 16 if v > 128 else 0
    E8 = torch.empty(v, d + pad, dtype=F8, device="cuda")[:, :d]
    es = torch.empty(-(-v // 128), -(-d // 128) + pad, device="cuda")[:, :-(-d // 128)]
    fh.flashhead_quantize_fp8(E, E8, es)
    torch.cuda.synchronize()
    # the values are the inputs themselves: no step before the scale's
    ref.check_codes(E8, es, ref.f64(E), 128, 0)


def test_quantize_reproduces_codes_and_handles_extremes(fh):
    # every e4m3 value, times a power of two, comes back as itself
    codes = torch.arange(256, dtype=torch.uint8).view(F8).float()
    codes = codes[torch.isfinite(codes)]
    E = torch.zeros(128, 128)
    E.view(-1)[:codes.numel()] = codes * 2.0 ** -9
    E = E.cuda()
    E8, es = torch.empty(128, 128, dtype=F8, device="cuda"), torch.empty(1, 1, device="cuda")
    fh.flashhead_quantize_fp8(E, E8, es)
    assert float(es) == 2.0 ** -9
    assert torch.equal(E8.float() * es, E)
    for x in (0.0, 1e-45, 1e-38, 3e38):
        E = torch.full((3, 8), x, device="cuda")
        E8 = torch.empty(3, 8, dtype=F8, device="cuda")
        fh.flashhead_quantize_fp8(E, E8, es)
        ref.check_codes(E8, es, ref.f64(E), 128, 0)
