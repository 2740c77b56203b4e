"""The calls around the head without a GPU: every refusal is decided on the
host before any device work, by the C ABI and by the binding."""
from __future__ import annotations

import ctypes as C
import os

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "two_stage_retrieval_amd", "libflashhead.so")
P = 0x10000   # aligned, never dereferenced: each call fails its checks first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fh():
    if not os.path.exists(LIB):
        pytest.fail("libflashhead.so is not built (run __graft_entry__.build())")
    from two_stage_retrieval_amd import binding
    return binding


def caller(fn, order, good):
    def call(**kw):
        a = dict(good, **kw)
        return fn(*[a[n] for n in order])
    return call


def test_rmsnorm_refusals(fh):
    inv, uns = fh.FH_ERR_INVALID_ARG, fh.FH_ERR_UNSUPPORTED
    order = ("x ldx r ldr w rows d dtype eps off ro ldro y ldy y8 ldy8 s lds stream").split()
    good = dict(x=P, ldx=256, r=P, ldr=256, w=P, rows=4, d=256, dtype=fh.FH_DTYPE_BF16, eps=1e-6,
                off=0.0, ro=P, ldro=256, y=P, ldy=256, y8=P, ldy8=256, s=P, lds=2, stream=None)
    call = caller(fh.lib.flashhead_rmsnorm, order, good)
    assert call(rows=0) == fh.FH_OK
    for kw in (dict(x=None), dict(rows=-1), dict(d=0), dict(eps=-1.0), dict(eps=NAN),
               dict(eps=INF), dict(off=NAN), dict(y8=None), dict(s=None), dict(ldx=255),
               dict(ldr=8), dict(ldro=0), dict(ldy=-256), dict(ldy8=200), dict(lds=1),
               dict(y=None, y8=None, s=None, ro=None)):
        assert call(**kw) == inv, kw
    for kw in (dict(dtype=7), dict(d=8200, ldx=8200, ldr=8200, ldro=8200, ldy=8200, ldy8=8200,
                                   lds=65), dict(d=252), dict(x=P + 8), dict(r=P + 2),
               dict(w=P + 4), dict(ro=P + 8), dict(y=P + 8), dict(y8=P + 4), dict(s=P + 2),
               dict(ldx=260), dict(ldr=260), dict(ldro=260), dict(ldy=260), dict(ldy8=260),
               dict(rows=1 << 24), dict(dtype=fh.FH_DTYPE_F32, d=254)):
        assert call(**kw) == uns, kw


def test_quantize_refusals(fh):
    inv, uns = fh.FH_ERR_INVALID_ARG, fh.FH_ERR_UNSUPPORTED
    order = "E v d dtype lde E8 lde8 s lds stream".split()
    good = dict(E=P, v=300, d=256, dtype=fh.FH_DTYPE_BF16, lde=256, E8=P, lde8=256, s=P, lds=2,
                stream=None)
    call = caller(fh.lib.flashhead_quantize_fp8, order, good)
    for kw in (dict(E=None), dict(E8=None), dict(s=None), dict(v=0), dict(d=0), dict(lde=200),
               dict(lde8=255), dict(lds=1)):
        assert call(**kw) == inv, kw
    for kw in (dict(dtype=2), dict(d=252), dict(E=P + 8), dict(E8=P + 4), dict(s=P + 1),
               dict(lde=260), dict(lde8=260), dict(v=65535 * 128 + 1)):
        assert call(**kw) == uns, kw


def test_logits_refusals(fh):
    inv, uns = fh.FH_ERR_INVALID_ARG, fh.FH_ERR_UNSUPPORTED
    order = "h ldh hs lds rows E lde es ldes v d out dtype ldo stream".split()
    good = dict(h=P, ldh=256, hs=P, lds=2, rows=4, E=P, lde=256, es=P, ldes=2, v=300, d=256, out=P,
                dtype=fh.FH_DTYPE_BF16, ldo=304, stream=None)
    call = caller(fh.lib.dense_logits_fp8, order, good)
    assert call(rows=0) == fh.FH_OK
    for kw in (dict(h=None), dict(hs=None), dict(E=None), dict(es=None), dict(out=None),
               dict(rows=-1), dict(v=0), dict(d=0), dict(ldh=128), dict(lde=128), dict(lds=1),
               dict(ldes=1), dict(ldo=296)):
        assert call(**kw) == inv, kw
    for kw in (dict(dtype=3), dict(d=248), dict(h=P + 8), dict(E=P + 4), dict(out=P + 8),
               dict(hs=P + 2), dict(es=P + 2), dict(ldh=264), dict(lde=264), dict(ldo=300),
               dict(v=2 ** 28 + 8, ldo=2 ** 29), dict(rows=65535 * 16 + 1), dict(ldh=1 << 22),
               dict(lde=1 << 22), dict(lds=1 << 22), dict(ldes=1 << 22)):
        assert call(**kw) == uns, kw


VERIFY = ("z rows v dtype ldl start B tok n q ldq mode tau ua us m out acc logp ws wsb "
          "stream").split()


def verify_good(fh):
    return dict(z=P, rows=12, v=1000, dtype=fh.FH_DTYPE_BF16, ldl=1000, start=P, B=4, tok=P, n=8,
                q=P, ldq=1000, mode=fh.FH_MODE_SAMPLE, tau=1.0, ua=P, us=P, m=3, out=P, acc=P,
                logp=P, ws=P, wsb=1 << 20, stream=None)


def test_verify_refusals(fh):
    inv, uns = fh.FH_ERR_INVALID_ARG, fh.FH_ERR_UNSUPPORTED
    call = caller(fh.lib.flashhead_verify, VERIFY, verify_good(fh))
    assert call(B=0) == fh.FH_OK
    for kw in (dict(z=None), dict(rows=-1), dict(v=0), dict(start=None), dict(B=-1),
               dict(tok=None), dict(n=-1), dict(mode=2), dict(tau=0.0), dict(tau=NAN),
               dict(tau=INF), dict(tau=-1.0), dict(ua=None), dict(us=None), dict(m=0),
               dict(out=None), dict(acc=None), dict(ws=None), dict(wsb=0), dict(ldl=992),
               dict(ldq=996), dict(mode=fh.FH_MODE_GREEDY)):
        assert call(**kw) == inv, kw
    n = fh.flashhead_verify_workspace_bytes(4, 12, 1000)
    assert call(wsb=n - 1) == inv
    for kw in (dict(dtype=5), dict(z=P + 8), dict(q=P + 8), dict(ws=P + 8), dict(ldl=1004),
               dict(ldq=1001), dict(v=2 ** 31, ldl=2 ** 31, ldq=2 ** 31), dict(rows=1 << 24),
               dict(B=1 << 24), dict(B=1 << 23), dict(rows=1 << 20, v=65536, ldl=65536, ldq=65536),
               dict(B=1 << 19, v=65536, ldl=65536, ldq=65536)):
        assert call(**kw) == uns, kw


def test_verify_workspace_size(fh):
    size = fh.flashhead_verify_workspace_bytes
    assert size(1, 1, 0) == 0 and size(-1, 1, 8) == 0 and size(1, -1, 8) == 0
    assert size(1, 1, 2 ** 31) == 0
    for v in (1, 2048, 5003, 128256, 262144):
        last = 0
        # never less for more rows or sequences: one workspace serves smaller calls
        for rows in (0, 1, 2, 5, 16, 17, 40, 64, 100, 256, 300, 512, 1000, 4096, 20000):
            n = size(max(1, rows // 5), rows, v)
            assert n >= last and n % 16 == 0
            last = n


def test_binding_refuses_host_tensors_shapes_and_types(fh):
    # a CPU tensor is refused before its address is used
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        fh.flashhead_rmsnorm(x, y=torch.empty_like(x))
    with pytest.raises(TypeError):
        fh.flashhead_rmsnorm(x.half(), y=torch.empty_like(x))
    with pytest.raises(ValueError):
        fh.flashhead_rmsnorm(x[0], y=x)
    with pytest.raises(ValueError):
        fh.flashhead_rmsnorm(x.t(), y=x)
    E8 = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        fh.flashhead_quantize_fp8(x, E8, torch.zeros(1, 2))
    with pytest.raises(TypeError):
        fh.dense_logits_fp8(x, torch.zeros(4, 2), E8, torch.zeros(1, 2), x)
    with pytest.raises(ValueError):
        fh.flashhead_verify(x, torch.zeros(2, dtype=torch.int32),
                            torch.zeros(3, dtype=torch.int32),
                            torch.zeros(1, 4, dtype=torch.int32),
                            torch.zeros(1, dtype=torch.int32), torch.zeros(1 << 16))


class FakeDevice:
    """Stands for a tensor on a second device (none is needed to refuse it)."""

    def __init__(self, t, index):
        self._t, self.device = t, torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_binding_refuses_other_devices(fh, monkeypatch):
    monkeypatch.setattr(fh, "_current_device", lambda: 0)
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="current device"):
        fh.flashhead_rmsnorm(FakeDevice(x, 1), y=FakeDevice(x, 1))
    with pytest.raises(ValueError, match="other arguments"):
        fh.flashhead_rmsnorm(FakeDevice(x, 0), y=FakeDevice(x, 1))
