"""Host-side refusals of the append and of the 4-bit cache's entry points:
answered before any launch, without a device where no device is asked about."""
import ctypes

import pytest

from paged_kv_cache_72_gb300 import _lib
from paged_kv_cache_72_gb300.build import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096   # a 16-byte aligned address that is never read: every call here is refused or empty


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def _append(lib, **kw):
    a = dict(q=P, qs=8 * 128, k=P, ks=2 * 128, v=P, vs=2 * 128, src=1, cs=P, rot=128, max_pos=64,
             inter=0, qn=None, kn=None, eps=1e-6, bt=P, stride=4, nseq=2, seq=P, pos=P, n=3,
             q_out=P, kc=P, vc=P, nb=9, B=16, Hq=8, H=2, D=128, dt=1, ksc=1.0, vsc=1.0)
    a.update(kw)
    return lib.pa_append_rope(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["src"], a["cs"],
                              a["rot"], a["max_pos"], a["inter"], a["qn"], a["kn"], a["eps"],
                              a["bt"], a["stride"], a["nseq"], a["seq"], a["pos"], a["n"],
                              a["q_out"], a["kc"], a["vc"], a["nb"], a["B"], a["Hq"], a["H"],
                              a["D"], a["dt"], a["ksc"], a["vsc"], None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(n=0, q=None, q_out=None, cs=None), OK),
    (dict(n=-1), INVALID),
    (dict(D=96), UNSUPPORTED),
    (dict(B=12), UNSUPPORTED),
    (dict(B=512), UNSUPPORTED),
    (dict(B=2, dt=3), UNSUPPORTED),            # 4-bit blocks hold at least 4 tokens
    (dict(src=2), UNSUPPORTED),
    (dict(src=0, dt=1), UNSUPPORTED),          # 16-bit pools are of the inputs' type
    (dict(rot=24), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED),
    (dict(cs=None), INVALID),
    (dict(q=None), INVALID),
    (dict(q_out=None), INVALID),
    (dict(k=None), INVALID),
    (dict(bt=None), INVALID),
    (dict(ks=2 * 128 - 8), INVALID),           # tokens would overlap
    (dict(ks=2 * 128 + 4), INVALID),
    (dict(qs=8 * 128 + 1), INVALID),
    (dict(k=P + 2), INVALID),
    (dict(kc=P + 8), INVALID),
    (dict(qn=P, eps=-1.0), INVALID),
    (dict(kn=P, eps=float("nan")), INVALID),
    (dict(dt=2, ksc=0.0), INVALID),
    (dict(dt=3, vsc=float("inf")), INVALID),
    (dict(dt=3, vsc=3e38), INVALID),           # 6 * scale overflows
    (dict(H=0), UNSUPPORTED),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(), INVALID),                          # no pointers
    (dict(n=-1), INVALID),
    (dict(B=2), UNSUPPORTED),
    (dict(D=80), UNSUPPORTED),
    (dict(dt=2), UNSUPPORTED),
    (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID),
])
def test_fp4_write_and_read_refusals(lib, kw, status):
    a = dict(n=3, B=16, D=128, dt=1, scale=1.0)
    a.update(kw)
    assert lib.pa_cache_write_fp4(None, None, a["dt"], None, a["n"], None, None, 9, a["B"], 2,
                                  a["D"], a["scale"], 1.0, None, None) == status
    assert lib.pa_cache_write_fp4_mapped(None, None, a["dt"], None, 4, 2, None, None, a["n"], None,
                                         None, 9, a["B"], 2, a["D"], a["scale"], 1.0, None, None,
                                         None) == status
    assert lib.pa_cache_read_fp4(None, a["n"], None, None, 9, a["B"], 2, a["D"], a["scale"], 1.0,
                                 None, None, a["dt"], None, None) == status


def test_fp4_decode_and_block_refusals(lib):
    n = ctypes.c_size_t(0)

    def size(Hq, H, D, B, flags=0, ctas=0):
        return lib.pa_decode_workspace_size(Hq, H, D, B, _lib.PA_FP4_E2M1, flags, ctas,
                                            ctypes.byref(n))
    assert size(8, 8, 96, 16) == UNSUPPORTED
    assert size(8, 8, 128, 2) == UNSUPPORTED
    assert size(8, 8, 128, 512) == UNSUPPORTED
    assert size(8, 8, 128, 16, flags=_lib.PA_DECODE_SIMT) == UNSUPPORTED
    assert size(8, 8, 128, 16, flags=7) == INVALID
    assert size(6, 4, 128, 16) == INVALID
    assert size(64, 2, 128, 16) == UNSUPPORTED          # 32 query heads a KV head
    assert size(8, 8, 128, 16, ctas=_lib.PA_DECODE_MAX_CTAS + 1) == INVALID

    def decode(window=0, ks=1.0, vs=1.0, dt=1, nseq=2):
        return lib.pa_decode_fp4(None, None, None, None, 4, None, nseq, 8, 2, 128, 16, 9, dt, 0.1,
                                 ks, vs, window, None, None, 0, 0, 0, None, None)
    assert decode(window=-1) == INVALID
    assert decode(ks=0.0) == INVALID
    assert decode(vs=float("nan")) == INVALID
    assert decode(dt=2) == UNSUPPORTED
    assert decode(nseq=-1) == INVALID
    # block copies and swaps of 4-bit pools need blocks of at least 4 tokens
    assert lib.pa_copy_blocks(None, 0, None, None, 9, 4, 2, 64, _lib.PA_FP4_E2M1, None, None) == OK
    assert lib.pa_copy_blocks(None, 0, None, None, 9, 2, 2, 64, _lib.PA_FP4_E2M1, None,
                              None) == UNSUPPORTED
