"""Host-side refusals of the quantized prefills and of the append with positions of several
axes: answered before any launch, without a device where no device is asked about."""
import ctypes

import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from paged_kv_cache_72_gb300 import _lib
from paged_kv_cache_72_gb300.build import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096   # 16-byte aligned addresses that are never read: every call here is refused or empty
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


@pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])
@pytest.mark.parametrize("kw,status", [
    (dict(nseq=0), OK),
    (dict(total=0), OK),
    (dict(total=0, q=None, out=None, ws=None, kc=None, bt=None, lens=None), OK),
    (dict(nseq=-1), INVALID),
    (dict(total=-1), INVALID),
    (dict(stride=-1), INVALID),
    (dict(stride=0), INVALID),
    (dict(nb=-1), INVALID),
    (dict(nb=0), INVALID),
    (dict(nb=2 ** 31), INVALID),
    (dict(total=2 ** 31), INVALID),
    (dict(window=-1), INVALID),
    (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID),
    (dict(ks=0.0), INVALID),
    (dict(ks=-1.0), INVALID),
    (dict(vs=NAN), INVALID),
    (dict(vs=INF), INVALID),
    (dict(dt=2), UNSUPPORTED),
    (dict(dt=3), UNSUPPORTED),
    (dict(B=2), UNSUPPORTED),
    (dict(B=12), UNSUPPORTED),
    (dict(B=512), UNSUPPORTED),
    (dict(B=0), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED),
    (dict(H=0), INVALID),
    (dict(Hq=0), INVALID),
    (dict(Hq=9), INVALID),
    (dict(Hq=34), UNSUPPORTED),                # 17 query heads a KV head
    (dict(Hq=2 ** 17, H=2 ** 17, B=256), UNSUPPORTED),   # a block's bytes pass 31 bits
    (dict(q=None), INVALID),
    (dict(kc=None), INVALID),
    (dict(vc=None), INVALID),
    (dict(bt=None), INVALID),
    (dict(lens=None), INVALID),
    (dict(start=None), INVALID),
    (dict(out=None), INVALID),
    (dict(ws=None), INVALID),
    (dict(out=P), INVALID),                    # in place
    (dict(q=P + 8), INVALID),
    (dict(kc=P + 4), INVALID),
    (dict(vc=P + 8), INVALID),
    (dict(out=2 * P + 2), INVALID),
    (dict(ws=P + 8), INVALID),
])
def test_prefill_refusals(lib, four, kw, status):
    a = dict(q=P, kc=P, vc=P, bt=P, stride=4, lens=P, start=P, nseq=2, total=5, Hq=8, H=2, D=128,
             B=16, nb=9, dt=1, scale=0.1, ks=1.0, vs=1.0, window=0, out=2 * P, ws=P, bytes=1 << 40)
    a.update(kw)
    call = lib.pa_prefill_fp4 if four else lib.pa_prefill_fp8
    assert call(a["q"], a["kc"], a["vc"], a["bt"], a["stride"], a["lens"], a["start"], a["nseq"],
                a["total"], a["Hq"], a["H"], a["D"], a["B"], a["nb"], a["dt"], a["scale"], a["ks"],
                a["vs"], a["window"], a["out"], a["ws"], a["bytes"], None, None) == status


def test_workspace_size_refusals(lib):
    n = ctypes.c_size_t(0)
    size = lib.pa_prefill_quant_workspace_size
    assert size(8, 2, 128, None) == INVALID
    assert size(8, 2, 96, ctypes.byref(n)) == UNSUPPORTED
    assert size(8, 0, 128, ctypes.byref(n)) == INVALID
    assert size(0, 2, 128, ctypes.byref(n)) == INVALID
    assert size(9, 2, 128, ctypes.byref(n)) == INVALID
    assert size(34, 2, 128, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(n=-1), INVALID),
    (dict(axes=0), UNSUPPORTED),
    (dict(axes=5), UNSUPPORTED),
    (dict(axes=-1), UNSUPPORTED),
    (dict(axis_of=None), INVALID),
    (dict(axis_of=P + 4), INVALID),
    (dict(rot_pos=None), INVALID),
    (dict(cs=None), INVALID),
    (dict(rot=0), INVALID),
    (dict(rot=24), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(B=12), UNSUPPORTED),
    (dict(B=2, dt=3), UNSUPPORTED),
    (dict(src=0), UNSUPPORTED),
    (dict(q=None), INVALID),
    (dict(q_out=None), INVALID),
    (dict(k=P + 2), INVALID),
    (dict(ks=2 * 128 - 8), INVALID),
    (dict(kn=P, eps=NAN), INVALID),
    (dict(dt=2, ksc=0.0), INVALID),
])
def test_append_axes_refusals(lib, kw, status):
    a = dict(q=P, qs=8 * 128, k=P, ks=2 * 128, v=P, vs=2 * 128, src=1, cs=P, rot=128, max_pos=64,
             axis_of=P, rot_pos=P, axes=3, inter=0, qn=None, kn=None, eps=1e-6, bt=P, stride=4,
             nseq=2, seq=P, pos=P, n=3, q_out=P, kc=P, vc=P, nb=9, B=16, Hq=8, H=2, D=128, dt=1,
             ksc=1.0, vsc=1.0)
    a.update(kw)
    assert lib.pa_append_rope_axes(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["src"], a["cs"], a["rot"],
        a["max_pos"], a["axis_of"], a["rot_pos"], a["axes"], a["inter"], a["qn"], a["kn"], a["eps"],
        a["bt"], a["stride"], a["nseq"], a["seq"], a["pos"], a["n"], a["q_out"], a["kc"], a["vc"],
        a["nb"], a["B"], a["Hq"], a["H"], a["D"], a["dt"], a["ksc"], a["vsc"], None, None,
        None) == status


@pytest.mark.gpu
def test_host_tensors_are_refused():
    """The Python calls take CUDA tensors alone."""
    D, B, H, Hq = 64, 16, 2, 8
    q = torch.zeros(3, Hq, D, dtype=torch.float16)
    i32 = torch.zeros(3, dtype=torch.int32)
    bt = torch.zeros(2, 4, dtype=torch.int32)
    pool8 = torch.zeros(5, B, H, D, dtype=torch.uint8)
    pool4 = torch.zeros(pa.pa_fp4_pool_shape(5, B, H, D), dtype=torch.uint8)
    ws = torch.zeros(16, dtype=torch.uint8)
    for call, pool in ((pa.pa_prefill_fp8, pool8), (pa.pa_prefill_fp4, pool4)):
        with pytest.raises((TypeError, ValueError)):
            call(q, pool, pool, bt, i32[:2], i32, 0.1, 1.0, 1.0, out=torch.empty_like(q),
                 workspace=ws)
    k = torch.zeros(3, H, D, dtype=torch.float16)
    kc = torch.zeros(5, B, H, D, dtype=torch.float16)
    with pytest.raises((TypeError, ValueError)):
        pa.pa_append_rope_axes(q, k, k, torch.zeros(8, D), torch.zeros(D // 2, dtype=torch.uint8),
                               torch.zeros(3, 3, dtype=torch.int32), bt, i32, i32, kc, kc)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])
def test_python_refusals(four):
    """Tensors of other types and shapes, workspaces that are too small: refused, nothing runs."""
    D, B, H, Hq = 64, 16, 2, 8
    dev = "cuda"
    shape = pa.pa_fp4_pool_shape(5, B, H, D) if four else (5, B, H, D)
    good = dict(q=torch.ones(3, Hq, D, dtype=torch.float16, device=dev),
                k=torch.zeros(shape, dtype=torch.uint8, device=dev),
                v=torch.zeros(shape, dtype=torch.uint8, device=dev),
                bt=torch.zeros(2, 4, dtype=torch.int32, device=dev),
                lens=torch.tensor([2, 1], dtype=torch.int32, device=dev),
                start=torch.tensor([0, 2, 3], dtype=torch.int32, device=dev), scale=0.1, ks=1.0,
                vs=1.0, window=0, out=torch.full((3, Hq, D), 7.0, dtype=torch.float16, device=dev),
                ws=torch.zeros(pa.pa_prefill_quant_workspace_size(Hq, H, D), dtype=torch.uint8,
                               device=dev))

    def call(**kw):
        a = dict(good)
        a.update(kw)
        return (pa.pa_prefill_fp4 if four else pa.pa_prefill_fp8)(
            a["q"], a["k"], a["v"], a["bt"], a["lens"], a["start"], a["scale"], a["ks"], a["vs"],
            window=a["window"], out=a["out"], workspace=a["ws"])

    wide = torch.zeros(3, 2 * Hq, D, dtype=torch.float16, device=dev)
    for kw in (dict(q=good["q"].float()), dict(q=wide[:, ::2]), dict(q=good["q"][:, :, :32]),
               dict(q=good["q"][0]), dict(k=good["k"].half()), dict(v=good["v"][:4]),
               dict(bt=good["bt"].long()), dict(bt=good["bt"][:1]), dict(bt=good["bt"][0]),
               dict(lens=good["lens"].long()), dict(lens=good["lens"][:1]),
               dict(start=good["start"][:2]), dict(start=good["start"].long()),
               dict(out=good["out"].bfloat16()), dict(out=good["out"][:2]),
               dict(window=2 ** 40), dict(scale="x"), dict(q=good["q"].cpu()),
               dict(ws=good["ws"].cpu())):
        with pytest.raises((TypeError, ValueError, OverflowError)):
            call(**kw)
    for kw in (dict(window=-1), dict(ks=0.0), dict(vs=float("nan")), dict(scale=float("inf")),
               dict(out=good["q"]), dict(ws=good["ws"][:-16]), dict(ws=good["ws"][8:])):
        with pytest.raises(pa.PAError):
            call(**kw)
    torch.cuda.synchronize()
    assert bool((good["out"] == 7).all())
