"""The 4-bit (E2M1) KV cache on the GPU against the fp64 oracle.

The quantizing write must give the oracle's codes (bit for bit, up to the sign
of zeros), the read-back the oracle's values rounded once to fp32 and once to 16
bits, and the decode must stay within
    |g - o| <= ulp(g) / 2 + u_p spread (1 + 2^-6) + 2^-14 (|o| + spread)
of the oracle's decode of the same codes (harness.rounding_report): u_p is the
rounding of the softmax weights, 2^-11 for one binary16 value (bfloat16
outputs), 2^-21 for a pair of them (binary16 outputs).  K, V and the queries
enter the products exactly, but for elements of a bfloat16 query below 2^-14 of
its head's largest, which lose less than 2^-24 of that: inside the fp32 term.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_72_gb300 as pa
import workloads as W
from harness import assert_close, bits_of, bits_to_f64, rounding_report, to_dev, ulp_spacing

pytestmark = pytest.mark.gpu


def _u_p(dtype):
    return 2.0 ** -11 if dtype == W.BF16 else 2.0 ** -21


class State:
    """Pools of quantized normal values, queries and tables, on both sides.
    Rows and blocks that no query attends to hold NaN scales."""

    def __init__(self, seed, dtype, Hq, H, D, B, lens, window=0, sigma=1.0, q_sigma=1.0, spare=5,
                 scales=(0.3, 0.4)):
        rng = np.random.default_rng(seed)
        self.dtype, self.H, self.D, self.B, self.window = dtype, H, D, B, window
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens.astype(np.int64) // B)
        first = np.maximum(0, self.lens - window) if window else np.zeros_like(self.lens)
        nb = int(need.sum()) + spare
        perm = rng.permutation(nb).astype(np.int32)
        self.bt = np.full((self.lens.size, max(1, int(need.max()))), -1, np.int32)
        self.k_scale, self.v_scale = scales
        self.scale = float(np.float32(D ** -0.5))
        pools = np.full((2, nb, H, B * 9 * D // 16), 0x7F, np.uint8)   # NaN scale codes
        at = 0
        for i, n in enumerate(need):
            rows = perm[at:at + n]
            at += n
            if n == 0:
                continue
            lo = int(first[i]) // B
            self.bt[i, lo:n] = rows[lo:]          # blocks before the window are released
            for p, sc in zip(pools, scales):
                x = (sigma * rng.standard_normal((n, H, B, D))).astype(np.float32)
                codes, s16 = oracle.fp4_quantize(x, sc)
                live = (np.arange(n)[:, None] * B + np.arange(B))[:, None, :] < self.lens[i]
                live &= (np.arange(n)[:, None] * B + np.arange(B))[:, None, :] >= first[i]
                s16 = np.where(live[..., None], s16, 0x7F)
                p[rows, :, :B * D // 2] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(
                    n, H, -1)
                p[rows, :, B * D // 2:] = s16.reshape(n, H, B // 4, 4, D // 16).transpose(
                    0, 1, 2, 4, 3).reshape(n, H, -1)
        self.k, self.v = (p.reshape(nb, H, B, 9 * D // 16) for p in pools)
        q = (q_sigma * rng.standard_normal((self.lens.size, Hq, D))).astype(np.float32)
        self.q = W.to_bits(q, dtype)
        self.dev = dict(q=to_dev(self.q, dtype), k=torch.from_numpy(self.k).cuda(),
                        v=torch.from_numpy(self.v).cuda(), bt=torch.from_numpy(self.bt).cuda(),
                        lens=torch.from_numpy(self.lens).cuda())
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def decode(self, **kw):
        d = self.dev
        kw.setdefault("window", self.window)
        return pa.pa_decode_fp4(d["q"], d["k"], d["v"], d["bt"], d["lens"], self.scale,
                                self.k_scale, self.v_scale, err=self.err, **kw)

    def expected(self):
        return oracle.paged_decode_fp4(bits_to_f64(self.q, self.dtype), self.k, self.v,
                                       self.k_scale, self.v_scale, self.bt, self.lens, self.scale,
                                       window=self.window)

    def check(self, out, ref=None, what=""):
        o, spread = self.expected() if ref is None else ref
        rounding_report(bits_of(out), o, spread, self.dtype, _u_p(self.dtype), what)
        assert pa.pa_get_error(self.err) == 0


EDGE_LENS = [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200, 777]
CASES = [
    # dtype, Hq, H, D, B
    (W.F16, 8, 8, 64, 4),         # the tiny workload's heads
    (W.F16, 32, 32, 128, 16),     # no grouped heads
    (W.BF16, 32, 8, 128, 16),
    (W.BF16, 64, 8, 128, 16),
    (W.F16, 14, 2, 64, 16),       # 7 heads a KV head
    (W.BF16, 16, 2, 128, 8),
    (W.BF16, 32, 2, 128, 32),     # 16 heads a KV head: two head tiles
    (W.F16, 24, 2, 64, 64),       # 12
    (W.F16, 9, 1, 128, 256),      # 9
    (W.BF16, 15, 3, 64, 8),
    (W.BF16, 5, 5, 128, 4),
]


@pytest.mark.parametrize("dtype,Hq,H,D,B", CASES)
def test_decode_parity_sweep(cuda_device, dtype, Hq, H, D, B):
    st = State(400 + Hq + D + B, dtype, Hq, H, D, B, EDGE_LENS)
    ref = st.expected()
    for ctas in (0, 1, 7):
        st.check(st.decode(num_ctas=ctas), ref, "ctas=%d" % ctas)


@pytest.mark.parametrize("window", [1, 3, 16, 33, 100, 5000])
@pytest.mark.parametrize("dtype,Hq,H,D,B", [CASES[0], CASES[2], CASES[6], CASES[7]])
def test_decode_window_over_released_blocks(cuda_device, dtype, Hq, H, D, B, window):
    st = State(500 + window, dtype, Hq, H, D, B, EDGE_LENS, window=window)
    ref = st.expected()
    for ctas in (0, 3):
        st.check(st.decode(num_ctas=ctas), ref, "window=%d ctas=%d" % (window, ctas))


@pytest.mark.parametrize("num_ctas", [0, 1, 2, 5, 64, 1000])
@pytest.mark.parametrize("dtype,Hq,H,D", [(W.BF16, 8, 2, 128), (W.F16, 16, 1, 64)])
def test_decode_split_contexts(cuda_device, dtype, Hq, H, D, num_ctas):
    # contexts cut between warps, between blocks, and over many blocks
    st = State(600, dtype, Hq, H, D, 16, [3000, 1, 64, 0, 65, 9000, 5, 4096])
    st.check(st.decode(num_ctas=num_ctas), what="ctas=%d" % num_ctas)


def test_decode_one_long_context(cuda_device):
    st = State(601, W.BF16, 4, 1, 128, 16, [60000])
    ref = st.expected()
    ws = torch.zeros(pa.pa_decode_workspace_size(4, 1, 128, 16, pa.PA_FP4_E2M1), dtype=torch.uint8,
                     device="cuda")
    a = st.decode(workspace=ws)
    st.check(a, ref)
    # the workspace is left ready, and the result does not depend on the order of arrival
    for _ in range(5):
        assert torch.equal(st.decode(workspace=ws), a)


def test_decode_empty_invalid_and_many_sequences(cuda_device):
    # zero lengths give zero rows; a length outside its table is reported and
    # gives zero rows; more sequences than a block has threads
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 40, 700)
    lens[[0, 1, 300, 699]] = 0
    st = State(602, W.BF16, 4, 2, 64, 8, lens)
    out = st.decode(out=torch.full_like(st.dev["q"], float("nan")))
    st.check(out)
    assert not out[[0, 1, 300, 699]].any()
    good = out.clone()
    bad = st.dev["lens"].clone()
    bad[5], bad[6] = -3, 8 * st.bt.shape[1] + 1
    st.dev["lens"] = bad
    out = st.decode(out=torch.full_like(good, float("nan")))
    assert pa.pa_get_error(st.err) == pa.PA_DEVERR_SEQ_LEN
    assert not out[[5, 6]].any()
    keep = [i for i in range(700) if i not in (5, 6)]
    # the cuts moved, so sums may round differently: held to the oracle
    o, spread = st.expected()
    rounding_report(bits_of(out[keep].contiguous()), o[keep], spread[keep], W.BF16, 2.0 ** -11)
    # nothing at all
    none = pa.pa_decode_fp4(st.dev["q"][:0], st.dev["k"], st.dev["v"], st.dev["bt"][:0],
                            st.dev["lens"][:0], st.scale, 1.0, 1.0)
    assert none.shape == (0, 4, 64)


def test_decode_leaves_out_blocks_with_bad_entries(cuda_device):
    st = State(603, W.BF16, 8, 2, 128, 16, [100, 40, 16])
    bt = st.bt.copy()
    bt[0, 2], bt[2, 0] = len(st.k) + 3, -1     # one block of sequence 0, all of sequence 2
    st.dev["bt"] = torch.from_numpy(bt).cuda()
    out = st.decode()
    assert pa.pa_get_error(st.err) == pa.PA_DEVERR_BLOCK_ID
    assert not out[2].any()
    # sequence 0 without tokens 32 .. 47: the same blocks with that one dropped
    st.bt[0, 2:6] = st.bt[0, 3:7]
    st.lens[0] = 84
    o, spread = st.expected()
    rounding_report(bits_of(out[:2].contiguous()), o[:2], spread[:2], W.BF16, 2.0 ** -11)


@pytest.mark.parametrize("dtype,q_sigma", [(W.BF16, 1e30), (W.BF16, 1e-30), (W.F16, 3000.0),
                                           (W.F16, 1e-6), (W.BF16, 0.0)])
def test_decode_query_magnitudes(cuda_device, dtype, q_sigma):
    # a bfloat16 query beyond binary16's range is scaled by a power of two
    st = State(604, dtype, 8, 2, 128, 16, [300, 17, 64], q_sigma=q_sigma)
    st.scale = float(np.float32(0.1 / max(q_sigma, 1e-30)))
    st.check(st.decode())


def test_decode_peaked_and_long_tailed_weights(cuda_device):
    # one token far above 20,000 others whose weights are all small
    st = State(605, W.F16, 8, 1, 64, 16, [20000], q_sigma=0.5)
    st.scale = 1.5
    st.check(st.decode())
    st = State(606, W.BF16, 8, 1, 64, 16, [20000], q_sigma=0.5)
    st.scale = 1.5
    st.check(st.decode())


def test_decode_graphs_share_a_workspace_and_streams(cuda_device):
    a = State(607, W.BF16, 8, 2, 128, 16, [3000, 700])
    b = State(608, W.F16, 16, 1, 64, 8, [5000, 1, 900])
    size = max(pa.pa_decode_workspace_size(8, 2, 128, 16, pa.PA_FP4_E2M1),
               pa.pa_decode_workspace_size(16, 1, 64, 8, pa.PA_FP4_E2M1))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(s.dev["q"]) for s in (a, b)]
    for s, o in ((a, outs[0]), (b, outs[1])):
        s.decode(workspace=ws, out=o)          # plans are looked up before the capture
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for s, o in ((a, outs[0]), (b, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.decode(workspace=ws, out=o, flags=pa.PA_DECODE_TABLES_READY)
        graphs.append(g)
    want = [s.expected() for s in (a, b)]
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:                       # one after the other on one stream
            g.replay()
        torch.cuda.synchronize()
        for s, o, w in ((a, outs[0], want[0]), (b, outs[1], want[1])):
            s.check(o, w)


def test_offsets_past_32_bits(cuda_device):
    # a pool of more than 4 GiB whose used blocks lie at its end
    st = State(609, W.BF16, 8, 2, 128, 16, [200, 33])
    nb = (5 << 30) // (2 * 16 * 72)
    big_k = torch.zeros((nb,) + st.k.shape[1:], dtype=torch.uint8, device="cuda")
    big_v = torch.zeros_like(big_k)
    off = nb - len(st.k)
    big_k[off:] = st.dev["k"]
    big_v[off:] = st.dev["v"]
    bt = torch.where(st.dev["bt"] >= 0, st.dev["bt"] + off, st.dev["bt"])
    out = pa.pa_decode_fp4(st.dev["q"], big_k, big_v, bt, st.dev["lens"], st.scale, st.k_scale,
                           st.v_scale, err=st.err)
    st.check(out)
    # the write and the read-back address the same rows
    x = torch.randn(3, 2, 128, device="cuda").bfloat16()
    slots = torch.tensor([nb * 16 - 1, nb * 16 - 17, 5], dtype=torch.int64, device="cuda")
    pa.pa_cache_write_fp4(x, x, slots, big_k, big_v, 0.3, 0.3, err=st.err)
    k, v = pa.pa_cache_read_fp4(slots, big_k, big_v, 0.3, 0.3)
    small = torch.zeros((1,) + st.k.shape[1:], dtype=torch.uint8, device="cuda")
    s3 = torch.arange(3, device="cuda")
    small_v = small.clone()
    pa.pa_cache_write_fp4(x, x, s3, small, small_v, 0.3, 0.3)
    k3, _ = pa.pa_cache_read_fp4(s3, small, small_v, 0.3, 0.3)
    assert torch.equal(k, k3) and torch.equal(v, k3)
    assert pa.pa_get_error(st.err) == 0


# ---------------------------------------------------------------------------
# write, read-back, block copies and swaps
# ---------------------------------------------------------------------------

def _pools(nb, B, H, D, fill=0):
    return [torch.full(pa.pa_fp4_pool_shape(nb, B, H, D), fill, dtype=torch.uint8, device="cuda")
            for _ in range(2)]


def _tie_rows(rng, n, H, D, scale):
    """float32 rows rich in exact ties: products of codes' midpoints with a
    power-of-two scale, zeros, tiny groups and saturating ones."""
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], np.float32)
    x = grid[rng.integers(0, 16, (n, H, D // 16, 16))] * rng.choice([-1, 1], (n, H, D // 16, 16))
    x = x * 2.0 ** rng.integers(-3, 4, (n, H, D // 16, 1))
    x[0, 0, 0] = 0                             # a group of zeros
    x[0, 0, 1] = scale * 2.0 ** -9             # a group that becomes zeros
    x[0, 0, 2] = scale * 6 * 2.0 ** -9         # one that keeps E4M3's smallest scale
    x[0, 0, 3] = 4 * 448 * 6 * scale           # one beyond the format's range
    return (x.reshape(n, H, D) * np.float32(1)).astype(np.float32)


@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
@pytest.mark.parametrize("H,D,B", [(8, 128, 16), (2, 64, 4), (3, 128, 8), (1, 64, 256)])
def test_write_and_read_back(cuda_device, dtype, H, D, B):
    rng = np.random.default_rng(700 + H)
    n, nb = 53, max(2, 80 // B + 2)
    for scales in ((1.0, 0.5), (0.0371, 0.811)):
        k = W.to_bits(_tie_rows(rng, n, H, D, scales[0]), dtype)
        v = W.to_bits(rng.standard_normal((n, H, D)).astype(np.float32), dtype)
        slots = rng.permutation(nb * B)[:n].astype(np.int64)
        slots[[3, 17]] = -1                    # padding
        kc, vc = _pools(nb, B, H, D, fill=0x5A)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_cache_write_fp4(to_dev(k, dtype), to_dev(v, dtype), torch.from_numpy(slots).cuda(),
                              kc, vc, *scales, err=err)
        want = [np.full(kc.shape, 0x5A, np.uint8) for _ in range(2)]
        f = [bits_to_f64(b, dtype).astype(np.float32) for b in (k, v)]
        oracle.cache_write_fp4(want[0], want[1], f[0], f[1], slots, *scales)
        for got, w in zip((kc, vc), want):
            got = got.cpu().numpy()
            assert np.array_equal(oracle.fp4_dequant(got, D), oracle.fp4_dequant(w, D))
            planes = [p.reshape(nb, H, -1)[..., B * D // 2:] for p in (got, w)]
            assert np.array_equal(*planes)     # the scale codes, untouched ones among them
        # back: rounded once to fp32 and once to 16 bits; padding rows as they were
        k_out = to_dev(np.full((n, H, D), 0x1234, np.uint16), dtype)
        v_out = k_out.clone()
        pa.pa_cache_read_fp4(torch.from_numpy(slots).cuda(), kc, vc, *scales, k_out=k_out,
                             v_out=v_out, err=err)
        for got, w, sc in zip((k_out, v_out), want, scales):
            rows = oracle.fp4_dequant(w, D).reshape(-1, H, D)[np.maximum(slots, 0)]
            val = (rows.astype(np.float32) * np.float32(sc)).astype(np.float32)
            assert np.all(np.isfinite(val))
            ok = slots >= 0
            if dtype == W.F16:                 # beyond binary16's range: infinities
                with np.errstate(over="ignore"):
                    ref = val.astype(np.float16).view(np.uint16)
            else:
                ref = W.to_bits(val, dtype)
            g = bits_of(got)
            zero = rows == 0
            assert np.array_equal(g[ok] & np.where(zero[ok], 0x7FFF, 0xFFFF),
                                  ref[ok] & np.where(zero[ok], 0x7FFF, 0xFFFF))
            assert np.all(g[~ok] == 0x1234)
        assert pa.pa_get_error(err) == 0


def test_mapped_write_equals_the_two_calls_and_reports(cuda_device):
    rng = np.random.default_rng(710)
    H, D, B, nb = 4, 128, 16, 20
    bt = torch.from_numpy(rng.permutation(nb)[:12].reshape(3, 4).astype(np.int32)).cuda()
    seq = torch.tensor([0, 1, 2, 2, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 17, 63, 62, 33, 5], dtype=torch.int32, device="cuda")
    k = torch.randn(6, H, D, device="cuda").half()
    v = torch.randn(6, H, D, device="cuda").half()
    a, b = _pools(nb, B, H, D), _pools(nb, B, H, D)
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    pa.pa_cache_write_fp4_mapped(k, v, bt, seq, pos, *a, 0.3, 0.2, slot_mapping=slots)
    s2 = pa.pa_slot_mapping(bt, seq, pos, B, nb)
    pa.pa_cache_write_fp4(k, v, s2, *b, 0.3, 0.2)
    assert torch.equal(slots, s2) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # slots beyond the pool are reported and skipped, by the write and the read
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    far = s2.clone()
    far[2] = nb * B
    c = _pools(nb, B, H, D)
    pa.pa_cache_write_fp4(k, v, far, *c, 0.3, 0.2, err=err)
    assert pa.pa_get_error(err) == pa.PA_DEVERR_SLOT
    back, _ = pa.pa_cache_read_fp4(far, *c, 0.3, 0.2, dtype=torch.float16, err=err)
    assert pa.pa_get_error(err) == pa.PA_DEVERR_SLOT
    assert not back[2].any() and back[[0, 1, 3, 4, 5]].any(-1).all()
    # a bad table entry; padding
    bt[1, 2] = -7
    seq[0] = -1
    d = _pools(nb, B, H, D)
    pa.pa_cache_write_fp4_mapped(k, v, bt, seq, pos, *d, 0.3, 0.2, slot_mapping=slots, err=err)
    assert pa.pa_get_error(err) == pa.PA_DEVERR_BLOCK_ID
    assert slots[[0, 4]].tolist() == [-1, -1] and torch.equal(slots[[1, 2, 3, 5]], s2[[1, 2, 3, 5]])
    # nothing to do
    pa.pa_cache_write_fp4(k[:0], v[:0], s2[:0], *d, 0.3, 0.2)
    assert pa.pa_cache_read_fp4(s2[:0], *d, 0.3, 0.2)[0].shape == (0, H, D)


@pytest.mark.parametrize("H,D,B", [(2, 64, 4), (3, 128, 16)])
def test_block_copy_and_swap(cuda_device, H, D, B):
    kc, vc = (torch.randint(0, 256, pa.pa_fp4_pool_shape(12, B, H, D), dtype=torch.uint8,
                            device="cuda") for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    pairs = torch.tensor([[0, 7], [3, 8], [0, 11]], dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks(pairs, kc, vc)
    for src, dst in pairs.tolist():
        k0[dst], v0[dst] = k0[src], v0[src]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    hk, hv = (torch.zeros(pa.pa_fp4_pool_shape(6, B, H, D), dtype=torch.uint8).pin_memory()
              for _ in range(2))
    out = torch.tensor([[7, 0], [2, 5]], dtype=torch.int32, device="cuda")
    pa.pa_swap_blocks(out, kc, vc, hk, hv)
    torch.cuda.synchronize()
    assert torch.equal(hk[0], k0[7].cpu()) and torch.equal(hv[5], v0[2].cpu())
    assert not hk[1:5].any()
    back = torch.tensor([[5, 1], [0, 4]], dtype=torch.int32, device="cuda")
    pa.pa_swap_blocks(back, hk, hv, kc, vc)
    k0[1], v0[1], k0[4], v0[4] = k0[2], v0[2], k0[7], v0[7]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

def test_steps_of_append_and_decode(cuda_device):
    """A prompt and ten decode steps: append (norm, rotation, 4-bit store), then
    decode, every step against the oracle's decode of the pool's own codes."""
    rng = np.random.default_rng(800)
    Hq, H, D, B, N, nb = 8, 2, 128, 16, 3, 40
    perm = rng.permutation(nb)[:12 * N].astype(np.int32).reshape(N, 12)
    bt = torch.from_numpy(perm).cuda()
    ang = np.arange(200)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    cs = torch.from_numpy(np.concatenate((np.cos(ang), np.sin(ang)), -1).astype(np.float32)).cuda()
    kc, vc = _pools(nb, B, H, D, fill=0x7F)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(pa.pa_decode_workspace_size(Hq, H, D, B, pa.PA_FP4_E2M1), dtype=torch.uint8,
                     device="cuda")
    lens = np.zeros(N, np.int64)
    for step in range(11):
        new = np.array([150, 1, 31]) if step == 0 else np.ones(N, np.int64)
        seq = np.repeat(np.arange(N), new).astype(np.int32)
        pos = np.concatenate([np.arange(p, p + c) for p, c in zip(lens, new)]).astype(np.int32)
        lens = lens + new
        x = torch.from_numpy(rng.standard_normal((seq.size, (Hq + 2 * H) * D)).astype(np.float32))
        x = x.cuda().bfloat16()
        q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, H * D, H * D], 1))
        q = pa.pa_append_rope(q, k, v, cs, bt, torch.from_numpy(seq).cuda(),
                              torch.from_numpy(pos).cuda(), kc, vc, q_norm=w, k_norm=w,
                              k_scale=0.25, v_scale=0.25, err=err)
        last = torch.from_numpy(np.cumsum(new) - 1).cuda()
        q = q[last].contiguous()
        out = pa.pa_decode_fp4(q, kc, vc, bt, torch.from_numpy(lens.astype(np.int32)).cuda(),
                               D ** -0.5, 0.25, 0.25, workspace=ws, err=err)
        o, spread = oracle.paged_decode_fp4(bits_to_f64(bits_of(q), W.BF16), kc.cpu().numpy(),
                                            vc.cpu().numpy(), 0.25, 0.25, perm, lens, D ** -0.5)
        rounding_report(bits_of(out), o, spread, W.BF16, 2.0 ** -11, "step %d" % step)
    assert pa.pa_get_error(err) == 0


def test_prefill_over_rows_read_back(cuda_device):
    """A prompt chunk over a 4-bit context: its rows read back into a 16-bit
    pool, the chunk appended there, and the prefill over both."""
    rng = np.random.default_rng(801)
    Hq, H, D, B, T, L = 8, 2, 128, 16, 96, 40
    kc, vc = _pools(10, B, H, D)
    table = torch.tensor([[7, 2, 9, 0, 4, 5]], dtype=torch.int32, device="cuda")
    zeros = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    k = torch.randn(T, H, D, device="cuda").bfloat16()
    v = torch.randn(T, H, D, device="cuda").bfloat16()
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    pa.pa_cache_write_fp4_mapped(k, v, table, zeros, pos, kc, vc, 0.25, 0.25, slot_mapping=slots)
    kp = torch.zeros(9, B, H, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    pa.pa_cache_read_fp4(slots, kc, vc, 0.25, 0.25, k_out=kp.view(-1, H, D)[:T],
                         v_out=vp.view(-1, H, D)[:T])
    bt = torch.arange(9, dtype=torch.int32, device="cuda")[None].contiguous()
    ang = np.arange(200)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    cs = torch.from_numpy(np.concatenate((np.cos(ang), np.sin(ang)), -1).astype(np.float32)).cuda()
    x = torch.randn(L, Hq + 2 * H, D, device="cuda").bfloat16()
    q = pa.pa_append_rope(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], cs, bt, zeros[:L],
                          pos[:L] + T, kp, vp)
    out = pa.pa_prefill(q, kp, vp, bt, torch.tensor([T + L], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, L], dtype=torch.int32, device="cuda"), D ** -0.5)
    K = np.concatenate((oracle.fp4_dequant(kc.cpu().numpy(), D)[table[0].cpu()].reshape(-1, H, D)
                        * 0.25, bits_to_f64(bits_of(kp.view(-1, H, D)[T:T + L]), W.BF16)))
    V = np.concatenate((oracle.fp4_dequant(vc.cpu().numpy(), D)[table[0].cpu()].reshape(-1, H, D)
                        * 0.25, bits_to_f64(bits_of(x[:, Hq + H:]), W.BF16)))
    got = out.float().cpu().numpy()
    for j in (0, 1, L - 1):
        ref = oracle.contiguous_decode(bits_to_f64(bits_of(q[j]), W.BF16), K[:T + j + 1],
                                       V[:T + j + 1], D ** -0.5)
        # with a power of two as scale every value that was read back is exact
        assert_close(got[j], ref, "row %d" % j)


def test_argument_checks(cuda_device):
    st = State(620, W.BF16, 8, 2, 128, 16, [30, 5])
    d = st.dev

    def call(**kw):
        a = dict(q=d["q"], k_cache=d["k"], v_cache=d["v"], block_tables=d["bt"],
                 seq_lens=d["lens"], scale=0.1, k_scale=1.0, v_scale=1.0)
        a.update(kw)
        return pa.pa_decode_fp4(**a)
    call()
    half_k, half_v = (d[p][..., :64].contiguous() for p in "kv")
    for kw, exc in ((dict(q=d["q"].float()), TypeError),
                    (dict(q=d["q"][..., :64].contiguous()), ValueError),
                    (dict(k_cache=half_k, v_cache=half_v), ValueError),
                    (dict(seq_lens=d["lens"].long()), TypeError),
                    (dict(block_tables=d["bt"][:1].contiguous()), ValueError),
                    (dict(out=d["q"][:1]), ValueError), (dict(q=d["q"].cpu()), ValueError),
                    (dict(k_cache=d["k"].transpose(0, 1)), ValueError)):
        with pytest.raises(exc):
            call(**kw)
    small = torch.zeros(64, dtype=torch.uint8, device="cuda")
    for kw, status in ((dict(window=-1), 1), (dict(k_scale=0.0), 1),
                       (dict(flags=pa.PA_DECODE_SIMT), 2), (dict(workspace=small), 3),
                       (dict(num_ctas=pa.PA_DECODE_MAX_CTAS + 1), 1)):
        with pytest.raises(pa.PAError) as e:
            call(**kw)
        assert e.value.status == status, kw
    with pytest.raises(ValueError):
        pa.pa_cache_read_fp4(torch.zeros(2, dtype=torch.int64, device="cuda"), d["k"], d["v"], 1.0,
                             1.0, k_out=torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda"))
    # ulp_spacing is what the bounds count: one bfloat16 step above 1 is 2^-7
    assert ulp_spacing(W.to_bits(np.float32(1.0), W.BF16), W.BF16) == 2.0 ** -7


# ---------------------------------------------------------------------------
# the largest calls, and several calls at once
# ---------------------------------------------------------------------------

def _constant_pools(blocks, B, D, seed):
    """One KV head; keys zero, every row's values the same vector of E2M1 values
    with unit scales.  Every attended mean is that vector, and every product and
    partial sum of the decode a multiple of 2^12 below 2^36: exact in fp32 up to
    the joins of partial sums."""
    rng = np.random.default_rng(seed)
    row = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[rng.integers(0, 8, D)] * rng.choice([-1, 1], D)
    code = oracle.e2m1_encode(row).astype(np.uint8)
    v = np.zeros((blocks, 1, B * 9 * D // 16), np.uint8)
    v[..., :B * D // 2] = np.tile(code[0::2] | (code[1::2] << 4), B)
    v[..., B * D // 2:] = 0x38               # E4M3 one
    k = np.zeros_like(v)
    k[..., B * D // 2:] = 0x38
    return row, k, v


@pytest.mark.parametrize("window", [0, 40])
def test_decode_longest_context(cuda_device, window):
    # 2^31 - 1 tokens, the most an int32 length says; the row behind the last
    # token has NaN scales
    B, D, T = 256, 64, 2 ** 31 - 1
    row, k, v = _constant_pools(2, B, D, 620)
    for p in (k, v):
        p[1, 0, B * D // 2:].reshape(B // 4, D // 16, 4)[-1, :, 3] = 0x7F
    bt = torch.zeros((1, 2 ** 23), dtype=torch.int32, device="cuda")
    bt[0, -1] = 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, D, device="cuda").bfloat16()
    pools = [torch.from_numpy(p.reshape(2, 1, B, 9 * D // 16)).cuda() for p in (k, v)]
    out = pa.pa_decode_fp4(q, *pools, bt, torch.tensor([T], dtype=torch.int32, device="cuda"), 1.0,
                           1.0, 1.0, window=window, err=err)
    assert pa.pa_get_error(err) == 0
    # the joins leave relative errors below 2^-12, the values need 2 of 8 bits
    assert np.array_equal(bits_to_f64(bits_of(out), W.BF16)[0], np.tile(row, (4, 1)))


def test_decode_quarter_million_sequences(cuda_device):
    n, B, D = 2 ** 18 + 1500, 4, 64
    row, k, v = _constant_pools(64, B, D, 621)
    sizes = np.arange(64) % 4                 # block b: its values times 2^(b % 4)
    v[..., B * D // 2:] = (0x38 + 8 * sizes)[:, None, None]
    rng = np.random.default_rng(622)
    lens = rng.integers(0, 4, n).astype(np.int32)
    bt = rng.integers(0, 64, (n, 1)).astype(np.int32)
    pools = [torch.from_numpy(p.reshape(64, 1, B, 9 * D // 16)).cuda() for p in (k, v)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.pa_decode_fp4(torch.randn(n, 1, D, device="cuda").bfloat16(), *pools,
                           torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 1.0, 1.0,
                           1.0, out=torch.full((n, 1, D), float("nan"), dtype=torch.bfloat16,
                                               device="cuda"), err=err)
    assert pa.pa_get_error(err) == 0
    want = torch.from_numpy(row * (2.0 ** sizes[bt] * (lens[:, None] > 0))).cuda()
    assert torch.equal(out[:, 0].double(), want)


def test_decodes_of_three_caches_share_a_workspace(cuda_device):
    st = State(623, W.BF16, 8, 2, 128, 16, [2000, 1, 300])
    nb = len(st.k)
    gen = torch.Generator(device="cuda").manual_seed(624)
    k16, v16 = (torch.randn((nb, 16, 2, 128), device="cuda", generator=gen).bfloat16()
                for _ in range(2))
    k8, v8 = (torch.randint(0, 0x70, (nb, 16, 2, 128), dtype=torch.uint8, device="cuda",
                            generator=gen) for _ in range(2))
    d = st.dev
    ws = torch.zeros(max(pa.pa_decode_workspace_size(8, 2, 128, 16, t)
                         for t in (pa.PA_BF16, pa.PA_FP8_E4M3, pa.PA_FP4_E2M1)),
                     dtype=torch.uint8, device="cuda")

    def run16(w):
        return pa.pa_decode(d["q"], k16, v16, d["bt"], d["lens"], st.scale, workspace=w)

    def run8(w):
        return pa.pa_decode_fp8(d["q"], k8, v8, d["bt"], d["lens"], st.scale, 0.1, 0.1, workspace=w)

    runs = (run16, run8, lambda w: st.decode(workspace=w))
    alone = [f(None) for f in runs]
    ref = st.expected()
    for order in ((0, 1, 2), (2, 0, 2, 1), (1, 2, 0)):
        for i in order:
            out = runs[i](ws)
            assert torch.equal(out, alone[i]), i
            if i == 2:
                st.check(out, ref)


def test_decodes_on_two_streams_at_once(cuda_device):
    # a workspace each
    states = [State(625, W.BF16, 32, 8, 128, 16, [4000, 900]), State(626, W.F16, 8, 2, 64, 8, [7000])]
    alone = [st.decode() for st in states]
    ws = [torch.zeros(pa.pa_decode_workspace_size(st.q.shape[1], st.H, st.D, st.B, pa.PA_FP4_E2M1),
                      dtype=torch.uint8, device="cuda") for st in states]
    streams = [torch.cuda.Stream() for _ in states]
    kept = [[torch.zeros_like(st.dev["q"]) for _ in range(20)] for st in states]
    torch.cuda.synchronize()
    for n in range(20):
        for st, s, w, out in zip(states, streams, ws, kept):
            with torch.cuda.stream(s):
                st.decode(workspace=w, out=out[n])
    torch.cuda.synchronize()
    for a, out, st in zip(alone, kept, states):
        assert all(torch.equal(o, a) for o in out)
        assert pa.pa_get_error(st.err) == 0


@pytest.mark.parametrize("B", [4, 8, 32, 128])
@pytest.mark.parametrize("window", [0, 150])
def test_decode_leaves_out_bad_blocks_of_every_size(cuda_device, B, window):
    # of 300 tokens, whole blocks drop out at both ends and inside a tile; the rest is
    # attended to as if their weights were zero
    st = State(630 + B, W.F16, 4, 2, 64, B, [300, 300, 5], window=window)
    lost = [299 // B] if B > 32 else sorted({180 // B, 180 // B + 2, 299 // B})
    bt = st.bt.copy()
    bt[0, lost] = [len(st.k), -7, 1 << 30][:len(lost)]
    st.dev["bt"] = torch.from_numpy(bt).cuda()
    out = st.decode()
    assert pa.pa_get_error(st.err) == pa.PA_DEVERR_BLOCK_ID
    q = bits_to_f64(st.q, W.F16)
    k, v = oracle.fp4_dequant(st.k, 64) * st.k_scale, oracle.fp4_dequant(st.v, 64) * st.v_scale
    rows = [t for t in range(max(0, 300 - window) if window else 0, 300) if t // B not in lost]
    blk, off = st.bt[0, np.array(rows) // B], np.array(rows) % B
    o, spread = st.expected()
    for h in range(4):
        kk, vv = k[blk, off, h // 2], v[blk, off, h // 2]
        w = np.exp(st.scale * (kk @ q[0, h]) - (st.scale * (kk @ q[0, h])).max())
        w /= w.sum()
        o[0, h] = w @ vv
        spread[0, h] = w @ np.abs(vv - o[0, h])
    rounding_report(bits_of(out), o, spread, W.F16, _u_p(W.F16), "B=%d" % B)
