"""The append (head norms, position rotation, store at the slots) on the GPU.

Without norms the kernel computes each product and sum of the rotation in
binary32, rounded one by one, as the oracle does in numpy: queries, 16-bit pools
and the quantized pools' bytes must be equal bit for bit.  With norms the
binary32 sum of squares depends on its order, so the 16-bit results are held to
the formula in 64 bits:
    |g - y| <= ulp16(g) / 2 + 2^-19 (|a| + |b|)
with a, b the normed pair in 64 bits.  Half an ulp is the one rounding to 16
bits.  The rest is binary32 work: a row's sum of at most 128 squares in a chain
of 8 and 4 tree levels is within 12 * 2^-24 relative, the mean, the sum with
eps, the root and its reciprocal add 4 roundings, half of all that reaches the
root; the two products of the norm and the rotation's two roundings add 4:
under 14 * 2^-24 < 2^-20 of |a| + |b|, doubled for the angles' products.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_72_gb300 as pa
import workloads as W
from harness import bits_of, bits_to_f64, to_dev, ulp_spacing

pytestmark = pytest.mark.gpu

KINDS = ("16", "e4m3", "e2m1")


def _table(max_pos, rot, base=10000.0):
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate((np.cos(ang), np.sin(ang)), -1).astype(np.float32)


class Step:
    """One step's inputs on the host and the GPU: ragged sequences, tokens in a
    random order, q, k, v views of one projection's output."""

    def __init__(self, seed, dtype, Hq, H, D, B, past, new, kind, rot, norm="", spare=3, pad=()):
        rng = np.random.default_rng(seed)
        self.dtype, self.Hq, self.H, self.D, self.B, self.kind, self.rot = (dtype, Hq, H, D, B,
                                                                            kind, rot)
        lens = np.asarray(past) + np.asarray(new)
        need = -(-lens // B)
        self.nb = int(need.sum()) + spare
        perm = rng.permutation(self.nb).astype(np.int32)
        self.bt = np.full((lens.size, max(1, int(need.max()))), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.bt[i, :n] = perm[at:at + n]
            at += n
        seq = np.repeat(np.arange(lens.size), new)
        pos = np.concatenate([np.arange(p, p + c) for p, c in zip(past, new)])
        order = rng.permutation(seq.size)
        self.seq, self.pos = seq[order].astype(np.int32), pos[order].astype(np.int32)
        for n in pad:
            self.seq[n] = -1
        self.n = seq.size
        self.width = (Hq + 2 * H) * D + 24      # rows further apart than they are long
        x = rng.standard_normal((self.n, self.width)).astype(np.float32)
        self.x = W.to_bits(x, dtype)
        self.dx = to_dev(self.x, dtype)
        self.max_pos = int(lens.max()) + 5
        self.cs = _table(self.max_pos, rot) if rot else None
        self.qn = W.to_bits(1 + 0.3 * rng.standard_normal(D).astype(np.float32), dtype)
        self.kn = W.to_bits(1 + 0.3 * rng.standard_normal(D).astype(np.float32), dtype)
        self.norm = norm
        self.k_scale, self.v_scale = {"16": (1.0, 1.0), "e4m3": (0.011, 2.0 ** -7),
                                      "e2m1": (0.3, 0.5)}[kind]
        if kind == "16":
            self.pool0 = rng.integers(0, 1 << 14, (2, self.nb, B, H, D)).astype(np.uint16)
        elif kind == "e4m3":
            self.pool0 = rng.integers(0, 127, (2, self.nb, B, H, D), dtype=np.uint8)
        else:
            self.pool0 = rng.integers(0, 127, (2, self.nb, H, B, 9 * D // 16), dtype=np.uint8)
        self.k_cache, self.v_cache = (self._dev(p) for p in self.pool0)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _dev(self, p):
        return to_dev(p, self.dtype) if self.kind == "16" else torch.from_numpy(p).cuda()

    def rows(self, part, x=None):
        x = self.x if x is None else x
        Hq, H, D = self.Hq, self.H, self.D
        lo, hi, h = {"q": (0, Hq * D, Hq), "k": (Hq * D, (Hq + H) * D, H),
                     "v": ((Hq + H) * D, (Hq + 2 * H) * D, H)}[part]
        return x[:, lo:hi].reshape(x.shape[0], h, D) if isinstance(x, np.ndarray) else \
            x[:, lo:hi].unflatten(-1, (h, D))

    def call(self, interleaved=False, **kw):
        args = dict(interleaved=interleaved, k_scale=self.k_scale, v_scale=self.v_scale,
                    err=self.err, eps=1e-5)
        if "q" in self.norm:
            args["q_norm"] = to_dev(self.qn, self.dtype)
        if "k" in self.norm:
            args["k_norm"] = to_dev(self.kn, self.dtype)
        args.update(kw)
        cs = None if self.cs is None else torch.from_numpy(self.cs).cuda()
        q = self.rows("q", self.dx) if self.Hq else None
        return pa.pa_append_rope(q, self.rows("k", self.dx), self.rows("v", self.dx), cs,
                                 torch.from_numpy(self.bt).cuda(),
                                 torch.from_numpy(self.seq).cuda(),
                                 torch.from_numpy(self.pos).cuda(), self.k_cache, self.v_cache,
                                 **args)

    def slots(self):
        live = self.seq >= 0
        blk = self.bt[np.maximum(self.seq, 0), self.pos // self.B].astype(np.int64)
        return np.where(live, blk * self.B + self.pos % self.B, -1)

    def rotated(self, part, interleaved):
        """16-bit patterns of the rotated rows, every operation in binary32."""
        x = bits_to_f64(self.rows(part), self.dtype).astype(np.float32)
        if self.rot:
            x = oracle.rotate(x, self.cs[self.pos], interleaved)
        assert x.dtype == np.float32
        return W.to_bits(x, self.dtype)

    def stored(self, k_bits, v_bits):
        """The pools after k_bits, v_bits [n, H, D] are stored at the slots."""
        kc, vc = self.pool0[0].copy(), self.pool0[1].copy()
        s = self.slots()
        if self.kind == "16":
            oracle.cache_write(kc, vc, k_bits, v_bits, s)
        elif self.kind == "e4m3":
            oracle.cache_write_fp8(kc, vc, k_bits, v_bits, self.dtype, s, self.k_scale,
                                   self.v_scale)
        else:
            f = [bits_to_f64(b, self.dtype).astype(np.float32) for b in (k_bits, v_bits)]
            oracle.cache_write_fp4(kc, vc, f[0], f[1], s, self.k_scale, self.v_scale)
        return kc, vc

    def pools(self):
        return [bits_of(p) if self.kind == "16" else p.cpu().numpy()
                for p in (self.k_cache, self.v_cache)]


def _same_pools(st, want):
    for got, w, pool in zip(st.pools(), want, "KV"):
        if st.kind == "e2m1":   # a zero may carry either sign
            D = st.D
            assert np.array_equal(oracle.fp4_dequant(got, D), oracle.fp4_dequant(w, D)), pool
        else:
            assert np.array_equal(got, w), pool


SHAPES = [
    # dtype, Hq, H, D, B, past, new
    (W.F16, 8, 8, 64, 4, [6, 7, 8, 32], [1, 1, 1, 1]),            # the tiny workload's step
    (W.BF16, 32, 8, 128, 16, [0, 15, 16, 400, 33], [1, 1, 1, 1, 1]),
    (W.BF16, 14, 2, 64, 16, [1800, 5], [37, 300]),                # many tokens, two passes
    (W.F16, 5, 5, 128, 8, [3], [1]),                              # one token
    (W.BF16, 7, 1, 128, 256, [250, 0], [9, 2]),
    (W.F16, 3, 3, 64, 32, [0, 0, 31], [5, 1, 2]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_is_bit_exact_without_norms(cuda_device, shape, interleaved, kind):
    dtype, Hq, H, D, B, past, new = SHAPES[shape]
    for rot in (D, D // 2, 16, 0):
        st = Step(100 + shape + rot, dtype, Hq, H, D, B, past, new, kind, rot)
        slots = torch.full((st.n,), 7, dtype=torch.int64, device="cuda")
        q = st.call(interleaved, slot_mapping=slots)
        assert np.array_equal(bits_of(q), st.rotated("q", interleaved)), rot
        assert np.array_equal(slots.cpu().numpy(), st.slots())
        _same_pools(st, st.stored(st.rotated("k", interleaved), st.rows("v")))
        assert pa.pa_get_error(st.err) == 0


@pytest.mark.parametrize("norm", ["q", "k", "qk"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_norms(cuda_device, shape, norm):
    dtype, Hq, H, D, B, past, new = SHAPES[shape]
    interleaved = bool(shape % 2)
    for rot in (D, D // 2, 0):
        st = Step(200 + shape + rot, dtype, Hq, H, D, B, past, new, "16", rot, norm)
        q = st.call(interleaved)
        s = st.slots()
        k = st.pools()[0].reshape(-1, H, D)[s]
        for part, got, w in (("q", bits_of(q), st.qn), ("k", k, st.kn)):
            y = bits_to_f64(st.rows(part), dtype)
            if part in norm:
                y = oracle.head_norm(y, bits_to_f64(w, dtype), 1e-5)
            mag = np.abs(y)
            if rot:
                cs = st.cs[st.pos].astype(np.float64)
                one = np.concatenate((np.ones(rot // 2), np.zeros(rot // 2)))[None].repeat(st.n, 0)
                mag = (np.abs(oracle.rotate(y, one, interleaved))
                       + np.abs(oracle.rotate(y, np.roll(one, rot // 2, 1), interleaved)))
                y = oracle.rotate(y, cs, interleaved)
            bound = 0.5 * ulp_spacing(got, dtype) + 2.0 ** -19 * mag
            assert np.all(np.abs(bits_to_f64(got, dtype) - y) <= bound), (part, rot)
        # values are neither normed nor rotated, and nothing else is written
        want = st.stored(k, st.rows("v"))
        _same_pools(st, want)
        # a quantized pool stores the 16-bit pool's keys, quantized
        for kind in ("e4m3", "e2m1"):
            qt = Step(200 + shape + rot, dtype, Hq, H, D, B, past, new, kind, rot, norm)
            assert np.array_equal(bits_of(qt.call(interleaved)), bits_of(q))
            _same_pools(qt, qt.stored(k, qt.rows("v")))


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
def test_quantized_stores_of_every_16_bit_value(cuda_device, dtype, kind):
    """Every finite 16-bit pattern as a key, in groups of any neighbours and in
    groups of like magnitudes, at scales in and far outside the common range:
    the quotients are the correctly rounded ones, so every code is the oracle's."""
    rng = np.random.default_rng(9)
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    with np.errstate(invalid="ignore"):
        finite = np.isfinite(bits_to_f64(bits, dtype))
    bits[~finite] = W.to_bits(np.float32(1.0), dtype)
    near = bits[np.argsort(np.abs(bits_to_f64(bits, dtype)), kind="stable")]
    k = np.concatenate((rng.permutation(bits), near)).reshape(256, 4, 128)
    n = len(k)
    zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None].contiguous()
    dk = to_dev(k, dtype)
    for scale in (1.0, 0.0371, 2.0 ** -20, 1.5e-30, 3e-37, 7.7e8, 2e30, 5e37):
        scale = float(np.float32(scale))
        shape = pa.pa_fp4_pool_shape(n // 16, 16, 4, 128)
        if kind == "e4m3":
            shape = (n // 16, 16, 4, 128)
        kc, vc = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        pa.pa_append_rope(None, dk, dk, None, table, zeros, pos, kc, vc, k_scale=scale, v_scale=1.0)
        want = [np.full(shape, 0x7F, np.uint8) for _ in range(2)]
        if kind == "e4m3":
            oracle.cache_write_fp8(want[0], want[1], k, k, dtype, np.arange(n), scale, 1.0)
            assert np.array_equal(kc.cpu().numpy() & 0x7F, want[0] & 0x7F), scale
            assert np.array_equal(oracle.e4m3_decode(vc.cpu().numpy()), oracle.e4m3_decode(want[1]))
        else:
            x = bits_to_f64(k, dtype).astype(np.float32)
            oracle.cache_write_fp4(want[0], want[1], x, x, np.arange(n), scale, 1.0)
            got = kc.cpu().numpy()
            assert np.array_equal(got.reshape(n // 16, 4, -1)[..., 16 * 64:],
                                  want[0].reshape(n // 16, 4, -1)[..., 16 * 64:]), scale
            assert np.array_equal(oracle.fp4_dequant(got, 128),
                                  oracle.fp4_dequant(want[0], 128)), scale


def test_append_padding_and_bad_tokens_write_nothing(cuda_device):
    for kind in KINDS:
        st = Step(301, W.BF16, 8, 2, 128, 16, [5, 20, 100], [4, 30, 7], kind, 128, pad=(0, 11, 40))
        q_out = torch.full((st.n, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        slots = torch.full((st.n,), 7, dtype=torch.int64, device="cuda")
        st.call(q_out=q_out, slot_mapping=slots)
        assert pa.pa_get_error(st.err) == 0        # padding is no error
        want = st.rotated("q", False)
        want[[0, 11, 40]] = W.to_bits(np.float32(3.0), W.BF16)
        assert np.array_equal(bits_of(q_out), want)
        assert np.array_equal(slots.cpu().numpy(), st.slots())
        _same_pools(st, st.stored(st.rotated("k", False), st.rows("v")))
    # bad tokens: reported, nothing written, the others stored
    for what, bit in (("seq", pa.PA_DEVERR_POSITION), ("neg", pa.PA_DEVERR_POSITION),
                      ("pos", pa.PA_DEVERR_POSITION), ("far", pa.PA_DEVERR_POSITION),
                      ("table", pa.PA_DEVERR_BLOCK_ID), ("block", pa.PA_DEVERR_BLOCK_ID)):
        st = Step(302, W.F16, 4, 2, 64, 8, [5, 20], [4, 13], "16", 64)
        bad = 6
        pos = st.pos.copy()
        if what == "seq":
            st.seq[bad] = 2
        elif what == "neg":
            st.seq[bad] = -2
        elif what == "pos":
            st.pos[bad] = -1
        elif what == "far":
            st.cs = st.cs[:20]                       # the angle table ends at position 20
        else:
            i, p = st.seq[bad], st.pos[bad] // 8
            hit = (st.seq == i) & (st.pos // 8 == p)
            good_bt = st.bt.copy()
            st.bt[i, p] = -1 if what == "table" else st.nb
        q_out = torch.full((st.n, 4, 64), 3.0, dtype=torch.float16, device="cuda")
        st.call(q_out=q_out)
        assert pa.pa_get_error(st.err) == bit, what
        gone = np.zeros(st.n, bool)
        if what == "far":
            gone = st.pos >= 20
            st.cs = _table(st.max_pos, 64)
        elif what in ("table", "block"):
            gone = hit
            st.bt = good_bt
        else:
            gone[bad] = True
        assert gone.any() and not gone.all()
        st.pos = pos
        st.seq[gone] = -1                            # for the oracle: not there
        want = st.rotated("q", False)
        want[gone] = W.to_bits(np.float32(3.0), W.F16)
        assert np.array_equal(bits_of(q_out), want), what
        _same_pools(st, st.stored(st.rotated("k", False), st.rows("v")))


def test_append_without_queries_in_place_and_empty(cuda_device):
    st = Step(303, W.BF16, 0, 4, 64, 16, [3, 9], [20, 1], "16", 64)
    assert st.call() is None
    _same_pools(st, st.stored(st.rotated("k", False), st.rows("v")))
    # q_out may be q itself
    st = Step(304, W.BF16, 6, 2, 128, 16, [3, 9], [200, 111], "16", 128)
    q = st.rows("q", st.dx).contiguous()
    pa.pa_append_rope(q, st.rows("k", st.dx), st.rows("v", st.dx), torch.from_numpy(st.cs).cuda(),
                      torch.from_numpy(st.bt).cuda(), torch.from_numpy(st.seq).cuda(),
                      torch.from_numpy(st.pos).cuda(), st.k_cache, st.v_cache, q_out=q, err=st.err)
    assert np.array_equal(bits_of(q), st.rotated("q", False))
    assert pa.pa_get_error(st.err) == 0
    # no tokens
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    k = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    before = bits_of(st.k_cache)
    out = pa.pa_append_rope(k, k, k, torch.from_numpy(st.cs).cuda(),
                            torch.from_numpy(st.bt).cuda(), none, none, st.k_cache, st.v_cache)
    assert out.shape == (0, 2, 128) and np.array_equal(bits_of(st.k_cache), before)


def test_append_passes_non_finite_values_through(cuda_device):
    # an infinity or NaN stays within its own pair (and its own head)
    st = Step(305, W.F16, 2, 1, 64, 16, [0], [3], "16", 32)
    x = st.dx.clone()
    x[0, 3] = float("inf")         # element 3 of query head 0: pairs with 19
    x[1, 64 + 50] = float("nan")   # element 50 of query head 1: not rotated
    st.dx = x
    q = st.call().float().cpu().numpy()
    bad = ~np.isfinite(q)
    want = np.zeros_like(bad)
    want[0, 0, [3, 19]] = True
    want[1, 1, 50] = True
    # position 0 has sin = 0: inf * 0 is NaN, in the pair all the same
    assert np.array_equal(bad, want)


def test_append_far_positions_and_graph_replay(cuda_device):
    # position 131,071 of a table computed in 64 bits; captured once, replayed
    # with new contents in the same buffers, on another stream
    st = Step(306, W.BF16, 8, 2, 128, 256, [131071, 70000], [1, 1], "e2m1", 128)
    q_out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    cs = torch.from_numpy(st.cs).cuda()
    bt, seq, pos = (torch.from_numpy(t).cuda() for t in (st.bt, st.seq, st.pos))
    args = (st.rows("q", st.dx), st.rows("k", st.dx), st.rows("v", st.dx), cs, bt, seq, pos,
            st.k_cache, st.v_cache)
    kw = dict(k_scale=st.k_scale, v_scale=st.v_scale, q_out=q_out, err=st.err)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pa.pa_append_rope(*args, **kw)
    for seed in (1, 2):
        st.x = W.to_bits(np.random.default_rng(seed).standard_normal(st.x.shape).astype(np.float32),
                         W.BF16)
        st.dx.copy_(to_dev(st.x, W.BF16))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(q_out), st.rotated("q", False))
        _same_pools(st, st.stored(st.rotated("k", False), st.rows("v")))
    assert pa.pa_get_error(st.err) == 0


def test_append_argument_checks(cuda_device):
    st = Step(307, W.BF16, 4, 2, 64, 16, [3], [5], "16", 64)
    q, k, v = (st.rows(p, st.dx) for p in "qkv")
    cs, bt, seq, pos = (torch.from_numpy(t).cuda() for t in (st.cs, st.bt, st.seq, st.pos))

    def call(**kw):
        a = dict(q=q, k=k, v=v, cos_sin=cs, block_tables=bt, token_seq=seq, token_pos=pos,
                 k_cache=st.k_cache, v_cache=st.v_cache)
        a.update(kw)
        return pa.pa_append_rope(**a)
    call()
    for kw, exc in ((dict(k=k.half()), TypeError), (dict(q=q.transpose(1, 2)), ValueError),
                    (dict(q=q[..., :32]), ValueError), (dict(token_seq=seq.long()), TypeError),
                    (dict(token_pos=pos[:4]), ValueError), (dict(cos_sin=cs.double()), TypeError),
                    (dict(k=k.cpu()), ValueError), (dict(q_norm=torch.ones(64).cuda()), ValueError),
                    (dict(q_out=q), ValueError), (dict(q=None, q_out=q), ValueError),
                    (dict(slot_mapping=seq), ValueError), (dict(block_tables=bt[0]), ValueError),
                    (dict(err=torch.zeros(1).cuda()), ValueError),
                    (dict(k_cache=st.k_cache.half(), v_cache=st.v_cache.half()), TypeError)):
        with pytest.raises(exc):
            call(**kw)
    # a token stride that is no multiple of 8 elements is refused by the library
    odd = torch.zeros(5, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    odd = odd[:, :128].unflatten(1, (2, 64))
    with pytest.raises(pa.PAError) as e:
        call(k=odd)
    assert e.value.status == 1
