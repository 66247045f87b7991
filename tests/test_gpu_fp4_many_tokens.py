"""The 4-bit write and read-back where blocks of threads take several tokens, and on
both sides of the row count from which the write takes a warp or more a token.

A block takes several tokens as long as two blocks an SM remain (from 608 tokens on
152 SMs), and the last block may hold fewer.  Codes, scales, slots and rows that no
token names are compared with the oracle's; the slots of the mapped write with the
plain slot mapping's.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_72_gb300 as pa
import workloads as W
from harness import bits_of, bits_to_f64, to_dev

pytestmark = pytest.mark.gpu

SHAPES = [
    # H, D, tokens
    (1, 64, 8191), (2, 64, 607), (2, 64, 608), (3, 64, 1801), (15, 64, 913), (16, 64, 912),
    (33, 64, 321), (1, 128, 4099), (2, 128, 1216), (5, 128, 1801), (7, 128, 609), (8, 128, 608),
    (8, 128, 1201), (15, 128, 307),
]


class Rows:
    """n tokens' K and V rows and the slots of all but some of them."""

    def __init__(self, seed, dtype, H, D, n, B=16):
        rng = np.random.default_rng(seed)
        self.dtype, self.H, self.D, self.n, self.B = dtype, H, D, n, B
        self.nb = -(-n // B) + 3
        self.k, self.v = (W.to_bits(rng.standard_normal((n, H, D)).astype(np.float32), dtype)
                          for _ in range(2))
        self.slots = rng.permutation(self.nb * B)[:n].astype(np.int64)
        self.pad = np.array([0, 5, n // 2, n - 1])
        self.far = np.array([3, n // 3, n - 2])
        self.scales = (0.3, 0.7)
        self.pools = [torch.full(pa.pa_fp4_pool_shape(self.nb, B, H, D), 0x5A, dtype=torch.uint8,
                                 device="cuda") for _ in range(2)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self):
        return to_dev(self.k, self.dtype), to_dev(self.v, self.dtype)

    def check_pools(self, slots):
        """the pools, byte for byte, after a write at `slots` (below 0: nothing)"""
        for pool, bits, sc in zip(self.pools, (self.k, self.v), self.scales):
            B, D, H = self.B, self.D, self.H
            codes, s16 = oracle.fp4_quantize(bits_to_f64(bits, self.dtype).astype(np.float32), sc)
            w = np.full((self.nb, H, B * 9 * D // 16), 0x5A, np.uint8)
            c = w[..., :B * D // 2].reshape(self.nb, H, B, D // 2)
            s = w[..., B * D // 2:].reshape(self.nb, H, B // 4, D // 16, 4)
            live = slots >= 0
            blk, row = slots[live] // B, slots[live] % B
            c[blk, :, row] = codes[live][..., 0::2] | (codes[live][..., 1::2] << 4)
            s[blk, :, row // 4, :, row % 4] = s16[live]
            w = np.concatenate((c.reshape(self.nb, H, -1), s.reshape(self.nb, H, -1)), -1)
            assert np.array_equal(pool.cpu().numpy().reshape(w.shape), w)

    def check_read(self, slots, k_out, v_out, before):
        """rows of `slots`, rounded once to fp32 and once to 16 bits; others as they were"""
        for out, pool, sc in zip((k_out, v_out), self.pools, self.scales):
            rows = oracle.fp4_dequant(pool.cpu().numpy(), self.D).reshape(-1, self.H, self.D)
            val = rows[np.maximum(slots, 0)].astype(np.float32) * np.float32(sc)
            want = (val.astype(np.float16).view(np.uint16) if self.dtype == W.F16
                    else W.to_bits(val, self.dtype))
            got, ok = bits_of(out), slots >= 0
            assert np.array_equal(got[ok], want[ok]) and np.all(got[~ok] == before)


@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
@pytest.mark.parametrize("H,D,n", SHAPES)
def test_write_and_read_of_many_tokens(cuda_device, H, D, n, dtype):
    r = Rows(1000 + H + n, dtype, H, D, n)
    slots = r.slots.copy()
    slots[r.pad] = -1
    given = slots.copy()
    given[r.far] = [r.nb * r.B, r.nb * r.B + 100, 2 ** 40]
    slots[r.far] = -1
    dev = torch.from_numpy(given).cuda()
    pa.pa_cache_write_fp4(*r.dev(), dev, *r.pools, *r.scales, err=r.err)
    assert pa.pa_get_error(r.err) == pa.PA_DEVERR_SLOT
    r.check_pools(slots)
    outs = [to_dev(np.full((n, H, D), 0x1234, np.uint16), dtype) for _ in range(2)]
    pa.pa_cache_read_fp4(dev, *r.pools, *r.scales, k_out=outs[0], v_out=outs[1], err=r.err)
    assert pa.pa_get_error(r.err) == pa.PA_DEVERR_SLOT
    r.check_read(slots, *outs, 0x1234)


@pytest.mark.parametrize("B", [4, 16, 256])
@pytest.mark.parametrize("H,D,n", SHAPES)
def test_mapped_write_of_many_tokens(cuda_device, H, D, n, B):
    rng = np.random.default_rng(1100 + H + n + B)
    r = Rows(1200 + H + n + B, W.BF16, H, D, n, B)
    lens = np.array([n // 3, n - n // 3 - n // 7, n // 7])
    need = -(-lens // B)
    r.nb = int(need.sum()) + 2
    r.pools = [torch.full(pa.pa_fp4_pool_shape(r.nb, B, H, D), 0x5A, dtype=torch.uint8,
                          device="cuda") for _ in range(2)]
    perm = rng.permutation(r.nb).astype(np.int32)
    bt = np.full((3, int(need.max())), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        bt[i, :m] = perm[at:at + m]
        at += m
    order = rng.permutation(n)
    seq = np.repeat(np.arange(3), lens)[order].astype(np.int32)
    pos = np.concatenate([np.arange(m) for m in lens])[order].astype(np.int32)
    slots = bt[seq, pos // B].astype(np.int64) * B + pos % B

    def write():
        out = torch.full((n,), 7, dtype=torch.int64, device="cuda")
        pa.pa_cache_write_fp4_mapped(*r.dev(), *(torch.from_numpy(t).cuda() for t in (bt, seq, pos)),
                                     *r.pools, *r.scales, slot_mapping=out, err=r.err)
        return out.cpu().numpy()

    seq[r.pad] = -1
    slots[r.pad] = -1
    assert np.array_equal(write(), slots)
    assert pa.pa_get_error(r.err) == 0
    r.check_pools(slots)
    # a sequence beyond the table, then a bad entry: no slot, nothing written, reported
    for p in r.pools:
        p.fill_(0x5A)
    seq[r.far] = [3, -2, 1 << 30]
    slots[r.far] = -1
    assert np.array_equal(write(), slots)
    assert pa.pa_get_error(r.err) == pa.PA_DEVERR_POSITION
    r.check_pools(slots)
    for p in r.pools:
        p.fill_(0x5A)
    bt[1, 0] = r.nb
    slots[(seq == 1) & (pos < B)] = -1
    assert np.array_equal(write(), slots)
    assert pa.pa_get_error(r.err) == pa.PA_DEVERR_POSITION | pa.PA_DEVERR_BLOCK_ID
    r.check_pools(slots)
