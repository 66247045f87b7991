"""The longest context an int32 length can say, 2^31 - 1 tokens, over both caches and in both
kernels of the quantized prefills: a table of 2^23 entries on two blocks of the pool."""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa

pytestmark = pytest.mark.gpu

B, D, T = 256, 64, 2 ** 31 - 1
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def constant_pools(four, seed):
    """Two blocks, one KV head: keys zero, every row's values the same vector of E2M1 values.
    Every attended mean is that vector.  The row behind the last token, the last block's last
    one, is NaN in K and V."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 8, D).astype(np.uint8)
    sign = rng.integers(0, 2, D).astype(np.uint8)
    row = E2M1[code] * (1.0 - 2.0 * sign)
    if four:
        x = code | sign << 3
        v = np.zeros((2, 1, B * 9 * D // 16), np.uint8)
        v[..., :B * D // 2] = np.tile(x[0::2] | (x[1::2] << 4), B)
        v[..., B * D // 2:] = 0x38               # E4M3 one
        k = np.zeros_like(v)
        k[..., B * D // 2:] = 0x38
        for p in (k, v):
            p[1, 0, B * D // 2:].reshape(B // 4, D // 16, 4)[-1, :, 3] = 0x7F
        k, v = (p.reshape(2, 1, B, 9 * D // 16) for p in (k, v))
    else:
        x = torch.from_numpy(row.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
        v = np.tile(x.numpy(), (2, B, 1, 1))
        k = np.zeros_like(v)
        for p in (k, v):
            p[1, B - 1] = 0x7F
    return row, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()


# at most 16 rows and more, 4 heads a KV head; 70 tokens are two pairs of tiles
@pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])
@pytest.mark.parametrize("L,window", [(1, 0), (4, 0), (5, 0), (1, 1), (4, 40), (5, 40), (70, 1),
                                      (70, 300), (70, 2 ** 31 - 1)])
def test_longest_context(four, L, window):
    row, k, v = constant_pools(four, 61)
    bt = torch.zeros((1, 2 ** 23), dtype=torch.int32, device="cuda")
    bt[0, -1] = 1
    q = torch.randn(L, 4, D, device="cuda").bfloat16()
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = pa.pa_prefill_fp4 if four else pa.pa_prefill_fp8
    out = call(q, k, v, bt, lens, start, 1.0, 1.0, 1.0, window=window, err=err)
    assert pa.pa_get_error(err) == 0
    # Weights are equal, 2^7 each, and their sums, 2^13 a stage, exact.  A value's sum in a block
    # is one of N equal products; the tensor cores cut a product at 2^-25 of the power of two of
    # the sum that it joins.  A power of two stays whole up to N = 2^25; 1.5 * 2^j, whose last bit
    # is 2^(j-1), while the sum is below 2^(j+25), that is for N0 = 2^25 / 1.5 products, and
    # counts 2/3 from there to 2 N0.  A block has T / sms tokens, with two pairs of tiles (L = 70
    # without a window that cuts) twice that for the first pair's rows: the joined mean keeps
    # (N0 + 2/3 (N - N0)) / N of such a value.  Joins leave relative errors below 2^-12, and the
    # values need 2 of 8 bits, so that what is exact before the rounding is exact behind it.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N, N0 = (2 if L == 70 and window > 300 else 1) * (T + 384) / sms, 2 ** 25 / 1.5
    lost = max(0.0, (N - N0) / (3 * N))
    got, want = out.double().cpu(), torch.from_numpy(row).expand(L, 4, D)
    whole = torch.from_numpy(np.isin(np.abs(row), (0, .5, 1, 2, 4))).expand(L, 4, D)
    assert N < 2 ** 25 and torch.equal(got[whole], want[whole])
    if lost == 0.0:
        assert torch.equal(got, want)
    else:
        assert bool(((got - want).abs() <= want.abs() * (lost + 2.0 ** -8)).all())
