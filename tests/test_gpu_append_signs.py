"""What the append stores into a quantized pool is, byte for byte, what the pool's
own write stores of the same 16-bit rows: signs of zeros and of values that round
to zero among them."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_72_gb300 as pa
import workloads as W
from harness import bits_to_f64, to_dev

pytestmark = pytest.mark.gpu

SCALES = (1.0, 0.0371, 2.0 ** -20, 1.5e-30, 3e-37, 7.7e8, 2e30, 5e37)


def _every_value(dtype):
    """Every finite 16-bit pattern, [256, 4, 128]: in groups of any neighbours,
    then in groups of like magnitudes."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    with np.errstate(invalid="ignore"):
        bits[~np.isfinite(bits_to_f64(bits, dtype))] = 0x8000     # a negative zero
    near = bits[np.argsort(np.abs(bits_to_f64(bits, dtype)), kind="stable")]
    return np.concatenate((np.random.default_rng(9).permutation(bits), near)).reshape(256, 4, 128)


def _place(n):
    zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None].contiguous()
    return table, zeros, pos


@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
def test_e4m3_bytes_are_the_plain_writes(cuda_device, dtype):
    k = _every_value(dtype)
    n, dk = len(k), to_dev(k, dtype)
    slots = torch.arange(n, device="cuda")
    for scale in SCALES:
        got, want = ([torch.full((n // 16, 16, 4, 128), 0x55, dtype=torch.uint8, device="cuda")
                      for _ in range(2)] for _ in range(2))
        pa.pa_append_rope(None, dk, dk, None, *_place(n), *got, k_scale=scale, v_scale=0.3)
        pa.pa_cache_write_fp8(dk, dk, slots, *want, scale, 0.3)
        for a, b in zip(got, want):
            assert torch.equal(a, b), scale


@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
@pytest.mark.parametrize("way", ["append", "write", "write, few rows"])
def test_e2m1_bytes_are_the_oracles(cuda_device, dtype, way):
    k = _every_value(dtype)
    if way == "write, few rows":
        k = k.reshape(512, 2, 128)
    n, H = k.shape[:2]
    dk = to_dev(k, dtype)
    x = bits_to_f64(k, dtype).astype(np.float32)
    for scale in SCALES:
        pools = [torch.zeros(pa.pa_fp4_pool_shape(n // 16, 16, H, 128), dtype=torch.uint8,
                             device="cuda") for _ in range(2)]
        if way == "append":
            pa.pa_append_rope(None, dk, dk, None, *_place(n), *pools, k_scale=scale, v_scale=0.3)
        else:
            pa.pa_cache_write_fp4(dk, dk, torch.arange(n, device="cuda"), *pools, scale, 0.3)
        want = [np.zeros(pools[0].shape, np.uint8) for _ in range(2)]
        oracle.cache_write_fp4(want[0], want[1], x, x, np.arange(n), scale, 0.3)
        for got, w in zip(pools, want):
            assert np.array_equal(got.cpu().numpy(), w), scale
