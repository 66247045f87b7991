"""Scales that the append takes: those of the pool's own write."""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
import workloads as W
from harness import to_dev
from paged_kv_cache_72_gb300 import _lib
from paged_kv_cache_72_gb300.build import build

P = 4096   # a 16-byte aligned address that is never read: every call is empty or refused


@pytest.mark.parametrize("cache,scale,status", [
    # 6 * scale need not be finite for E4M3 codes, whose quotient is x / scale
    (2, 1e38, 0), (2, 3e38, 0), (2, float(np.float32(1e-45)), 0),
    (2, 0.0, 1), (2, -1.0, 1), (2, float("inf"), 1), (2, float("nan"), 1),
    (3, 5e37, 0), (3, 1e38, 1), (3, 0.0, 1), (3, float("nan"), 1),
])
@pytest.mark.parametrize("which", ["k", "v"])
def test_append_scale_range(cache, scale, status, which):
    build()
    ks, vs = (scale, 1.0) if which == "k" else (1.0, scale)
    got = _lib.load().pa_append_rope(P, 1024, P, 256, P, 256, 1, P, 128, 64, 0, None, None, 1e-6, P,
                                     4, 2, P, P, 0, P, P, P, 9, 16, 8, 2, 128, cache, ks, vs, None,
                                     None, None)
    assert got == status


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e38, 3e38])
def test_e4m3_append_at_the_largest_scales(cuda_device, scale):
    rng = np.random.default_rng(3)
    x = (rng.choice([-1, 1], (32, 2, 64)) * 2.0 ** rng.uniform(110, 127, (32, 2, 64)))
    dk = to_dev(W.to_bits(x.astype(np.float32), W.BF16), W.BF16)
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None].contiguous()
    pos = torch.arange(32, dtype=torch.int32, device="cuda")
    got, want = ([torch.zeros((2, 16, 2, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
                 for _ in range(2))
    pa.pa_append_rope(None, dk, dk, None, table, torch.zeros_like(pos), pos, *got, k_scale=scale,
                      v_scale=scale)
    pa.pa_cache_write_fp8(dk, dk, torch.arange(32, device="cuda"), *want, scale, scale)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and (a & 0x7F).any()
