"""Lengths that change while the 4-bit decode reads them are a caller's error: the
results of that call mean nothing, but every access stays inside the buffers, the
call ends, and with a zeroed workspace the next one is right.

Guarded places, each reached when a thread reads a length that its block's count did
not hold: the walk past the last sequence (loads and products), and the count and
join of contexts cut between blocks, whose block numbers come from those lengths.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
import workloads as W
from test_gpu_fp4 import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flags", [pa.PA_DECODE_AUTO, pa.PA_DECODE_TABLES_READY])
def test_lengths_that_change_during_the_call(cuda_device, flags):
    rng = np.random.default_rng(5)
    n, most = 400, 1500
    st = State(640, W.BF16, 8, 2, 64, 16, [most] * 3 + [1] * (n - 3))
    d = st.dev
    # every entry of every row is a block of the pool
    d["bt"] = torch.from_numpy(rng.integers(0, len(st.k), st.bt.shape).astype(np.int32)).cuda()
    variants = [torch.from_numpy(rng.integers(0, hi + 1, n).astype(np.int32)).cuda()
                for hi in (0, 3, 40, 200, most, most)]
    size = pa.pa_decode_workspace_size(8, 2, 64, 16, pa.PA_FP4_E2M1)
    ws = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    ws[size:] = 0x5A
    out = torch.full((n + 8, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lens = variants[3].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(150):
        with torch.cuda.stream(b):
            for j in range(6):
                lens.copy_(variants[(i * 5 + j) % len(variants)])
        with torch.cuda.stream(a):
            pa.pa_decode_fp4(d["q"], d["k"], d["v"], d["bt"], lens, st.scale, st.k_scale, st.v_scale,
                             out=out[:n], workspace=ws[:size], flags=flags, err=err)
    torch.cuda.synchronize()
    assert pa.pa_get_error(err) in (0, pa.PA_DEVERR_SEQ_LEN)
    # nothing behind the workspace and the output
    assert bool((ws[size:] == 0x5A).all()) and bool((out[n:] == 3.0).all())
    ws[:size].zero_()
    for lens in variants:
        first = pa.pa_decode_fp4(d["q"], d["k"], d["v"], d["bt"], lens, st.scale, st.k_scale,
                                 st.v_scale, workspace=ws[:size], err=err)
        alone = pa.pa_decode_fp4(d["q"], d["k"], d["v"], d["bt"], lens, st.scale, st.k_scale,
                                 st.v_scale, err=err)
        # (NaN scales of the pool's unused rows are among what is read)
        assert torch.equal(first.view(torch.int16), alone.view(torch.int16))
    assert pa.pa_get_error(err) == 0
