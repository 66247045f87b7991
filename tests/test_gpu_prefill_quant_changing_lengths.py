"""Lengths that change while a quantized prefill reads them are a caller's error: the results of
that call mean nothing, but every access stays inside the buffers, the block's threads stay
together, the call ends, and with zeroed counters the next one is right.

A block takes a sequence's words once: the kernel of few rows by one thread that walks for all,
the other by one lane of the warp that walks.  What a thread computes from other reads of the
lengths (the line's cuts) only says where a block begins and ends.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from quant_reference import Chunks, assert_within

pytestmark = pytest.mark.gpu

POOLS = pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])


def splits(rng, n, rows):
    """Row ranges of n sequences: some empty, some of many rows, `rows` in all."""
    cut = np.sort(rng.integers(0, rows + 1, n - 1))
    return np.concatenate([[0], cut, [rows]]).astype(np.int32)


# sequences, new tokens in all, longest context: both kernels (4 heads a KV head), the one with
# tiles of 128 rows alone, the one of few rows alone
@POOLS
@pytest.mark.parametrize("n,rows,most", [(300, 1500, 1500), (5, 700, 4000), (3, 4, 6000)],
                         ids=["both", "tiles", "few"])
def test_lengths_that_change_during_the_call(four, n, rows, most):
    rng = np.random.default_rng(n)
    Hq, H, D, B = 8, 2, 64, 16
    base = Chunks(51, four, torch.bfloat16, Hq, H, D, B, [rows], [max(rows, 400)])
    nb = base.k.shape[0]
    width = -(-most // B)
    # every entry of every row is a block of the pool that holds values
    used = base.bt[0].cpu().numpy()
    used = used[used >= 0][:max(rows, 400) // B]
    bt = torch.from_numpy(rng.choice(used, (n, width)).astype(np.int32)).cuda()
    assert int(bt.max()) < nb
    cases = []
    for hi in (0, 3, 40, 200, most, most):
        start = splits(rng, n, rows) if hi else np.zeros(n + 1, np.int32)
        new = np.diff(start)
        lens = np.minimum(new + rng.integers(0, hi + 1, n), most).astype(np.int32)
        cases.append((torch.from_numpy(lens).cuda(), torch.from_numpy(start).cuda()))
    size = pa.pa_prefill_quant_workspace_size(Hq, H, D)
    ws = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    ws[size:] = 0x5A
    out = torch.full((rows + 8, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lens, start = (x.clone() for x in cases[3])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(150):
        with torch.cuda.stream(b):
            for j in range(6):
                k = (i * 5 + j) % len(cases)
                lens.copy_(cases[k][0])
                start.copy_(cases[(k + (j == 2)) % len(cases)][1])
        with torch.cuda.stream(a):
            base.run(pa, bt=bt, lens=lens, start=start, out=out[:rows], workspace=ws[:size])
        if i % 25 == 24:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert pa.pa_get_error(base.err) in (0, pa.PA_DEVERR_SEQ_LEN)
    # nothing behind the workspace and the output
    assert bool((ws[size:] == 0x5A).all()) and bool((out[rows:] == 3.0).all())
    ws[:pa.PA_PREFILL_QUANT_COUNTERS].zero_()
    for lens, start in cases:
        first = base.run(pa, bt=bt, lens=lens, start=start, workspace=ws[:size])
        alone = base.run(pa, bt=bt, lens=lens, start=start)
        assert torch.equal(first, alone) and not bool(first.isnan().any())
    assert pa.pa_get_error(base.err) == 0
    want, tol = base.reference()
    assert_within(base.run(pa, workspace=ws[:size]), want, tol)
