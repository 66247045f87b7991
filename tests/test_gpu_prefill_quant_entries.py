"""Table entries that name no block of the pool, whatever their value: their tokens are left out
of the softmax and reported, over both caches and in both kernels of the quantized prefills."""
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from quant_reference import Chunks, assert_within

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
POOLS = pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])
# new tokens and lengths: tiles of 128 rows, and sequences of at most 16 rows (2 heads a KV head)
ROWS = pytest.mark.parametrize("new,lens", [([30, 40, 11], [400, 300, 290]),
                                            ([3, 8, 1], [400, 300, 290])], ids=["many", "few"])


@POOLS
@ROWS
@pytest.mark.parametrize("B", [4, 16, 128])
@pytest.mark.parametrize("entry", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1, None])
def test_entries_of_any_value_are_left_out(four, new, lens, B, entry):
    c = Chunks(41, four, BF16, 4, 2, 64, B, new, lens)
    if entry is None:
        entry = c.k.shape[0]                      # the first that is past the pool
    left = {}
    for i, cols in {0: [0, 399 // B], 1: [140 // B], 2: [0, 1, 288 // B]}.items():
        for b in cols:
            c.bt[i, b] = entry
            left.setdefault(i, set()).update(range(b * B, (b + 1) * B))
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    want, tol = c.reference(left_out=left)
    assert_within(out, want, tol)
    # nothing left of a sequence: zeros
    c.bt[1] = entry
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    assert bool((out[new[0]:new[0] + new[1]] == 0).all())


@POOLS
@ROWS
def test_entries_that_are_not_needed_are_not_looked_at(four, new, lens):
    """Before the window and past the end an entry may hold anything."""
    for entry in (-2, -2 ** 31, 2 ** 31 - 1):
        c = Chunks(42, four, BF16, 4, 2, 64, 16, new, lens, window=50)
        c.bt[c.bt < 0] = entry
        want, tol = c.reference()
        assert_within(c.run(pa), want, tol)
        assert pa.pa_get_error(c.err) == 0
