"""NaN codes around a sliding window's edge, in blocks that the table holds: a row reads none of
the tokens before its own window, whichever other rows of the tile attend to them."""
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from quant_reference import Chunks, assert_within

pytestmark = pytest.mark.gpu

WINDOW = 20


# (heads a KV head, new tokens, length): at most 16 rows; one tile of 128 rows; three
@pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])
@pytest.mark.parametrize("G,L,T", [(2, 8, 160), (4, 20, 180), (4, 90, 250)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("before", [3, 1, 0, -1, -4, -19])
def test_nan_at_the_windows_edge(four, G, L, T, which, before):
    """A NaN `before` tokens ahead of the first row's window (0 and less: inside it)."""
    c = Chunks(71, four, torch.bfloat16, G, 1, 128, 16, [L], [T], window=WINDOW)
    want, tol = c.reference()
    first = T - L - WINDOW + 1
    t = first - before
    b, r = int(c.bt[0, t // 16]), t % 16
    assert b >= 0                                  # read, or read around, not skipped
    pool = getattr(c, which)
    if four:
        pool.view(pool.shape[0], 1, -1)[b, 0, 16 * 64 + (r // 4) * 32 + r % 4] = 0x7F
    else:
        pool[b, r, 0, 3] = 0xFF
    out = c.run(pa)
    p = torch.arange(T - L, T, device="cuda")
    hit = (p >= t) & (p < t + WINDOW)
    assert bool(hit.any()) == (before <= 0)
    assert bool(out[hit].isnan().all())
    assert_within(out[~hit], want[~hit], tol[~hit])
    assert pa.pa_get_error(c.err) == 0
