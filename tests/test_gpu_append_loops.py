"""The append where a warp takes several passes of a token's rows: more tokens than
a step has, few shares of a token's rows, remainders in the passes, in the batches
of query rows and in the key and value rows.

The launch splits a token's rows between warps only until there are six warps an SM
(or 32, beyond 20 passes a warp), so about a thousand tokens leave a warp all of a
token's rows, or half of them.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
import test_gpu_append as one_pass
import workloads as W
from harness import bits_of
from test_gpu_append import Step, _same_pools

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, Hq, H, D, B, past, new
    (W.BF16, 32, 8, 128, 16, [0, 500], [401, 600]),         # 16 and 4 passes
    (W.F16, 14, 2, 64, 8, [3, 0, 77], [500, 500, 3]),       # 4 and 1, with remainders
    (W.BF16, 7, 5, 128, 4, [0, 9], [950, 41]),              # 4 and 3, odd
    (W.F16, 33, 11, 128, 32, [100], [1001]),                # two shares: 9 and 3
    (W.BF16, 33, 11, 64, 16, [0, 64], [903, 100]),           # 9 and 3 of four rows
    (W.F16, 64, 8, 128, 16, [10, 0], [100, 200]),           # four shares: 8 and 1
    (W.BF16, 12, 12, 64, 16, [31], [1200]),                 # no grouped heads: 3 and 3
    (W.F16, 4, 32, 128, 128, [0], [930]),                   # more key than query rows
]


@pytest.mark.parametrize("kind", one_pass.KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_loops_are_bit_exact_without_norms(cuda_device, monkeypatch, shape, interleaved,
                                                  kind):
    monkeypatch.setattr(one_pass, "SHAPES", SHAPES)
    one_pass.test_append_is_bit_exact_without_norms(cuda_device, shape, interleaved, kind)


@pytest.mark.parametrize("norm", ["q", "k", "qk"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_loops_with_norms(cuda_device, monkeypatch, shape, norm):
    monkeypatch.setattr(one_pass, "SHAPES", SHAPES)
    one_pass.test_append_norms(cuda_device, shape, norm)


@pytest.mark.parametrize("norm", ["", "qk"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_loops_in_place(cuda_device, shape, norm):
    # q_out may be q itself: a warp stores rows before it loads later ones
    dtype, Hq, H, D, B, past, new = SHAPES[shape]
    args = (700 + shape, dtype, Hq, H, D, B, past, new, "16", D, norm)
    want = Step(*args).call(bool(shape % 2))
    st = Step(*args)
    width = (Hq + 2 * H) * D
    st.dx = st.dx[:, :width].contiguous()
    q = st.rows("q", st.dx).contiguous()
    kw = {n + "_norm": torch.from_numpy(w.view(np.int16)).cuda().view(q.dtype)
          for n, w in (("q", st.qn), ("k", st.kn)) if n in norm}
    cs, bt, seq, pos = (torch.from_numpy(t).cuda() for t in (st.cs, st.bt, st.seq, st.pos))
    out = pa.pa_append_rope(q, st.rows("k", st.dx), st.rows("v", st.dx), cs, bt, seq, pos,
                            st.k_cache, st.v_cache, interleaved=bool(shape % 2), eps=1e-5,
                            q_out=q, err=st.err, **kw)
    assert out is q and np.array_equal(bits_of(q), bits_of(want))
    assert pa.pa_get_error(st.err) == 0


@pytest.mark.parametrize("kind", one_pass.KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_loops_without_queries_and_with_padding(cuda_device, shape, kind):
    dtype, _, H, D, B, past, new = SHAPES[shape]
    n = sum(new)
    st = Step(800 + shape, dtype, 0, H, D, B, past, new, kind, D // 2, pad=(0, 1, 17, n - 1))
    slots = torch.full((n,), 7, dtype=torch.int64, device="cuda")
    assert st.call(slot_mapping=slots) is None
    assert np.array_equal(slots.cpu().numpy(), st.slots())
    _same_pools(st, st.stored(st.rotated("k", False), st.rows("v")))
    assert pa.pa_get_error(st.err) == 0
