"""Chunks of new tokens over E4M3 and 4-bit paged caches against the formula in 64 bits
(quant_reference.py, which derives the bound)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from quant_reference import Chunks, assert_within

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
POOLS = pytest.mark.parametrize("four", [False, True], ids=["e4m3", "4bit"])


def check(c, **kw):
    out = c.run(pa, **kw)
    want, tol = c.reference()
    rows = int(c.start[-1])
    assert_within(out[:rows], want[:rows], tol[:rows])
    assert pa.pa_get_error(c.err) == 0
    return out


@POOLS
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(4, 4), (8, 2), (7, 1), (9, 3), (16, 1), (12, 1)])
def test_head_layouts(four, dtype, D, Hq, H):
    check(Chunks(1, four, dtype, Hq, H, D, 16, [5, 70, 1, 33], [5, 131, 64, 200]))


@POOLS
@pytest.mark.parametrize("B", [4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_block_sizes(four, B, D):
    check(Chunks(2, four, BF16, 8, 2, D, B, [1, min(40, 3 * B - 1), 3], [B + 1, 3 * B - 1, 259]))


@POOLS
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 66, 127, 128, 129, 191, 193])
def test_lengths(four, T):
    """Every kind of length as one new token, as a fresh prompt and in between."""
    new = sorted({1, (T + 1) // 2, T})
    check(Chunks(3, four, F16, 8, 2, 128, 4, new, [T] * len(new)))


@POOLS
@pytest.mark.parametrize("L", [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 66, 97, 129, 130])
def test_chunk_lengths(four, L):
    """Row tiles of one and two kinds, their last one full or not (32 tokens a tile here)."""
    check(Chunks(4, four, BF16, 4, 1, 64, 16, [L], [L + 77]))


@POOLS
@pytest.mark.parametrize("window", [1, 2, 5, 63, 64, 65, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,D", [(F16, 64), (BF16, 128)], ids=["fp16", "bf16"])
def test_windows(four, window, dtype, D):
    check(Chunks(5, four, dtype, 8, 2, D, 8, [1, 3, 90, 201], [300, 131, 90, 450], window=window))


@POOLS
def test_sequences_without_tokens(four):
    """No new tokens, no tokens at all, in any place."""
    check(Chunks(6, four, BF16, 8, 2, 128, 16, [0, 3, 0, 0, 1, 50, 0], [9, 30, 0, 77, 1, 50, 0]))
    c = Chunks(6, four, BF16, 8, 2, 128, 16, [0, 0], [9, 0], tail_rows=4)
    out = torch.full_like(c.q, 3.0)
    c.run(pa, out=out)
    assert bool((out == 3.0).all())


@POOLS
@pytest.mark.parametrize("n", [1, 513, 1200])
def test_many_sequences(four, n):
    rng = np.random.default_rng(n)
    new = rng.integers(0, 3, size=n)
    lens = new + rng.integers(0, 20, size=n)
    check(Chunks(7, four, F16, 2, 1, 64, 4, new, lens))


@POOLS
@pytest.mark.parametrize("L,T", [(1, 20001), (3, 20000), (40, 9000), (130, 5000)])
@pytest.mark.parametrize("G", [1, 8])
def test_long_contexts(four, L, T, G):
    """Contexts that are cut between thread blocks."""
    check(Chunks(8, four, BF16, G, 1, 128, 16, [L], [T]))


@POOLS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [3, 70])
def test_many_stages_a_block(four, D, L):
    """Many stages in every thread block, tiles that take them in turn or together, the same
    result every time."""
    rng = np.random.default_rng(L)
    n = 8
    c = Chunks(24, four, BF16, 8, 8, D, 16, [L, 1] * (n // 2), rng.integers(8000, 12000, size=n))
    out = check(c)
    ws = torch.zeros(pa.pa_prefill_quant_workspace_size(8, 8, D), dtype=torch.uint8,
                     device="cuda")
    for _ in range(10):
        assert torch.equal(c.run(pa, workspace=ws), out)
    assert pa.pa_get_error(c.err) == 0


@POOLS
def test_ragged_long_and_short(four):
    rng = np.random.default_rng(9)
    lens = np.concatenate([rng.integers(1, 90, size=40), [6000, 3000, 1, 2]])
    new = np.minimum(lens, rng.integers(0, 80, size=44))
    new[40:42] = [70, 1]
    check(Chunks(9, four, F16, 8, 2, 64, 16, new, lens))


@POOLS
@pytest.mark.parametrize("sigma,q_sigma", [(1e-2, 1e-2), (30.0, 1.0), (4.0, 12.0)])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_score_ranges(four, sigma, q_sigma, dtype):
    """Flat and peaked weights; the reference of the exponentials moves often."""
    check(Chunks(10, four, dtype, 4, 1, 128, 16, [50, 1], [700, 500], sigma=sigma,
                 q_sigma=q_sigma, scales=(0.3 * sigma, 0.02 * sigma)))


@POOLS
@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_other_scales(four, scale):
    c = Chunks(11, four, F16, 4, 2, 64, 16, [40, 2], [200, 100])
    out = c.run(pa, scale=scale)
    want, tol = c.reference(scale=scale)
    assert_within(out, want, tol)


def test_wide_bfloat16_queries():
    """Rows whose magnitudes lie far outside binary16's range."""
    for power in (-60, -30, 20, 60):
        c = Chunks(12, True, BF16, 4, 1, 128, 16, [9, 1], [100, 70])
        c.q = (c.q.double() * 2.0 ** power).to(BF16)
        scale = c.scale * 2.0 ** -power
        out = c.run(pa, scale=scale)
        want, tol = c.reference(scale=scale)
        assert_within(out, want, tol)


@POOLS
def test_rows_rising_over_the_context(four):
    """Scores that grow with the position: every stage moves the reference."""
    c = Chunks(13, four, BF16, 4, 1, 128, 16, [33], [600])
    c.q[:] = 1.0
    t = torch.arange(608, device="cuda")
    if four:    # codes 1, scales rising in steps of the format
        flat = c.k.view(c.k.shape[0], 1, -1)
        rows = c.bt[0].long()
        flat[rows, :, :16 * 64] = 0x22
        s = (8 + t * 100 // 608).to(torch.uint8).view(38, 4, 1, 4).expand(38, 4, 8, 4)
        flat[rows, 0, 16 * 64:] = s.reshape(38, -1)
    else:
        c.k[c.bt[0].long()] = (8 + t * 100 // 608).to(torch.uint8).view(38, 16, 1, 1)
    check(c)


@POOLS
@pytest.mark.parametrize("B", [4, 16, 128])
def test_bad_table_entries_are_left_out(four, B):
    c = Chunks(14, four, BF16, 8, 2, 64, B, [30, 2, 3 * B + 1], [400, 300, 4 * B])
    nb = c.k.shape[0]
    bad = {0: [1, 300 // B], 1: [0], 2: [3]}
    left = {}
    for i, cols in bad.items():
        for n, b in enumerate(cols):
            c.bt[i, b] = -5 if (i + n) % 2 else nb
            left.setdefault(i, set()).update(range(b * B, (b + 1) * B))
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    want, tol = c.reference(left_out=left)
    assert_within(out, want, tol)
    # nothing left: zeros
    c.bt[1] = -1
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    assert bool((out[30:32] == 0).all())
    left[1] = set(range(300))
    want, tol = c.reference(left_out=left)
    assert_within(out, want, tol)


@POOLS
def test_bad_lengths(four):
    """Their rows get zeros, the others are not touched by them."""
    c = Chunks(15, four, F16, 4, 2, 128, 16, [3, 4, 5, 2], [50, 60, 70, 10], tail_rows=3)
    want, tol = c.reference()
    for value in (-1, 3, 16 * c.bt.shape[1] + 1, 2 ** 31 - 1):
        lens = c.lens.clone()
        lens[1] = value                                # 4 new tokens
        out = torch.full_like(c.q, 7.0)
        c.run(pa, lens=lens, out=out)
        assert pa.pa_get_error(c.err) == pa.PA_DEVERR_SEQ_LEN
        assert bool((out[3:7] == 0).all()) and bool((out[14:] == 7.0).all())
        keep = [0, 1, 2] + list(range(7, 14))
        assert_within(out[keep], want[keep], tol[keep])
    for start in ([0, 3, 7, 12, 18], [-2, 3, 7, 12, 14]):       # past q, before it
        out = torch.full_like(c.q, 7.0)
        c.run(pa, start=torch.tensor(start, dtype=torch.int32, device="cuda"), out=out)
        assert pa.pa_get_error(c.err) == pa.PA_DEVERR_SEQ_LEN
        assert_within(out[3:12], want[3:12], tol[3:12])


@POOLS
@pytest.mark.parametrize("G", [1, 4])
def test_nan_reaches_its_readers_alone(four, G):
    """A NaN value row makes the rows that attend to it NaN, and no others; a NaN key its own
    weight's rows; neither reaches rows before it or past the window."""
    for window in (0, 40):
        for which in ("v", "k"):
            c = Chunks(16, four, BF16, G, 1, 128, 16, [100], [180], window=window)
            want, tol = c.reference()
            t = 130                                   # attended by positions 130 ..
            b, r = int(c.bt[0, t // 16]), t % 16
            pool = getattr(c, which)
            if four:
                pool.view(pool.shape[0], 1, -1)[b, 0, 16 * 64 + (r // 4) * 32 + r % 4] = 0x7F
            else:
                pool[b, r, 0, 3] = 0xFF
            out = c.run(pa)
            p = torch.arange(80, 180, device="cuda")
            hit = (p >= t) & (p < t + window if window else p >= 0)
            assert bool(out[hit].isnan().all())
            assert_within(out[~hit], want[~hit], tol[~hit])


@POOLS
def test_placement_and_repetition_change_nothing(four):
    c = Chunks(17, four, BF16, 8, 2, 128, 16, [70, 1, 5], [900, 5000, 40])
    one = c.run(pa)
    ws = torch.zeros(pa.pa_prefill_quant_workspace_size(8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    for _ in range(3):
        assert torch.equal(c.run(pa, workspace=ws), one)
    perm = torch.randperm(c.k.shape[0], device="cuda")
    k, v = torch.empty_like(c.k), torch.empty_like(c.v)
    k[perm], v[perm] = c.k, c.v
    bt = torch.where(c.bt >= 0, perm[c.bt.clamp(min=0).long()].int(), c.bt)
    c.k, c.v = k, v
    assert torch.equal(c.run(pa, workspace=ws, bt=bt), one)
    assert int(ws[:pa.PA_PREFILL_QUANT_COUNTERS].max()) == 0


def test_one_workspace_for_calls_of_any_shape():
    ws = None
    for seed, (four, Hq, H, D) in enumerate([(True, 8, 2, 128), (False, 4, 4, 64),
                                             (True, 16, 1, 64), (False, 32, 8, 128)]):
        c = Chunks(30 + seed, four, BF16, Hq, H, D, 16, [2, 40], [3000, 100])
        if ws is None:
            ws = torch.zeros(max(pa.pa_prefill_quant_workspace_size(8, 2, d) for d in (64, 128)),
                             dtype=torch.uint8, device="cuda")
        check(c, workspace=ws)


@POOLS
def test_captured_and_replayed(four):
    """A captured call reads what its inputs hold at the replay."""
    c = Chunks(18, four, F16, 8, 2, 64, 16, [33, 1, 1], [400, 3000, 9])
    ws = torch.zeros(pa.pa_prefill_quant_workspace_size(8, 2, 64), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros_like(c.q)
    c.run(pa, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(pa, out=out, workspace=ws)
        c.run(pa, out=out, workspace=ws)
    for step in range(3):
        c.q.copy_(torch.randn_like(c.q))
        c.lens.copy_(torch.tensor([400 - step, 3000 - 700 * step, 9 - step], dtype=torch.int32))
        out.zero_()
        graph.replay()
        want, tol = c.reference()
        assert_within(out, want, tol)
    assert pa.pa_get_error(c.err) == 0


# Sequences of few rows (tokens times heads of a KV head), alone and beside others: they have
# a kernel of their own.

@POOLS
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (8, 2), (7, 1), (16, 1), (24, 3)])
def test_few_rows(four, dtype, D, Hq, H):
    G = Hq // H
    most = 16 // G
    lens = [1, 2, 31, 32, 33, 95, 128, 700, 2500]
    new = [min(T, 1 + i % most) for i, T in enumerate(lens)]
    check(Chunks(31, four, dtype, Hq, H, D, 16, new, lens))
    check(Chunks(32, four, dtype, Hq, H, D, 16, [most], [1000]))
    check(Chunks(33, four, dtype, Hq, H, D, 16, [0, 1, most + 1, 0, most, 40], [0, 77, 300, 5, 90, 70]))


@POOLS
@pytest.mark.parametrize("B", [4, 8, 32, 64, 256])
@pytest.mark.parametrize("window", [0, 1, 31, 33, 500])
def test_few_rows_blocks_and_windows(four, B, window):
    check(Chunks(34, four, BF16, 4, 2, 128, B, [1, 3, 8, 2, 1], [600, 3, 41, 1300, 32],
                 window=window))


@POOLS
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_of_many_sequences(four, D):
    rng = np.random.default_rng(35)
    lens = rng.integers(1, 200, 700)
    new = np.minimum(rng.integers(0, 5, 700), lens)
    check(Chunks(35, four, F16, 4, 2, D, 16, new, lens))


@POOLS
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("t", [70, 150, 155])
def test_few_rows_nan_reaches_its_readers_alone(four, window, which, t):
    c = Chunks(36, four, BF16, 2, 1, 128, 16, [8], [160], window=window)
    want, tol = c.reference()
    b, r = int(c.bt[0, t // 16]), t % 16
    if b < 0:
        return                                        # before every row's window
    pool = getattr(c, which)
    if four:
        pool.view(pool.shape[0], 1, -1)[b, 0, 16 * 64 + (r // 4) * 32 + r % 4] = 0x7F
    else:
        pool[b, r, 0, 3] = 0xFF
    out = c.run(pa)
    p = torch.arange(152, 160, device="cuda")
    hit = (p >= t) & (p < t + window if window else p >= 0)
    assert bool(out[hit].isnan().all())
    assert_within(out[~hit], want[~hit], tol[~hit])
    assert pa.pa_get_error(c.err) == 0


@POOLS
@pytest.mark.parametrize("B", [4, 16, 128])
def test_few_rows_bad_table_entries_are_left_out(four, B):
    c = Chunks(37, four, BF16, 4, 2, 64, B, [3, 2], [400, 300])
    nb = c.k.shape[0]
    left = {}
    for i, cols in {0: [1, 399 // B], 1: [0, 150 // B]}.items():
        for n, b in enumerate(cols):
            c.bt[i, b] = -5 if (i + n) % 2 else nb
            left.setdefault(i, set()).update(range(b * B, (b + 1) * B))
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    want, tol = c.reference(left_out=left)
    assert_within(out, want, tol)
    c.bt[1] = -1
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_BLOCK_ID
    assert bool((out[3:5] == 0).all())


@POOLS
def test_few_rows_bad_lengths(four):
    """One sequence that contradicts itself: its rows cleared, the others unharmed."""
    c = Chunks(38, four, F16, 4, 4, 64, 16, [2, 1, 3], [40, 50, 60])
    want, tol = c.reference()
    c.lens[1] = -7
    out = c.run(pa)
    assert pa.pa_get_error(c.err) == pa.PA_DEVERR_SEQ_LEN
    assert bool((out[2] == 0).all())
    keep = [0, 1, 3, 4, 5]
    assert_within(out[keep], want[keep], tol[keep])


@POOLS
def test_many_calls(four):
    """Thousands of calls, in bursts: none gives up a wait, all give the same bits."""
    chunks = [Chunks(21 + k, four, dt, 8, 2, D, 16, [33, 1, 1], [400, 3000, 9])
              for k, (D, dt) in enumerate([(64, F16), (128, BF16)])]
    ws = torch.zeros(pa.pa_prefill_quant_workspace_size(8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    wants = [c.run(pa, workspace=ws).clone() for c in chunks]
    outs = [torch.empty_like(c.q) for c in chunks]
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for step in range(1000):
        for c, out, want in zip(chunks, outs, wants):
            for _ in range(3):
                c.run(pa, out=out, workspace=ws)
            differ += (out != want).sum()
        if step % 50 == 0:
            torch.cuda.synchronize()
    assert int(differ) == 0
    for c in chunks:
        assert pa.pa_get_error(c.err) == 0


def test_two_streams():
    """Two calls at once, each with a workspace of its own."""
    cs = [Chunks(19 + i, bool(i), BF16, 8, 2, 128, 16, [40, 1], [700, 4000]) for i in range(2)]
    refs = [c.reference() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    n = pa.pa_prefill_quant_workspace_size(8, 2, 128)
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in cs]
    outs = [torch.zeros_like(c.q) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, w, o in zip(cs, streams, ws, outs):
            with torch.cuda.stream(s):
                c.run(pa, workspace=w, out=o)
    torch.cuda.synchronize()
    for o, (want, tol) in zip(outs, refs):
        assert_within(o, want, tol)


@POOLS
def test_single_tokens_are_the_decode(four):
    """One new token a sequence: within both bounds of pa_decode_fp8 / pa_decode_fp4."""
    c = Chunks(21, four, F16, 8, 2, 128, 16, [1] * 6, [1, 17, 64, 100, 700, 33])
    out = c.run(pa)
    if four:
        dec = pa.pa_decode_fp4(c.q, c.k, c.v, c.bt, c.lens, c.scale, c.k_scale, c.v_scale)
    else:
        dec = pa.pa_decode_fp8(c.q, c.k, c.v, c.bt, c.lens, c.scale, c.k_scale, c.v_scale)
    want, tol = c.reference()
    assert_within(out, want, tol)
    assert_within(dec, want, 2 * tol)


@POOLS
def test_chunks_add_up_to_the_prompt(four):
    """A prompt in chunks gives what it gives at once, up to both bounds."""
    c = Chunks(22, four, BF16, 4, 2, 64, 16, [150], [150])
    whole = c.run(pa)
    want, tol = c.reference()
    assert_within(whole, want, tol)
    at = 0
    for n in (1, 64, 20, 65):
        part = c.run(pa, q=c.q[at:at + n],
                     start=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                     lens=torch.tensor([at + n], dtype=torch.int32, device="cuda"))
        assert_within(part, want[at:at + n], tol[at:at + n])
        at += n


def test_large_offsets():
    """A pool of more than 2^31 bytes: blocks at its end."""
    H, D, B = 8, 128, 16
    nb = (2 ** 32) // (B * H * D) + 40
    c = Chunks(23, False, BF16, 8, 8, D, B, [20, 1], [100, 260])
    k = torch.full((nb, B, H, D), 0x7F, dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, 0x7F)
    small = c.k.shape[0]
    k[nb - small:], v[nb - small:] = c.k, c.v
    want, tol = c.reference()
    c.k, c.v = k, v
    out = c.run(pa, bt=torch.where(c.bt >= 0, c.bt + (nb - small), c.bt))
    assert_within(out, want, tol)
