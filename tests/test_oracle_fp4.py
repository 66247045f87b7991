"""The 4-bit cache's oracle against values worked by hand, and its layout
against the byte offsets that include/pa.h states."""
import numpy as np

import oracle


def test_e2m1_codes_and_ties():
    # the eight magnitudes, then every midpoint: ties go to the even code
    assert oracle.e2m1_encode(oracle._E2M1).tolist() == list(range(8))
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert oracle.e2m1_encode(mids).tolist() == [0, 2, 2, 4, 4, 6, 6]
    # just past the midpoints
    assert oracle.e2m1_encode(np.array(mids) * (1 + 2.0 ** -20)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert oracle.e2m1_encode(np.array(mids) * (1 - 2.0 ** -20)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert oracle.e2m1_encode([7.0, 1e9, -6.5, -0.5]).tolist() == [7, 7, 15, 9]
    assert oracle.e2m1_encode([1e30, -3e38, np.inf, -np.inf]).tolist() == [7, 15, 7, 15]
    assert np.array_equal(oracle.e2m1_decode(range(16))[8:], -oracle._E2M1)


def test_quantize_worked_example():
    # one group: max 3, scale 1/2: 3 / (6 * .5) = 1 -> s16 = 1 (E4M3 0x38); d = .5,
    # so the values are codes of x / .5
    x = np.zeros(32, np.float32)
    x[:6] = [3.0, -1.5, 0.25, 0.126, -0.124, 1.0]
    codes, s16 = oracle.fp4_quantize(x, 0.5)
    assert s16.tolist() == [0x38, 0]
    assert codes[:6].tolist() == [7, 8 | 5, 1, 1, 8, 4]
    assert not codes[16:].any()
    # a group whose scale rounds to zero in E4M3 stores zeros
    codes, s16 = oracle.fp4_quantize(np.full(16, 6 * 2.0 ** -11, np.float32), 1.0)
    assert s16.tolist() == [0] and not codes.any()


def test_layout_offsets():
    B, H, D = 8, 2, 64
    pool = np.zeros((3, H, B, 9 * D // 16), np.uint8)
    codes = np.arange(D, dtype=np.uint8) % 16
    oracle.fp4_put(pool, 2, 5, 1, codes, np.array([1, 2, 3, 4], np.uint8))
    flat = pool.reshape(-1)
    plane = (2 * H + 1) * B * 36
    # the even element in the low nibble
    assert flat[plane + 5 * 32] == 0x10 and flat[plane + 5 * 32 + 7] == 0xFE
    # scales after the codes: quad 1, position 1
    for g in range(4):
        assert flat[plane + B * 32 + (1 * 4 + g) * 4 + 1] == g + 1
    assert np.count_nonzero(pool) == 32 + 4
    v = oracle.fp4_dequant(pool, D)
    assert v.shape == (3, B, H, D)
    want = oracle.e2m1_decode(codes) * np.repeat(oracle.e4m3_decode([1, 2, 3, 4]), 16)
    assert np.array_equal(v[2, 5, 1], want)


def test_decode_matches_contiguous_attention():
    rng = np.random.default_rng(3)
    H, G, D, B = 2, 3, 64, 4
    k = rng.integers(0, 128, (9, H, B, 36), dtype=np.uint8) & 0x77
    v = rng.integers(0, 128, (9, H, B, 36), dtype=np.uint8) & 0x77
    q = rng.standard_normal((2, H * G, D))
    bt = np.array([[8, 0, 3, 5], [1, 2, -1, -1]])
    out, spread = oracle.paged_decode_fp4(q, k, v, 0.5, 0.25, bt, [13, 6], 0.125)
    K = oracle.fp4_dequant(k, D)[bt[0]].reshape(16, H, D)[:13] * 0.5
    V = oracle.fp4_dequant(v, D)[bt[0]].reshape(16, H, D)[:13] * 0.25
    np.testing.assert_allclose(out[0], oracle.contiguous_decode(q[0], K, V, 0.125), rtol=1e-12,
                               atol=1e-12)
    assert (spread >= 0).all()
    # a window of 3 reads the last 3 tokens
    win, _ = oracle.paged_decode_fp4(q, k, v, 0.5, 0.25, bt, [13, 6], 0.125, window=3)
    np.testing.assert_allclose(win[0], oracle.contiguous_decode(q[0], K[10:], V[10:], 0.125),
                               rtol=1e-12, atol=1e-12)


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 2, 64))
    ang = rng.standard_normal((3, 8))
    rows = np.concatenate((np.cos(ang), np.sin(ang)), -1)
    for inter in (False, True):
        y = oracle.rotate(x, rows, inter)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        back = oracle.rotate(y, np.concatenate((np.cos(ang), -np.sin(ang)), -1), inter)
        np.testing.assert_allclose(back, x, rtol=1e-12, atol=1e-12)
    y = oracle.rotate(x, rows, False)
    np.testing.assert_allclose(y[1, 0, 2], x[1, 0, 2] * np.cos(ang[1, 2])
                               - x[1, 0, 10] * np.sin(ang[1, 2]))
    unit = oracle.head_norm(x, np.ones(64), 0.0)
    np.testing.assert_allclose((unit ** 2).mean(-1), 1.0)
