"""The softmax weights of the 4-bit decode carry 21 bits into the value products,
whatever the output's type: each is a pair of binary16 values.

A kernel's result x before its one rounding to 16 bits is a mean of the value rows
whose weights are off by relative errors of at most e, so |x - o| <= e spread, and
its fp32 sums add their own errors:
    |g - o| <= ulp(g) / 2 + F (|o| + spread),
    F = 2^-22 ((D / 16 + 2) A + T / 16 + 12)
with A the largest sum_d |q_d K_td| of the row's scores in units of log2.  A matrix
instruction's sum is taken to be within 2^-22 of its terms' magnitudes: D / 16 of
them make a score, T / 16 a value, and an error of the score is one of its weight
(times ln 2 < 1).  The factor and the base add 2 A 2^-23; the exponential 2^-22, the
pair 2^-21, the sum of weights, the joins of parts and the last product the rest of
the 12.  Elements of a bfloat16 query under 2^-14 of its row's largest lose 2^-25 of
that, inside the same terms.
"""
import numpy as np
import pytest

import oracle
import workloads as W
from harness import bits_of, bits_to_f64, ulp_spacing
from test_gpu_fp4 import State

pytestmark = pytest.mark.gpu

LENS = list(range(1, 25)) + [31, 33, 48, 64, 90]


@pytest.mark.parametrize("num_ctas", [0, 1])
@pytest.mark.parametrize("window", [0, 7])
@pytest.mark.parametrize("dtype", [W.BF16, W.F16])
@pytest.mark.parametrize("Hq,H,D,B", [(8, 8, 64, 4), (32, 8, 128, 16), (24, 3, 128, 16),
                                      (14, 2, 64, 8), (32, 2, 128, 32), (18, 2, 64, 16)])
def test_weights_are_pairs(cuda_device, dtype, Hq, H, D, B, window, num_ctas):
    st = State(900 + Hq + D, dtype, Hq, H, D, B, LENS, window=window)
    st.scale = float(np.float32(0.25 * D ** -0.5))
    o, spread = st.expected()
    q = np.abs(bits_to_f64(st.q, dtype))
    F = np.zeros(o.shape[:2] + (1,))
    for i, T in enumerate(LENS):
        first = max(0, T - window) if window else 0
        lo = first // B
        K = np.abs(oracle.fp4_dequant(st.k[st.bt[i, lo:-(-T // B)]], D)) * st.k_scale
        K = K.reshape(-1, H, D)[first - lo * B:T - lo * B]
        for h in range(Hq):
            A = (K[:, h // (Hq // H)] @ q[i, h]).max() * st.scale / np.log(2)
            F[i, h] = 2.0 ** -22 * ((D / 16 + 2) * A + T / 16 + 12)
    g_bits = bits_of(st.decode(num_ctas=num_ctas))
    g = bits_to_f64(g_bits, dtype)
    bound = 0.5 * ulp_spacing(g_bits, dtype) + F * (np.abs(o) + spread)
    use = np.abs(g - o) / bound
    assert np.all(use <= 1), "%d of %d past the bound, worst %.3g of it" % (
        (use > 1).sum(), use.size, use.max())
