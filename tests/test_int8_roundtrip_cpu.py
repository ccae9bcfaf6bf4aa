"""What quantizing restored values again does (the oracle; no GPU).

Restored values are BF16: each is off its code * scale by at most 2^-8 of it
(d1, and d2 for the group's largest).  So the new scale is within 2^-8, and the
roundings of two FP32 divisions, of the old one, and a code c becomes the
nearest integer to c (1 + d1) / (1 + d2), at most |c| (2 * 2^-8 + 2^-14) from c:
the same code up to |c| = 62, one off at most above.  Where every code * scale is exact
in BF16 (power-of-two scales: codes have seven bits) both come back as they
were."""
import numpy as np
import pytest

from oracle import oracle as O


def again(codes, scales, group):
    return O.quantize_int8(O.dequantize_int8(codes, scales, group), group)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("seed", range(4))
def test_scales_and_small_codes_come_back(group, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (16, 400)) * np.exp(rng.uniform(-20, 20, (16, 1)))
    codes, scales = O.quantize_int8(O.f32_to_bf16_bits(x.astype(np.float32)), group)
    c2, s2 = again(codes, scales, group)
    assert (np.abs(s2.astype(np.float64) - scales) <= (2.0 ** -8 + 2.0 ** -22) * scales).all()
    off = np.abs(c2.astype(int) - codes)
    assert off.max() <= 1 and not off[np.abs(codes.astype(int)) <= 62].any()


@pytest.mark.parametrize("group", [0, 128])
def test_exact_values_come_back_exactly(group):
    rng = np.random.default_rng(9)
    g = group or 384
    codes = rng.integers(-127, 128, (12, 384)).astype(np.int8)
    codes[:, ::g] = 127
    scales = (2.0 ** rng.integers(-100, 100, (384 // g, 12))).astype(np.float32)
    c2, s2 = again(codes, scales, group)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
