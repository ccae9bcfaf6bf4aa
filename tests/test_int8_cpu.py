"""The 8-bit format, its oracle and the argument checks of its entry points,
without a GPU.  No test here launches a kernel."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import oracle as O

FAKE = 0x10000   # never dereferenced: every call below fails validation, or does nothing, first
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_20_b200 import build
    build.build()
    from bit_nf4_quantized_20_b200 import _lib
    return _lib.lib()


def bf16(x):
    return O.f32_to_bf16_bits(np.asarray(x, np.float32))


# --------------------------------------------------------------------------
# the oracle
# --------------------------------------------------------------------------
@pytest.mark.parametrize("group", [0, 128])
def test_codes_are_the_nearest_integers(group):
    """Every code against exact rational arithmetic: |x inv - code| <= 1/2, and
    an exact half goes to the even code."""
    rng = np.random.default_rng(5)
    x = bf16(rng.normal(0, 1, (6, 272)) * np.array([1, 1e-3, 40, 1e30, 1e-30, 1])[:, None])
    codes, scales = O.quantize_int8(x, group)
    xf = O.bf16_bits_to_f32(x)
    g = group or 272
    for i in range(6):
        for j in range(272):
            inv = Fraction(float(np.float32(1) / scales[j // g, i]))
            d = Fraction(float(xf[i, j])) * inv - int(codes[i, j])
            assert abs(d) < Fraction(1, 2) or (abs(d) == Fraction(1, 2) and codes[i, j] % 2 == 0)
    assert np.abs(codes.astype(int)).max() == 127


def test_ties_go_to_even():
    """amax = 127 gives scale 1: halves are exact ties."""
    x = np.zeros((1, 16), np.float32)
    x[0, :9] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5, -126.5]
    codes, scales = O.quantize_int8(bf16(x))
    assert scales[0, 0] == 1.0
    assert codes[0, :9].tolist() == [127, 0, 2, 2, 0, -2, -2, 64, -126]


def test_special_groups():
    x = np.zeros((5, 256), np.float32)
    x[1, 3] = np.inf
    x[2, 200] = np.nan
    x[3, :] = 2.0 ** -133             # the smallest BF16 subnormal
    x[4, 7] = 3.3895314e38            # the largest finite BF16
    codes, scales = O.quantize_int8(bf16(x), 128)
    assert scales[0, 0] == np.float32(2.0 ** -126) and not codes[0].any()
    assert np.isnan(scales[0, 1]) and not np.isnan(scales[1, 1])
    assert np.isnan(scales[1, 2]) and not np.isnan(scales[0, 2])
    assert not codes[3].any() and scales[0, 3] == np.float32(2.0 ** -126)   # 2^-133 / 2^-126 rounds to 0
    assert codes[4, 7] == 127 and np.isfinite(scales[0, 4])
    v = O.values_int8(codes, scales, 128)
    assert np.isnan(v[1, :128]).all() and (v[1, 128:] == 0).all()


def test_round_trip_error_is_half_a_step():
    """|x - code scale| <= scale / 2 plus the rounding of inv (2^-24 of x, and x
    is at most 127 scale (1 + 2^-23))."""
    rng = np.random.default_rng(6)
    x = bf16(rng.normal(0, 1, (9, 400)))
    for group in (0, 128):
        codes, scales = O.quantize_int8(x, group)
        g = group or 400
        s = np.repeat(scales.astype(np.float64).T, g, axis=1)[:, :400]
        err = np.abs(O.bf16_bits_to_f32(x).astype(np.float64) - O.values_int8(codes, scales, group))
        assert (err <= s * (0.5 + 130 * 2.0 ** -22)).all()
        # writing the values again gives them back (the largest code of a group is 127)
        c2, s2 = O.quantize_int8(O.dequantize_int8(codes, scales, group), group)
        assert (np.abs(c2.astype(int) - codes) <= 1).all()


def test_linear_int8_oracle_is_the_integer_sum():
    rng = np.random.default_rng(7)
    xq = rng.integers(-127, 128, (3, 48)).astype(np.int8)
    wq = rng.integers(-127, 128, (8, 48)).astype(np.int8)
    sx, sw = rng.uniform(0.1, 1, 3).astype(np.float32), rng.uniform(0.1, 1, 8).astype(np.float32)
    got = O.bf16_bits_to_f32(O.linear_int8(xq, sx, wq, sw)).astype(np.float64)
    for t in range(3):
        for n in range(8):
            acc = sum(int(a) * int(b) for a, b in zip(xq[t], wq[n]))
            ref = acc * float(sx[t]) * float(sw[n])
            # one BF16 rounding (2^-8) and two FP32 roundings (2^-24 each)
            assert abs(got[t, n] - ref) <= (2.0 ** -8 + 2.0 ** -22) * abs(ref)


# --------------------------------------------------------------------------
# the C ABI
# --------------------------------------------------------------------------
def matrix(rows=32, cols=128, codes=FAKE, scales=FAKE, group=0):
    from bit_nf4_quantized_20_b200._lib import Int8Matrix
    return Int8Matrix(codes, scales, rows, cols, group)


def weight(rows=128, cols=128):
    from bit_nf4_quantized_20_b200._lib import NF4Weight
    w = NF4Weight()
    w.codes, w.scales, w.c2 = 0x1000, 0x2000, 0x3000
    w.rows, w.cols, w.blocksize, w.dq_block = rows, cols, 64, 256
    for i, v in enumerate(O.nf4_codebook()):
        w.codebook[i] = float(v)
    return w


def test_storage_bytes(L):
    a, b = C.c_size_t(), C.c_size_t()
    f = L.qlora_int8_storage_bytes
    assert f(7, 272, 0, C.byref(a), C.byref(b)) == 0 and (a.value, b.value) == (7 * 272, 28)
    assert f(7, 272, 128, C.byref(a), C.byref(b)) == 0 and (a.value, b.value) == (7 * 272, 3 * 28)
    assert f(0, 272, 0, C.byref(a), C.byref(b)) == 0 and (a.value, b.value) == (0, 0)
    assert f(7, 264, 0, C.byref(a), C.byref(b)) == 2          # cols % 16
    assert f(7, 272, 64, C.byref(a), C.byref(b)) == 2         # group
    assert f(-1, 272, 0, C.byref(a), C.byref(b)) == 1
    assert f(7, 0, 0, C.byref(a), C.byref(b)) == 1
    assert f(7, 272, 0, None, C.byref(b)) == 1
    assert f(1 << 31, 272, 0, C.byref(a), C.byref(b)) == 2


def test_quantize_int8_validation(L):
    f, P = L.qlora_quantize_int8, FAKE
    assert f(None, 32, 128, 0, C.byref(matrix()), None) == 1
    assert f(P, 32, 128, 0, None, None) == 1
    assert f(P, 32, 128, 0, C.byref(matrix(codes=None)), None) == 1
    assert f(P, 32, 128, 0, C.byref(matrix(scales=None)), None) == 1
    assert f(P, -1, 128, 0, C.byref(matrix()), None) == 1
    assert f(P, 32, 120, 0, C.byref(matrix()), None) == 2
    assert f(P, 32, 128, 32, C.byref(matrix()), None) == 2
    assert f(P + 8, 32, 128, 0, C.byref(matrix()), None) == 3
    assert f(P, 32, 128, 0, C.byref(matrix(codes=FAKE + 8)), None) == 3
    assert f(P, 32, 128, 0, C.byref(matrix(scales=FAKE + 4)), None) == 3
    m = matrix(rows=9, cols=9)
    assert f(None, 0, 128, 128, C.byref(m), None) == 0                 # no rows: nothing to do
    assert (m.rows, m.cols, m.group) == (0, 128, 128)
    d = L.qlora_dequantize_int8
    assert d(None, P, None) == 1
    assert d(C.byref(matrix()), None, None) == 1
    assert d(C.byref(matrix()), P + 2, None) == 3
    assert d(C.byref(matrix(cols=100)), P, None) == 2
    assert d(C.byref(matrix(group=1)), P, None) == 2
    assert d(C.byref(matrix(rows=0)), None, None) == 0


def test_linear_int8_validation(L):
    f, P = L.qlora_linear_int8, FAKE
    w = matrix(rows=64, cols=256)

    def call(x=P, T=5, w=w, y=P, scratch=P, nbytes=BIG, status=P):
        return f(x, T, C.byref(w) if w is not None else None, y, scratch, nbytes, status, None)

    assert call(x=None) == 1
    assert call(T=-1) == 1
    assert call(w=None) == 1
    assert call(y=None) == 1
    assert call(w=matrix(rows=0, cols=256)) == 1
    assert call(w=matrix(rows=60, cols=256)) == 2             # N % 8
    assert call(w=matrix(rows=64, cols=256, group=128)) == 2  # one scale per output channel
    assert call(w=matrix(rows=64, cols=131072 + 16)) == 2     # INT32 sums
    assert call(T=65535 * 256 + 1) == 2
    assert call(T=65535 * 256, w=matrix(rows=1 << 30, cols=16)) == 2   # more tiles than the kernels count
    assert call(x=P + 2) == 3
    assert call(y=P + 8) == 3
    assert call(status=P + 1) == 3
    assert call(w=matrix(rows=64, cols=256, codes=FAKE + 1)) == 3
    assert call(T=17, scratch=None) == 4
    assert call(T=17, scratch=P + 8) == 4
    assert call(T=17, nbytes=17 * 256 + 255) == 4
    assert call(x=None, T=0, y=None, scratch=None, nbytes=0, status=None) == 0
    s = L.qlora_linear_int8_scratch_bytes
    assert s(17, 64, 256) == 17 * 256 + 256
    assert s(4, 64, 256) == 0                                 # quantized inside the product
    assert s(5, 64, 256) == 1280 + 256
    assert s(4, 8, 131072) == 4 * 131072 + 256                # too long a range for that: 64 KiB of codes a CTA
    assert s(1, 65536, 1024) == 1024 + 256                    # a long stream of weights
    assert s(0, 64, 256) == 0 and s(-1, 64, 256) == 0 and s(17, 64, 250) == 0 and s(17, 64, 131088) == 0
    assert s(17, 60, 256) == 0
    g = L.qlora_linear_int8_q
    x = matrix(rows=5, cols=256)
    assert g(None, C.byref(w), P, P, None) == 1
    assert g(C.byref(x), None, P, P, None) == 1
    assert g(C.byref(x), C.byref(w), None, P, None) == 1
    assert g(C.byref(matrix(rows=5, cols=128)), C.byref(w), P, P, None) == 1     # K differs
    assert g(C.byref(matrix(rows=5, cols=256, group=128)), C.byref(w), P, P, None) == 2
    assert g(C.byref(matrix(rows=0, cols=256)), C.byref(w), None, None, None) == 0


def test_linear_bwd_saved_int8_validation(L):
    f, P = L.qlora_linear_bwd_saved_int8, FAKE
    w, x = weight(), matrix(rows=16, cols=128, group=128)

    def call(dy=P, x=x, w=w, A=P, B=P, r=8, s=2.0, u=P, dx=P, dA=P, dB=P, ws=P, nbytes=BIG, status=P):
        return f(dy, C.byref(x) if x is not None else None, C.byref(w), A, B, r, s, u, dx, dA, dB, ws, nbytes, status,
                 None)

    for k in ("dy", "x", "A", "B", "u", "dx", "dA", "dB"):
        assert call(**{k: None}) == 1, k
    assert call(r=0) == 1 and call(r=129) == 1 and call(s=float("nan")) == 1
    assert call(x=matrix(rows=16, cols=256)) == 1             # K differs from the weight's
    assert call(x=matrix(rows=16, cols=128, group=2)) == 2
    assert call(w=weight(rows=100)) == 2
    for k in ("dy", "A", "B", "u", "dx", "dA", "dB"):
        assert call(**{k: P + 8}) == 3, k
    assert call(status=P + 2) == 3
    assert call(x=matrix(rows=16, cols=128, scales=FAKE + 8)) == 3
    assert call(ws=None) == 4 and call(ws=P + 16) == 4 and call(nbytes=1024) == 4


def test_kernel_names(L):
    assert L.qlora_kernel_name(16) == b"quantize_int8"
    assert L.qlora_kernel_name(17) == b"dequantize_int8"
    assert L.qlora_kernel_name(18) == b"int8_gemm"
    assert L.qlora_kernel_name(19) == b"lora_dA_int8"
    assert L.qlora_kernel_name(20) == b"int8_decode"


# --------------------------------------------------------------------------
# the Python entry points refuse what the kernels do not take
# --------------------------------------------------------------------------
def test_python_refuses_cpu_tensors():
    import bit_nf4_quantized_20_b200 as q
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.quantize_int8(x)
    with pytest.raises(ValueError):
        q.QuantizedInt8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        q.linear_int8(x, x)
    with pytest.raises(ValueError):
        q.linear_bwd_saved_int8(x, x, None, x, x, 1.0, x)
