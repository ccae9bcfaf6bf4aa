"""Cases of the 8-bit operators whose results are exact, so that nothing can
hide in a tolerance: the second planes of dU, and codes of -128."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from bit_nf4_quantized_20_b200 import inputs

pytestmark = pytest.mark.gpu


def Q():
    import bit_nf4_quantized_20_b200 as q
    return q


def bits(t):
    return inputs.bf16_bits(t)


def f64(t):
    return O.bf16_bits_to_f32(bits(t)).astype(np.float64)


def dev_bf16(a):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    assert np.array_equal(t.float().numpy(), a), "not exact in BF16"
    return t.cuda()


def bf16_of(a):
    """The BF16 bits of exactly representable FP32 sums, rounded once."""
    f = a.astype(np.float32)
    assert np.array_equal(f.astype(np.float64), a), "not exact in FP32"
    return O.f32_to_bf16_bits(f)


# --------------------------------------------------------------------------
# dA where it comes from the low planes alone
# --------------------------------------------------------------------------
def cancelling(T, N, K, r, group, seed):
    """Tokens in pairs with equal codes.  dU is a b_j (1 + e) for the first and
    -a b_j for the second, e = m 2^-14 with |m| < 64: 1 + e has 15 significant
    bits, so BF16 holds it in two planes and no fewer, and in dA = dU^T x the
    halves of a pair cancel down to e.  a = +-1, b_j = +-1 or +-2, s = 1, and
    scales 1, 2 or 4 (a code of +-127 in every group: RN(127 s / 127) = s), so
    every product is a multiple of 2^-14.

    Products of the high planes are multiples of 2^-8 (|dU| > 1/2, where BF16 has
    a step of 2^-8 at least) of at most 2032, those of the low planes multiples
    of 2^-14 of at most 4.  The test checks that the sums over any run of tokens,
    and any sixteen tokens beside them, stay below 2^24 such steps: then every
    FP32 sum is exact, in whatever order it is taken."""
    rng = np.random.default_rng(seed)
    P = T // 2
    a = rng.choice([-1.0, 1.0], P)
    m = rng.integers(1, 64, P) * rng.choice([-1, 1], P)
    b = rng.choice([-2.0, -1.0, 1.0, 2.0], r)
    dY = np.zeros((T, N))
    dY[0:2 * P:2, 0], dY[1:2 * P:2, 0] = a, -a
    dY[0:2 * P:2, N - 1] = a * m * 2.0 ** -14
    B = np.zeros((N, r))
    B[0], B[N - 1] = b, b
    g = group or K
    codes = rng.integers(-126, 127, (P, K)).astype(np.float64)
    scale = np.empty((P, K))
    for k0 in range(0, K, g):
        codes[:, k0 + rng.integers(0, min(g, K - k0))] = rng.choice([-127, 127], P)
        scale[:, k0:k0 + g] = rng.choice([1.0, 2.0, 4.0], (P, 1))
    x = np.zeros((T, K))
    x[0:2 * P:2] = x[1:2 * P:2] = codes * scale
    return dY, B, x


def planes(v):
    hi = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()
    lo = torch.from_numpy((v - hi).astype(np.float32)).to(torch.bfloat16).double().numpy()
    return hi, lo


SHAPES = [(300, 64, 192, 13), (300, 64, 192, 16), (130, 136, 320, 32), (258, 64, 320, 24), (300, 128, 256, 33),
          (510, 64, 192, 64), (300, 72, 320, 65), (96, 264, 448, 128), (1003, 512, 320, 100), (16, 512, 512, 8)]


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_dA_from_the_low_planes_alone(T, N, K, r, group):
    q = Q()
    dY, B, x = cancelling(T, N, K, r, group, 7 * T + r + group)
    dU = dY @ B
    want = dU.T @ x
    # the oracle's own check of what the docstring says, and that dropping the
    # low plane could not go unnoticed: without it almost every element is wrong
    hi, lo = planes(dU)
    assert np.array_equal(hi + lo, dU)
    for p, step, largest in ((hi, 2.0 ** -8, 2032), (lo, 2.0 ** -14, 4)):
        for j in range(r):
            run = np.cumsum(p[:, j:j + 1] * x, axis=0)
            assert np.array_equal(run / step, np.round(run / step))
            assert 2 * np.abs(run).max() + 16 * largest < 2 ** 24 * step
    planted = hi.T @ x
    assert (np.abs(planted - want) > 2.0 ** -7 * np.abs(want))[want != 0].mean() > 0.9

    A = np.zeros((r, K))
    A[:, 0] = 1.0
    qw = q.quantize_nf4(inputs.normal_bf16((N, K), 0.02, 3, "cuda"))
    X, tA, tB, tY = dev_bf16(x), dev_bf16(A), dev_bf16(B), dev_bf16(dY)
    x8 = q.quantize_int8(X, group=group)
    assert np.array_equal(f64(q.dequantize_int8(x8)), x), "the codes stand for x itself"
    _, u = q.linear_fwd_save(X, qw, tA, tB, 1.0)
    _, dA, _ = q.linear_bwd_saved_int8(tY, x8, qw, tA, tB, 1.0, u)
    q.get_error()
    assert np.array_equal(bits(dA), bf16_of(want)), f"{(bits(dA) != bf16_of(want)).sum()} of {dA.numel()} differ"


# --------------------------------------------------------------------------
# the whole range of a signed byte
# --------------------------------------------------------------------------
def low_codes(rows, cols, seed, everywhere):
    """Given codes with -128, which quantize_int8 never writes."""
    rng = np.random.default_rng(seed)
    c = np.full((rows, cols), -128) if everywhere else rng.integers(-128, 128, (rows, cols))
    c[:, :3] = -128
    s = (2.0 ** rng.integers(-12, -2, (1, rows))).astype(np.float32)
    return c.astype(np.int8), s


def given(c, s, group=0):
    return Q().QuantizedInt8(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), group)


@pytest.mark.parametrize("everywhere", [False, True])
@pytest.mark.parametrize("T,N,K", [(3, 16, 131056), (40, 16, 131056), (100, 264, 1040), (600, 520, 2064)])
def test_product_of_given_codes(T, N, K, everywhere):
    """Sums up to 16384 K: inside INT32 for every K but the largest."""
    q = Q()
    (xc, xs), (wc, ws) = low_codes(T, K, 1, everywhere), low_codes(N, K, 2, everywhere)
    y = q.linear_int8(given(xc, xs), given(wc, ws))
    q.get_error()
    assert np.array_equal(bits(y), O.linear_int8(xc, xs[0], wc, ws[0]))
    if everywhere and K == 131056:
        assert (np.abs(f64(y)) > 0).all() and (y > 0).all()


def test_largest_length_of_codes_that_quantize_writes():
    """K = 131072 with -128 on one side alone: 128 x 127 x K is inside INT32."""
    q = Q()
    T, N, K = 33, 8, 131072
    xc, xs = low_codes(T, K, 1, True)
    wc, ws = np.full((N, K), 127, np.int8), np.full((1, N), 2.0 ** -6, np.float32)
    wc[1::2] = -127
    y = q.linear_int8(given(xc, xs), given(wc, ws))
    assert np.array_equal(bits(y), O.linear_int8(xc, xs[0], wc, ws[0]))
    # tokens quantized in the call against -128 in the weight
    x = torch.ones(2, K, dtype=torch.bfloat16, device="cuda")
    wl = given(np.full((N, K), -128, np.int8), ws)
    want = O.linear_int8(np.full((2, K), 127, np.int8), np.full(2, np.float32(1) / np.float32(127), np.float32),
                         np.full((N, K), -128, np.int8), ws[0])
    assert np.array_equal(bits(q.linear_int8(x, wl)), want)


@pytest.mark.parametrize("group", [0, 128])
def test_restored_and_backward_of_given_codes(group):
    """-128 in a checkpoint: restored, and in dA, as what it stands for.  dU is
    1 or -1 and the scales are powers of two, so the sums are exact."""
    q = Q()
    T, N, K, r = 70, 64, 192, 9
    rng = np.random.default_rng(5)
    c, _ = low_codes(T, K, 3, False)
    groups = -(-K // 128) if group else 1
    s = (2.0 ** rng.integers(-3, 3, (groups, T))).astype(np.float32)
    x8 = given(c, s, group)
    x = c * np.repeat(s.T.astype(np.float64), group or K, axis=1)[:, :K]
    assert np.array_equal(f64(q.dequantize_int8(x8)), x)
    dY, B, A = np.zeros((T, N)), np.zeros((N, r)), np.zeros((r, K))
    dY[:, 5], B[5] = rng.choice([-1.0, 1.0], T), rng.choice([-1.0, 1.0], r)
    qw = q.quantize_nf4(inputs.normal_bf16((N, K), 0.02, 3, "cuda"))
    u = torch.zeros(q.saved_u_bytes(T, r), dtype=torch.uint8, device="cuda")
    _, dA, dB = q.linear_bwd_saved_int8(dev_bf16(dY), x8, qw, dev_bf16(A), dev_bf16(B), 1.0, u)
    q.get_error()
    assert np.array_equal(bits(dA), bf16_of((dY @ B).T @ x)) and not dB.any()
