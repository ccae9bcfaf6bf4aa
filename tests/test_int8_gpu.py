"""The 8-bit operators on the GPU against plain 64-bit implementations.

Codes, scales and restored values are bit-exact.  The int8 product is
bit-exact too: integer sums are exact and every rounding after them is defined.
The backward's dX and dB are those of linear_bwd_saved bit for bit (they do not
depend on x), and dA is bounded below from the roundings it makes.
"""
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


def from_f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).cuda()


def activation(T, K, seed, dev="cuda"):
    x = inputs.normal_bf16((T, K), 1.0, seed, dev)
    x[:, 5::256] *= 20   # outlier channels
    return x


def equal_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


# --------------------------------------------------------------------------
# quantize / dequantize
# --------------------------------------------------------------------------
def check_quantize(x, group):
    q = Q()
    q8 = q.quantize_int8(x, group=group)
    back = q.dequantize_int8(q8)
    torch.cuda.synchronize()
    codes, scales = O.quantize_int8(bits(x), group)
    got_s = q8.scales.cpu().numpy()
    nan = np.isnan(scales)
    assert np.array_equal(np.isnan(got_s), nan)
    assert np.array_equal(got_s[~nan].view(np.uint32), scales[~nan].view(np.uint32)), "scales"
    got = q8.codes.cpu().numpy()
    assert np.array_equal(got, codes), f"codes differ at {np.argwhere(got != codes)[:5]}"
    ref = O.dequantize_int8(codes, scales, group)
    g = bits(back)
    isnan = np.isnan(O.bf16_bits_to_f32(ref))
    assert np.array_equal(np.isnan(O.bf16_bits_to_f32(g)), isnan)
    assert np.array_equal(g[~isnan], ref[~isnan])
    return q8


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,cols", [
    (1, 16), (1, 64), (3, 80), (7, 128), (9, 144), (17, 1024), (5, 1040), (33, 4096), (2, 4112), (4, 14336), (3, 16400),
    (2, 22016), (2, 40000), (1000, 272), (1027, 1040), (1025, 2048),
])
def test_quantize_dequantize_bitexact(rows, cols, group):
    check_quantize(activation(rows, cols, rows * 100003 + cols), group)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("cols", [256, 2064, 33024])
def test_quantize_special_rows(cols, group):
    """Zeros, subnormals, the largest values, exact ties, infinities and NaN."""
    rng = np.random.default_rng(cols)
    x = rng.normal(0, 1, (12, cols)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2] = 2.0 ** -133
    x[3] = rng.normal(0, 1e-38, cols)
    x[4] = rng.normal(0, 5e37, cols)
    x[5] = 0.5 * rng.integers(-254, 255, cols)
    x[5, ::64] = 127                      # scale 1: every odd half is a tie
    x[6, cols - 1] = np.inf
    x[7, 0] = -np.inf
    x[8, cols // 2] = np.nan
    x[9] = 0
    x[9, 17] = -3.0
    check_quantize(from_f32(x), group)


def test_quantize_into_and_strided_refusal():
    q = Q()
    x = activation(40, 512, 1)
    q8 = q.quantize_int8(x, group=128)
    y = activation(40, 512, 2)
    q.quantize_int8_into(y, q8)
    ref = q.quantize_int8(y, group=128)
    assert torch.equal(q8.codes, ref.codes) and torch.equal(q8.scales, ref.scales)
    with pytest.raises(ValueError):
        q.quantize_int8(x[:, ::2])
    with pytest.raises(ValueError):
        q.quantize_int8_into(y[:39], q8)
    with pytest.raises(ValueError):
        q.quantize_int8_into(y, q8.codes)
    with pytest.raises(ValueError):
        q.dequantize_int8(q8.codes)
    with pytest.raises(ValueError):
        q.quantize_int8(x.float())
    with pytest.raises(ValueError):
        q.quantize_int8(x, group=64)
    with pytest.raises(q.QLoraError):
        q.quantize_int8(x[:, :40].contiguous())          # cols % 16
    with pytest.raises(q.QLoraError):
        q.quantize_int8(torch.zeros(2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 64))   # misaligned


def test_rows_behind_the_last_are_left_alone():
    q = Q()
    for group in (0, 128):
        x = activation(21, 656, 3)
        cbuf = torch.full((40, 656), 77, dtype=torch.int8, device="cuda")
        n = 6 if group else 1
        sbuf = torch.full((n * 21 + 64,), 9.0, device="cuda")
        q8 = q.QuantizedInt8(cbuf[:21], sbuf[:n * 21].view(n, 21), group)
        q.quantize_int8_into(x, q8)
        ref = q.quantize_int8(x, group=group)
        assert torch.equal(q8.codes, ref.codes) and torch.equal(q8.scales, ref.scales)
        assert (cbuf[21:] == 77).all() and (sbuf[n * 21:] == 9).all()
        obuf = torch.full((30, 656), 5.0, dtype=torch.bfloat16, device="cuda")
        q.dequantize_int8(q8, out=obuf[:21])
        assert equal_bits(obuf[:21], q.dequantize_int8(ref)) and (obuf[21:] == 5).all()


# --------------------------------------------------------------------------
# the int8 product
# --------------------------------------------------------------------------
def check_linear(x, w):
    q = Q()
    w8 = q.quantize_int8(w)
    y = q.linear_int8(x, w8)
    x8 = q.quantize_int8(x)
    y2 = q.linear_int8(x8, w8)
    q.get_error()
    torch.cuda.synchronize()
    xc, sx = O.quantize_int8(bits(x))
    wc, sw = O.quantize_int8(bits(w))
    ref = O.linear_int8(xc, sx[0], wc, sw[0])
    g = bits(y)
    assert np.array_equal(g, ref), f"{(g != ref).sum()} of {g.size} differ, first {np.argwhere(g != ref)[:4]}"
    assert equal_bits(y, y2)


@pytest.mark.parametrize("T,N,K", [
    (1, 8, 16), (1, 8, 128), (2, 136, 48), (1, 1024, 4096), (3, 40, 320), (4, 1032, 4112), (4, 4096, 4096), (1, 512, 14336),
    (2, 24, 32784), (1, 8, 32768), (4, 16400, 1040), (5, 1024, 4096), (1, 14336, 4096), (15, 256, 144), (16, 512, 512),
    (17, 264, 1040), (31, 128, 2048), (32, 136, 4096), (33, 640, 256), (64, 1024, 272), (65, 248, 1024), (100, 384, 4112),
    (127, 136, 128), (128, 256, 512), (129, 264, 256), (200, 1032, 656), (256, 512, 128), (257, 256, 1024), (300, 384, 320),
    (511, 1000, 528), (513, 520, 2048), (700, 2056, 1104), (1025, 4096, 512), (2000, 2040, 784), (2049, 1024, 4096),
])
def test_linear_int8_bitexact(T, N, K):
    check_linear(activation(T, K, T * 7 + K), inputs.normal_bf16((N, K), 0.02, N, "cuda"))


def test_linear_int8_largest_sums():
    """K = 131072 codes of +-127: the INT32 sums reach 2.114e9 of 2.147e9."""
    for T in (2, 40):
        x = torch.ones(T, 131072, dtype=torch.bfloat16, device="cuda")
        x[1] = -1
        w = torch.full((16, 131072), 0.5, dtype=torch.bfloat16, device="cuda")
        w[3] = -0.5
        check_linear(x, w)


@pytest.mark.parametrize("T", [2, 150, 600])
def test_linear_int8_non_finite_rows(T):
    """A token with a NaN or an infinity gives NaN for that token alone, an
    output channel with one NaN in that column alone."""
    q = Q()
    x, w = activation(T, 256, 4), inputs.normal_bf16((264, 256), 0.02, 5, "cuda")
    clean = q.linear_int8(x, q.quantize_int8(w))
    x[1, 3] = float("nan")
    w[200, 7] = float("inf")
    y = q.linear_int8(x, q.quantize_int8(w)).float()
    assert y[1].isnan().all() and y[:, 200].isnan().all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[:, 200] = False, False
    assert torch.equal(y[keep], clean.float()[keep])


@pytest.mark.parametrize("T", [0, 1, 30, 260, 600])
def test_linear_int8_out_buffer_and_zero_tokens(T):
    q = Q()
    w8 = q.quantize_int8(inputs.normal_bf16((520, 336), 0.02, 6, "cuda"))
    x = activation(T, 336, 7)
    buf = torch.full((T + 40, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    y = q.linear_int8(x, w8, out=buf[:T])
    assert y.shape == (T, 520) and (buf[T:] == 3).all()
    assert equal_bits(buf[:T], q.linear_int8(x, w8))
    assert q.linear_int8(q.quantize_int8(x), w8).shape == (T, 520)


def test_linear_int8_refusals():
    q = Q()
    w = inputs.normal_bf16((64, 256), 0.02, 8, "cuda")
    w8, x = q.quantize_int8(w), activation(5, 256, 9)
    with pytest.raises(ValueError):
        q.linear_int8(x, q.quantize_int8(w, group=128))
    with pytest.raises(ValueError):
        q.linear_int8(q.quantize_int8(x, group=128), w8)
    with pytest.raises(ValueError):
        q.linear_int8(x[:, :240].contiguous(), w8)
    with pytest.raises(ValueError):
        q.linear_int8(x, w8, out=torch.empty(4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        q.linear_int8(x.cpu(), w8)
    with pytest.raises(ValueError):
        q.linear_int8(x, w)
    with pytest.raises(q.QLoraError):
        q.linear_int8(x, q.quantize_int8(w[:60].contiguous()))    # N % 8


# --------------------------------------------------------------------------
# the backward from an 8-bit activation
# --------------------------------------------------------------------------
def layer(T, N, K, r, s, seed=50, b_std=0.05):
    W, X, A, B, dY = inputs.layer_inputs(seed, 0, 0, T, N, K, r, device="cuda", b_std=b_std)
    X[:, 5::256] *= 20
    return W, X, A, B, dY


def check_backward(T, N, K, r, s, group, seed=50):
    q = Q()
    W, X, A, B, dY = layer(T, N, K, r, s, seed)
    qw = q.quantize_nf4(W)
    _, u = q.linear_fwd_save(X, qw, A, B, s)
    x8 = q.quantize_int8(X, group=group)
    dx0, dA0, dB0 = q.linear_bwd_saved(dY, X, qw, A, B, s, u)
    dx, dA, dB = q.linear_bwd_saved_int8(dY, x8, qw, A, B, s, u)
    q.get_error()
    torch.cuda.synchronize()
    assert equal_bits(dx, dx0) and equal_bits(dB, dB0)
    f = lambda t: O.bf16_bits_to_f32(bits(t)).astype(np.float64)
    dy64, b64 = f(dY), f(B)
    xh = O.values_int8(*O.quantize_int8(bits(X), group), group)
    dU = s * (dy64 @ b64)
    ref = dU.T @ xh
    # dU: FP32 sums of exact products over N features (at most 2^-23 a step),
    # kept as hi + lo twice (before and after the scale, 2^-16 each); dA: FP32
    # sums of two planes over T tokens and the cluster, then one BF16 rounding
    S = (abs(s) * (np.abs(dy64) @ np.abs(b64))).T @ np.abs(xh)
    bound = 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -16 + (N + 2 * T + 16) * 2.0 ** -23) * S
    err = np.abs(f(dA) - ref)
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size}, worst {np.max(err - bound)}"
    # and, far tighter than that worst case, the error of the whole gradient
    assert np.linalg.norm(f(dA) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    return dA


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,N,K,r,s", [
    (1, 64, 64, 1, 1.0), (2, 8, 64, 3, 2.0), (16, 512, 512, 8, 2.0), (63, 136, 192, 13, 0.5), (65, 256, 128, 128, 0.25),
    (129, 264, 320, 17, 1.0), (300, 384, 320, 24, 0.5), (257, 128, 256, 65, 1.0), (512, 1024, 768, 16, 2.0),
    (1003, 640, 1088, 36, 1.0), (777, 1024, 4096, 64, 0.25), (2047, 512, 1024, 100, 1.0),
])
def test_backward_int8(T, N, K, r, s, group):
    check_backward(T, N, K, r, s, group)


def test_backward_int8_8b_q_projection():
    check_backward(4096, 4096, 4096, 16, 2.0, 128)


def test_backward_int8_against_differences():
    """dA against central differences, in 64 bits, of <dY, s (x A^T) B^T> with x
    the values the codes stand for (linear in A, so the difference is exact but
    for its own rounding)."""
    T, N, K, r, s = 37, 64, 192, 5, 1.5
    dA = O.bf16_bits_to_f32(bits(check_backward(T, N, K, r, s, 128, seed=51))).astype(np.float64)
    _, X, A, B, dY = layer(T, N, K, r, s, 51)
    xh = O.values_int8(*O.quantize_int8(bits(X), 128), 128)
    a, b, dy = (O.bf16_bits_to_f32(bits(t)).astype(np.float64) for t in (A, B, dY))
    loss = lambda a: float((dy * (s * (xh @ a.T) @ b.T)).sum())
    for j in range(r):
        for k in (0, 1, 64, 127, 128, 191):
            e = np.zeros_like(a)
            e[j, k] = 1.0
            diff = (loss(a + e) - loss(a - e)) / 2
            S = (abs(s) * (np.abs(dy) @ np.abs(b)))[:, j] @ np.abs(xh[:, k])
            assert abs(dA[j, k] - diff) <= 2.0 ** -8 * abs(diff) + (2 * 2.0 ** -16 + (N + 2 * T + 16) * 2.0 ** -23) * S


def test_backward_int8_zero_tokens_and_non_finite():
    q = Q()
    W, X, A, B, dY = layer(70, 128, 256, 8, 2.0)
    qw = q.quantize_nf4(W)
    e = q.quantize_int8(X[:0])
    dx, dA, dB = q.linear_bwd_saved_int8(dY[:0], e, qw, A, B, 2.0, torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert dx.shape == (0, 256) and not dA.any() and not dB.any()
    _, u = q.linear_fwd_save(X, qw, A, B, 2.0)
    clean = q.linear_bwd_saved_int8(dY, q.quantize_int8(X, group=128), qw, A, B, 2.0, u)
    X[69, 200] = float("inf")
    dx, dA, dB = q.linear_bwd_saved_int8(dY, q.quantize_int8(X, group=128), qw, A, B, 2.0, u)
    assert dA[:, 128:].isnan().all()                       # the group of the infinity
    assert equal_bits(dA[:, :128].contiguous(), clean[1][:, :128].contiguous())
    assert equal_bits(dx, clean[0]) and equal_bits(dB, clean[2])


def test_backward_int8_refusals():
    q = Q()
    W, X, A, B, dY = layer(16, 128, 256, 8, 2.0)
    qw = q.quantize_nf4(W)
    _, u = q.linear_fwd_save(X, qw, A, B, 2.0)
    x8 = q.quantize_int8(X)
    with pytest.raises(ValueError):
        q.linear_bwd_saved_int8(dY, X, qw, A, B, 2.0, u)                   # not in 8 bits
    with pytest.raises(ValueError):
        q.linear_bwd_saved_int8(dY[:15], x8, qw, A, B, 2.0, u)
    with pytest.raises(ValueError):
        q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u[:100])
    with pytest.raises(ValueError):
        q.linear_bwd_saved_int8(dY, q.quantize_int8(X[:, :128].contiguous()), qw, A, B, 2.0, u)
    with pytest.raises(q.QLoraError):
        q.linear_bwd_saved_int8(dY, x8, qw, A, B, float("inf"), u)


# --------------------------------------------------------------------------
# the operators as a program uses them
# --------------------------------------------------------------------------
def test_training_and_serving_run():
    """Forward, checkpoint, backward, Adam, merge, quantize, serve: the served
    product is the oracle's on the merged weight, and the restored activation is
    what the backward saw."""
    q = Q()
    T, N, K, r, s, lr = 192, 256, 320, 8, 2.0, 1e-2
    W, X, A, B, dY = layer(T, N, K, r, s)
    qw = q.quantize_nf4(W)
    pA, mA, vA = A.float(), torch.zeros_like(A, dtype=torch.float32), torch.zeros_like(A, dtype=torch.float32)
    _, u = q.linear_fwd_save(X, qw, A, B, s)
    x8 = q.quantize_int8(X, group=128)
    xr = q.dequantize_int8(x8)
    dx, dA, dB = q.linear_bwd_saved_int8(dY, x8, qw, A, B, s, u)
    ref = q.linear_bwd_saved(dY, xr, qw, A, B, s, u)[1].float()
    # the restored activation is BF16 (2^-8 a value), each result BF16
    assert (dA.float() - ref).norm() <= 2 * 2.0 ** -8 * ref.norm()
    A2 = torch.empty_like(A)
    q.adam_step(pA, mA, vA, dA, A2, step=1, lr=lr)
    w8 = q.quantize_int8(q.merge_adapter(qw, A2, B, s))
    for t in (1, 9, T):
        y = q.linear_int8(X[:t], w8)
        wc, sw = O.quantize_int8(bits(q.merge_adapter(qw, A2, B, s)))
        xc, sx = O.quantize_int8(bits(X[:t]))
        assert np.array_equal(bits(y), O.linear_int8(xc, sx[0], wc, sw[0]))
    q.get_error()


def test_captured_replayed_and_interleaved():
    """Two graphs captured on one stream, replayed at once on two streams with
    new inputs, give what eager calls give; eager calls run between them."""
    q = Q()
    T, N, K, r, s = 320, 512, 640, 16, 2.0
    W, X, A, B, dY = layer(T, N, K, r, s)
    qw, w8 = q.quantize_nf4(W), q.quantize_int8(W)
    _, u = q.linear_fwd_save(X, qw, A, B, s)
    cap = torch.cuda.Stream()
    graphs = []
    for i in range(2):
        x, dy = X.clone(), dY.clone()
        with torch.cuda.stream(cap):
            q.linear_int8(x, w8)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            y = q.linear_int8(x, w8)
            x8 = q.quantize_int8(x, group=128)
            grads = q.linear_bwd_saved_int8(dy, x8, qw, A, B, s, u)
        graphs.append((g, x, dy, y, grads))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for step in range(4):
        want = []
        for i, (g, x, dy, _, _) in enumerate(graphs):
            x.copy_(activation(T, K, 100 + 10 * step + i))
            dy.copy_(inputs.normal_bf16((T, N), 1.0, 200 + 10 * step + i, "cuda"))
            want.append((q.linear_int8(x, w8),
                         q.linear_bwd_saved_int8(dy, q.quantize_int8(x, group=128), qw, A, B, s, u)))
        torch.cuda.synchronize()
        for st, (g, *_) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for (g, x, dy, y, grads), (wy, wg) in zip(graphs, want):
            assert equal_bits(y, wy)
            assert all(equal_bits(a, b) for a, b in zip(grads, wg))
    q.get_error()
    del graphs


def test_random_shapes():
    """Sizes drawn over the whole range, each operator: bit-exact codes, values
    and products, bounded gradients."""
    import random
    rng = random.Random(20)
    log = lambda lo, hi, m: max(m, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi))))) // m * m)
    for _ in range(25):
        check_quantize(activation(log(1, 3000, 1), log(16, 9000, 16), rng.randrange(1 << 20)), rng.choice((0, 128)))
        T, N, K = log(1, 3000, 1), log(8, 3000, 8), log(16, 6000, 16)
        check_linear(activation(T, K, rng.randrange(1 << 20)),
                     inputs.normal_bf16((N, K), 0.02, rng.randrange(1 << 20), "cuda"))
    for _ in range(8):
        check_backward(log(1, 1500, 1), log(8, 1000, 8), log(64, 3000, 64), rng.randint(1, 128), 1.0,
                       rng.choice((0, 128)))


def test_scratch_and_workspace_need_no_initialisation():
    """The per-call buffers come from the allocator as they are: all ones here
    (NaN, and every counter and flag set)."""
    q = Q()
    for r in (16, 100):
        W, X, A, B, dY = layer(300, 520, 640, r, 2.0)
        qw, w8 = q.quantize_nf4(W), q.quantize_int8(W)
        _, u = q.linear_fwd_save(X, qw, A, B, 2.0)
        x8 = q.quantize_int8(X, group=128)
        first = (q.linear_int8(X, w8), *q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u))
        torch.cuda.synchronize()
        for _ in range(3):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 20, 1 << 22, 1 << 24)]
            del junk
            again = (q.linear_int8(X, w8), *q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u))
            assert all(equal_bits(a, b) for a, b in zip(first, again))
    q.get_error()


def test_quantized_int8_object():
    import io
    q = Q()
    x8 = q.quantize_int8(activation(5, 272, 1), group=128)
    with pytest.raises(AttributeError):
        x8.codes = torch.zeros(5, 272, dtype=torch.int8, device="cuda")
    assert x8.nbytes() == 5 * 272 + 4 * 3 * 5
    f = io.BytesIO()
    torch.save(x8, f)
    f.seek(0)
    y8 = torch.load(f, weights_only=False)
    assert torch.equal(y8.codes, x8.codes) and torch.equal(y8.scales, x8.scales) and y8.group == 128
    assert equal_bits(q.dequantize_int8(y8), q.dequantize_int8(x8))
    for bad in (dict(scales=torch.zeros(1, 5, device="cuda")), dict(codes=torch.zeros(5, 272, device="cuda")),
                dict(codes=x8.codes.t()), dict(group=64)):
        with pytest.raises(ValueError):
            q.QuantizedInt8(**{**dict(codes=x8.codes, scales=x8.scales, group=128), **bad})


def test_status_word():
    """A recorded timeout of the 8-bit calls is raised once by get_error; the
    calls run without a status word too."""
    import ctypes as C
    q = Q()
    x, w = activation(40, 256, 1), inputs.normal_bf16((64, 256), 0.02, 2, "cuda")
    w8, x8 = q.quantize_int8(w), q.quantize_int8(x)
    want = q.linear_int8(x8, w8)
    q.get_error()
    q._STATUS[x.device][0] = 2        # DEV_TIMEOUT
    with pytest.raises(q.QLoraError) as e:
        q.get_error()
    assert e.value.status == 7
    q.get_error()
    q._STATUS[x.device][0] = 2
    with pytest.raises(q.QLoraError):
        q.get_error("cuda")           # the current device
    q.get_error()
    y = torch.empty_like(want)
    st = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert q.lib().qlora_linear_int8_q(x8._ref, w8._ref, y.data_ptr(), None, st) == 0
    assert equal_bits(y, want)


def test_two_streams_at_once():
    """The same weight and the same token batch from two streams at once."""
    q = Q()
    w8 = q.quantize_int8(inputs.normal_bf16((1024, 4096), 0.02, 1, "cuda"))
    xs = [activation(t, 4096, t) for t in (1, 20, 333)]
    want = [q.linear_int8(x, w8) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                got.append([q.linear_int8(x, w8) for x in xs])
    torch.cuda.synchronize()
    for ys in got:
        assert all(equal_bits(a, b) for a, b in zip(ys, want))
    q.get_error()


# --------------------------------------------------------------------------
# matrices of more than 2^31 elements: the last rows, against calls on them alone
# --------------------------------------------------------------------------
def test_format_past_31_bits():
    q = Q()
    x = torch.empty(131200, 16400, dtype=torch.bfloat16, device="cuda").normal_()
    for group in (0, 128):
        q8, tail = q.quantize_int8(x, group), q.quantize_int8(x[-300:], group)
        assert torch.equal(q8.codes[-300:], tail.codes) and torch.equal(q8.scales[:, -300:], tail.scales)
        assert equal_bits(q.dequantize_int8(q8)[-300:], q.dequantize_int8(tail))
        del q8


def test_linear_int8_past_31_bits():
    q = Q()
    g = torch.Generator(device="cuda").manual_seed(5)

    def rows8(rows, cols):
        codes = torch.empty(rows, cols, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
        return q.QuantizedInt8(codes, torch.rand(1, rows, device="cuda", generator=g) * 0.01)

    def last(m, n):
        return q.QuantizedInt8(m.codes[-n:], m.scales[:, -n:].clone())

    w, x = rows8(40008, 65536), rows8(300, 65536)         # the weight
    w_end = last(w, 264)
    for T in (1, 40, 300):
        xt = last(x, T)
        assert equal_bits(q.linear_int8(xt, w)[:, -264:], q.linear_int8(xt, w_end))
    w, x = rows8(16392, 64), rows8(131200, 64)            # y
    assert equal_bits(q.linear_int8(x, w)[-300:], q.linear_int8(last(x, 300), w))
    x, w = rows8(131200, 16400), rows8(24, 16400)         # x
    assert equal_bits(q.linear_int8(x, w)[-300:], q.linear_int8(last(x, 300), w))
    q.get_error()


def test_backward_int8_past_31_bits():
    """Only the last 200 tokens have a gradient, so dA is theirs alone: apart by
    the BF16 rounding of both results (2^-8 each) and the order of FP32 sums of
    200 terms and of dU's 128 (2^-24 x 328 of the terms' sizes, dU's planes 2^-16)."""
    q = Q()
    T, N, K, r = 131200, 128, 16384, 8
    qw = q.quantize_nf4(inputs.normal_bf16((N, K), 0.02, 1, "cuda"))
    A, B = inputs.normal_bf16((r, K), K ** -0.5, 2, "cuda"), inputs.normal_bf16((N, r), 0.01, 3, "cuda")
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    dy[-200:] = inputs.normal_bf16((200, N), 1.0, 4, "cuda")
    u = torch.zeros(q.saved_u_bytes(T, r), dtype=torch.uint8, device="cuda")
    for group in (0, 128):
        x8 = q.quantize_int8(x, group)
        tail = q.quantize_int8(x[-200:], group)
        dx, dA, dB = q.linear_bwd_saved_int8(dy, x8, qw, A, B, 2.0, u)
        tx, tA, _ = q.linear_bwd_saved_int8(dy[-200:], tail, qw, A, B, 2.0, u)
        q.get_error()
        du = 2.0 * dy[-200:].double() @ B.double()
        size = du.abs().T @ q.dequantize_int8(tail).double().abs()
        diff = (dA.double() - tA.double()).abs()
        assert (diff <= 2 * 2.0 ** -8 * tA.double().abs() + (2.0 ** -15 + 328 * 2.0 ** -24) * size).all()
        assert dA.abs().max() > 0 and (dx[:-200] == 0).all()
        ddx = (dx[-200:].double() - tx.double()).abs()
        assert (ddx <= 2 * 2.0 ** -8 * tx.double().abs() + 1e-5).all()
        del dx, x8
