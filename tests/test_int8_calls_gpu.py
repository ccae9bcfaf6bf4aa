"""Ways of calling the 8-bit operators that their other tests do not take: a
caller's gradient buffers, inside a captured graph too, and one checkpoint for
several projections."""
import pytest
import torch

from bit_nf4_quantized_20_b200 import inputs

pytestmark = pytest.mark.gpu


def Q():
    import bit_nf4_quantized_20_b200 as q
    return q


def equal_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def guarded(*shape):
    """A buffer with rows behind it that no call may touch."""
    buf = torch.full((shape[0] + 9, *shape[1:]), 3.0, dtype=torch.bfloat16, device="cuda")
    return buf, buf[:shape[0]]


@pytest.mark.parametrize("T,N,K,r", [(0, 64, 128, 4), (1, 64, 128, 4), (77, 136, 320, 13), (300, 520, 640, 100)])
def test_backward_into_given_buffers(T, N, K, r):
    q = Q()
    W, X, A, B, dY = inputs.layer_inputs(70, 0, 0, max(T, 1), N, K, r, device="cuda", b_std=0.05)
    X, dY = X[:T], dY[:T]
    qw = q.quantize_nf4(W)
    u = q.linear_fwd_save(X, qw, A, B, 1.5)[1] if T else torch.empty(16, dtype=torch.uint8, device="cuda")
    x8 = q.quantize_int8(X, group=128)
    want = q.linear_bwd_saved_int8(dY, x8, qw, A, B, 1.5, u)
    bufs = [guarded(T, K), guarded(r, K), guarded(N, r)]
    outs = tuple(v for _, v in bufs)
    got = q.linear_bwd_saved_int8(dY, x8, qw, A, B, 1.5, u, outs=outs)
    assert all(a is b for a, b in zip(got, outs))
    assert all(equal_bits(a, b) for a, b in zip(got, want))
    assert all((buf[v.shape[0]:] == 3).all() for buf, v in bufs)
    dx, dA, dB = outs
    for bad in ((dx, dA, dB[:-1]), (dx, dA.float(), dB), (dx, torch.empty(K, r, dtype=torch.bfloat16, device="cuda").t(), dB),
                (dx, dA.cpu(), dB)):
        with pytest.raises(ValueError):
            q.linear_bwd_saved_int8(dY, x8, qw, A, B, 1.5, u, outs=bad)
    q.get_error()


def test_captured_into_given_buffers():
    """A captured backward writes the caller's buffers at every replay, from the
    gradient and the checkpoint as they are then."""
    q = Q()
    T, N, K, r = 200, 264, 320, 16
    W, X, A, B, dY = inputs.layer_inputs(71, 0, 0, T, N, K, r, device="cuda", b_std=0.05)
    qw = q.quantize_nf4(W)
    _, u = q.linear_fwd_save(X, qw, A, B, 2.0)
    x8 = q.quantize_int8(X, group=128)
    outs = tuple(torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((T, K), (r, K), (N, r)))
    q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u, outs=outs)
    for k in range(3):
        X.copy_(inputs.normal_bf16((T, K), 1.0, 80 + k, "cuda"))
        dY.copy_(inputs.normal_bf16((T, N), 1.0, 90 + k, "cuda"))
        q.quantize_int8_into(X, x8)
        want = q.linear_bwd_saved_int8(dY, x8, qw, A, B, 2.0, u)
        g.replay()
        assert all(equal_bits(a, b) for a, b in zip(outs, want))
    q.get_error()
    del g


def test_one_checkpoint_for_several_projections_and_streams():
    """Projections of different widths share one checkpoint, each backward on a
    stream of its own at the same time."""
    q = Q()
    T, K, r = 333, 640, 16
    X = inputs.normal_bf16((T, K), 1.0, 5, "cuda")
    x8 = q.quantize_int8(X, group=128)
    layers = []
    for i, N in enumerate((64, 264, 1024)):
        W, _, A, B, dY = inputs.layer_inputs(72 + i, 0, 0, T, N, K, r, device="cuda", b_std=0.05)
        qw = q.quantize_nf4(W)
        layers.append((dY, x8, qw, A, B, 2.0, q.linear_fwd_save(X, qw, A, B, 2.0)[1]))
    want = [q.linear_bwd_saved_int8(*a) for a in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for _ in range(10):
        for st, a in zip(streams, layers):
            with torch.cuda.stream(st):
                got.append(q.linear_bwd_saved_int8(*a))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(equal_bits(a, b) for a, b in zip(g, want[i % len(want)]))
    q.get_error()
