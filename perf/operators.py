"""The 8-bit operators as they are measured: their cases, inputs, plain forms
and 64-bit values.

Three operators of the library, built on one format.  An int8 matrix holds for
each row (group 0) or for each 128 consecutive columns of a row (group 128)

    amax  = max |x| over the group
    scale = max(RN32(amax / 127), 2^-126),  inv = RN32(1 / scale)
    code  = the integer nearest to x * inv (the exact product), ties to even

and stands for code * scale.

  checkpoint   an activation written in 8 bits and read back as BF16
  linear       y = xq wq^T with x quantized per token, w per output channel
  backward     the NF4 layer's backward whose activation is an 8-bit
               checkpoint: dX = dY W' + dU A, dU = s dY B,
               dA = dU^T xq, dB = dY^T U, U = s X A^T saved by the forward

`own` selects the library's kernels; without it every operator is computed in
elementary torch operations in 32 bits (64 for the borders of the rounding).
"""
import math
import statistics

import torch

own = False

DEV = "cuda"
GROUP = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _ckpt(name, T, K, group):
    return {"name": name, "op": "checkpoint", "T": T, "K": K, "group": group}


def _lin(name, T, N, K):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K}


def _bwd(name, T, N, K, r, s, group):
    return {"name": name, "op": "backward", "T": T, "N": N, "K": K, "r": r, "s": s, "group": group}


def listed():
    return [
        # the tiny layer's input: nothing but launch latency
        _ckpt("ckpt_16x512_g128", 16, 512, 128),
        # one token batch of the 8B block's hidden state, kept for the backward
        _ckpt("ckpt_4096x4096_g128", 4096, 4096, 128),
        # the 8B down projection's input, an odd token count, one scale a row (as the int8 product takes it)
        _ckpt("ckpt_4095x14336_row", 4095, 14336, 0),
        # one token through the 8B k / v projection: the smallest serving call
        _lin("lin_T1_1024x4096", 1, 1024, 4096),
        # a small decode batch through the 8B gate / up projection
        _lin("lin_T16_14336x4096", 16, 14336, 4096),
        # an odd batch between decode and prefill, long contraction (8B down)
        _lin("lin_T101_4096x14336", 101, 4096, 14336),
        # a ragged prefill on a 65B-shaped hidden projection
        _lin("lin_T1531_8192x8192", 1531, 8192, 8192),
        # a full 8B gate / up prefill: the largest product
        _lin("lin_T4096_14336x4096", 4096, 14336, 4096),
        # the tiny layer's training step
        _bwd("bwd_T16_512x512_r8_g128", 16, 512, 512, 8, 2.0, 128),
        # four short sequences of the 65B-shaped hidden projection, rank 64, per-row scales
        _bwd("bwd_T2048_8192x8192_r64_row", 2048, 8192, 8192, 64, 0.25, 0),
        # an odd token count on the 8B down projection (a wide checkpoint)
        _bwd("bwd_T1003_4096x14336_r16_g128", 1003, 4096, 14336, 16, 2.0, 128),
        # a full training batch of the 8B q / o projection
        _bwd("bwd_T4096_4096x4096_r16_g128", 4096, 4096, 4096, 16, 2.0, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(("checkpoint", "linear", "linear", "backward"))
    while True:
        if op == "checkpoint":
            c = {"op": op, "T": _log(rng, 1, 16384), "K": _mult(rng, 64, 22016, 16), "group": rng.choice((0, 128))}
            if c["T"] * c["K"] <= 4095 * 14336:
                return c
        elif op == "linear":
            c = {"op": op, "T": _log(rng, 1, 8192), "N": _mult(rng, 64, 22016, 8), "K": _mult(rng, 64, 22016, 16)}
            if c["T"] * c["N"] * c["K"] <= 4096 * 14336 * 4096 and c["N"] * c["K"] <= 8192 * 22016:
                return c
        else:
            c = {"op": op, "T": _log(rng, 1, 4096), "N": _mult(rng, 64, 14336, 8), "K": _mult(rng, 64, 14336, 64),
                 "r": rng.choice((1, 4, 8, 13, 16, 32, 64, 128)), "s": rng.choice((0.25, 1.0, 2.0)),
                 "group": rng.choice((0, 128))}
            if c["T"] * c["N"] * c["K"] <= 2048 * 8192 * 8192:
                return c


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "checkpoint":
        # BF16 in, BF16 out, and the codes and scales between (written, then read)
        groups = 1 if case["group"] == 0 else -(-K // case["group"])
        return {"bytes": 2 * T * K + 2 * (T * K + 4 * T * groups) + 2 * T * K, "flops": 2 * T * K}
    N = case["N"]
    if case["op"] == "linear":
        return {"bytes": 2 * T * K + N * K + 4 * N + 2 * T * N, "flops": 2 * T * N * K}
    r = case["r"]
    groups = 1 if case["group"] == 0 else -(-K // case["group"])
    nf4 = N * K // 2 + N * K // 64 + 4 * (-(-(N * K) // 16384))
    return {"bytes": 2 * T * N + T * K + 4 * T * groups + nf4 + 2 * r * (N + K) + 4 * r * T + 2 * T * K + 2 * r * (N + K),
            "flops": 2 * T * N * K + 2 * T * r * (2 * N + 2 * K)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(shape, std, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _activation(T, K, g):
    """Activations as a decoder layer has them: unit normal, one channel in 256
    twenty times larger (the outlier channels that per-row scales feel)."""
    x = _randn((T, K), 1.0, g)
    gain = torch.where(torch.rand((K,), generator=g, device=DEV) < 1.0 / 256, 20.0, 1.0)
    return (x * gain).to(torch.bfloat16)


def _make(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * seed + 17)
    T, K = case["T"], case["K"]
    d = {"x": _activation(T, K, g)}
    if case["op"] == "checkpoint":
        return d
    N = case["N"]
    d["w"] = _randn((N, K), 0.02, g).to(torch.bfloat16)
    if case["op"] == "linear":
        return d
    r = case["r"]
    d["A"] = _randn((r, K), 1.0 / math.sqrt(K), g).to(torch.bfloat16)
    d["B"] = _randn((N, r), 0.01, g).to(torch.bfloat16)
    d["dy"] = _randn((T, N), 1.0, g).to(torch.bfloat16)
    return d


def _nf4_levels():
    q = [statistics.NormalDist().inv_cdf((i - 0.5) / 16) for i in range(9, 17)]
    pos = [v / q[-1] for v in q]
    return torch.tensor([-v for v in reversed(pos)] + pos, dtype=torch.float32)


def _nf4(w):
    """A frozen NF4 weight of w: packed codes, E4M3 scale bytes, second-level scales, levels."""
    levels = _nf4_levels().to(w.device)
    blocks = w.float().reshape(-1, 64)
    c1 = blocks.abs().amax(1)
    n = c1.numel()
    groups = -(-n // 256)
    padded = torch.zeros(groups * 256, device=w.device)
    padded[:n] = c1
    c2 = padded.reshape(groups, 256).amax(1) / 448.0
    f8 = (c1 / c2.repeat_interleave(256)[:n]).to(torch.float8_e4m3fn)
    mid = (levels[1:] + levels[:-1]) / 2
    code = torch.bucketize(blocks / c1[:, None], mid, right=True).to(torch.uint8).reshape(-1)
    return (code[0::2] | (code[1::2] << 4)).contiguous(), f8.view(torch.uint8), c2, levels


def _saved_u(x, A, s, T, r):
    """U = s x A^T as the forward saves it: two BF16 planes U^T [r, ceil8(T)], hi then lo."""
    u = s * (x.float() @ A.float().t())
    hi = u.to(torch.bfloat16)
    lo = (u - hi.float()).to(torch.bfloat16)
    Tp = -(-T // 8) * 8
    plane = -(-(r * Tp * 2) // 256) * 256
    buf = torch.zeros(2 * plane, dtype=torch.uint8, device=x.device)
    for i, p in enumerate((hi, lo)):
        v = buf[i * plane:i * plane + r * Tp * 2].view(torch.bfloat16).view(r, Tp)
        v[:, :T] = p.t()
    return buf


def _u_planes(buf, T, r):
    Tp = -(-T // 8) * 8
    plane = buf.numel() // 2
    hi, lo = (buf[i * plane:i * plane + r * Tp * 2].view(torch.bfloat16).view(r, Tp)[:, :T] for i in (0, 1))
    return hi, lo


def prepare(case, seed):
    d = _make(case, seed)
    op = case["op"]
    st = {"op": op, "group": case.get("group", 0)}
    if own:
        import bit_nf4_quantized_20_b200 as q
        st["q"] = q
    if op == "checkpoint":
        st["x"] = d["x"]
    elif op == "linear":
        # the weight is quantized once, per output channel; activations arrive per call
        st["x"] = d["x"]
        if own:
            st["w8"] = st["q"].quantize_int8(d["w"])
        else:
            st["w8"] = _plain_quantize(d["w"], 0)
    else:
        codes, scales, c2, levels = _nf4(d["w"])
        st.update(A=d["A"], B=d["B"], dy=d["dy"], s=case["s"], N=case["N"], K=case["K"], T=case["T"], r=case["r"])
        st["u"] = _saved_u(d["x"], d["A"], case["s"], case["T"], case["r"])
        if own:
            q = st["q"]
            st["qw"] = q.QuantizedNF4(codes, scales, c2, case["N"], case["K"], [float(v) for v in levels.tolist()])
            st["x8"] = q.quantize_int8(d["x"], group=case["group"])
        else:
            st["qw"] = (codes, scales, c2, levels)
            st["x8"] = _plain_quantize(d["x"], case["group"])
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_quantize(x, group):
    """codes as FP32 integers [R, C], scales FP32 [R, groups]."""
    R, C = x.shape
    g = C if group == 0 else group
    n = -(-C // g)
    xf = x.float()
    if n * g != C:
        xf = torch.nn.functional.pad(xf, (0, n * g - C))
    xg = xf.reshape(R, n, g)
    scale = torch.clamp(xg.abs().amax(2) / 127.0, min=2.0 ** -126)
    inv = 1.0 / scale
    # the border of the rounding needs the exact product: 8 x 24 bits fit in 64
    q = torch.round(xg.double() * inv.double()[:, :, None]).float()
    return q.reshape(R, n * g)[:, :C], scale


def _plain_value(q, scale, group):
    """FP32 values code * scale."""
    R, C = q.shape
    g = C if group == 0 else group
    return q * scale.repeat_interleave(g, 1)[:, :C]


def _plain_nf4(qw, N, K):
    codes, scales, c2, levels = qw
    c = torch.stack((codes & 15, codes >> 4), 1).reshape(-1).long()
    sb = scales.view(torch.float8_e4m3fn).float() * c2.repeat_interleave(256)[:scales.numel()]
    # W' is BF16 by definition of the layer
    return (levels[c].reshape(-1, 64) * sb[:, None]).to(torch.bfloat16).float().reshape(N, K)


def run(state):
    op = state["op"]
    if own:
        q = state["q"]
        if op == "checkpoint":
            return q.dequantize_int8(q.quantize_int8(state["x"], group=state["group"]))
        if op == "linear":
            return q.linear_int8(state["x"], state["w8"])
        return q.linear_bwd_saved_int8(state["dy"], state["x8"], state["qw"], state["A"], state["B"], state["s"],
                                       state["u"])
    if op == "checkpoint":
        c, s = _plain_quantize(state["x"], state["group"])
        return _plain_value(c, s, state["group"]).to(torch.bfloat16)
    if op == "linear":
        xq, sx = _plain_quantize(state["x"], 0)
        wq, sw = state["w8"]
        return ((xq @ wq.t()) * sx * sw.t()).to(torch.bfloat16)
    dy, A, B = state["dy"].float(), state["A"].float(), state["B"].float()
    w = _plain_nf4(state["qw"], state["N"], state["K"])
    hi, lo = _u_planes(state["u"], state["T"], state["r"])
    du = state["s"] * (dy @ B)
    dx = dy @ w + du @ A
    dA = du.t() @ _plain_value(*state["x8"], state["group"])
    dB = dy.t() @ (hi.float() + lo.float()).t()
    return dx.to(torch.bfloat16), dA.to(torch.bfloat16), dB.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# 64-bit values, from the definitions
# ---------------------------------------------------------------------------
def _exact_int8(x, group):
    """The values an int8 matrix of x stands for, in 64 bits, group by group."""
    x64 = x.double()
    R, C = x64.shape
    g = group if group else C
    out = torch.empty_like(x64)
    for c0 in range(0, C, g):
        blk = x64[:, c0:c0 + g]
        top = blk.abs().max(1, keepdim=True).values
        # scale and its inverse are FP32 numbers by definition
        scale = torch.maximum((top / 127).float().double(), torch.full_like(top, 2.0 ** -126))
        p = blk * (1 / scale).float().double()
        lower = torch.floor(p)
        frac = p - lower
        up = (frac > 0.5) | ((frac == 0.5) & (torch.remainder(lower, 2) == 1))
        out[:, c0:c0 + g] = (lower + up.double()) * scale
    return out


def exact(case, seed):
    d = _make(case, seed)
    if case["op"] == "checkpoint":
        return _exact_int8(d["x"], case["group"])
    if case["op"] == "linear":
        return torch.einsum("tk,nk->tn", _exact_int8(d["x"], 0), _exact_int8(d["w"], 0))
    T, N, K, r, s = (case[k] for k in ("T", "N", "K", "r", "s"))
    codes, scales, c2, levels = _nf4(d["w"])
    blk = torch.empty(N * K // 64, 64, dtype=torch.float64, device=DEV)
    lv = levels.double()
    b = codes.reshape(-1, 32)
    # block scale and W' are rounded to FP32 and BF16 by the layer's definition
    sb = (scales.view(torch.float8_e4m3fn).double() *
          c2.double()[torch.arange(scales.numel(), device=DEV) // 256]).float().double()
    for nib in (0, 1):
        v = lv[((b >> (4 * nib)) & 15).long()] * sb[:, None]
        blk[:, nib::2] = v.float().to(torch.bfloat16).double()
    w = blk.reshape(N, K)
    hi, lo = _u_planes(_saved_u(d["x"], d["A"], s, T, r), T, r)
    dy = d["dy"].double()
    du = torch.einsum("tn,nj->tj", dy, d["B"].double()) * s
    dx = torch.einsum("tn,nk->tk", dy, w) + torch.einsum("tj,jk->tk", du, d["A"].double())
    dA = torch.einsum("tj,tk->jk", du, _exact_int8(d["x"], case["group"]))
    dB = torch.einsum("tn,jt->nj", dy, hi.double() + lo.double())
    return dx, dA, dB
