"""Plain 64-bit forms of the fused-epilogue and expert operators, and how far a kernel's output
may be from them. Shared by the tests of those operators; no part of the library.

Tolerance of one output y = act(p + bias) * mul + residual, with u = eps / 2 of the type, from
the arithmetic alone, worst case:
  * p is a sum of K products x w. One operand of each is rounded to 16 bits at most once (the
    dequantized weight in the tensor-core kernel, x * inv_s in the decode kernels), so a
    product is off by at most u |x w| (and 2^-25, half the smallest fp16 subnormal, times the
    other factor where the rounded one is subnormal); the fp32 accumulation adds at most
    (K / 16 + 32) 2^-23 of sum |x w| (one truncation per 16-wide step of the tensor cores, the
    adds across warps or slices).
  * the M = 1 decode kernel multiplies the codes offset by 1024 (128 in bf16) and takes the
    offset off afterwards: fp32 roundings relative to 1024 s |x| instead of |x w|, at most
    (128 / 16 + 8) 2^-23 of it.
  * |act'| <= 1.13 (gelu_tanh's and gelu's largest slope; silu's is 1.1), so act carries an
    error on by that much, and evaluating it in fp32 adds at most 16 roundings of its argument.
  * mul scales the error, and the last rounding adds u |y| (or half a subnormal step).
"""
import numpy as np
import torch

import oracle as O

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def act64(v, act):
    if act == "none":
        return v
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    t = torch.from_numpy(np.ascontiguousarray(v))
    if act == "silu":
        return (t * torch.sigmoid(t)).numpy()
    if act == "gelu":
        return (t * 0.5 * torch.erfc(-t * 0.5 ** 0.5)).numpy()
    assert act == "gelu_tanh"
    return (t * torch.sigmoid(2.0 * (2.0 / np.pi) ** 0.5 * (t + 0.044715 * t ** 3))).numpy()


def packed(rng, N, K, bits, scale=0.02):
    """A packed weight of random codes: (qweight uint32, scales fp16 [G, N], zeros u8 [G, N])."""
    codes = rng.integers(0, 2 ** bits, (N, K)).astype(np.uint32)
    G = K // 128
    sc = (scale * rng.uniform(0.5, 1.5, (G, N))).astype(np.float16)
    z = rng.integers(0, 2 ** bits, (G, N)).astype(np.uint8)
    return O.pack(codes, bits), sc, z


def linear64(X, qw, sc, z, N, K, bits, inv_s=None, bias=None, act="none", mul=None, residual=None,
             dtype=torch.float16):
    """(y, tolerance) of the fused product for one packed weight, from fp64 numpy inputs."""
    W = O.dequantize(O.unpack(qw, bits, K), sc, z, 128).astype(np.float64)
    x = X if inv_s is None else X * inv_s.astype(np.float64)[None, :]
    u = U[dtype]
    p = x @ W.T
    size = np.abs(x) @ np.abs(W).T
    step = np.repeat(np.abs(sc.astype(np.float64)).T, 128, axis=1)        # |scale| per weight
    tol = (u + (K / 16 + 32) * 2.0 ** -23) * size + TINY[dtype] * (np.abs(x).sum(1)[:, None] +
                                                                   np.abs(W).sum(1)[None, :])
    if X.shape[0] == 1:
        base = 1024.0 if dtype == torch.float16 else 128.0
        tol += 16 * 2.0 ** -23 * 16 * base * (np.abs(x) @ step.T)
    v = p if bias is None else p + bias[None, :]
    y = act64(v, act)
    if act != "none":
        tol = 1.13 * tol
    tol = tol + 16 * 2.0 ** -24 * np.abs(v)
    if mul is not None:
        y, tol = y * mul, tol * np.abs(mul)
    if residual is not None:
        y = y + residual
    return y, tol + u * (np.abs(y) + tol) + TINY[dtype] + 2.0 ** -23 * np.abs(y)


def assert_within(got, want, tol, what=""):
    got = f64(got)
    off = np.abs(got - want) - tol
    assert np.isfinite(got).all(), what
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 0, (what, i, got[i], want[i], tol[i])
    # as a whole: the roundings are independent, so the norm of the error is far below the sum
    # of the bounds; three roundings of u each are the most any path makes
    norm = np.linalg.norm(want)
    return np.linalg.norm(got - want) / norm if norm else 0.0
