"""The fused-epilogue and expert entry points with every output and workspace between sentinel
bytes, on the release build and on the bounds-checking debug build: no byte outside what the
call may write changes, and the debug build reports no index outside the shapes."""
import numpy as np
import pytest
import torch

import oracle as O
from expert_reference import assert_within, linear64, packed
from test_gpu_guards import Guarded, L, P, _no_violation, _ok, _stream  # noqa: F401 (L: fixture)

pytestmark = pytest.mark.gpu

F16 = torch.float16


def half(rng, *shape):
    return (rng.standard_normal(shape) * 0.7).astype(np.float16)


# M, N, K, bits, inv: the decode, the streaming (N odd; long K) and the tensor-core kernel (K
# split; several tiles; 3 bits)
@pytest.mark.parametrize("M,N,K,bits,inv", [
    (1, 48, 256, 4, True), (7, 112, 384, 3, False), (3, 37, 2176, 4, True), (8, 70, 256, 3, True),
    (6, 4400, 7808, 4, False), (12, 41, 384, 4, True), (33, 130, 4096, 4, True),
    (70, 258, 640, 3, False), (300, 200, 384, 4, True)])
def test_epilogue_guarded(L, M, N, K, bits, inv):  # noqa: F811
    rng = np.random.default_rng([M, N, K])
    qw, sc, z = packed(rng, N, K, bits)
    X, mul, res, bias = half(rng, M, K), half(rng, M, N), half(rng, M, N), half(rng, N)
    s = rng.uniform(0.5, 2.0, K).astype(np.float32)
    g = {k: Guarded(v.nbytes, v) for k, v in
         dict(x=X, q=qw, sc=sc, z=z, mul=mul, res=res, bias=bias, s=s).items()}
    y = Guarded(2 * M * N)
    need = L.awq_gemm_epilogue_workspace_size(M, N, K, bits, inv, 0)
    ws = Guarded(need) if need else None
    for flags in (0, 1):
        _ok(L, L.awq_gemm_w4a16_epilogue(
            g["x"].ptr, M, g["q"].ptr, g["sc"].ptr, g["z"].ptr, N, K, bits, 128,
            g["s"].ptr if inv else None, g["bias"].ptr, 2, g["mul"].ptr, g["res"].ptr, flags, y.ptr,
            ws.ptr if ws else None, ws.n if ws else 0, _stream()))
        _no_violation(L)
        y.assert_intact("Y")
        if ws:
            ws.assert_intact("workspace")
        want, tol = linear64(X.astype(np.float64), qw, sc, z, N, K, bits, s if inv else None,
                             bias.astype(np.float64), "silu", mul.astype(np.float64),
                             res.astype(np.float64), F16)
        assert_within(torch.from_numpy(y.host(np.float16).reshape(M, N).copy()), want, tol)


@pytest.mark.parametrize("counts,N,K,bits", [
    ([2, 0, 3, 1], 37, 384, 4), ([0, 8, 9, 0], 144, 256, 3), ([40, 1, 0, 7], 130, 640, 4),
    ([33, 70, 0], 77, 256, 3), ([200, 150, 300], 40, 128, 4)])
def test_grouped_guarded(L, counts, N, K, bits):  # noqa: F811
    rng = np.random.default_rng([N, K, len(counts)])
    E = len(counts)
    off = np.concatenate([[1], 1 + np.cumsum(counts)]).astype(np.int32)   # a row before, two behind
    T = int(off[-1]) + 2
    ws_ = [packed(rng, N, K, bits) for _ in range(E)]
    qw, sc, z = (np.stack([w[i] for w in ws_]) for i in range(3))
    X, s = half(rng, T, K), rng.uniform(0.5, 2.0, (E, K)).astype(np.float32)
    g = {k: Guarded(v.nbytes, v) for k, v in dict(x=X, o=off, q=qw, sc=sc, z=z, s=s).items()}
    y = Guarded(2 * T * N, np.full(T * N, 7, np.float16))
    need = L.awq_gemm_grouped_workspace_size(T, E, N, K, bits, 1, 0)
    ws = Guarded(need) if need else None
    _ok(L, L.awq_gemm_w4a16_grouped(g["x"].ptr, T, g["o"].ptr, E, g["q"].ptr, g["sc"].ptr, g["z"].ptr,
                                    N, K, bits, 128, g["s"].ptr, None, 0, None, None, 0, y.ptr,
                                    ws.ptr if ws else None, ws.n if ws else 0, _stream()))
    _no_violation(L)
    y.assert_intact("Y")
    if ws:
        ws.assert_intact("workspace")
    got = y.host(np.float16).reshape(T, N)
    assert (got[:1] == 7).all() and (got[off[-1]:] == 7).all()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            want, tol = linear64(X[a:b].astype(np.float64), *ws_[e], N, K, bits, s[e], dtype=F16)
            assert_within(torch.from_numpy(got[a:b].copy()), want, tol)


@pytest.mark.parametrize("counts,K", [([5, 0, 90, 1], 264), ([1], 8), ([700, 3, 0, 0, 40], 520)])
def test_stats_and_silu_guarded(L, counts, K):  # noqa: F811
    rng = np.random.default_rng([K, len(counts)])
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(off[-1])
    X = half(rng, T, K)
    x, o, out = Guarded(X.nbytes, X), Guarded(off.nbytes, off), Guarded(4 * E * K)
    ws = Guarded(L.awq_act_stats_grouped_workspace_size(T, E, K))
    _ok(L, L.awq_act_stats_grouped(x.ptr, T, o.ptr, E, K, out.ptr, ws.ptr, ws.n, _stream()))
    _no_violation(L)
    out.assert_intact("s_x")
    ws.assert_intact("workspace")
    got = out.host(np.float32).reshape(E, K)
    for e in range(E):
        rows = X[off[e]:off[e + 1]]
        np.testing.assert_array_equal(got[e], O.act_stats(rows) if len(rows) else np.zeros(K, np.float32))
    I, K2 = 50, 128
    X2, Wg, Wu = half(rng, T, K2), half(rng, E, I, K2), half(rng, E, I, K2)
    x2, wg, wu, h = (Guarded(v.nbytes, v) for v in (X2, Wg, Wu, np.full((T, I), 7, np.float16)))
    _ok(L, L.awq_silu_mul_gemm_grouped(x2.ptr, T, o.ptr, E, wg.ptr, wu.ptr, I, K2, h.ptr, _stream()))
    _no_violation(L)
    h.assert_intact("H")
    got = h.host(np.float16).reshape(T, I).astype(np.float64)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            want = O.silu_mul(X2[a:b], Wg[e], Wu[e])
            # fp16's rounding, and fp32 accumulation of K2 / 16 steps in each factor
            assert np.linalg.norm(got[a:b] - want) <= 2.0 ** -11 * 2 * np.linalg.norm(want) + 1e-6
