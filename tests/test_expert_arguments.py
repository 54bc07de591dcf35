"""Refusals of the fused-epilogue and expert entry points, on the host before any launch (the
pointers below are never dereferenced), and the binding's checks."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, FAKE, ODD = 0, P(1 << 20), P((1 << 20) + 2)
INVALID, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def L():
    from weight_only_int4_stats_b200 import build
    build.build()
    import weight_only_int4_stats_b200 as awq
    return awq.lib()


def epilogue(L, M=4, N=16, K=128, bits=4, group=128, inv=None, bias=None, act=0, mul=None, res=None,
             flags=0, x=FAKE, qw=FAKE, sc=FAKE, z=FAKE, y=FAKE, ws=FAKE, n=1 << 40):
    return L.awq_gemm_w4a16_epilogue(x, M, qw, sc, z, N, K, bits, group, inv, bias, act, mul, res,
                                     flags, y, ws, n, None)


def grouped(L, T=4, E=2, N=16, K=128, bits=4, group=128, inv=None, bias=None, act=0, mul=None,
            res=None, flags=0, x=FAKE, off=FAKE, qw=FAKE, sc=FAKE, z=FAKE, y=FAKE, ws=FAKE, n=1 << 40):
    return L.awq_gemm_w4a16_grouped(x, T, off, E, qw, sc, z, N, K, bits, group, inv, bias, act, mul,
                                    res, flags, y, ws, n, None)


@pytest.mark.parametrize("call", [epilogue, grouped])
@pytest.mark.parametrize("bad", [
    dict(K=0), dict(K=200), dict(K=-128), dict(N=-1), dict(N=1 << 31), dict(bits=2), dict(bits=8),
    dict(group=64), dict(act=-1), dict(act=5), dict(flags=4), dict(flags=1 << 31), dict(x=None),
    dict(qw=None), dict(sc=None), dict(z=None), dict(y=None), dict(x=ODD), dict(qw=ODD), dict(sc=ODD),
    dict(z=ODD), dict(y=ODD), dict(inv=ODD), dict(bias=ODD), dict(mul=ODD), dict(res=ODD)])
def test_products_refuse(L, call, bad):
    assert call(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(E=-1),
                                 dict(off=None), dict(off=ODD), dict(E=1024, N=1 << 21),
                                 dict(E=1024, K=1 << 28)])
def test_grouped_product_refuses(L, bad):
    assert grouped(L, **bad) == INVALID


def test_nothing_to_do(L):
    assert epilogue(L, M=0) == OK and epilogue(L, N=0) == OK
    assert grouped(L, T=0) == OK and grouped(L, N=0) == OK
    assert L.awq_silu_mul_gemm_grouped(FAKE, 0, FAKE, 2, FAKE, FAKE, 8, 128, FAKE, None) == OK
    assert L.awq_silu_mul_gemm_grouped(FAKE, 4, FAKE, 2, FAKE, FAKE, 0, 128, FAKE, None) == OK
    assert L.awq_act_stats_grouped(FAKE, 4, FAKE, 2, 0, FAKE, None, 0, None) == OK
    # bad arguments are refused all the same
    assert epilogue(L, M=0, act=9) == INVALID and grouped(L, T=0, E=0) == INVALID


def test_workspace_missing_or_small(L):
    M, N, K = 64, 4096, 4096
    need = L.awq_gemm_epilogue_workspace_size(M, N, K, 4, 0, 0)
    if need:
        assert epilogue(L, M=M, N=N, K=K, ws=None, n=0) == WORKSPACE
        assert epilogue(L, M=M, N=N, K=K, n=need - 1) == WORKSPACE
        assert epilogue(L, M=M, N=N, K=K, ws=ODD, n=need) == WORKSPACE
    need = L.awq_act_stats_grouped_workspace_size(1000, 4, 256)
    assert need > 0
    for ws, n in ((None, 0), (FAKE, need - 1), (ODD, need)):
        assert L.awq_act_stats_grouped(FAKE, 1000, FAKE, 4, 256, FAKE, ws, n, None) == WORKSPACE


@pytest.mark.parametrize("T,E,K,x,off,out", [
    (-1, 2, 8, FAKE, FAKE, FAKE), (4, 0, 8, FAKE, FAKE, FAKE), (4, 1025, 8, FAKE, FAKE, FAKE),
    (4, 2, 12, FAKE, FAKE, FAKE), (4, 2, -8, FAKE, FAKE, FAKE), (4, 2, 8, None, FAKE, FAKE),
    (4, 2, 8, FAKE, None, FAKE), (4, 2, 8, FAKE, FAKE, None), (4, 2, 8, ODD, FAKE, FAKE),
    (4, 2, 8, FAKE, ODD, FAKE), (4, 2, 8, FAKE, FAKE, ODD)])
def test_stats_refuse(L, T, E, K, x, off, out):
    assert L.awq_act_stats_grouped(x, T, off, E, K, out, FAKE, 1 << 40, None) == INVALID


@pytest.mark.parametrize("T,E,I,K,x,off,g,u,h", [
    (-1, 2, 8, 128, FAKE, FAKE, FAKE, FAKE, FAKE), (4, 0, 8, 128, FAKE, FAKE, FAKE, FAKE, FAKE),
    (4, 1025, 8, 128, FAKE, FAKE, FAKE, FAKE, FAKE), (4, 2, 8, 64, FAKE, FAKE, FAKE, FAKE, FAKE),
    (4, 2, 8, 0, FAKE, FAKE, FAKE, FAKE, FAKE), (4, 2, -1, 128, FAKE, FAKE, FAKE, FAKE, FAKE),
    (4, 1024, 1 << 21, 128, FAKE, FAKE, FAKE, FAKE, FAKE),
    (4, 2, 8, 128, None, FAKE, FAKE, FAKE, FAKE), (4, 2, 8, 128, FAKE, None, FAKE, FAKE, FAKE),
    (4, 2, 8, 128, FAKE, FAKE, ODD, FAKE, FAKE), (4, 2, 8, 128, FAKE, FAKE, FAKE, None, FAKE),
    (4, 2, 8, 128, FAKE, FAKE, FAKE, FAKE, ODD)])
def test_silu_mul_refuses(L, T, E, I, K, x, off, g, u, h):
    assert L.awq_silu_mul_gemm_grouped(x, T, off, E, g, u, I, K, h, None) == INVALID


def test_binding_refuses_what_is_no_cuda_tensor_of_the_shape():
    import weight_only_int4_stats_b200 as awq
    X = torch.zeros(4, 128, dtype=torch.float16)
    qw, sc = torch.zeros(16, 16, dtype=torch.int32), torch.zeros(1, 16, dtype=torch.float16)
    z, off = torch.zeros(1, 16, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    good = dict(X=X, qweight=qw, scales=sc, zeros=z, N=16, K=128)
    with pytest.raises(TypeError, match="CUDA"):
        awq.awq_gemm_w4a16_epilogue(**good)
    with pytest.raises(ValueError, match="act"):
        awq.awq_gemm_w4a16_epilogue(**good, act="tanh")
    for name, t in (("X", X.float()), ("X", X.t()), ("X", X[:, ::2]), ("qweight", qw[:8]),
                    ("qweight", qw.long()), ("scales", sc.float()), ("zeros", z[:, :8]),
                    ("bias", torch.zeros(16)), ("bias", torch.zeros(8, dtype=torch.float16)),
                    ("mul", torch.zeros(4, 32, dtype=torch.float16)[:, ::2]),
                    ("residual", torch.zeros(3, 16, dtype=torch.float16)),
                    ("inv_s", torch.zeros(128, dtype=torch.float16)),
                    ("out", torch.zeros(4, 16, dtype=torch.bfloat16))):
        with pytest.raises(TypeError, match=name):
            awq.awq_gemm_w4a16_epilogue(**{**good, name: t})
    two = dict(X=X, offsets=off, qweight=qw.expand(2, -1, -1).contiguous(),
               scales=sc.expand(2, -1, -1).contiguous(), zeros=z.expand(2, -1, -1).contiguous(),
               N=16, K=128)
    with pytest.raises(TypeError, match="CUDA"):
        awq.awq_gemm_w4a16_grouped(**two)
    for name, t in (("offsets", off.long()), ("qweight", qw), ("scales", sc),
                    ("bias", torch.zeros(16, dtype=torch.float16))):
        with pytest.raises(TypeError, match=name):
            awq.awq_gemm_w4a16_grouped(**{**two, name: t})
    with pytest.raises(TypeError, match="offsets"):
        awq.awq_act_stats_grouped(X, off.long())
    W = torch.zeros(2, 16, 128, dtype=torch.float16)
    with pytest.raises(TypeError, match="W_up"):
        awq.awq_silu_mul_gemm_grouped(X, off, W, W[:1])
    with pytest.raises(TypeError, match="CUDA"):
        awq.awq_silu_mul_gemm_grouped(X, off, W, W)
