"""The products with a fused epilogue and the expert operators where their rules meet: inputs that
the kernel just before writes, the ends of the value ranges, each path's own precision."""
import numpy as np
import pytest
import torch

import oracle as O
from expert_reference import TINY, U, assert_within, f64
from test_gpu_experts import (BF16, F16, Layer, awq, cu, dense, grouped, offsets_of,  # noqa: F401
                              silu_mul_tolerance, tokens)   # (awq: fixture)

pytestmark = pytest.mark.gpu


# M, N, K, bits, dtype: the streaming kernel, then the tensor-core kernel with and without slices of
# K, at each size of its token tile
@pytest.mark.parametrize("M,N,K,bits,dtype", [
    (1, 512, 2048, 4, F16), (3, 512, 2048, 3, F16), (8, 512, 2048, 4, BF16), (6, 512, 2048, 4, F16),
    (30, 512, 4096, 3, F16), (64, 4096, 1024, 4, F16), (77, 512, 11008, 4, F16),
    (128, 512, 1024, 3, F16), (300, 1024, 1024, 4, F16), (40, 512, 1024, 4, BF16)])
def test_inv_s_from_the_kernel_just_before(awq, M, N, K, bits, dtype):  # noqa: F811
    """weights_ready speaks of the packed weights alone: factors that the preceding kernel is
    still writing when this call's kernels start (the statistics let the next launch start before
    they store) are read after it has stored them."""
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, 1, N, K, bits, dtype)
    X = tokens(rng, M, K, dtype)
    rows = tokens(rng, 2048, K, F16)
    sides, off = (rows, rows * 4), cu(np.array([0, 2048], np.int32))
    inv = torch.empty(1, K, device="cuda")

    def product():
        return awq.awq_gemm_w4a16_epilogue(X, layer.qw[0], layer.sc[0], layer.z[0], N, K, bits,
                                           inv_s=inv[0], weights_ready=True)

    want = []
    for side in sides:
        awq.awq_act_stats_grouped(side, off, out=inv)
        torch.cuda.synchronize()
        want.append(product())
        torch.cuda.synchronize()
    assert torch.allclose(want[1].float(), 4 * want[0].float(), rtol=2.0 ** -6, atol=1e-2)
    assert not torch.equal(want[0], want[1])
    for turn in range(24):
        awq.awq_act_stats_grouped(sides[turn % 2], off, out=inv)
        y = product()
        assert torch.equal(y, want[turn % 2]), turn
    awq.awq_check_error()


# the streaming kernel (one and two rows a token), the tensor-core kernel with and without slices of K
@pytest.mark.parametrize("M,N,K,bits,inv", [(3, 144, 1024, 4, True), (8, 37, 384, 3, True),
                                            (5, 4400, 7808, 4, False), (40, 130, 512, 4, True),
                                            (77, 512, 4096, 4, False), (300, 257, 256, 3, True)])
@pytest.mark.parametrize("e", [118, 70, -70, -112])
def test_bf16_rows_at_the_ends_of_the_range(awq, M, N, K, bits, inv, e):  # noqa: F811
    """Rows times 2^e give outputs times 2^e: every step is a product or a sum, and none leaves the
    range of fp32 on the way (|P| < 2^9 here). Outputs that become subnormal are off by a step."""
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, 1, N, K, bits, BF16, inv)
    X = tokens(rng, M, K, BF16).clamp(-8, 8)
    base = dense(awq, layer, X).float()
    assert base.abs().max() < 512
    y = dense(awq, layer, X * 2.0 ** e).float()
    awq.awq_check_error()
    back = y.double() * 2.0 ** -e   # (a Python power: exact)
    step = 2.0 ** (-133 - e)   # of bf16's subnormals, seen from the base's scale
    assert ((back - base.double()).abs() <= (step if e < -100 else 0)).all()


def test_a_row_of_each_size_beside_the_others(awq):  # noqa: F811
    """Each row has its own power of two: a tiny and a huge row do not notice one another."""
    rng = np.random.default_rng(1)
    layer = Layer(rng, 1, 96, 256, 4, BF16)
    for M in (7, 50):
        X = tokens(rng, M, 256, BF16).clamp(-8, 8)
        X[-1] = 0
        e = np.linspace(-100, 118, M).round().astype(int)   # (powers of two by ldexp: exact)
        up, down = (torch.from_numpy(np.ldexp(1.0, k)[:, None]).cuda() for k in (e, -e))
        y = dense(awq, layer, (X.double() * up).to(BF16))
        want = dense(awq, layer, X)
        assert torch.equal(y.double() * down, want.double())
        assert (y[-1] == 0).all()


def output_rounding_alone(layer, e, X):
    """(y, bound of one output, the norm that the rounding to y's type leaves) of expert e's product
    where nothing but the output is rounded to 16 bits: codes, scales, zero points, x and x * inv_s
    enter in fp32 or exactly. The sums of q x and of z x are apart, so their fp32 roundings (one a
    16-wide step, the joins across groups and warps) go by |x| (q + z) scale; two-part x * inv_s
    adds 2^-22 of that."""
    qw, sc, z = layer.host[e]
    scale, zero = (np.repeat(v.astype(np.float64).T, 128, axis=1) for v in (sc, z))
    q = O.unpack(qw, layer.bits, layer.K).astype(np.float64)
    x = f64(X) if layer.inv is None else f64(X) * f64(layer.inv[e])[None, :]
    y = x @ ((q - zero) * scale).T
    size = np.abs(x) @ ((q + zero) * scale).T
    u, t = U[layer.dtype], layer.dtype
    tol = ((layer.K / 16 + 32) * 2.0 ** -23 + 2.0 ** -22) * size
    rounded = f64(torch.from_numpy(y).to(t))
    return y, tol + u * (np.abs(y) + tol) + TINY[t], np.linalg.norm(rounded - y)


def assert_rounded_once(got, want, tol, left):
    """Each output within its bound, and the whole within 2 % of the rounding's own norm: of the fp32
    roundings, each group's are some 2^-23 sqrt(128 * 8) |x| q scale, which over all groups is
    below a hundredth of fp16's 2^-11 of the output."""
    got = f64(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()
    norm = np.linalg.norm(got - want)
    assert norm <= 1.02 * left, (norm / left, norm / np.linalg.norm(want))


# the decode kernel (one token; more), then the streaming kernel (N odd; with inv_s: two parts a token)
@pytest.mark.parametrize("M,N,K,bits,dtype,inv", [
    (1, 4096, 4096, 4, F16, False), (1, 2048, 2176, 3, F16, False), (1, 1024, 384, 4, F16, False),
    (2, 2048, 4096, 4, F16, False), (8, 512, 1024, 3, F16, False), (1, 2001, 2176, 4, F16, False),
    (7, 333, 1024, 3, F16, False), (1, 4096, 4096, 4, F16, True), (3, 1001, 2176, 3, F16, True),
    (4, 512, 1024, 4, F16, True), (1, 4096, 4096, 4, BF16, False), (5, 1001, 1024, 4, BF16, False),
    (5, 1001, 2176, 4, F16, True), (6, 4096, 1024, 3, F16, True), (8, 512, 4096, 4, F16, True)])
@pytest.mark.parametrize("e", [0, -6, -12])
def test_few_rows_are_rounded_once(awq, M, N, K, bits, dtype, inv, e):  # noqa: F811
    """Up to 8 rows nothing is rounded to 16 bits before the output, small activations included."""
    rng = np.random.default_rng([M, N, K, bits])
    layer = Layer(rng, 1, N, K, bits, dtype, inv)
    X = tokens(rng, M, K, dtype) * 2.0 ** e
    y = dense(awq, layer, X)
    awq.awq_check_error()
    assert_rounded_once(y, *output_rounding_alone(layer, 0, X))


@pytest.mark.parametrize("counts,N,K,bits,dtype,inv", [
    ([1] * 24, 512, 1024, 4, F16, True), ([1] * 24, 500, 2176, 3, F16, False),
    ([0, 2, 0, 1, 5, 0, 1, 1], 512, 1024, 4, F16, False), ([8, 7, 9, 5], 300, 1024, 4, F16, True),
    ([30, 0, 1, 0], 512, 384, 3, F16, True), ([1, 0, 0, 2], 512, 2048, 4, BF16, False),
    ([4] * 12, 512, 1024, 3, BF16, False)])
def test_experts_of_few_rows_are_rounded_once(awq, counts, N, K, bits, dtype, inv):  # noqa: F811
    """Up to 8 rows an expert on average, however they are spread; the norm is taken over the
    whole call, so that experts of one row count in it."""
    rng = np.random.default_rng([N, K, len(counts)])
    layer = Layer(rng, len(counts), N, K, bits, dtype, inv)
    off = offsets_of(counts, 0)
    X = tokens(rng, int(off[-1]), K, dtype)
    y = grouped(awq, layer, X, off)
    awq.awq_check_error()
    each = [output_rounding_alone(layer, e, X[off[e]:off[e + 1]]) for e in range(len(counts))
            if counts[e]]
    want, tol = (np.concatenate([v[i] for v in each]) for i in range(2))
    assert_rounded_once(y, want, tol, np.sqrt(sum(v[2] ** 2 for v in each)))


@pytest.mark.parametrize("M,N,K,bits,dtype,inv", [
    (5, 67, 11008, 4, BF16, False), (3, 40, 14336, 3, F16, True), (40, 130, 8320, 4, BF16, True),
    (33, 64, 16512, 3, BF16, False)])
def test_rows_longer_than_the_preparation_keeps_in_registers(awq, M, N, K, bits, dtype, inv):  # noqa: F811
    """K past 8192: the preparation reads the rest of a row twice. Its last part alone holds the
    row's largest values in every second row, so both passes have to see it."""
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, 1, N, K, bits, dtype, inv)
    X = tokens(rng, M, K, dtype)
    X[::2, 8192:] *= 64
    y = dense(awq, layer, X)
    awq.awq_check_error()
    if M <= 8 and not (inv and dtype == BF16):
        assert_rounded_once(y, *output_rounding_alone(layer, 0, X))
    else:
        want, tol = layer.want(0, X)
        assert assert_within(y, want, tol) <= 3 * U[dtype]


@pytest.mark.parametrize("M", [2, 5, 8])
def test_product_without_parts_has_the_plain_products_bits(awq, M):  # noqa: F811
    """From 2 rows to 8 both are the decode kernel with exact q - z (bf16: from one row on)."""
    rng = np.random.default_rng(M)
    for dtype, bits, rows in ((F16, 4, M), (F16, 3, M), (BF16, 4, M), (BF16, 4, 1)):
        layer = Layer(rng, 1, 512, 1024, bits, dtype)
        X = tokens(rng, rows, 1024, dtype)
        plain = awq.awq_gemm_w4a16(X, layer.qw[0], layer.sc[0], layer.z[0], 512, 1024, bits)
        assert torch.equal(dense(awq, layer, X), plain)


@pytest.mark.parametrize("counts,I,K", [([3000, 0, 2900], 14336, 4096), ([2700, 40, 0, 1500], 2000, 1024)])
def test_silu_mul_of_many_rows_an_expert(awq, counts, I, K):  # noqa: F811
    """Token tiles of 256 rows with a deep and a short K; sampled outputs, every tile's and
    expert's borders among the rows."""
    rng = np.random.default_rng([I, K])
    E, off = len(counts), offsets_of(counts, 0)
    X = tokens(rng, int(off[-1]), K, F16)
    g = torch.Generator(device="cuda").manual_seed(K)
    Wg, Wu = (torch.randn(E, I, K, generator=g, device="cuda").mul_(K ** -0.5).to(F16) for _ in range(2))
    h = awq.awq_silu_mul_gemm_grouped(X, cu(off), Wg, Wu)
    awq.awq_check_error()
    cols = cu(np.unique(np.concatenate([rng.integers(0, I, 200), [0, 63, 64, 127, 128, I - 1]])))
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        at = np.concatenate([rng.integers(a, b, 60), [a, b - 1], np.arange(a + 255, b, 256),
                             np.arange(a + 256, b, 256)])
        rows = cu(np.unique(at))
        want, tol = silu_mul_tolerance(X[rows], Wg[e][cols], Wu[e][cols])
        got = h[rows][:, cols]
        assert_within(got, want, tol, e)
        # as a whole: fp16's rounding, and what fp32 sums of K / 16 steps add to it
        assert np.linalg.norm(f64(got) - want) <= 1.05 * 2.0 ** -11 * 3 ** -0.5 * np.linalg.norm(want)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 11008), (4, 1001, 4096), (8, 40, 4096)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_plain_product_of_few_rows_and_an_odd_width(awq, M, N, K, dtype):  # noqa: F811
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, 1, N, K, 4, dtype)
    X = tokens(rng, M, K, dtype)
    y = awq.awq_gemm_w4a16(X, layer.qw[0], layer.sc[0], layer.z[0], N, K, 4)
    awq.awq_check_error()
    want, tol = layer.want(0, X)
    assert assert_within(y, want, tol) <= 3 * U[dtype]
