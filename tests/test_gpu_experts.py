"""The products with a fused epilogue and the operators of expert layers against plain 64-bit
forms: types, odd sizes, empty experts, rows of no expert, aliased operands, offsets out of
order, graphs and streams."""
import numpy as np
import pytest
import torch

import oracle as O
from expert_reference import U, act64, assert_within, f64, linear64, packed

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_stats_b200 import build
    build.build()
    import weight_only_int4_stats_b200 as m
    return m


def cu(a, dtype=None):
    a = np.ascontiguousarray(a)
    t = torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a)
    return (t if dtype is None else t.to(dtype)).cuda()


def tokens(rng, M, K, dtype):
    m = rng.lognormal(0, 0.5, K)
    return cu(rng.standard_normal((M, K)) * m, dtype)


class Layer:
    """E experts' packed weights with optional inv_s and bias, on the GPU and the host."""

    def __init__(self, rng, E, N, K, bits, dtype, inv=False, bias=False):
        self.E, self.N, self.K, self.bits, self.dtype = E, N, K, bits, dtype
        self.host = [packed(rng, N, K, bits) for _ in range(E)]
        self.qw, self.sc, self.z = (cu(np.stack([h[i] for h in self.host])) for i in range(3))
        self.inv = cu(rng.uniform(0.3, 3.0, (E, K)).astype(np.float32)) if inv else None
        self.bias = cu(rng.standard_normal((E, N)) * 0.3, dtype) if bias else None

    def want(self, e, X, act="none", mul=None, residual=None):
        qw, sc, z = self.host[e]
        return linear64(f64(X), qw, sc, z, self.N, self.K, self.bits,
                        None if self.inv is None else f64(self.inv[e]),
                        None if self.bias is None else f64(self.bias[e]), act,
                        f64(mul), f64(residual), self.dtype)


def dense(awq, layer, X, **kw):
    return awq.awq_gemm_w4a16_epilogue(
        X, layer.qw[0], layer.sc[0], layer.z[0], layer.N, layer.K, layer.bits,
        inv_s=None if layer.inv is None else layer.inv[0],
        bias=None if layer.bias is None else layer.bias[0], **kw)


def grouped(awq, layer, X, offsets, **kw):
    off = offsets if torch.is_tensor(offsets) else cu(np.asarray(offsets, np.int32))
    return awq.awq_gemm_w4a16_grouped(X, off, layer.qw, layer.sc, layer.z, layer.N, layer.K,
                                      layer.bits, inv_s=layer.inv, bias=layer.bias, **kw)


# ----------------------------------------------------------------------------- fused epilogue

EPILOGUES = [   # M, N, K, bits, dtype, inv_s, bias, act, mul, residual
    (1, 16, 128, 4, F16, False, True, "none", False, False),
    (1, 1000, 2176, 4, BF16, True, False, "gelu", False, True),
    (1, 4096, 4096, 4, F16, True, True, "silu", True, True),
    (1, 48, 256, 3, BF16, False, False, "relu", False, False),
    (2, 37, 384, 4, F16, False, True, "gelu_tanh", True, False),
    (5, 1, 128, 4, BF16, True, True, "none", False, True),
    (8, 258, 2048, 3, F16, True, False, "silu", True, False),
    (8, 512, 4096, 4, BF16, False, False, "silu", True, False),
    (9, 512, 1024, 4, F16, True, True, "relu", False, True),
    (16, 130, 1152, 4, BF16, False, True, "gelu", True, True),
    (16, 256, 2048, 3, F16, True, True, "none", True, False),
    (17, 1001, 512, 4, F16, True, False, "none", False, True),
    (33, 128, 4096, 3, BF16, True, True, "silu", False, False),
    (64, 640, 1024, 4, F16, False, True, "gelu_tanh", False, True),
    (77, 512, 11008, 4, F16, True, False, "none", False, True),
    (129, 300, 768, 4, BF16, False, False, "relu", True, False),
    (300, 384, 1024, 4, F16, False, True, "gelu", True, True),
    (513, 257, 256, 3, F16, True, False, "silu", True, False),
    (1000, 1024, 512, 4, BF16, True, True, "gelu_tanh", False, False),
]


@pytest.mark.parametrize("M,N,K,bits,dtype,inv,bias,act,mul,res", EPILOGUES)
def test_epilogue_against_64_bits(awq, M, N, K, bits, dtype, inv, bias, act, mul, res):
    rng = np.random.default_rng([M, N, K, bits])
    layer = Layer(rng, 1, N, K, bits, dtype, inv, bias)
    X = tokens(rng, M, K, dtype)
    mu = cu(rng.standard_normal((M, N)), dtype) if mul else None
    re = cu(rng.standard_normal((M, N)), dtype) if res else None
    y = dense(awq, layer, X, act=act, mul=mu, residual=re)
    assert y.dtype == dtype and y.shape == (M, N)
    want, tol = layer.want(0, X, act, mu, re)
    rel = assert_within(y, want, tol)
    assert rel <= 3 * U[dtype]
    awq.awq_check_error()
    for ready in (False, True):   # the same bits again
        again = dense(awq, layer, X, act=act, mul=mu, residual=re, weights_ready=ready)
        assert torch.equal(y, again)


@pytest.mark.parametrize("M", [1, 4, 12, 40, 200])
def test_epilogue_operands_may_be_the_output(awq, M):
    rng = np.random.default_rng(M)
    layer = Layer(rng, 1, 272, 512, 4, F16)
    X = tokens(rng, M, 512, F16)
    mu, re = (cu(rng.standard_normal((M, 272)), F16) for _ in range(2))
    y = dense(awq, layer, X, act="silu", mul=mu, residual=re)
    for alias in ("mul", "residual"):
        kw = {"mul": mu.clone(), "residual": re.clone()}
        got = dense(awq, layer, X, act="silu", out=kw[alias], **kw)
        assert got.data_ptr() == kw[alias].data_ptr() and torch.equal(got, y)


@pytest.mark.parametrize("M", [1, 3, 16, 50])
def test_epilogue_keeps_nan_and_infinity_in_their_rows(awq, M):
    rng = np.random.default_rng(M)
    layer = Layer(rng, 1, 144, 256, 4, F16, bias=True)
    X = tokens(rng, M, 256, F16)
    clean = dense(awq, layer, X, act="relu")
    bad = X.clone()
    bad[M // 2, 7] = float("nan")
    y = dense(awq, layer, bad, act="relu")
    assert y[M // 2].isnan().all()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[keep], clean[keep])
    mu = torch.ones(M, 144, dtype=F16, device="cuda")
    mu[0, 3], mu[M - 1, 143] = float("inf"), float("nan")
    y = dense(awq, layer, X, mul=mu)
    assert y[0, 3].isinf() and y[M - 1, 143].isnan()
    assert y.isfinite().sum() == M * 144 - 2


def test_epilogue_without_parts_is_the_plain_product(awq):
    rng = np.random.default_rng(3)
    layer = Layer(rng, 1, 512, 1024, 4, F16)
    for M in (1, 8, 16):   # the same decode kernel, the same bits
        X = tokens(rng, M, 1024, F16)
        plain = awq.awq_gemm_w4a16(X, layer.qw[0], layer.sc[0], layer.z[0], 512, 1024, 4)
        want, tol = layer.want(0, X)
        assert_within(dense(awq, layer, X), want, tol)
        assert_within(plain, want, tol)


def test_activations_far_out(awq):
    # large arguments: silu and gelu run to v or to 0 without an overflow on the way
    K, N = 128, 64
    codes = np.zeros((N, K), np.uint32)
    codes[:, 0] = np.arange(N) % 16
    qw, sc, z = O.pack(codes, 4), np.ones((1, N), np.float16), np.zeros((1, N), np.uint8)
    z[:] = 8
    codes[:, 1:] = 8
    qw = O.pack(codes, 4)
    X = torch.zeros(2, K, dtype=F16, device="cuda")
    X[0, 0], X[1, 0] = 100.0, 3000.0
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        y = awq.awq_gemm_w4a16_epilogue(X, cu(qw), cu(sc), cu(z), N, K, 4, act=act)
        v = f64(X[:, :1]) * (codes[:, 0].astype(np.float64) - 8)[None, :]
        want = act64(v, act)
        assert np.abs(f64(y) - want).max() <= 2.0 ** -11 * np.abs(want).max()
        assert (f64(y)[v < -90] == 0).all()


# ----------------------------------------------------------------------------- experts

GROUPS = [   # counts of rows, before the first expert's and behind the last one's
    ([3], 0, 0),
    ([1], 0, 0),
    ([0, 5, 0, 0, 17, 1, 0], 0, 0),
    ([0, 0, 0], 4, 3),
    ([2, 0, 1], 1, 6),
    ([40, 3, 0, 129, 16], 0, 5),
    ([300, 1, 31, 0, 33, 260], 2, 0),
    ([1] * 40, 0, 0),
    ([0, 1, 2] * 43 + [7], 3, 1),
    ([600, 0, 0, 0], 0, 0),
]
KINDS = [   # N, K, bits, dtype, inv_s, bias, act, mul, residual
    (144, 384, 4, F16, True, False, "silu", True, False),
    (1000, 256, 4, BF16, False, True, "none", False, True),
    (37, 2176, 3, F16, False, False, "none", False, False),
    (512, 1024, 3, BF16, True, True, "gelu", True, True),
    (130, 128, 4, F16, False, True, "relu", False, False),
]


def offsets_of(counts, before):
    return np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("group", range(len(GROUPS)))
def test_grouped_against_64_bits(awq, group, kind):
    counts, before, behind = GROUPS[group]
    N, K, bits, dtype, inv, bias, act, mul, res = KINDS[kind]
    rng = np.random.default_rng([group, kind])
    E = len(counts)
    layer = Layer(rng, E, N, K, bits, dtype, inv, bias)
    off = offsets_of(counts, before)
    T = int(off[-1]) + behind
    X = tokens(rng, T, K, dtype)
    mu = cu(rng.standard_normal((T, N)), dtype) if mul else None
    re = cu(rng.standard_normal((T, N)), dtype) if res else None
    out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    y = grouped(awq, layer, X, off, act=act, mul=mu, residual=re, out=out)
    assert y is out
    awq.awq_check_error()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        want, tol = layer.want(e, X[a:b], act, None if mu is None else mu[a:b],
                               None if re is None else re[a:b])
        rel = assert_within(y[a:b], want, tol, (e, a, b))
        assert b - a < 8 or rel <= 3 * U[dtype]
    assert (y[:off[0]] == 7).all() and (y[off[-1]:] == 7).all()   # rows of no expert
    again = grouped(awq, layer, X, off, act=act, mul=mu, residual=re, out=torch.empty_like(out),
                    weights_ready=True)
    assert torch.equal(again[off[0]:off[-1]], y[off[0]:off[-1]])


def test_grouped_most_experts(awq):
    rng = np.random.default_rng(5)
    layer = Layer(rng, 1, 32, 128, 4, F16)
    E = 1024
    counts = rng.integers(0, 3, E)
    off = offsets_of(counts, 0)
    X = tokens(rng, int(off[-1]), 128, F16)
    y = awq.awq_gemm_w4a16_grouped(X, cu(off), layer.qw.expand(E, -1, -1).contiguous(),
                                   layer.sc.expand(E, -1, -1).contiguous(),
                                   layer.z.expand(E, -1, -1).contiguous(), 32, 128, 4)
    s = awq.awq_act_stats_grouped(X, cu(off))
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            assert_within(y[a:b], *layer.want(0, X[a:b]), e)
        np.testing.assert_array_equal(s[e].cpu().numpy(),
                                      O.act_stats(f16(X[a:b])) if b > a else np.zeros(128, np.float32))


def f16(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("T", [6, 60, 600])
def test_grouped_offsets_out_of_order_stay_inside(awq, T):
    # any offsets: values that mean nothing, but no row outside the arguments is touched, and a
    # good call afterwards is as good as ever
    rng = np.random.default_rng(T)
    N, K = 80, 256
    layer = Layer(rng, 5, N, K, 4, F16)
    X = tokens(rng, T, K, F16)
    guard = torch.full((T + 512, N), 7.0, dtype=F16, device="cuda")
    for off in ([T, 0, T, 0, T, 0], [-5, T + 9, -2 ** 31, 2 ** 31 - 1, 3, T], [2, 1, 0, T, T, 2],
                [T + 1] * 6, [-1] * 6):
        o = cu(np.asarray(off, np.int32))
        grouped(awq, layer, X, o, out=guard[256:256 + T])
        awq.awq_act_stats_grouped(X, o)
        awq.awq_check_error()
        assert (guard[:256] == 7).all() and (guard[256 + T:] == 7).all()
    good = offsets_of([T - 3, 0, 1, 2, 0], 0)
    y = grouped(awq, layer, X, good)
    for e in range(5):
        a, b = good[e], good[e + 1]
        if b > a:
            want, tol = layer.want(e, X[a:b])
            assert_within(y[a:b], want, tol)


@pytest.mark.parametrize("T,K,counts", [
    (1, 8, [1]), (700, 264, [0, 300, 1, 0, 399, 0]), (5000, 1024, [2500, 7] + [1] * 60 + [2400]),
    (4099, 2056, [0, 0, 4000, 0]), (64, 16384, [64]), (0, 64, [0, 0])])
def test_stats_grouped_bitexact(awq, T, K, counts):
    rng = np.random.default_rng([T, K])
    X = tokens(rng, T, K, F16)
    off = offsets_of(counts, 0)
    out = torch.full((len(counts), K), -1.0, device="cuda")
    got = awq.awq_act_stats_grouped(X, cu(off), out=out).cpu().numpy()
    for e in range(len(counts)):
        rows = f16(X[off[e]:off[e + 1]])
        want = O.act_stats(rows) if len(rows) else np.zeros(K, np.float32)
        np.testing.assert_array_equal(got[e], want)
    if len(counts) == 1:
        np.testing.assert_array_equal(got[0], awq.awq_act_stats(X).cpu().numpy())


def test_stats_grouped_keeps_nan_and_infinity_apart(awq):
    rng = np.random.default_rng(0)
    X = tokens(rng, 90, 256, F16)
    X[10, 3], X[50, 4] = float("nan"), float("-inf")
    X[89, 5] = float("nan")   # behind the last expert
    s = awq.awq_act_stats_grouped(X, cu(np.array([0, 30, 60, 88], np.int32)))
    bad = ~s.isfinite()
    assert s[0, 3].isnan() and s[1, 4] == float("inf") and bad.sum() == 2


def silu_mul_tolerance(X, Wg, Wu):
    """Both sums exact but for fp32 accumulation (one truncation per 16-wide step), silu's slope
    at most 1.1, a few fp32 roundings, then one to fp16."""
    x, g, u = f64(X), f64(Wg), f64(Wu)
    acc = (x.shape[1] / 16 + 16) * 2.0 ** -23
    G, U_ = x @ g.T, x @ u.T
    dG, dU = acc * (np.abs(x) @ np.abs(g).T), acc * (np.abs(x) @ np.abs(u).T)
    h = act64(G, "silu") * U_
    tol = 1.1 * dG * (np.abs(U_) + dU) + np.abs(act64(G, "silu")) * dU
    return h, tol + 8 * 2.0 ** -24 * np.abs(G * U_) + 2.0 ** -11 * (np.abs(h) + tol) + 2.0 ** -25


# small layers (tiles of 64 rows of each weight), then layers whose tiles of 128 rows fill the GPU
# once, for each token tile
SILU = [(c, b, e, I, K) for c, b, e in GROUPS for I, K in ((144, 256), (37, 384), (300, 1024))] + [
    ([64, 1, 0, 33, 200], 2, 1, 3000, 256), ([400, 300], 0, 0, 5000, 128),
    ([10, 0, 7, 30], 0, 3, 4500, 128), ([150, 100, 140], 1, 0, 5000, 128)]


@pytest.mark.parametrize("case", range(len(SILU)))
def test_silu_mul_grouped_against_64_bits(awq, case):
    counts, before, behind, I, K = SILU[case]
    rng = np.random.default_rng([case, I, K])
    E = len(counts)
    off = offsets_of(counts, before)
    T = int(off[-1]) + behind
    X = tokens(rng, T, K, F16)
    Wg, Wu = (cu(rng.standard_normal((E, I, K)) * K ** -0.5, F16) for _ in range(2))
    out = torch.full((T, I), 7.0, dtype=F16, device="cuda")
    h = awq.awq_silu_mul_gemm_grouped(X, cu(off), Wg, Wu, out=out)
    awq.awq_check_error()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            assert_within(h[a:b], *silu_mul_tolerance(X[a:b], Wg[e], Wu[e]), (e, a, b))
    assert (h[:off[0]] == 7).all() and (h[off[-1]:] == 7).all()


# ----------------------------------------------------------------------------- together

def test_expert_layer_calibrated_and_served(awq):
    """An expert layer from full-precision weights: per-expert statistics, the gated products
    that calibrate the down projections, search and packing of every expert, then the packed
    layer in three grouped products; against the same steps in 64 bits with the same codes."""
    rng = np.random.default_rng(11)
    E, I, K, counts = 4, 256, 384, [90, 0, 31, 150]
    off = offsets_of(counts, 0)
    T = int(off[-1])
    X, o = tokens(rng, T, K, F16), cu(off)
    Wg, Wu = (cu(rng.standard_normal((E, I, K)) * 0.05, F16) for _ in range(2))
    Wd = cu(rng.standard_normal((E, K, I)) * 0.05, F16)
    alphas = cu(O.alpha_grid(20))

    s_in = awq.awq_act_stats_grouped(X, o)
    H = awq.awq_silu_mul_gemm_grouped(X, o, Wg, Wu)
    s_mid = awq.awq_act_stats_grouped(H, o)
    sides = {"gate": (Wg, X, s_in), "up": (Wu, X, s_in), "down": (Wd, H, s_mid)}
    packs = {}
    for name, (W, inp, s) in sides.items():
        N, Kin = W.shape[1:]
        qw = torch.empty(E, N, Kin // 8, dtype=torch.int32, device="cuda")
        sc = torch.empty(E, Kin // 128, N, dtype=F16, device="cuda")
        z = torch.empty(E, Kin // 128, N, dtype=torch.uint8, device="cuda")
        inv = torch.ones(E, Kin, device="cuda")
        for e in range(E):
            best = None
            if counts[e]:   # an expert no calibration row reached is rounded unscaled
                rows = inp[off[e]:off[e + 1]].contiguous()
                _, _, best, _, inv[e] = awq.awq_search_scale(W[e], rows, s[e], alphas, inv=True)
            awq.awq_quantize_pack(W[e], best, out=(qw[e], sc[e], z[e]))
        packs[name] = (qw, sc, z, inv)

    def product(x, name, N, Kin, **kw):
        qw, sc, z, inv = packs[name]
        return awq.awq_gemm_w4a16_grouped(x, o, qw, sc, z, N, Kin, inv_s=inv, **kw)

    def want(x, name, e, **kw):
        qw, sc, z, inv = (t[e] for t in packs[name])
        N, Kin = z.shape[1], inv.shape[0]
        return linear64(f64(x), qw.cpu().numpy().view(np.uint32), sc.cpu().numpy(), z.cpu().numpy(),
                        N, Kin, 4, f64(inv), **kw)

    up = product(X, "up", I, K)
    mid = product(X, "gate", I, K, act="silu", mul=up)
    y = product(mid, "down", K, I)
    awq.awq_check_error()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        assert_within(up[a:b], *want(X[a:b], "up", e))
        assert_within(mid[a:b], *want(X[a:b], "gate", e, act="silu", mul=f64(up[a:b])))
        assert_within(y[a:b], *want(mid[a:b], "down", e))
        # and the packed layer is near the full-precision one: 4-bit weights of group 128
        full = f64(H[a:b]) @ f64(Wd[e]).T
        assert np.linalg.norm(f64(y[a:b]) - full) <= 0.35 * np.linalg.norm(full)


@pytest.mark.parametrize("M", [1, 6, 16, 40])
def test_captured_and_replayed_with_new_inputs(awq, M):
    rng = np.random.default_rng(M)
    dense_layer = Layer(rng, 1, 256, 512, 4, F16, bias=True)
    experts = Layer(rng, 6, 512, 256, 4, F16, inv=True)
    X = tokens(rng, M, 512, F16)
    off = cu(np.zeros(7, np.int32))

    def step():
        h = dense(awq, dense_layer, X, act="gelu")
        y = grouped(awq, experts, h, off, residual=X)
        return h, y, awq.awq_act_stats_grouped(h, off)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for k in range(3):
        X.copy_(tokens(rng, M, 512, F16))
        cuts = np.sort(rng.integers(0, M + 1, 5))
        off.copy_(cu(np.concatenate([[0], cuts, [M]]).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        eager = step()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
    awq.awq_check_error()


def test_two_streams_at_once(awq):
    rng = np.random.default_rng(2)
    layer = Layer(rng, 8, 512, 1024, 4, BF16, inv=True)
    sets = []
    for k, T in enumerate((5, 120)):
        off = offsets_of(rng.multinomial(T, np.ones(8) / 8), 0)
        X = tokens(rng, T, 1024, BF16)
        sets.append((X, cu(off), torch.cuda.Stream()))
    want = [(grouped(awq, layer, X, o), dense(awq, layer, X)) for X, o, _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, (X, o, s) in enumerate(sets):
            got[k].append((grouped(awq, layer, X, o, stream=s), dense(awq, layer, X, stream=s)))
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in got[k]:
            assert torch.equal(a, want[k][0]) and torch.equal(b, want[k][1])
