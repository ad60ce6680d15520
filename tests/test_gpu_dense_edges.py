"""The dense products on the GPU at the edges of their contract, against the plain float64 forms of dense_ref."""
import math

import pytest
import torch

import dense_ref as ref
from block_ref import U, check

pytestmark = pytest.mark.gpu

from test_gpu_dense import BF16, F32, FN, dense, gen, mx8, nan, rand, scratch

if torch.cuda.is_available():
    import routed_expert_ffn_router_amd as m      # must load: no fallback path exists


def h8_outputs(T, N):
    return (torch.full((T, N), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda"))


# columns in whole blocks of 32 that end in each quarter of a step: few tokens, small and large tiles
@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("T,N", [(1, 64), (17, 264), (50, 96), (300, 520), (3593, 1824)])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 1056])
def test_mxfp8_columns_in_whole_blocks(T, N, K, act):
    g = gen(600 + K)
    (x, xs), (w, ws) = mx8(g, T, K), mx8(g, 2 * N, K, std=0.1)
    X, W = ref.values(x, xs), ref.values(w, ws)
    how, fn = ("mx8" if act == BF16 else "bf16"), FN[K // 32 % 4]
    d = dense(N, K, act, fn, True)
    bias, residual, y = rand(g, N), rand(g, T, N, dtype=act), nan(T, N, dtype=act)
    m.moe_matmul(d, x, xs, T, w[:N].contiguous(), ws[:N].contiguous(), bias, residual, None, y, scratch(d, T))
    check(y, ref.matmul(X, W[:N], how, fn, bias, residual)[1], act, "y")
    pre, h = nan(T, 2 * N, dtype=act), nan(T, N, dtype=act)
    m.moe_gated(d, x, xs, T, w, ws, pre, h, None, scratch(d, T))
    v, want = ref.gated(X, W, how, fn)
    check(pre, v, act, "pre")
    check(h, want, act, "h")
    if N % 32 == 0:
        codes, scales = h8_outputs(T, N)
        m.moe_gated(d, x, xs, T, w, ws, None, codes, scales, scratch(d, T))
        ref.check_mx8(codes, scales, want, "h8")


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("f", [32, 96, 1056])
def test_gated_into_a_product_in_8_bits(f, T):
    """h in MXFP8 of any rows that the gated block writes is an operand of the product behind it."""
    g, K, N = gen(610 + f), 160, 72
    (x, xs), (w, ws), (wd, wds) = mx8(g, T, K), mx8(g, 2 * f, K, std=0.1), mx8(g, N, f, std=0.1)
    gate, down = dense(f, K, BF16, "silu", True), dense(N, f, BF16, "none", True)
    (h, hs), y = h8_outputs(T, f), nan(T, N, dtype=BF16)
    m.moe_gated(gate, x, xs, T, w, ws, None, h, hs, scratch(gate, T))
    m.moe_matmul(down, h, hs, T, wd, wds, None, None, None, y, scratch(down, T))
    check(y, ref.matmul(ref.values(h, hs), ref.values(wd, wds), "mx8", "none")[1], BF16, "y")


@pytest.mark.parametrize("T", [3, 50, 700])
@pytest.mark.parametrize("act", [BF16, F32])
def test_mxfp8_nan_in_the_last_block(act, T):
    N, K = 520, 160
    g = gen(620)
    (x, xs), (w, ws) = mx8(g, T, K), mx8(g, N, K)
    xs[2, 4], ws[9, 4] = 255, 255
    d, y = dense(N, K, act, "none", True), nan(T, N, dtype=act)
    m.moe_matmul(d, x, xs, T, w, ws, None, None, None, y, scratch(d, T))
    want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    want[2], want[:, 9] = True, True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("T", [1, 300])
def test_mxfp8_blocks_replayed(T):
    """The copy of the scales is made in every replay, from what the operands hold then."""
    N, K = 96, 96
    g = gen(630)
    (x, xs), (w, ws) = mx8(g, T, K), mx8(g, N, K)
    d = dense(N, K, BF16, "none", True)
    got, want, ws1, ws2 = nan(T, N, dtype=BF16), nan(T, N, dtype=BF16), scratch(d, T), scratch(d, T)
    m.moe_matmul(d, x, xs, T, w, ws, None, None, None, got, ws1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_matmul(d, x, xs, T, w, ws, None, None, None, got, ws1)
    for seed in range(3):
        for t, new in zip((x, xs), mx8(gen(640 + seed), T, K)):
            t.copy_(new)
        graph.replay()
        m.moe_matmul(d, x, xs, T, w, ws, None, None, None, want, ws2)
        torch.cuda.synchronize()
        assert torch.equal(got, want), seed


def _rows_alike(got, want, what):
    """Infinite and NaN in the same places, with the same signs."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN"
    assert torch.equal(got == math.inf, want == math.inf) and torch.equal(got == -math.inf, want == -math.inf), f"{what}: infinities"


# one product of a row is left by the weight's columns that are zeros; the rest of the sum is of order one
@pytest.mark.parametrize("T,N,K", [(40, 136, 200), (70, 136, 200), (300, 264, 72), (700, 1032, 2056), (3593, 3600, 136)])
def test_fp32_infinities_and_the_largest_values(T, N, K):
    """What an fp32 sum that an infinity or a value near the type's end enters is does not depend on the call's length."""
    g = gen(650)
    d, lowest = dense(N, K, F32), torch.finfo(F32).min
    x, w = rand(g, T, K), rand(g, N, K)
    x[3, 5], x[9, 7], x[12, 1], x[12, 2], x[20, 0], x[T - 1, K - 1] = math.inf, -math.inf, math.inf, -math.inf, lowest, math.inf
    w[:, [0, 5, 7, 1, 2, K - 1]] = 0.0
    w[N // 2:, [5, 7, 1, K - 1]] = w[N // 2:, [5, 7, 1, K - 1]] + 0.25   # zeros times an infinity below, numbers above
    w[N // 2:, 2] = w[N // 2:, 1]
    w[N // 2:, 0] = 2.0 ** -3
    w[N - 1, 3] = -math.inf
    y, ws = nan(T, N), scratch(d, T)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, ws)
    # (in 64 bits the infinities are the same and the lowest value's products are no infinities)
    want = torch.matmul(x.double().cpu(), w.double().cpu().t().contiguous()).cuda()
    _rows_alike(y, want, "y")
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[3, 9, 12, T - 1]] = False
    v = ref.matmul(x[rows].double(), w[:N - 1].double(), "f32", "none")[1]
    check(y[rows][:, :N - 1], v, F32, "y")                     # the lowest value's row too


@pytest.mark.parametrize("T,N,K", [(50, 72, 136), (300, 264, 328), (1500, 776, 640)])
def test_fp32_infinities_in_gradients(T, N, K):
    g = gen(660)
    d = dense(N, K, F32)
    x, w, dy = rand(g, T, K), rand(g, N, K), rand(g, T, N)
    x[5, 8], dy[7, 3], w[2, 9] = math.inf, torch.finfo(F32).min, -math.inf
    w[3], dy[5] = 2.0 ** -4, 0.0
    dx, dw = nan(T, K), nan(N, K)
    m.moe_matmul_backward(d, x, T, w, None, dy, dx, dw, None, scratch(d, T))
    wx = torch.matmul(dy.double().cpu(), w.double().cpu()).cuda()
    ww = torch.matmul(dy.double().cpu().t().contiguous(), x.double().cpu()).cuda()
    _rows_alike(dx, wx, "dx")
    x7 = x[7].double()
    ww[3] = torch.where(x7.abs() * -torch.finfo(F32).min > torch.finfo(F32).max, -torch.sign(x7) * math.inf, ww[3])
    ww[3, 8] = math.nan
    _rows_alike(dw, ww, "dw")


@pytest.mark.parametrize("T", [20, 48, 200])
def test_fp32_gated_near_the_types_end(T):
    N, K = 64, 136
    g = gen(670)
    x, w = rand(g, T, K), rand(g, 2 * N, K, std=0.1)
    x[1, 4] = 3.4028e38
    w[:N, 4], w[N:, 4] = 0.0, 2.0 ** -100
    d, (codes, scales), h = dense(N, K, F32, "silu"), h8_outputs(T, N), nan(T, N)
    v, want = ref.gated(x.double(), w.double(), "f32", "silu")
    m.moe_gated(d, x, None, T, w, None, None, h, None, scratch(d, T))
    check(h, want, F32, "h")
    m.moe_gated(d, x, None, T, w, None, None, codes, scales, scratch(d, T))
    ref.check_mx8(codes, scales, want, "h8")


def points():
    """Pre-activations of every size: dense around zero, out to where the functions leave the type's range."""
    v = torch.cat([torch.linspace(-20, 20, 4001), torch.linspace(-110, 110, 551), 2.0 ** torch.linspace(-40, 6, 93), -2.0 ** torch.linspace(-40, 6, 93)])
    return v[:v.numel() // 8 * 8].to(F32).cuda()


def forward_at(v, fn, T=None):
    """The activation of exact pre-activations, from a product with one value a row; with 8 or with T tokens a call."""
    x, w, d = torch.zeros(v.numel(), 8, device="cuda"), torch.zeros(8, 8, device="cuda"), dense(8, 8, F32, fn)
    x[:, 0], w[:, 0] = v, 1.0
    y, T = nan(v.numel(), 8), T or v.numel()
    for t in range(0, v.numel(), T):
        n = min(T, v.numel() - t)
        m.moe_matmul(d, x[t:t + n], None, n, w, None, None, None, None, y[t:t + n], scratch(d, n))
    assert torch.equal(y, y[:, :1].expand(-1, 8))
    return y[:, 0].double()


def slope_at(v, fn):
    """The activation's derivative as the bias gradient of one token, which is summed from nothing else."""
    N, d_bias = v.numel(), nan(v.numel())
    d = dense(N, 8, F32, fn)
    m.moe_matmul_backward(d, None, 1, None, v, torch.ones(1, N, device="cuda"), None, None, d_bias, scratch(d, 1))
    return d_bias.double()


def within(got, want, bound, what):
    off = (got - want).abs() - bound
    k = off.argmax()
    assert off.max() <= 0, f"{what}: {got[k]} for {want[k]}, bound {bound[k]}"


def test_the_logistic_function_relative_to_itself():
    """exp off by a unit (2 U), the sum, the reciprocal's rounding and one product: 6 U for either side, with what the sum
    passes on; one more product with v for SiLU.  Its slope p (1 + v q) is taken against the sum of its parts' sizes: 12 U
    with the product and sum of 1 and v q; the sigmoid's p q relative to itself, 13 U.  Below 2^-126 the steps are 2^-149."""
    v = points()
    x = v.double()
    p, q = torch.sigmoid(x), torch.sigmoid(-x)
    tiny = 2.0 ** -140
    for T in (32, 600, None):
        within(forward_at(v, "sigmoid", T), p, 6 * U * p + tiny, "sigmoid")
        within(forward_at(v, "silu", T), x * p, 7 * U * (x * p).abs() + tiny, "silu")
    within(slope_at(v, "sigmoid"), p * q, 13 * U * p * q + tiny, "sigmoid's slope")
    within(slope_at(v, "silu"), p * (1 + x * q), 20 * U * p * (1 + x.abs() * q) + tiny, "SiLU's slope")


def test_the_logistic_functions_gradient_of_large_pre_activations():
    """bf16: a gradient that a rounding of its own is the only one of, half a step (2^-8)."""
    v = torch.linspace(4, 80, 1024, device="cuda").to(BF16).reshape(128, 8)
    d, dx = dense(8, 8, BF16, "sigmoid"), nan(128, 8, dtype=BF16)
    m.moe_matmul_backward(d, None, 128, torch.eye(8, dtype=BF16, device="cuda"), v, torch.ones(128, 8, dtype=BF16, device="cuda"), dx, None, None,
                          scratch(d, 128))
    want = torch.sigmoid(v.double()) * torch.sigmoid(-v.double())
    within(dx.double().flatten(), want.flatten(), (2.0 ** -8 * want * (1 + 2.0 ** -8)).flatten(), "dx")


def normal_cdf(x):
    """Relative to itself in the tail too (ndtr comes in steps of 2^-54 there)."""
    return 0.5 * torch.special.erfc(-x * math.sqrt(0.5))


def test_gelu_relative_to_itself():
    """The tail of the distribution function: 0.5 U of the approximation, nine steps of its polynomial that lose up to
    a third of their sizes' sum (1.3) as R falls to 0.03 (33 U in a replay of every step), and the exponential, a unit of its
    instruction (2 U) and three roundings: 40 U.  The function itself: the tail is at most a half, 1.2 U in that
    replay, a unit of each instruction and the rounding of 1 - tail: 3 U.  Its slope adds v times the density (the
    exponential's 5 U, two products, 8 U).  Below 2^-126 the exponential's instruction gives zero."""
    v = points()
    x = v.double()
    cdf, density = normal_cdf(x), torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    off = U * torch.minimum(40 * cdf, torch.full_like(cdf, 3.0))
    tiny = 2.0 ** -125 * (1 + x.abs())
    for T in (32, 600, None):
        within(forward_at(v, "gelu", T), x * cdf, x.abs() * off + 2 * U * (x * cdf).abs() + tiny, "gelu")
    within(slope_at(v, "gelu"), cdf + x * density, off + 8 * U * x.abs() * density + 2 * U * (cdf + x * density).abs() + tiny, "its slope")


def test_gelu_in_bf16_is_rounded_once():
    v = -torch.linspace(0.01, 13, 4096, device="cuda").to(BF16)
    x, w, d, y = torch.zeros(4096, 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda"), dense(8, 8, BF16, "gelu"), nan(4096, 8, dtype=BF16)
    x[:, 0], w[:, 0] = v, 1.0
    m.moe_matmul(d, x, None, 4096, w, None, None, None, None, y, scratch(d, 4096))
    want = v.double() * normal_cdf(v.double())
    within(y[:, 0].double(), want, 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -120, "y")


@pytest.mark.parametrize("T,h8", [(32, 1), (33, 1), (64, 0), (65, 0)])
def test_fp32_bits_below_bf16s_smallest(T, h8):
    """Values enter as they are up to 32 tokens with h in MXFP8 and up to 64 without; beyond, bits below 2^-133 are left out."""
    g = gen(680)
    N, K = 64, 136
    x, w = torch.zeros(T, K, device="cuda"), rand(g, 2 * N, K)
    x[:, 0] = 3 * 2.0 ** -134
    w[:N] = 0.0
    w[:N, 1], x[:, 1], w[N:, 0], w[N:, 1] = 1.0, 1.0, 2.0 ** 100, 0.0    # gate 1, up 3 * 2^-34
    d = dense(N, K, F32, "none")
    if h8:
        codes, scales = h8_outputs(T, N)
        m.moe_gated(d, x, None, T, w, None, None, codes, scales, scratch(d, T))
        h = ref.values(codes, scales)
    else:
        h = nan(T, N)
        m.moe_gated(d, x, None, T, w, None, None, h, None, scratch(d, T))
    as_they_are = T <= (32 if h8 else 64)
    assert ((h.double() - 3 * 2.0 ** -34).abs() <= (0 if as_they_are else 2.0 ** -34)).all()


@pytest.mark.parametrize("T", [3, 70, 300])
@pytest.mark.parametrize("act", [BF16, F32])
def test_gated_offsets_past_32_bits(act, T):
    """The up projection's rows start past 4 GiB, and the gate's last rows too with fp32."""
    K, last = 4096, 40
    N = (1 << 32) // (K * 2) + 1032
    g = gen(690)
    w = torch.zeros(2 * N, K, dtype=act, device="cuda")
    for end in (N, 2 * N):
        w[end - last:end] = rand(g, last, K, dtype=act, std=0.1)
    x = rand(g, T, K, dtype=act)
    d, h = dense(N, K, act, "silu"), nan(T, N, dtype=act)
    m.moe_gated(d, x, None, T, w, None, None, h, None, scratch(d, T))
    assert (h[:, :-last] == 0).all()
    rows = torch.cat([w[N - last:N], w[2 * N - last:]]).double()
    check(h[:, -last:], ref.gated(x.double(), rows, "bf16" if act == BF16 else "f32", "silu")[1], act, "h")


@pytest.mark.parametrize("T", [3, 70, 300])
@pytest.mark.parametrize("K", [8192, 8224])
def test_mxfp8_offsets_past_32_bits(K, T):
    """Gated, more than 4 GiB of codes in either half, with the operands' own scales and with copied ones."""
    last = 40
    N = ((1 << 32) // K + 1032) // 8 * 8
    g = gen(695)
    w, ws = torch.zeros(2 * N, K, dtype=torch.uint8, device="cuda"), torch.full((2 * N, K // 32), 121, dtype=torch.uint8, device="cuda")
    for end in (N, 2 * N):
        w[end - last:end], ws[end - last:end] = mx8(g, last, K, std=0.1)
    x, xs = mx8(g, T, K)
    d, h = dense(N, K, BF16, "silu", True), nan(T, N, dtype=BF16)
    m.moe_gated(d, x, xs, T, w, ws, None, h, None, scratch(d, T))
    assert (h[:, :-last] == 0).all()
    rows = torch.cat([ref.values(w[e - last:e], ws[e - last:e]) for e in (N, 2 * N)])
    check(h[:, -last:], ref.gated(ref.values(x, xs), rows, "mx8", "silu")[1], BF16, "h")


def test_the_most_rows():
    """The gated block's gradient over 2^20 rows of h: sums over 2^21 values, rows of 2^23 bytes."""
    T, N, K = 70, 1 << 20, 8
    g = gen(698)
    d = dense(N, K, F32, "sigmoid")
    w, dh, pre = rand(g, 2 * N, K, std=0.1), rand(g, T, N), rand(g, T, 2 * N)
    dx = nan(T, K)
    m.moe_gated_backward(d, None, T, w, pre, dh, dx, None, scratch(d, T))
    grad = ref.gated_grad(dh, pre, "sigmoid")
    check(dx, ref.product(grad.v, w.double().t(), "f32", grad.e), F32, "dx")


@pytest.mark.parametrize("act", [BF16, F32])
def test_outputs_past_32_bits(act):
    """More than 4 GiB of y, residual and pre: rows from the ends and the middle, the residual in y's place."""
    T, N, K = 65536, 36872, 8
    g = gen(699)
    x, w, d = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act), dense(N, K, act, "silu")
    y, pre = torch.empty(T, N, dtype=act, device="cuda"), torch.empty(T, N, dtype=act, device="cuda")
    for t in range(0, T, 8192):
        y[t:t + 8192] = torch.randn(8192, 1, generator=g, device="cuda")
    rows = torch.tensor([0, 1, 29119, 29120, 32768, 58255, T - 2, T - 1], device="cuda")
    residual = y[rows].clone()
    m.moe_matmul(d, x, None, T, w, None, None, y, pre, y, scratch(d, T))
    v, want = ref.matmul(x[rows].double(), w.double(), "bf16" if act == BF16 else "f32", "silu", None, residual)
    check(pre[rows], v, act, "pre")
    check(y[rows], want, act, "y")
    dx = nan(T, K, dtype=act)
    m.moe_matmul_backward(d, None, T, w, pre, y, dx, None, None, scratch(d, T))
    grad = ref.matmul_grad(y[rows], pre[rows], "silu")
    check(dx[rows], ref.backward(grad, x[rows].double(), w.double(), "bf16" if act == BF16 else "f32")[0], act, "dx")
