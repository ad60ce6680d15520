"""The dense products beside the experts on the GPU, through the binding, against plain float64 forms with an error
bound carried along (dense_ref): the product with its epilogue, the gated block, their gradients, the norm to
8 bits, and a run of them as a dense block uses them."""
import math

import pytest
import torch

import block_ref
import dense_ref as ref
from block_ref import Val, check

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routed_expert_ffn_router_amd as m      # must load: no fallback path exists

F32, BF16 = torch.float32, torch.bfloat16
FN = ["none", "silu", "gelu", "sigmoid"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *size, dtype=F32, std=1.0):
    return (torch.randn(*size, generator=g, device="cuda") * std).to(dtype)


def dense(rows, cols, act, fn="none", mx8=False):
    return m.make_dense(rows, cols, m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32,
                        m.MOE_OPERANDS_MXFP8 if mx8 else m.MOE_OPERANDS_ACT, FN.index(fn))


def scratch(d, T):
    """A workspace full of NaN bytes: no call may read what it has not written."""
    return m.dense_workspace(d, T).fill_(255)


def nan(*size, dtype=F32):
    return torch.full(size, float("nan"), dtype=dtype, device="cuda")


def kind(act):
    return "bf16" if act == BF16 else "f32"


def mx8(g, rows, cols, std=1.0):
    """Random codes (every finite one) under random scales of about std."""
    codes = torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    top = round(math.log2(std)) - 6 + 127
    return codes, torch.randint(top - 3, top + 3, (rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8)


# few tokens: more tiles than workgroups, sums shorter than a wave's share and longer than its ring
FEW = [(1, 4424, 328), (16, 4424, 72), (32, 8264, 136), (33, 4424, 264), (64, 4104, 1096), (7, 8288, 8), (20, 8288, 456), (48, 6144, 2056), (2, 72, 8200)]
FEW8 = [(1, 8288, 128), (16, 4424, 640), (31, 8288, 1152), (33, 4424, 256), (64, 4104, 384), (48, 96, 8192)]
# T, rows, cols: single values, sizes that end inside tiles and steps, several tiles each way, sums in parts
SIZES = [(1, 8, 8), (2, 24, 40), (1, 4096, 1024), (3, 136, 64), (5, 40, 2056), (16, 64, 256), (17, 72, 200), (33, 264, 136), (64, 512, 1024),
         (100, 1000, 520), (128, 128, 128), (129, 384, 648), (257, 520, 1160), (300, 2048, 512), (1030, 328, 72),
         (513, 96, 4104), (2049, 264, 264), (600, 2056, 328), *FEW]
EPILOGUES = [("none", 0, 0, 0), ("silu", 1, 0, 1), ("gelu", 0, 1, 1), ("sigmoid", 1, 1, 0), ("none", 1, 1, 1)]


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_matmul(n, act):
    T, N, K = SIZES[n]
    g = gen(n)
    x, w = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act, std=0.1)
    for fn, has_bias, has_residual, has_pre in EPILOGUES if n % 3 == 0 else [EPILOGUES[n % 5]]:
        d = dense(N, K, act, fn)
        bias = rand(g, N) if has_bias else None
        residual = rand(g, T, N, dtype=act) if has_residual else None
        pre, y = nan(T, N, dtype=act) if has_pre else None, nan(T, N, dtype=act)
        m.moe_matmul(d, x, None, T, w, None, bias, residual, pre, y, scratch(d, T))
        v, want = ref.matmul(x.double(), w.double(), kind(act), fn, bias, residual)
        check(y, want, act, f"y {fn}")
        if has_pre:
            check(pre, v, act, f"pre {fn}")
        if has_residual:                          # in the residual's place
            m.moe_matmul(d, x, None, T, w, None, bias, residual, None, residual, scratch(d, T))
            assert torch.equal(residual, y)


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_gated(n, act):
    T, N, K = SIZES[n]
    g = gen(100 + n)
    x, w = rand(g, T, K, dtype=act), rand(g, 2 * N, K, dtype=act, std=0.1)
    for fn in FN if n % 3 == 0 else [FN[n % 4]]:
        d = dense(N, K, act, fn)
        pre, h = nan(T, 2 * N, dtype=act), nan(T, N, dtype=act)
        m.moe_gated(d, x, None, T, w, None, pre, h, None, scratch(d, T))
        v, want = ref.gated(x.double(), w.double(), kind(act), fn)
        check(pre, v, act, f"pre {fn}")
        check(h, want, act, f"h {fn}")
        only = nan(T, N, dtype=act)
        m.moe_gated(d, x, None, T, w, None, None, only, None, scratch(d, T))
        assert torch.equal(only, h)
        if N % 32 == 0:
            codes, scales = torch.full((T, N), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda")
            m.moe_gated(d, x, None, T, w, None, None, codes, scales, scratch(d, T))
            ref.check_mx8(codes, scales, want, f"h8 {fn}")


SIZES8 = [(1, 8, 128), (3, 40, 256), (1, 4096, 1024), (16, 64, 4096), (17, 96, 384), (65, 1032, 128), (130, 256, 1152), (300, 512, 640), (1025, 520, 256), (512, 1056, 2048), *FEW8]


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n", range(len(SIZES8)))
def test_mxfp8_operands(n, act):
    T, N, K = SIZES8[n]
    g = gen(200 + n)
    (x, xs), (w, ws) = mx8(g, T, K), mx8(g, 2 * N, K, std=0.1)
    X, W = ref.values(x, xs), ref.values(w, ws)
    how = "mx8" if act == BF16 else "bf16"
    fn = FN[n % 4]
    d = dense(N, K, act, fn, True)
    bias, residual, y = rand(g, N), rand(g, T, N, dtype=act), nan(T, N, dtype=act)
    m.moe_matmul(d, x, xs, T, w[:N].contiguous(), ws[:N].contiguous(), bias, residual, None, y, scratch(d, T))
    check(y, ref.matmul(X, W[:N], how, fn, bias, residual)[1], act, "y")
    pre, h = nan(T, 2 * N, dtype=act), nan(T, N, dtype=act)
    m.moe_gated(d, x.view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu), T, w, ws, pre, h, None, scratch(d, T))
    v, want = ref.gated(X, W, how, fn)
    check(pre, v, act, "pre")
    check(h, want, act, "h")
    if N % 32 == 0:
        codes, scales = torch.full((T, N), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda")
        m.moe_gated(d, x, xs, T, w, ws, None, codes, scales, scratch(d, T))
        ref.check_mx8(codes, scales, want, "h8")


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_matmul_backward(n, act):
    T, N, K = SIZES[n]
    g = gen(300 + n)
    x, w, dy = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act, std=0.1), rand(g, T, N, dtype=act)
    for fn in FN if n % 3 == 0 else [FN[n % 4]]:
        d = dense(N, K, act, fn)
        pre = rand(g, T, N, dtype=act, std=2.0) if fn != "none" else None
        dx, dw, db = nan(T, K, dtype=act), nan(N, K, dtype=act), nan(N)
        m.moe_matmul_backward(d, x, T, w, pre, dy, dx, dw, db, scratch(d, T))
        grad = ref.matmul_grad(dy, pre, fn)
        wx, ww = ref.backward(grad, x.double(), w.double(), kind(act))
        check(dx, wx, act, f"dx {fn}")
        check(dw, ww, act, f"dw {fn}")
        check(db, ref.bias_grad(grad), F32, f"d_bias {fn}")
        # each alone gives the same bits
        one = [torch.empty_like(t) for t in (dx, dw, db)]
        m.moe_matmul_backward(d, None, T, w, pre, dy, one[0], None, None, scratch(d, T))
        m.moe_matmul_backward(d, x, T, None, pre, dy, None, one[1], None, scratch(d, T))
        m.moe_matmul_backward(d, None, T, None, pre, dy, None, None, one[2], scratch(d, T))
        assert all(torch.equal(a, b) for a, b in zip(one, (dx, dw, db)))


@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_gated_backward(n, act):
    T, N, K = SIZES[n]
    g = gen(400 + n)
    x, w, dh = rand(g, T, K, dtype=act), rand(g, 2 * N, K, dtype=act, std=0.1), rand(g, T, N, dtype=act)
    pre = rand(g, T, 2 * N, dtype=act, std=1.5)
    for fn in FN if n % 3 == 0 else [FN[n % 4]]:
        d = dense(N, K, act, fn)
        dx, dw = nan(T, K, dtype=act), nan(2 * N, K, dtype=act)
        m.moe_gated_backward(d, x, T, w, pre, dh, dx, dw, scratch(d, T))
        wx, ww = ref.backward(ref.gated_grad(dh, pre, fn), x.double(), w.double(), kind(act))
        check(dx, wx, act, f"dx {fn}")
        check(dw, ww, act, f"dw {fn}")
        one = [torch.empty_like(t) for t in (dx, dw)]
        m.moe_gated_backward(d, None, T, w, pre, dh, one[0], None, scratch(d, T))
        m.moe_gated_backward(d, x, T, None, pre, dh, None, one[1], scratch(d, T))
        assert torch.equal(one[0], dx) and torch.equal(one[1], dw)


@pytest.mark.parametrize("act", [BF16, F32])
def test_large_products(act):
    """Many tiles each way, the last ones cut, and steps past the places that the operands have in LDS: the product and
    both gradients."""
    T, N, K = 3593, 3600, 3592
    g = gen(500)
    x, w, dy = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act, std=0.02), rand(g, T, N, dtype=act)
    d = dense(N, K, act, "silu")
    bias, residual, pre, y = rand(g, N), rand(g, T, N, dtype=act), nan(T, N, dtype=act), nan(T, N, dtype=act)
    m.moe_matmul(d, x, None, T, w, None, bias, residual, pre, y, scratch(d, T))
    v, want = ref.matmul(x.double(), w.double(), kind(act), "silu", bias, residual)
    check(pre, v, act, "pre")
    check(y, want, act, "y")
    dx, dw, db = nan(T, K, dtype=act), nan(N, K, dtype=act), nan(N)
    m.moe_matmul_backward(d, x, T, w, pre, dy, dx, dw, db, scratch(d, T))
    grad = ref.matmul_grad(dy, pre, "silu")
    wx, ww = ref.backward(grad, x.double(), w.double(), kind(act))
    check(dx, wx, act, "dx")
    check(dw, ww, act, "dw")
    check(db, ref.bias_grad(grad), F32, "d_bias")


@pytest.mark.parametrize("K", [64, 72, 128, 200, 264])
@pytest.mark.parametrize("act", [BF16, F32])
def test_large_products_of_few_steps(act, K):
    """Sums of one to five steps, some cut, for each layout of the operands."""
    g = gen(510)
    T, N = 3600, 3664
    x, w = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act, std=0.1)
    y = nan(T, N, dtype=act)
    d = dense(N, K, act)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, scratch(d, T))
    check(y, ref.matmul(x.double(), w.double(), kind(act), "none")[1], act, "y")
    d = dense(K, N, act)                                     # dx sums over K rows, dw over K tokens
    dy, w, dx = rand(g, T, K, dtype=act), rand(g, K, N, dtype=act, std=0.1), nan(T, N, dtype=act)
    m.moe_matmul_backward(d, None, T, w, None, dy, dx, None, None, scratch(d, T))
    check(dx, product_of(dy, w.t(), act), act, "dx")
    d = dense(T, N, act)
    dy, x, dw = rand(g, K, T, dtype=act), rand(g, K, N, dtype=act), nan(T, N, dtype=act)
    m.moe_matmul_backward(d, x, K, None, None, dy, None, dw, None, scratch(d, K))
    check(dw, product_of(dy.t(), x.t(), act), act, "dw")


def product_of(a, b, act):
    return ref.product(a.double(), b.double(), kind(act))


@pytest.mark.parametrize("act", [BF16, F32])
def test_large_gated(act):
    T, N, K = 3593, 1824, 456
    g = gen(501)
    x, w = rand(g, T, K, dtype=act), rand(g, 2 * N, K, dtype=act, std=0.1)
    d = dense(N, K, act, "gelu")
    pre, h = nan(T, 2 * N, dtype=act), nan(T, N, dtype=act)
    m.moe_gated(d, x, None, T, w, None, pre, h, None, scratch(d, T))
    v, want = ref.gated(x.double(), w.double(), kind(act), "gelu")
    check(pre, v, act, "pre")
    check(h, want, act, "h")
    codes, scales = torch.full((T, N), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda")
    m.moe_gated(d, x, None, T, w, None, None, codes, scales, scratch(d, T))
    ref.check_mx8(codes, scales, want, "h8")


@pytest.mark.parametrize("K", [128, 256, 384, 1152])
def test_large_mxfp8(K):
    T, N = 3593, 3616
    g = gen(502)
    (x, xs), (w, ws) = mx8(g, T, K), mx8(g, N, K, std=0.1)
    X, W = ref.values(x, xs), ref.values(w, ws)
    d, y = dense(N, K, BF16, "sigmoid", True), nan(T, N, dtype=BF16)
    m.moe_matmul(d, x, xs, T, w, ws, None, None, None, y, scratch(d, T))
    check(y, ref.matmul(X, W, "mx8", "sigmoid")[1], BF16, "y")
    half = N // 2
    d, h, pre = dense(half, K, BF16, "silu", True), nan(T, half, dtype=BF16), nan(T, N, dtype=BF16)
    m.moe_gated(d, x, xs, T, w, ws, pre, h, None, scratch(d, T))
    v, want = ref.gated(X, W, "mx8", "silu")
    check(pre, v, BF16, "pre")
    check(h, want, BF16, "h")


def test_gradients_against_differences():
    """The gradients of a sum of outputs, in fp32, along random directions: central differences of the calls themselves
    with step h are off by the curvature (h^2, with values of order one) and by the outputs' rounding over h."""
    T, N, K, h = 7, 40, 56, 2.0 ** -6
    g = gen(5)
    x, w, b, up = rand(g, T, K), rand(g, 2 * N, K, std=0.2), rand(g, N), rand(g, T, N)

    def loss(d, x, w, b):
        y = nan(T, N)
        if b is None:
            m.moe_gated(d, x, None, T, w, None, None, y, None, scratch(d, T))
        else:
            m.moe_matmul(d, x, None, T, w, None, b, None, None, y, scratch(d, T))
        return (y.double() * up.double()).sum().item()

    for fn in FN:
        d = dense(N, K, F32, fn)
        pre, y, dx, dw, db = nan(T, 2 * N), nan(T, N), torch.empty_like(x), torch.empty_like(w), nan(N)
        m.moe_gated(d, x, None, T, w, None, pre, y, None, scratch(d, T))
        m.moe_gated_backward(d, x, T, w, pre, up, dx, dw, scratch(d, T))
        w1 = w[:N].contiguous()
        pre1, dx1, dw1 = nan(T, N), torch.empty_like(x), torch.empty_like(w1)
        m.moe_matmul(d, x, None, T, w1, None, b, None, pre1, y, scratch(d, T))
        m.moe_matmul_backward(d, x, T, w1, pre1 if fn != "none" else None, up, dx1, dw1, db, scratch(d, T))
        for args, at, grad in [((x, w, None), 0, dx), ((x, w, None), 1, dw), ((x, w1, b), 0, dx1), ((x, w1, b), 1, dw1), ((x, w1, b), 2, db)]:
            v = rand(g, *grad.shape)
            v = v / v.norm()
            ends = []
            for s in (h, -h):
                moved = list(args)
                moved[at] = args[at] + s * v
                ends.append(loss(d, *moved))
            want = (grad.double() * v.double()).sum().item()
            size = grad.double().norm().item()
            assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 16 * h * h * size + 1e-3, (fn, at)


@pytest.mark.parametrize("act", [BF16, F32])
def test_no_tokens(act):
    """T = 0: nothing forward, zeros in the weights' gradients."""
    N, K = 24, 40
    d = dense(N, K, act, "silu")
    ws = scratch(d, 0)
    y = nan(4, N, dtype=act)
    m.moe_matmul(d, None, None, 0, None, None, None, None, None, y, ws)
    m.moe_gated(d, None, None, 0, None, None, None, y, None, ws)
    assert torch.isnan(y).all()
    dw, db, dw2 = nan(N, K, dtype=act), nan(N), nan(2 * N, K, dtype=act)
    m.moe_matmul_backward(d, None, 0, None, None, None, None, dw, db, ws)
    m.moe_gated_backward(d, None, 0, None, None, None, None, dw2, ws)
    assert (dw == 0).all() and (db == 0).all() and (dw2 == 0).all()


@pytest.mark.parametrize("act", [BF16, F32])
def test_not_finite(act):
    """A NaN or an infinity stays in the rows that it enters; an fp32 sum that an infinity enters is not finite."""
    T, N, K = 70, 136, 200
    g = gen(7)
    x, w = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act)
    x[3, 5], x[40, 199], w[130, 0] = float("nan"), float("inf"), float("nan")
    d = dense(N, K, act)
    y = nan(T, N, dtype=act)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, scratch(d, T))
    bad = ~torch.isfinite(y)
    want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    want[3], want[40], want[:, 130] = True, True, True
    assert torch.equal(bad, want)
    x = rand(g, T, K, dtype=act) * 0.01                      # values near the type's ends
    x[0, 0], x[1, 1] = 3.0e38, -3.38e38
    w = rand(g, N, K, dtype=act).clamp(-0.5, 0.5)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, scratch(d, T))
    check(y, ref.matmul(x.double(), w.double(), kind(act), "none")[1], act, "large")
    x, w = rand(g, T, K, dtype=act, std=1e-30), rand(g, N, K, dtype=act, std=1e-2)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, scratch(d, T))
    check(y, ref.matmul(x.double(), w.double(), kind(act), "none")[1], act, "small")


def test_mxfp8_nan_blocks():
    T, N, K = 33, 64, 256
    g = gen(8)
    for act in (BF16, F32):
        (x, xs), (w, ws) = mx8(g, T, K), mx8(g, N, K)
        xs[5, 3], ws[9, 0] = 255, 255
        d = dense(N, K, act, "none", True)
        y = nan(T, N, dtype=act)
        m.moe_matmul(d, x, xs, T, w, ws, None, None, None, y, scratch(d, T))
        want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
        want[5], want[:, 9] = True, True
        assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("T", [3, 20, 50, 200])
def test_mxfp8_scales_of_the_whole_range(T):
    N, K = 64, 256
    g = gen(17)
    for act in (BF16, F32):
        for sx, sw in ((0, 180), (1, 180), (180, 0), (246, 10), (10, 246), (246, 7)):
            (x, xs), (w, ws) = mx8(g, T, K), mx8(g, N, K)
            xs.fill_(sx), ws.fill_(sw)
            d, y = dense(N, K, act, "none", True), nan(T, N, dtype=act)
            m.moe_matmul(d, x, xs, T, w, ws, None, None, None, y, scratch(d, T))
            X, W = ref.values(x, xs), ref.values(w, ws)
            want = ref.product(X, W, "mx8" if act == BF16 else "bf16")
            # a value is right to half of bf16's smallest number, 2^-133
            tiny = 2.0 ** -134 * (X.abs().sum(1, keepdim=True) + W.abs().sum(1))
            check(y, Val(want.v, want.e + tiny), act, f"y {sx} {sw}")


NORMS = [(1, 128, BF16, "none", 1, 1), (3, 256, F32, "token", 0, 1), (1, 4096, BF16, "none", 1, 1), (70, 640, BF16, "element", 1, 1),
         (33, 4352, F32, "element", 1, 1), (5, 16384, BF16, "token", 0, 1), (2, 8320, F32, "none", 1, 0), (257, 2176, BF16, "none", 0, 0)]


@pytest.mark.parametrize("T,d,act,gate_kind,has_post,has_pre", NORMS)
def test_norm_to_8_bits(T, d, act, gate_kind, has_post, has_pre):
    g = gen(9)
    sh = m.make_shape(d, 128, 1, 1, act_dtype=m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32)
    x, y = rand(g, T, d, dtype=act, std=2.0), rand(g, T, d, dtype=act)
    post, pre = (1 + rand(g, d, std=0.1) if has_post else None), (1 + rand(g, d, std=0.1) if has_pre else None)
    gate = {"none": lambda: None, "token": lambda: torch.rand(T, generator=g, device="cuda"),
            "element": lambda: rand(g, T, d, dtype=act)}[gate_kind]()
    if T > 2:
        x[1], y[1] = 0, 0                                     # a row of zeros
        x[2, 7] = float("inf")                                # normed: inf / inf there, zeros elsewhere
    codes, scales = torch.full((T, d), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, d // 32, dtype=torch.uint8, device="cuda")
    x_out = nan(T, d, dtype=act)
    kinds = {"none": m.MOE_GATE_NONE, "token": m.MOE_GATE_TOKEN, "element": m.MOE_GATE_ELEMENT}
    m.moe_block_norm_mx8(sh, x, y, T, post, pre, gate, kinds[gate_kind], 0.7, 1e-5, x_out, codes, scales)
    u, normed = block_ref.norm_forward(x, Val(y), post, pre, None if gate is None else gate.reshape(T, -1), 0.7, 1e-5)
    fine = torch.ones(T, dtype=torch.bool, device="cuda")
    if T > 2:
        fine[2] = False
        assert scales[2, 0] == 255 and (codes[2, :32] == 0).all() and (scales[2, 1:] < 255).all()
        assert not has_pre or ((scales[2, 1:] == 1).all() and ((codes[2, 32:] & 127) == 0).all())
    check(x_out[fine], u[fine], act, "x_out")
    ref.check_mx8(codes[fine], scales[fine], (normed if has_pre else u)[fine], "normed")
    again = torch.empty_like(codes), torch.empty_like(scales)
    m.moe_block_norm_mx8(sh, x, y, T, post, pre, gate, kinds[gate_kind], 0.7, 1e-5, None, again[0].view(torch.float8_e4m3fn),
                         again[1].view(torch.float8_e8m0fnu))
    assert torch.equal(again[0], codes) and torch.equal(again[1], scales)
    here = x.clone()                                          # the stream in its own place
    m.moe_block_norm_mx8(sh, here, y, T, post, pre, gate, kinds[gate_kind], 0.7, 1e-5, here, *again)
    assert torch.equal(here[fine], x_out[fine]) and torch.equal(again[0], codes) and torch.equal(again[1], scales)


def test_rows_to_8_bits():
    """y and pre_gamma left out: rows as they are, at every magnitude."""
    g = gen(10)
    T, d = 40, 256
    x = rand(g, T, d) * 2.0 ** torch.randint(-140, 120, (T, d // 32), generator=g, device="cuda").float().repeat_interleave(32, 1)
    codes, scales = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, d // 32, dtype=torch.uint8, device="cuda")
    m.moe_block_norm_mx8(m.make_shape(d, 128, 1, 1, act_dtype=m.MOE_DT_F32), x, None, T, None, None, None, 0, 1.0, 1e-5, None, codes, scales)
    ref.check_mx8(codes, scales, Val(x), "rows")


def _block(T, d, f, act, g):
    return rand(g, T, d, dtype=act), 1 + rand(g, d, std=0.1), rand(g, 2 * f, d, dtype=act, std=0.05), rand(g, d, f, dtype=act, std=0.05)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_dense_block_and_its_gradient(T):
    """norm, gated block, down projection onto the stream, and back, in fp32 against autograd in 64 bits: every step is
    right to some 2^-20 of its size here, so that the whole is to 1e-4 of each gradient's largest value."""
    g, d, f = gen(11), 256, 384
    x, gamma, w, wd = _block(T, d, f, F32, g)
    up = rand(g, T, d)
    sh = m.make_shape(d, 128, 1, 1, act_dtype=m.MOE_DT_F32)
    gate, down = dense(f, d, F32, "silu"), dense(d, f, F32)
    ws = scratch(gate, T), scratch(down, T)
    normed, pre, h, y = nan(T, d), nan(T, 2 * f), nan(T, f), nan(T, d)
    m.moe_block_norm(sh, x, None, T, None, gamma, None, 0, 1.0, 1e-5, None, normed)
    m.moe_gated(gate, normed, None, T, w, None, pre, h, None, ws[0])
    m.moe_matmul(down, h, None, T, wd, None, None, x, None, y, ws[1])
    dh, dwd, dn, dw, dx, dg = nan(T, f), nan(d, f), nan(T, d), nan(2 * f, d), nan(T, d), nan(d)
    m.moe_matmul_backward(down, h, T, wd, None, up, dh, dwd, None, ws[1])
    m.moe_gated_backward(gate, normed, T, w, pre, dh, dn, dw, ws[0])
    m.moe_block_norm_backward(sh, x, None, T, None, gamma, None, 0, 1.0, 1e-5, up, dn, dx, None, None, None, dg, m.workspace(sh, T))
    X, G, W, WD = (t.double().cpu().requires_grad_() for t in (x, gamma, w, wd))
    n = X * torch.rsqrt(X.square().mean(-1, keepdim=True) + 1e-5) * G
    v = n @ W.t()
    out = X + (torch.nn.functional.silu(v[:, :f]) * v[:, f:]) @ WD.t()
    out.backward(up.double().cpu())
    for got, want in ((y, out.detach()), (dx, X.grad), (dg, G.grad), (dw, W.grad), (dwd, WD.grad)):
        assert (got.double().cpu() - want).abs().max() <= 1e-4 * want.abs().max()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_dense_block_in_8_bits(T):
    """norm, gated block and down projection through MXFP8 at every hand-over: each step against the plain form of what
    the step before wrote."""
    g, d, f = gen(12), 256, 384
    x, gamma, w, wd = _block(T, d, f, BF16, g)
    sh = m.make_shape(d, 128, 1, 1)

    def eight(rows, shape, pre=None):
        q = torch.empty(rows.shape, dtype=torch.uint8, device="cuda"), torch.empty(rows.shape[0], rows.shape[1] // 32, dtype=torch.uint8, device="cuda")
        m.moe_block_norm_mx8(shape, rows, None, rows.shape[0], None, pre, None, 0, 1.0, 1e-5, None, *q)
        return q

    (n8, ns), (w8, wss), (d8, ds) = eight(x, sh, gamma), eight(w, sh), eight(wd, m.make_shape(f, 128, 1, 1))
    ref.check_mx8(d8, ds, Val(wd), "weight")
    gate, down = dense(f, d, BF16, "silu", True), dense(d, f, BF16, "none", True)
    h8, hs, y = torch.empty(T, f, dtype=torch.uint8, device="cuda"), torch.empty(T, f // 32, dtype=torch.uint8, device="cuda"), x.clone()
    m.moe_gated(gate, n8, ns, T, w8, wss, None, h8, hs, scratch(gate, T))
    ref.check_mx8(h8, hs, ref.gated(ref.values(n8, ns), ref.values(w8, wss), "mx8", "silu")[1], "h")
    m.moe_matmul(down, h8, hs, T, d8, ds, None, y, None, y, scratch(down, T))
    check(y, ref.matmul(ref.values(h8, hs), ref.values(d8, ds), "mx8", "none", None, x)[1], BF16, "y")


@pytest.mark.parametrize("T", [1, 24, 200])
@pytest.mark.parametrize("act", [BF16, F32])
def test_streams_and_graph_replays_give_the_same_bits(act, T):
    """A forward and backward pass eagerly, on another stream, and captured: replays on new inputs, with eager calls of
    the same shapes and another workspace in between."""
    N, K = 264, 520
    g = gen(13)
    d = dense(N, K, act, "silu")
    x, w, up = rand(g, T, K, dtype=act), rand(g, 2 * N, K, dtype=act, std=0.1), rand(g, T, N, dtype=act)

    def step(x, out, ws):
        pre, h, dx, dw, y, db = out
        m.moe_gated(d, x, None, T, w, None, pre, h, None, ws)
        m.moe_gated_backward(d, x, T, w, pre, up, dx, dw, ws)
        m.moe_matmul(d, x, None, T, w[:N], None, None, up, None, y, ws)
        m.moe_matmul_backward(d, None, T, w[:N], h, up, None, None, db, ws)

    def outputs():
        return [nan(T, 2 * N, dtype=act), nan(T, N, dtype=act), nan(T, K, dtype=act), nan(2 * N, K, dtype=act), nan(T, N, dtype=act), nan(N)]

    want, ws = outputs(), scratch(d, T)
    step(x, want, ws)
    side, other, ws2 = torch.cuda.Stream(), outputs(), scratch(d, T)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, other, ws2)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    static, got, ws3 = x.clone(), outputs(), scratch(d, T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, got, ws3)
    for seed in range(3):
        new = rand(gen(50 + seed), T, K, dtype=act)
        static.copy_(new)
        graph.replay()
        step(new, want, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), seed


@pytest.mark.parametrize("T", [3, 70])
def test_offsets_past_32_bits(T):
    """A weight of more than 4 GiB: its last rows forward, and their share of the input's gradient and of their own."""
    K, last = 4096, 72
    N = (1 << 32) // (2 * K) + 1032
    g = gen(15)
    w = torch.zeros(N, K, dtype=BF16, device="cuda")
    w[-last:] = rand(g, last, K, dtype=BF16, std=0.1)
    x, dy = rand(g, T, K, dtype=BF16), rand(g, T, N, dtype=BF16)
    d = dense(N, K, BF16)
    ws, y, dx, dw = scratch(d, T), nan(T, N, dtype=BF16), nan(T, K, dtype=BF16), torch.empty_like(w)
    m.moe_matmul(d, x, None, T, w, None, None, None, None, y, ws)
    assert (y[:, :-last] == 0).all()
    check(y[:, -last:], ref.product(x.double(), w[-last:].double(), "bf16"), BF16, "y")
    m.moe_matmul_backward(d, x, T, w, None, dy, dx, dw, None, ws)
    wx = ref.product(dy[:, -last:].double(), w[-last:].double().t(), "bf16")
    check(dx, Val(wx.v, wx.e * (N // last)), BF16, "dx")      # (as many more additions, of zeros)
    check(dw[-last:], ref.product(dy[:, -last:].double().t(), x.double().t(), "bf16"), BF16, "dw")


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace and outputs."""
    g = gen(16)
    T, N, K = 300, 1032, 2056
    for act in (BF16, F32):
        d = dense(N, K, act, "gelu")
        xs, w = [rand(g, T, K, dtype=act) for _ in range(2)], rand(g, 2 * N, K, dtype=act, std=0.1)
        want = [nan(T, N, dtype=act) for _ in xs]
        for x, y in zip(xs, want):
            m.moe_gated(d, x, None, T, w, None, None, y, None, scratch(d, T))
        torch.cuda.synchronize()
        streams, got, ws = [torch.cuda.Stream() for _ in xs], [nan(T, N, dtype=act) for _ in xs], [scratch(d, T) for _ in xs]
        torch.cuda.synchronize()
        for _ in range(5):
            for k in range(2):
                m.moe_gated(d, xs[k], None, T, w, None, None, got[k], None, ws[k], stream=streams[k])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_past_the_last_token_are_left_alone():
    T, N, K = 5, 72, 136
    g = gen(14)
    for act in (BF16, F32):
        d = dense(N, K, act, "gelu")
        x, w = rand(g, T, K, dtype=act), rand(g, 2 * N, K, dtype=act)
        y, h, pre, dx = (torch.full((T + 3, n), 7.5, dtype=act, device="cuda") for n in (N, N, 2 * N, K))
        m.moe_matmul(d, x, None, T, w[:N], None, None, None, None, y, scratch(d, T))
        m.moe_gated(d, x, None, T, w, None, pre, h, None, scratch(d, T))
        m.moe_gated_backward(d, x, T, w, pre, h, dx, None, scratch(d, T))
        assert all((t[T:] == 7.5).all() and torch.isfinite(t).all() for t in (y, h, pre, dx))
