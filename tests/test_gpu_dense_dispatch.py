"""Every kernel that the dense products' rule can choose, at a size of dense_dispatch, against the plain float64 forms of
dense_ref."""
import math

import pytest
import torch

import dense_ref as ref
from block_ref import check
from dense_dispatch import CASES

pytestmark = pytest.mark.gpu

from test_gpu_dense import BF16, F32, FN, dense, gen, mx8, nan, rand, scratch

if torch.cuda.is_available():
    import routed_expert_ffn_router_amd as m      # must load: no fallback path exists

ALL = [(op, f, n, *size) for (op, f), sizes in CASES.items() for n, size in enumerate(sizes)]


def operands(g, T, R, K, f, act):
    """x, its scales, w, its scales, and both in 64 bits"""
    if f == "mx8":
        (x, xs), (w, ws) = mx8(g, T, K), mx8(g, R, K, std=0.1)
        return x, xs, w, ws, ref.values(x, xs), ref.values(w, ws)
    x, w = rand(g, T, K, dtype=act), rand(g, R, K, dtype=act, std=0.1)
    return x, None, w, None, x.double(), w.double()


def forward(op, f, act, how, n, T, N, K):
    g = gen(700 + n)
    fn, R = FN[n % 4], N if op == "matmul" else 2 * N
    x, xs, w, ws, X, W = operands(g, T, R, K, f, act)
    d = dense(N, K, act, fn, f == "mx8")
    if op == "matmul":
        bias, residual, pre, y = rand(g, N), rand(g, T, N, dtype=act), nan(T, N, dtype=act), nan(T, N, dtype=act)
        m.moe_matmul(d, x, xs, T, w, ws, bias, residual, pre, y, scratch(d, T))
        v, want = ref.matmul(X, W, how, fn, bias, residual)
        check(pre, v, act, "pre")
        check(y, want, act, "y")
        return
    v, want = ref.gated(X, W, how, fn)
    pre = nan(T, 2 * N, dtype=act)
    if op == "gated":
        h = nan(T, N, dtype=act)
        m.moe_gated(d, x, xs, T, w, ws, pre, h, None, scratch(d, T))
        check(h, want, act, "h")
    else:
        codes, scales = torch.full((T, N), 170, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda")
        m.moe_gated(d, x, xs, T, w, ws, pre, codes, scales, scratch(d, T))
        ref.check_mx8(codes, scales, want, "h8")
    check(pre, v, act, "pre")


@pytest.mark.parametrize("op,f,n,T,N,K", [c for c in ALL if c[0] not in ("dx", "dw")])
def test_forward(op, f, n, T, N, K):
    forward(op, f, F32 if f == "f32" else BF16, "bf16" if f == "bf16" else f, n, T, N, K)


@pytest.mark.parametrize("op,f,n,T,N,K", [c for c in ALL if c[1] == "mx8"])
def test_forward_of_copies(op, f, n, T, N, K):
    """MXFP8 operands of fp32 outputs: the bf16 kernels, on the copies."""
    forward(op, f, F32, "bf16", n, T, N, K)


@pytest.mark.parametrize("op,f,n,T,N,K", [c for c in ALL if c[0] in ("dx", "dw")])
def test_gradient(op, f, n, T, N, K):
    g, act = gen(800 + n), F32 if f == "f32" else BF16
    x, w, dy = rand(g, T, K, dtype=act), rand(g, N, K, dtype=act, std=0.1), rand(g, T, N, dtype=act)
    d = dense(N, K, act)
    if op == "dx":
        dx = nan(T, K, dtype=act)
        m.moe_matmul_backward(d, None, T, w, None, dy, dx, None, None, scratch(d, T))
        check(dx, ref.product(dy.double(), w.double().t(), f), act, "dx")
    else:
        dw = nan(N, K, dtype=act)
        m.moe_matmul_backward(d, x, T, None, None, dy, None, dw, None, scratch(d, T))
        check(dw, ref.product(dy.double().t(), x.double().t(), f), act, "dw")


@pytest.mark.parametrize("op,n,T,N,K", [(op, n, *size) for op, f, n, *size in ALL if f == "f32" and op in ("matmul", "dx", "dw")])
def test_fp32_infinity_in_every_tile(op, n, T, N, K):
    """An infinity in the first and the last row of one operand and a zero against it: infinite, NaN and finite sums."""
    g = gen(900 + n)
    d = dense(N, K, F32)
    a, b = {"matmul": ((T, K), (N, K)), "dx": ((T, N), (N, K)), "dw": ((T, N), (T, K))}[op]
    a, b = rand(g, *a), rand(g, *b)
    if op == "matmul":
        a[0, 0], a[-1, -1], b[3, 0] = math.inf, -math.inf, 0.0
        y, want = nan(T, N), a.double().cpu() @ b.double().cpu().t()
        m.moe_matmul(d, a, None, T, b, None, None, None, None, y, scratch(d, T))
    elif op == "dx":
        a[0, 0], a[-1, -1], b[0, 3] = math.inf, -math.inf, 0.0
        y, want = nan(T, K), a.double().cpu() @ b.double().cpu()
        m.moe_matmul_backward(d, None, T, b, None, a, y, None, None, scratch(d, T))
    else:
        a[0, 0], a[-1, -1], b[0, 3] = math.inf, -math.inf, 0.0
        y, want = nan(N, K), a.double().cpu().t() @ b.double().cpu()
        m.moe_matmul_backward(d, b, T, None, None, a, None, y, None, scratch(d, T))
    y = y.cpu()
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y == math.inf, want == math.inf)
    assert torch.equal(y == -math.inf, want == -math.inf) and want.isnan().sum() == 1 and want.isinf().any()
