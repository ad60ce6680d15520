"""The dense products on the GPU at the edges of their contract, against the plain float64 forms of dense_ref."""
import pytest
import torch

import dense_ref as ref
from block_ref import check

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
