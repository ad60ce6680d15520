"""What the dense products accept and refuse at the edges of their contract, on the host (fake device pointers that are
never dereferenced: every accepted call has no tokens)."""
import ctypes
import os

import pytest

m = pytest.importorskip("routed_expert_ffn_router_amd")

from test_dense_abi import (B, DW, DX, DY, INV, OK, P, R, UNS, W, WS, WSC, WSP, X, XS, Y, gated, gated_backward, matmul,
                            matmul_backward)


@pytest.mark.parametrize("f", [matmul, gated])
def test_mxfp8_columns_in_whole_blocks(f):
    for K in (32, 64, 96, 160, 1056):
        assert f(T=0, ops=1, K=K) == OK
        assert f(ops=1, K=K) == INV                            # no scales
        assert m.moe_dense_workspace_bytes(m.make_dense(256, K, operands=m.MOE_OPERANDS_MXFP8), 1) > 0
    for K in (8, 16, 48, 72, 1064):
        assert f(T=0, ops=1, K=K) == UNS and f(ops=1, xs=XS, ws=WSC, K=K) == UNS
        assert m.moe_dense_workspace_bytes(m.make_dense(256, K, operands=m.MOE_OPERANDS_MXFP8), 1) == 0


@pytest.mark.parametrize("f", [matmul, gated])
def test_operands_of_a_forward_call(f):
    assert f(T=0, x=None, w=None, y=None, s=None, n=0) == OK
    for bad in ({"x": None}, {"w": None}, {"y": None}, {"y": X}, {"y": W}, {"p": X}, {"p": Y}, {"y": Y + 8}, {"p": P + 8},
                {"xs": XS}, {"ws": WSC}, {"xs": XS, "ws": WSC}, {"ops": 1}, {"ops": 1, "xs": XS}, {"ops": 1, "ws": WSC},
                {"ops": 1, "xs": XS + 2, "ws": WSC}, {"ops": 1, "xs": XS, "ws": WSC + 1}):
        assert f(**bad) == INV, bad


@pytest.mark.parametrize("N,K,act", [(256, 32, 1), (264, 1056, 0), (32, 160, 1)])
def test_a_workspace_of_blocks_serves_every_call_with_fewer_tokens(N, K, act):
    d = m.make_dense(N, K, act, m.MOE_OPERANDS_MXFP8)
    sizes = [m.moe_dense_workspace_bytes(d, T) for T in [*range(600), *range(4000, 4100), 65535, 65536]]
    assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("act", [0, 1])
def test_few_tokens_bring_no_room_for_copies(act):
    """A decoded token's MXFP8 products read their operands where they are: a workspace of the scales' copies at most."""
    for N, K in ((8192, 4096), (8192, 4128)):
        d = m.make_dense(N, K, act, m.MOE_OPERANDS_MXFP8)
        scales = 0 if K % 128 == 0 else (2 * N + 32) * (K + 127) // 128 * 4
        for T in (1, 32):
            assert 0 < m.moe_dense_workspace_bytes(d, T) <= scales + 1024
        assert m.moe_dense_workspace_bytes(d, 33) > 1 << 20
        for f in (matmul, gated):
            size = m.moe_dense_workspace_bytes(d, 1)
            assert f(N=N, K=K, act=act, ops=1, xs=XS, ws=WSC, T=33, n=size) == WSP


#: bytes of the arrays of these calls: 3 tokens, 256 rows, 512 columns, bf16
WEIGHT, TOKENS, ROWS = 256 * 512 * 2, 3 * 512 * 2, 3 * 256 * 2


def test_outputs_that_meet_an_operand_half_way():
    """What only the first addresses' comparison let through: ranges that overlap."""
    for bad in ({"y": X + 16}, {"y": X - ROWS + 16}, {"y": W + WEIGHT - 16}, {"p": W + 4096}, {"y": P + 16}, {"p": Y + ROWS - 16},
                {"r": Y + 16}, {"r": Y - 16}, {"r": P + 16}, {"b": Y + 512}, {"p": B - 16}, {"s": X}, {"s": W + 256}, {"s": Y},
                {"x": WS + 256}, {"y": WS + 256}, {"b": WS + 512}, {"r": WS + 1024}, {"p": WS}):
        assert matmul(**bad) == INV, bad
    for bad in ({"y": X + 16}, {"y": W + 2 * WEIGHT - 16}, {"p": Y + 16}, {"p": Y - 2 * ROWS + 16}, {"y": P + 2 * ROWS - 16},
                {"ys": Y + 16}, {"ys": P + 1}, {"s": W + 2 * WEIGHT - 256}, {"x": WS + 256}, {"ys": WS + 3}):
        assert gated(**bad) == INV, bad
    for f in (matmul_backward, gated_backward):
        for bad in ({"dx": X + 16}, {"dw": W + 16}, {"dx": DW + 16}, {"dw": DX + TOKENS - 16}, {"dx": DY - TOKENS + 16}, {"dx": P + 16},
                    {"dw": P - 16}, {"s": DW}, {"s": DX - 256}, {"dx": WS + 256}, {"dy": WS + 256}):
            assert f(**bad) == INV, (f.__name__, bad)
    assert matmul_backward(db=DW + 16) == INV and matmul_backward(db=WS + 256) == INV and matmul_backward(T=0, db=DW + 16) == INV
    assert gated_backward(T=0, dw=W + 16) == INV


def test_norm_outputs_that_meet_an_operand_half_way():
    sh = m.make_shape(256, 128, 16, 2)

    def f(**kw):
        a = dict(x=X, y=Y, T=2, post=B, pre=R, gate=None, kind=0, out=P, c=W, s=XS) | kw
        return m.library().moe_block_norm_mx8(ctypes.byref(sh), a["x"], a["y"], a["T"], a["post"], a["pre"], a["gate"], a["kind"], 1.0, 1e-5,
                                              a["out"], a["c"], a["s"], 0)

    for bad in ({"c": X + 16}, {"c": Y - 496}, {"c": P + 1008}, {"s": X + 1}, {"s": W + 511}, {"s": P + 3}, {"c": B + 1008}, {"s": R + 4},
                {"kind": 2, "gate": W + 16}, {"kind": 1, "gate": W + 508}):
        assert f(**bad) == INV, bad


def test_a_forked_child_asks_torch_for_the_gpu_again():
    """torch refuses a GPU that was initialised before a fork; the binding keeps nothing that passes its check by."""
    kept, m._torch_c = m._torch_c, object()                     # as after a first call
    try:
        child = os.fork()
        if child == 0:
            os._exit(0 if m._torch_c is None else 1)
        assert os.waitstatus_to_exitcode(os.waitpid(child, 0)[1]) == 0
        assert m._torch_c is not None
    finally:
        m._torch_c = kept


def test_a_workspace_that_is_too_small_is_named_as_that():
    """... where its end meets the next array, too."""
    for f in (matmul, gated, matmul_backward, gated_backward):
        assert f(s=P - 256, n=256) == WSP, f.__name__
