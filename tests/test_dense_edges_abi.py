"""What the dense products accept and refuse at the edges of their contract, on the host (fake device pointers that are
never dereferenced: every accepted call has no tokens)."""
import pytest

m = pytest.importorskip("routed_expert_ffn_router_amd")

from test_dense_abi import INV, OK, P, UNS, W, WSC, WSP, X, XS, Y, gated, matmul


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
