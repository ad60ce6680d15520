"""Refusals of the dense products and of the norm to 8 bits, on the host: every bad argument gives its status before
anything is launched (fake device pointers that are never dereferenced), and the binding refuses tensors whose layout
the library cannot see."""
import ctypes

import pytest
import torch

m = pytest.importorskip("routed_expert_ffn_router_amd")

L = m.library()
INV, UNS, WSP, OK = m.MOE_ERR_INVALID, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE, m.MOE_OK
X, W, B, R, P, Y, WS, XS, WSC, HS, DY, DX, DW, DB = ((i + 1) << 24 for i in range(14))      # distinct fake device addresses
BIG = 1 << 40


def _dense(kw):
    names = dict(N=256, K=512, act=1, ops=0, fn=1)
    return ctypes.byref(m.make_dense(*(kw.pop(k, v) for k, v in names.items())))


def matmul(**kw):
    d = _dense(kw)
    a = dict(x=X, xs=None, T=3, w=W, ws=None, b=B, r=R, p=P, y=Y, s=WS, n=BIG) | kw
    return L.moe_matmul(d, a["x"], a["xs"], a["T"], a["w"], a["ws"], a["b"], a["r"], a["p"], a["y"], a["s"], a["n"], 0)


def gated(**kw):
    d = _dense(kw)
    a = dict(x=X, xs=None, T=3, w=W, ws=None, p=P, y=Y, ys=None, s=WS, n=BIG) | kw
    return L.moe_gated(d, a["x"], a["xs"], a["T"], a["w"], a["ws"], a["p"], a["y"], a["ys"], a["s"], a["n"], 0)


def matmul_backward(**kw):
    d = _dense(kw)
    a = dict(x=X, T=3, w=W, p=P, dy=DY, dx=DX, dw=DW, db=DB, s=WS, n=BIG) | kw
    return L.moe_matmul_backward(d, a["x"], a["T"], a["w"], a["p"], a["dy"], a["dx"], a["dw"], a["db"], a["s"], a["n"], 0)


def gated_backward(**kw):
    d = _dense(kw)
    a = dict(x=X, T=3, w=W, p=P, dy=DY, dx=DX, dw=DW, s=WS, n=BIG) | kw
    return L.moe_gated_backward(d, a["x"], a["T"], a["w"], a["p"], a["dy"], a["dx"], a["dw"], a["s"], a["n"], 0)


@pytest.mark.parametrize("f", [matmul, gated, matmul_backward, gated_backward])
def test_descriptions(f):
    for bad in ({"N": 0}, {"K": -8}, {"act": 2}, {"ops": 2}, {"ops": -1}, {"fn": 4}, {"fn": -1}, {"T": -1}):
        assert f(**bad) == INV, bad
    for bad in ({"N": 12}, {"K": 20}, {"T": 65537}, {"N": (1 << 20) + 8}, {"K": (1 << 20) + 8}, {"N": 1 << 17, "K": 1 << 17}):
        assert f(**bad) == UNS, bad
    for bad in ({"x": X + 8}, {"w": W + 4}, {"s": WS + 16}, {"s": None}):
        assert f(**bad) == INV, bad
    assert f(n=256) == WSP


def test_no_description():
    assert L.moe_matmul(None, X, None, 1, W, None, B, R, P, Y, WS, BIG, 0) == INV
    assert L.moe_gated(None, X, None, 1, W, None, P, Y, None, WS, BIG, 0) == INV
    assert L.moe_matmul_backward(None, X, 1, W, P, DY, DX, DW, DB, WS, BIG, 0) == INV
    assert L.moe_gated_backward(None, X, 1, W, P, DY, DX, DW, WS, BIG, 0) == INV
    assert L.moe_dense_workspace_bytes(None, 1) == 0


@pytest.mark.parametrize("f", [matmul, gated])
def test_forward(f):
    assert f(T=0, x=None, w=None, y=None, s=None, n=0) == OK
    for bad in ({"x": None}, {"w": None}, {"y": None}, {"y": X}, {"y": W}, {"p": X}, {"p": Y}, {"y": Y + 8}, {"p": P + 8},
                {"xs": XS}, {"ws": WSC}, {"xs": XS, "ws": WSC}, {"ops": 1}, {"ops": 1, "xs": XS}, {"ops": 1, "ws": WSC},
                {"ops": 1, "xs": XS + 2, "ws": WSC}, {"ops": 1, "xs": XS, "ws": WSC + 1}):
        assert f(**bad) == INV, bad
    assert f(ops=1, xs=XS, ws=WSC, K=64) == UNS


def test_epilogues():
    for bad in ({"b": B + 4}, {"r": R + 8}, {"y": B}, {"p": R}, {"p": B}):
        assert matmul(**bad) == INV, bad
    assert gated(N=264, ys=HS) == UNS                          # h in 8 bits has whole blocks of 32
    for bad in ({"ys": Y}, {"ys": P}, {"ys": X}):
        assert gated(**bad) == INV, bad


@pytest.mark.parametrize("f", [matmul_backward, gated_backward])
def test_backward(f):
    assert f(T=0, x=None, w=None, p=None, dy=None, dx=None, dw=None, s=None, n=0, **({"db": None} if f is matmul_backward else {})) == OK
    assert f(T=0, dw=DW + 4) == INV and f(T=0, dw=DX) == INV
    assert f(ops=1) == UNS
    for bad in ({"x": None}, {"w": None}, {"p": None}, {"dy": None}, {"dx": X}, {"dx": DY}, {"dw": W}, {"dw": DX}, {"dx": P},
                {"dy": DY + 8}, {"dx": DX + 8}, {"dw": DW + 8}, {"p": P + 8}):
        assert f(**bad) == INV, bad


def test_what_is_wanted():
    assert matmul_backward(dx=None, dw=None, db=None) == INV and gated_backward(dx=None, dw=None) == INV
    assert matmul_backward(fn=0) == INV                        # pre of no activation
    assert matmul_backward(db=DB + 4) == INV and matmul_backward(db=DW) == INV and matmul_backward(T=0, db=DW) == INV


def test_norm_to_8_bits():
    sh = m.make_shape(256, 128, 16, 2)

    def f(sh=sh, **kw):
        a = dict(x=X, y=Y, T=2, post=B, pre=R, gate=None, kind=0, alpha=1.0, eps=1e-5, out=P, c=W, s=XS) | kw
        return L.moe_block_norm_mx8(ctypes.byref(sh), a["x"], a["y"], a["T"], a["post"], a["pre"], a["gate"], a["kind"], a["alpha"],
                                    a["eps"], a["out"], a["c"], a["s"], 0)

    assert f(T=0, x=None, c=None, s=None) == OK
    assert f(T=-1) == INV and f(T=65537) == UNS and f(sh=m.make_shape(200, 128, 16, 2)) == UNS
    assert f(sh=m.make_shape(16512, 128, 16, 2)) == UNS
    for bad in ({"eps": 0.0}, {"alpha": float("nan")}, {"kind": 3, "gate": DY}, {"kind": 1}, {"gate": DY}, {"x": None}, {"c": None},
                {"s": None}, {"y": None}, {"c": X}, {"c": Y}, {"c": P}, {"s": W}, {"s": P}, {"c": W + 8}, {"x": X + 8}, {"post": B + 4},
                {"pre": R + 4}, {"out": P + 8}, {"kind": 2, "gate": DY + 8}, {"kind": 2, "gate": W}):
        assert f(**bad) == INV, bad


@pytest.mark.parametrize("N,K,act,ops", [(256, 512, 1, 0), (2048, 4096, 0, 0), (8, 8, 1, 0), (65536, 128, 1, 1), (264, 1152, 0, 1)])
def test_a_workspace_serves_every_call_with_fewer_tokens(N, K, act, ops):
    d = m.make_dense(N, K, act, ops)
    sizes = [m.moe_dense_workspace_bytes(d, T) for T in [*range(600), *range(4000, 4200), 65535, 65536]]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    assert m.moe_dense_workspace_bytes(d, -1) == 0 and m.moe_dense_workspace_bytes(m.make_dense(12, K, act, ops), 1) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """A host tensor, another dtype, a strided view and a short tensor, before any launch."""
    d, d8 = m.make_dense(64, 128), m.make_dense(64, 128, operands=m.MOE_OPERANDS_MXFP8)
    x, sh = torch.zeros(2, 128, dtype=torch.bfloat16), m.make_shape(128, 128, 1, 1)
    for call in (
        lambda: m.moe_matmul(d, x, None, 2, W, None, None, None, None, Y, WS, BIG, stream=0),
        lambda: m.moe_matmul(d, X, None, 2, x.float(), None, None, None, None, Y, WS, BIG, stream=0),
        lambda: m.moe_matmul(d8, X, x, 2, W, WSC, None, None, None, Y, WS, BIG, stream=0),
        lambda: m.moe_matmul(d, X, torch.zeros(2, 4, dtype=torch.uint8), 2, W, None, None, None, None, Y, WS, BIG, stream=0),
        lambda: m.moe_gated(d, X, None, 2, W, None, None, x[:, ::2], None, WS, BIG, stream=0),
        lambda: m.moe_gated(d, X, None, 2, W, None, None, x, HS, WS, BIG, stream=0),
        lambda: m.moe_matmul_backward(d, X, 2, W, None, x[:1], DX, DW, None, WS, BIG, stream=0),
        lambda: m.moe_gated_backward(d, X, 2, W, P, DY, x, DW, WS, BIG, stream=0),
        lambda: m.moe_block_norm_mx8(sh, x, None, 2, None, R, None, 0, 1.0, 1e-5, None, W, XS, stream=0),
        lambda: m.moe_block_norm_mx8(sh, X, None, 2, None, R, None, 0, 1.0, 1e-5, None, x, XS, stream=0),
    ):
        with pytest.raises(m.MoeError) as err:
            call()
        assert err.value.status == INV
