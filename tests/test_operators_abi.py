"""Refusals of the operators around the experts, on the host: every bad argument gives its status before
anything is launched (fake device pointers that are never dereferenced), and the binding refuses tensors
whose layout the library cannot see."""
import ctypes

import pytest
import torch

m = pytest.importorskip("routed_expert_ffn_router_amd")

A, B, C, D, E_, F = ((i + 1) << 24 for i in range(6))     # distinct fake device addresses
L = m.library()
SH = m.make_shape(256, 128, 16, 2)
INV, UNS, WSP, OK = m.MOE_ERR_INVALID, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE, m.MOE_OK


def r(s):
    return ctypes.byref(s)


BAD_SHAPE = m.make_shape(200, 128, 16, 2)


def test_dispatch():
    f = L.moe_dispatch
    assert f(r(SH), None, 0, None, None, 0) == OK
    assert f(None, A, 1, B, C, 0) == INV
    assert f(r(BAD_SHAPE), A, 1, B, C, 0) == UNS
    assert f(r(SH), A, -1, B, C, 0) == INV
    assert f(r(SH), A, 65537, B, C, 0) == UNS
    for bad in ((None, B, C), (A, None, C), (A, B, None), (A, B, A), (A + 8, B, C), (A, B, C + 8)):
        assert f(r(SH), bad[0], 1, bad[1], bad[2], 0) == INV


def test_dispatch_backward():
    f = L.moe_dispatch_backward
    assert f(r(SH), None, 0, None, None, 0) == OK
    assert f(r(BAD_SHAPE), A, 1, B, C, 0) == UNS
    for bad in ((None, B, C), (A, None, C), (A, B, None), (A, B, A), (A + 8, B, C), (A, B, C + 8)):
        assert f(r(SH), bad[0], 1, bad[1], bad[2], 0) == INV


def test_combine_backward():
    def f(dy=A, o=B, w=C, pos=D, T=1, do=E_, dw=F):
        return L.moe_combine_backward(r(SH), dy, o, w, pos, T, do, dw, 0)

    assert f(T=0, dy=None) == OK
    assert f(T=-1) == INV and f(T=65537) == UNS
    assert f(dy=None) == INV and f(pos=None) == INV
    assert f(do=None, dw=None) == INV                       # nothing wanted
    assert f(o=None) == INV                                 # d_w needs o
    assert f(w=None) == INV                                 # d_o needs the weights
    assert f(dy=A + 4) == INV and f(o=B + 4) == INV and f(do=E_ + 4) == INV
    assert f(do=A) == INV and f(dw=A) == INV and f(dw=E_) == INV and f(dw=B) == INV and f(dw=C) == INV


def _norm(fn=None, x=A, y=B, T=1, post=C, pre=D, gate=None, kind=0, alpha=1.0, eps=1e-5, x_out=E_, normed=F, sh=SH):
    return L.moe_block_norm(r(sh), x, y, T, post, pre, gate, kind, alpha, eps, x_out, normed, 0)


def _combine_norm(x=A, o=B, w=16 << 24, pos=17 << 24, T=1, post=C, pre=D, gate=None, kind=0, alpha=1.0, eps=1e-5, x_out=E_,
                  normed=F, sh=SH):
    return L.moe_combine_norm(r(sh), o, w, pos, x, T, post, pre, gate, kind, alpha, eps, x_out, normed, 0)


@pytest.mark.parametrize("f", [_norm, _combine_norm])
def test_norms(f):
    assert f(T=0, x=None) == OK
    assert f(T=-1) == INV and f(T=65537) == UNS
    assert f(sh=BAD_SHAPE) == UNS
    assert f(sh=m.make_shape(16512, 128, 16, 2)) == UNS     # rows longer than a workgroup holds
    assert f(eps=0.0) == INV and f(eps=-1.0) == INV and f(eps=float("nan")) == INV and f(eps=float("inf")) == INV
    assert f(alpha=float("inf")) == INV and f(alpha=float("nan")) == INV
    assert f(kind=3, gate=A) == INV and f(kind=-1) == INV
    assert f(kind=1) == INV and f(kind=2) == INV            # a kind without its gate
    assert f(gate=20 << 24) == INV                          # a gate without its kind
    assert f(x=None) == INV
    assert f(x_out=None, normed=None, pre=None) == INV      # nothing wanted
    assert f(x_out=E_, normed=E_) == INV
    assert f(pre=None) == INV and f(normed=None) == INV     # the pre-norm's weight and output go together
    for k in ("x", "post", "pre", "x_out", "normed"):
        assert f(**{k: (30 << 24) + 4}) == INV
    assert f(kind=2, gate=(30 << 24) + 4) == INV


def test_norm_rows():
    assert _norm(y=None) == INV                              # a post-norm of nothing
    assert _norm(y=None, post=None, gate=A, kind=1) == INV
    assert _norm(y=B + 4) == INV
    for bad in ({"o": None}, {"w": None}, {"pos": None}, {"o": B + 4}, {"x_out": B}, {"normed": B}):
        assert _combine_norm(**bad) == INV


def test_norm_backward():
    big = 1 << 40
    names = dict(x=A, y=B, T=4, post=C, pre=D, gate=None, kind=0, alpha=1.0, eps=1e-5, dxo=E_, dn=F, dx=7 << 24, dy=8 << 24,
                 dg=None, dpost=9 << 24, dpre=10 << 24, ws=11 << 24, nb=big)

    def f(sh=SH, **kw):
        a = names | kw
        return L.moe_block_norm_backward(r(sh), a["x"], a["y"], a["T"], a["post"], a["pre"], a["gate"], a["kind"], a["alpha"],
                                         a["eps"], a["dxo"], a["dn"], a["dx"], a["dy"], a["dg"], a["dpost"], a["dpre"],
                                         a["ws"], a["nb"], 0)

    assert f(T=0, dpost=None, dpre=None, x=None, ws=None) == OK
    assert f(T=-1) == INV and f(T=65537) == UNS
    assert f(sh=BAD_SHAPE) == UNS and f(sh=m.make_shape(16512, 128, 16, 2)) == UNS
    assert f(eps=0.0) == INV and f(alpha=float("nan")) == INV and f(kind=5) == INV and f(kind=1) == INV
    assert f(x=None) == INV and f(ws=None) == INV
    assert f(dxo=None, dn=None, pre=None, dpre=None) == INV          # no upstream gradient
    assert f(pre=None) == INV and f(dn=None) == INV                  # go together
    assert f(pre=None, dn=None) == INV                               # d_pre_gamma of no pre-norm
    assert f(y=None) == INV
    assert f(y=None, post=None, dpost=None) == INV                   # dy of no y
    assert f(post=None) == INV                                       # d_post_gamma of no post-norm
    assert f(dg=12 << 24) == INV                                     # d_gate of no gate
    assert f(dx=None, dy=None, dpost=None, dpre=None) == INV         # nothing wanted
    assert f(dx=8 << 24) == INV and f(dpre=9 << 24) == INV           # two outputs in one place
    assert f(ws=(11 << 24) + 16) == INV
    assert f(nb=256) == WSP
    for k in ("x", "y", "post", "pre", "dxo", "dn", "dx", "dy", "dpost", "dpre"):
        assert f(**{k: (30 << 24) + 4}) == INV


def test_linear():
    def f(N=16, K=256, wf=0, act=0, q=A, s=B, ts=1.0, x=C, T=1, bias=None, y=D):
        return L.moe_linear(r(m.make_matrix(N, K, wf, act)), q, s, ts, x, T, bias, y, 0)

    assert f(T=0, q=None) == OK
    assert L.moe_linear(None, A, B, 1.0, C, 1, None, D, 0) == INV
    assert f(N=0) == INV and f(K=0) == INV and f(T=-1) == INV
    assert f(wf=2) == INV and f(act=2) == INV and f(ts=float("nan")) == INV
    assert f(K=192) == UNS and f(T=65) == UNS and f(N=(1 << 24) + 1, K=128) == UNS and f(N=1 << 22, K=8192) == UNS
    for bad in ({"q": None}, {"s": None}, {"x": None}, {"y": None}, {"y": C}, {"q": A + 8}, {"s": B + 4}, {"x": C + 4},
                {"y": D + 4}, {"bias": E_ + 2}):
        assert f(**bad) == INV


@pytest.mark.parametrize("k,T", [(1, 1), (1, 700), (2, 3), (8, 4096)])
def test_workspace_holds_the_gradient_sums(k, T):
    sh = m.make_shape(256, 128, 16, k)
    # a group of rows per workgroup, up to eight workgroups for each of 256 CUs, two sums of 256 floats each
    assert m.moe_workspace_bytes(sh, T) >= 256 + 8 * 16 * 16 + (1 if T <= 2 else -(-T // -(-T // 2048))) * 8 * 256


@pytest.mark.parametrize("d,act", [(128, 1), (640, 0), (2176, 1)])
def test_a_workspace_serves_every_smaller_token_count(d, act):
    """One pick of one expert per token: the gradient sums are the largest part for many token counts."""
    sh = m.make_shape(d, 128, 1, 1, act_dtype=act)
    sizes = [m.moe_workspace_bytes(sh, T) for T in range(1, 2600)]
    assert sizes == sorted(sizes)


def test_binding_refuses_what_the_library_cannot_see():
    """A host tensor, another dtype, a strided view and a short tensor, before any launch."""
    d, T = SH.d_model, 2
    x = torch.zeros(T, d, dtype=torch.bfloat16)
    pos = torch.zeros(T, 2, dtype=torch.int32)
    calls = [
        lambda: m.moe_dispatch(SH, x, T, pos, torch.zeros(4, d, dtype=torch.bfloat16), stream=0),
        lambda: m.moe_dispatch_backward(SH, x, T, pos, x, stream=0),
        lambda: m.moe_combine_backward(SH, x, A, B, C, T, D, E_, stream=0),
        lambda: m.moe_block_norm(SH, x, None, T, None, A, None, 0, 1.0, 1e-5, None, B, stream=0),
        lambda: m.moe_combine_norm(SH, A, B, C, x, T, None, D, None, 0, 1.0, 1e-5, None, E_, stream=0),
        lambda: m.moe_block_norm_backward(SH, x, None, T, None, A, None, 0, 1.0, 1e-5, None, B, C, None, None, None, None, D,
                                          1 << 40, stream=0),
        lambda: m.moe_linear(m.make_matrix(16, d), A, B, 1.0, x, T, None, C, stream=0),
    ]
    for c in calls:
        with pytest.raises(m.MoeError) as err:
            c()
        assert err.value.status == INV
