"""What the operators around the experts and their workspace promise on the host: the same refusals whatever the
token count, and a workspace that serves every smaller call (fake device pointers, nothing is launched)."""
import ctypes

import pytest

m = pytest.importorskip("routed_expert_ffn_router_amd")

A, B = 1 << 24, 2 << 24                                      # distinct fake device addresses
L = m.library()
INV = m.MOE_ERR_INVALID


@pytest.mark.parametrize("T", [0, 4])
@pytest.mark.parametrize("dpost,dpre", [(A + 4, None), (None, A + 8), (A, B + 4), (A, A)])
def test_gamma_gradients_are_checked_for_no_tokens_too(T, dpost, dpre):
    """The gammas' gradients are written whatever T is: 16-byte aligned, and not both in one place."""
    sh, rows, gamma = m.make_shape(256, 128, 16, 2), 3 << 24, 4 << 24
    assert L.moe_block_norm_backward(ctypes.byref(sh), rows, rows, T, gamma, gamma, None, 0, 1.0, 1e-5, rows, rows, None, None,
                                     None, dpost, dpre, 5 << 24, 1 << 40, 0) == INV


@pytest.mark.parametrize("args,kw,top", [
    ((4096, 2048, 288, 8), dict(act_dtype=1), 1500), ((4096, 2048, 288, 8), dict(act_dtype=0, n_shared=1), 1500),
    ((6144, 2048, 256, 8, 1), dict(act_dtype=1, n_shared=1), 1500), ((4096, 2048, 64, 1), dict(act_dtype=1), 4500),
    ((4096, 1024, 1, 1), dict(act_dtype=1), 2600), ((256, 128, 16, 2), dict(act_dtype=0), 300), ((640, 128, 4, 1), dict(), 600)])
def test_a_workspace_serves_every_call_with_fewer_tokens(args, kw, top):
    """The size never falls as T grows, although the router's split of d_model and the tiles of the expert products do:
    with 288 experts, 672 tokens need more of both than 673."""
    sh = m.make_shape(*args, **kw)
    sizes = [m.moe_workspace_bytes(sh, T) for T in [*range(top), *range(10900, 11100), *range(32700, 32800), *range(65530, 65537)]]
    assert sizes[0] > 0 and sizes == sorted(sizes)
