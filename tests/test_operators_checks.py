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
