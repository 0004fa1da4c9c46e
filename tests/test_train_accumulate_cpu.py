"""The accumulate flag of a gradient call that asks for no weight gradient says
nothing: frozen experts in an accumulating program.  (With neither gradient
asked for, the call checks its arguments and queues nothing: no GPU needed.)"""
import ctypes as C

import pytest

import expert_routing_ffn_gb300 as moe

A, WS, N_WS = 0x10000, 1 << 20, 16 << 20  # addresses that are never followed


@pytest.mark.parametrize("wtype", ["bf16", "f32"])
@pytest.mark.parametrize("gtype", [moe.MOE_DTYPE_BF16, moe.MOE_DTYPE_F32])
def test_accumulate_without_a_weight_gradient_is_taken(wtype, gtype):
    D = moe.make_dims(4, 40, 8, 2, 24, wtype=wtype)
    L, r = moe.lib(), C.byref(D)
    expected = moe.MOE_ERR_UNSUPPORTED if (wtype, gtype) == ("f32", moe.MOE_DTYPE_BF16) else moe.MOE_OK
    assert L.moe_experts_up_grad(r, A, A, None, A, A, A, None, None, None, gtype, 1, WS, N_WS, None) == expected
    assert L.moe_experts_down_grad(r, A, None, A, A, A, A, None, None, None, gtype, 1, WS, N_WS, None) == expected
    if gtype == moe.MOE_DTYPE_BF16:  # with one, bf16 buffers cannot be added to
        assert L.moe_experts_up_grad(r, A, A, A, A, A, A, None, A, A, gtype, 1, WS, N_WS, None) == moe.MOE_ERR_UNSUPPORTED
        assert L.moe_experts_down_grad(r, A, A, A, A, A, A, None, None, A, gtype, 1, WS, N_WS, None) == moe.MOE_ERR_UNSUPPORTED
