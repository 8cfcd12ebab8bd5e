"""Sizes that do not fit the C interface's 32 bits are refused by the binding (ctypes would cut them to other sizes than
the tensors are checked for); no GPU is needed, the refusal comes before anything else."""
import pytest

import w4a16_routed_expert_moe_amd as moe

DESC = moe.MoeLayerDesc.make(512, 128, 8, 2, 1)
CALLS = {
    "moe_act_quant_int8": ((4, 64), 3), "moe_w8a8_prepack": ((1, 64, 64), 2), "moe_w8a8_gemm": ((4, 64, 64), 5),
    "moe_w8a8_linear": ((4, 64, 64), 6), "moe_w8a8_packed_bytes": ((1, 64, 64), 0),
    "moe_w8a8_experts": ((DESC, 4), 16), "moe_balance_workspace_bytes": ((DESC, 4, 2), 0),
    "moe_route_backward": ((DESC, 4, 2), 9),
}


@pytest.mark.parametrize("wide", [(1 << 32) + 4, 1 << 31, -(1 << 32) + 4, -(1 << 31) - 1, 1 << 63, 1 << 70])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_refused(name, wide):
    sizes, tensors = CALLS[name]
    for i, v in enumerate(sizes):
        if v is DESC:
            continue
        args = list(sizes) + [None] * tensors
        args[i] = wide
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            getattr(moe, name)(*args)


@pytest.mark.parametrize("wide", [(1 << 32) + 4, -(1 << 32) + 4])
def test_refused_between_tensors(wide):
    for at in (1, 5, 6, 7):
        args = [DESC, 4, None, None, None, 4, 128, 64, None, None, None, moe.MOE_ACT_NONE, None]
        args[at] = wide
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            moe.moe_w8a8_grouped_gemm(*args)
    with pytest.raises(ValueError, match="does not fit 32 bits"):  # (without a_gather a negative n_src is not refused)
        moe.moe_w8a8_grouped_gemm(DESC, wide, None, None, None, -1, 128, 64, None, None, None, moe.MOE_ACT_NONE, None)
    for at in (1, 2):
        args = [DESC, 4, 2, None, None, None, None, 0.1, None, None, None, None, None]
        args[at] = wide
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            moe.moe_balance_loss(*args)


def test_sizes_that_fit_reach_the_library():
    assert moe.moe_w8a8_packed_bytes(1, 64, 64) == 64 * 128
    for n in (-1, -(1 << 31), (1 << 31) - 1):
        assert moe.moe_w8a8_packed_bytes(n, 64, 64) == 0
        assert moe.moe_balance_workspace_bytes(DESC, n, 1) == 0
