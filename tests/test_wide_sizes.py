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
    "moe_route": ((DESC, 4), 6), "moe_workspace_bytes": ((DESC, 4), 0), "moe_permute": ((DESC, 4), 4),
    "moe_route_permute": ((DESC, 4), 10), "moe_route_permute_noalloc": ((DESC, 4), 9), "moe_row_sums": ((4, 128), 2),
    "moe_w4a16_down_combine": ((DESC, 4), 7), "moe_combine": ((DESC, 4), 4), "moe_w4a16_prepack": ((1, 128, 128), 2),
    "moe_mxfp4_prepack": ((1, 128, 128), 2), "moe_act_quant_fp8": ((4, 128), 3),
    "moe_act_quant_fp8_dequant": ((4, 128), 4), "moe_fp8_block_gemm": ((4, 128, 128), 5),
    "moe_fp8_prepack": ((128, 128), 2),
}
GROUPED = {  # name: sizes by position, arguments
    "moe_w8a8_grouped_gemm": ({1: 4, 5: 4, 6: 128, 7: 64, 11: 0}, 13),
    "moe_w4a8_grouped_gemm": ({1: 4, 5: 4, 6: 128, 7: 128, 11: 0}, 13),
    "moe_w4a16_grouped_gemm": ({1: 4, 4: 4, 6: 128, 7: 128, 11: 0}, 13),
    "moe_mxfp4_grouped_gemm": ({1: 4, 4: 4, 5: 128, 6: 128, 10: 0}, 12),
    "moe_gen_int4_codes": ({0: 1, 1: 0, 2: 0, 3: 1, 4: 0, 5: 128, 6: 128}, 8),
    "moe_gen_fp16_scales": ({0: 1, 1: 0, 2: 0, 3: 1, 4: 0, 5: 128, 6: 128}, 8),
    "moe_gen_ue8m0_scales": ({0: 1, 1: 0, 2: 0, 3: 1, 4: 0, 5: 128, 6: 128}, 8),
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
@pytest.mark.parametrize("name", sorted(GROUPED))
def test_refused_between_tensors(name, wide):
    sizes, n = GROUPED[name]
    for at in sizes:
        if name.startswith("moe_gen") and at not in (3, 5, 6):  # the others are numbers that the draw is made from
            continue
        args = [None] * n
        for i, v in sizes.items():
            args[i] = v
        if not name.startswith("moe_gen"):
            args[0] = DESC
        args[at] = wide
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            getattr(moe, name)(*args)


@pytest.mark.parametrize("wide", [(1 << 32) + 4, -(1 << 32) + 4])
def test_refused_beside_other_arguments(wide):
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
