"""Arguments of the 16-bit expert operators that are refused before any tensor is looked at, so without a GPU."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("flags", [moe.MOE_OP_FP16, moe.MOE_OP_FP16 | moe.MOE_OUT_FP32, moe.MOE_OP_TRANSPOSE, moe.MOE_NORM_INPUT,
                                   0x4, 1 << 31, 1 << 40, 1 << 80, -1, "2", None])
def test_adapter_flags(flags, dtype):
    """The operands' type is that of the tensors: a flag that names another type, or any flag but the two of the
    operator, is refused."""
    x, ids = torch.zeros(4, 64, dtype=dtype), torch.zeros(4, dtype=torch.int32)
    a, b = torch.zeros(1, 8, 64, dtype=dtype), torch.zeros(1, 32, 8, dtype=dtype)
    with pytest.raises(ValueError, match="flags"):
        moe.adapter_project(x, a, b, ids, flags=flags)
