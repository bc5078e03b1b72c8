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


P = 1 << 20  # a 16-byte aligned address (never read)
GRAD = dict(gu=P, ldgu=128, dh=2 * P, lddh=64, rows=5, f=64, rw=6 * P, n_rows=0, dgu=3 * P, lddgu=128, h=4 * P, ldh=64, drw=5 * P, flags=0)


@pytest.mark.parametrize("bad", [dict(dgu=P, lddgu=136), dict(dgu=2 * P), dict(h=P), dict(h=2 * P), dict(h=3 * P), dict(drw=6 * P)],
                         ids=str)
def test_swiglu_backward_over_an_operand(bad):
    """A result may be no operand, but dgu gu itself, at gu's pitch."""
    a = dict(GRAD, **bad)
    assert moe.lib().moe_swiglu_backward(a["gu"], a["ldgu"], a["dh"], a["lddh"], a["rows"], a["f"], a["rw"], a["n_rows"], a["dgu"],
                                         a["lddgu"], a["h"], a["ldh"], a["drw"], a["flags"], None) == 1


def test_swiglu_over_its_operand():
    assert moe.lib().moe_swiglu(P, 128, 5, 64, 0, 0, P, 128, 0, None) == 1


CALLS = {  # each operator with one tensor argument after the other requiring a gradient
    "grouped_matmul": lambda t: moe.grouped_matmul(t["x"], t["w"], t["ids"], out=t["out"]),
    "grouped_matmul_wgrad": lambda t: moe.grouped_matmul_wgrad(t["x"], t["w"], t["ids"], out=t["out"]),
    "swiglu": lambda t: moe.swiglu(t["x"], t["rw"], out=t["out"]),
    "swiglu_backward": lambda t: moe.swiglu_backward(t["x"], t["w"], t["rw"], dgu=t["out"]),
    "adapter_project": lambda t: moe.adapter_project(t["x"], t["w"], t["b"], t["ids"], scale=t["rw"], out=t["out"]),
}


@pytest.mark.parametrize("op", CALLS)
def test_a_tensor_that_requires_a_gradient(op):
    """No call records a gradient, so none takes a tensor that needs one while gradients are recorded."""
    t = {"x": torch.zeros(4, 64, dtype=torch.bfloat16), "w": torch.zeros(1, 8, 64, dtype=torch.bfloat16),
         "b": torch.zeros(1, 32, 8, dtype=torch.bfloat16), "ids": torch.zeros(4, dtype=torch.int32),
         "out": torch.zeros(4, 32, dtype=torch.bfloat16), "rw": torch.zeros(4)}
    t["x"].requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        CALLS[op](t)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        CALLS[op](t)


def test_adapter_check():
    """moe_adapter_check is moe_adapter_project's refusals, without the call."""
    import ctypes
    good = dict(x=P, ldx=64, tokens=10, n=32, k=64, w=0, a=P, b=P, scale=0, ids=P, n_adapters=3, rank=16, y=2 * P, ldy=32,
                workspace=3 * P, workspace_bytes=1 << 20)
    check = moe.lib().moe_adapter_check
    assert check(ctypes.byref(moe.MoeAdapterArgs(**good)), 0x3) == 0
    assert check(None, 0) == 1 and check(ctypes.byref(moe.MoeAdapterArgs(**good)), 0x4) == 1
    for bad in (dict(rank=12), dict(y=P), dict(a=P + 8), dict(ids=0), dict(n=4), dict(ldy=24), dict(workspace_bytes=8)):
        assert check(ctypes.byref(moe.MoeAdapterArgs(**dict(good, **bad))), 0) == 1


@pytest.mark.parametrize("bad", [dict(w=2 * P), dict(a=2 * P), dict(b=2 * P), dict(x=2 * P), dict(workspace=2 * P), dict(workspace=P)],
                         ids=str)
def test_adapters_over_an_operand(bad):
    """y is 2 P and x P: neither y nor the workspace may be an operand."""
    import ctypes
    good = dict(x=P, ldx=64, tokens=10, n=32, k=64, w=3 * P, a=4 * P, b=5 * P, scale=0, ids=P, n_adapters=3, rank=16, y=2 * P,
                ldy=32, workspace=6 * P, workspace_bytes=1 << 20)
    assert moe.lib().moe_adapter_check(ctypes.byref(moe.MoeAdapterArgs(**good)), 0) == 0
    assert moe.lib().moe_adapter_check(ctypes.byref(moe.MoeAdapterArgs(**dict(good, **bad))), 0) == 1
    assert moe.lib().moe_adapter_project(ctypes.byref(moe.MoeAdapterArgs(**dict(good, **bad))), 0, None) == 1
