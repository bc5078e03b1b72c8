"""The 16-bit expert operators beside torch's autograd, which they are no part of."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _tensors():
    t = {"x": torch.randn(6, 64, device="cuda").to(BF), "w": torch.randn(2, 32, 64, device="cuda").to(BF),
         "off": torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"), "dh": torch.randn(6, 32, device="cuda").to(BF),
         "a": torch.randn(2, 8, 64, device="cuda").to(BF), "b": torch.randn(2, 32, 8, device="cuda").to(BF),
         "ids": torch.zeros(6, dtype=torch.int32, device="cuda"), "w1": torch.randn(32, 64, device="cuda").to(BF),
         "scale": torch.rand(2, device="cuda"), "rw": torch.rand(6, device="cuda")}
    return t


CALLS = {
    "grouped_matmul": (lambda t, out: moe.grouped_matmul(t["x"], t["w"], t["off"], out=out), (6, 32), ("x", "w")),
    "grouped_matmul_wgrad": (lambda t, out: moe.grouped_matmul_wgrad(t["dh"], t["x"], t["off"], out=out), (2, 32, 64), ("dh", "x")),
    "swiglu": (lambda t, out: moe.swiglu(t["x"], t["rw"], out=out), (6, 32), ("x", "rw")),
    "swiglu_backward": (lambda t, out: moe.swiglu_backward(t["x"], t["dh"], t["rw"], dgu=out)[0], (6, 64), ("x", "dh", "rw")),
    "adapter_project": (lambda t, out: moe.adapter_project(t["x"], t["a"], t["b"], t["ids"], w=t["w1"], scale=t["scale"], out=out),
                        (6, 32), ("x", "a", "b", "w1", "scale")),
}


@pytest.mark.parametrize("op", CALLS)
def test_each_tensor_that_requires_a_gradient_is_refused(op):
    call, shape, names = CALLS[op]
    t = _tensors()
    ref = call(t, None)
    for name in names:
        t[name].requires_grad_(True)
        with pytest.raises(ValueError, match="gradient"):
            call(t, None)
        with torch.no_grad():
            assert torch.equal(call(t, None), ref)
        with torch.inference_mode():
            assert torch.equal(call(t, torch.zeros(shape, dtype=BF, device="cuda")), ref)
        t[name].requires_grad_(False)
    with pytest.raises(ValueError, match="gradient"):
        call(t, torch.zeros(shape, dtype=BF, device="cuda").requires_grad_(True))


@pytest.mark.parametrize("op", CALLS)
def test_a_graph_sees_that_its_tensor_was_overwritten(op):
    call, shape, _ = CALLS[op]
    t, out = _tensors(), torch.ones(shape, dtype=BF, device="cuda")
    p = torch.ones(shape, dtype=BF, device="cuda", requires_grad=True)
    loss = (p * out).sum()  # saves out
    call(t, out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_results_in_inference_mode_tensors():
    """A given result that is an inference tensor has no version to count, and is taken in either mode."""
    call, shape, _ = CALLS["grouped_matmul"]
    t = _tensors()
    with torch.inference_mode():
        out = torch.zeros(shape, dtype=BF, device="cuda")
        call(t, out)
    assert torch.equal(call(t, out), call(t, None))
