"""SwiGLU and its gradient in place and at the ends of the gate's range."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_expert_ffn_gemv_b200 import build
    build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,f", [(1, 8), (3, 2056), (300, 8208), (5000, 136), (5000, 1288), (5000, 4104)])
@pytest.mark.parametrize("wide", [False, True])
def test_gradient_in_place(rows, f, dtype, wide):
    """dgu over gu gives the bits of a call into another tensor, with h and drw, as one block and as a slice."""
    g = torch.Generator(device="cuda").manual_seed(rows + f)
    buf = torch.randn(rows, 2 * f + (32 if wide else 0), generator=g, device="cuda").to(dtype)
    gu = buf[:, 16:16 + 2 * f] if wide else buf
    dh = torch.randn(rows, f, generator=g, device="cuda").to(dtype)
    rw = torch.rand(rows, generator=g, device="cuda")
    ref, h, drw = moe.swiglu_backward(gu, dh, rw, with_h=True)
    edges = buf.clone()
    got, h2, drw2 = moe.swiglu_backward(gu, dh, rw, dgu=gu, with_h=True)
    assert got is gu and torch.equal(gu, ref) and torch.equal(h, h2) and torch.equal(drw, drw2)
    if wide:
        assert torch.equal(buf[:, :16], edges[:, :16]) and torch.equal(buf[:, -16:], edges[:, -16:])
