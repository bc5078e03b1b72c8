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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lo,hi", [(-110.0, -80.0), (-89.0, -87.0), (-80.0, -8.0), (8.0, 110.0)])
def test_gates_far_from_zero(lo, hi, dtype):
    """Gates at which the sigmoid is small, down to fp32's subnormal range, times values of u up to the type's largest.

    Bounds: half a step of the result, and fp32 arithmetic: the exponential within 2 + 1.2 |g| steps (2^-23), ten more for
    the other operations, and where s is subnormal two roundings of half its step, 2^-149 together.  The gate's gradient
    multiplies dh with the slope before u (their product with dh first overflows): one more of half a step, times u."""
    f32 = torch.float32
    n = 1024
    gate = torch.linspace(lo, hi, n, device="cuda").to(dtype)
    top = 3e38 if dtype == torch.bfloat16 else 6e4
    up = torch.cat([torch.logspace(0, torch.tensor(top).log10().item(), n // 2, device="cuda"), torch.full((n // 2,), top, device="cuda")])
    up = up[torch.randperm(n, generator=torch.Generator().manual_seed(1)).cuda()]
    if hi > 0:
        up = up.clamp(max=200.0)  # (h stays finite)
    gu = torch.cat([gate[None], up.to(dtype)[None]], 1).contiguous()
    dh = torch.linspace(-2, 2, n, device="cuda").to(dtype)[None].contiguous()
    rw = torch.full((1,), 0.75, device="cuda")
    g, u, d = gu[:, :n].double(), gu[:, n:].double(), dh.double()
    z = torch.exp(-g.abs())
    s = torch.where(g >= 0, 1 / (1 + z), z / (1 + z))
    rest = torch.where(g >= 0, z / (1 + z), 1 / (1 + z))
    arith, least = (12 + 1.2 * g.abs()) * 2.0 ** -23, 2.0 ** -149

    def near(got, ref, mag, scale):
        f = torch.finfo(got.dtype)
        bound = f.eps / 2 * ref.abs() + arith * mag + least * scale + f.smallest_normal * f.eps
        off = (got.double() - ref).abs()
        assert not bool((off > bound).any()), f"worst {float((off / bound).max()):.3g} bounds at {float(g.flatten()[int((off / bound).argmax()) % n])}"

    h = 0.75 * g * s * u
    near(moe.swiglu(gu, rw), h, h.abs(), (g * u).abs())
    dgu, h2, _ = moe.swiglu_backward(gu, dh, rw, with_h=True)
    near(h2, h, h.abs(), (g * u).abs())
    near(dgu[:, :n], 0.75 * d * u * s * (1 + g * rest), (d * u).abs() * s * (1 + g.abs() * rest), (d * u).abs() * (1 + g.abs()) + u.abs() / 2)
    near(dgu[:, n:], 0.75 * d * g * s, (d * g).abs() * s, (d * g).abs())
