"""Grouped products and their gradients at the edges of tiles and tables, against the formulas in 64 bits; the bounds are
those of the grouped products' other tests (half a step of the result's type, two fp32 steps per 16-wide step)."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_expert_ffn_gemv_b200 import build
    build.build()
    yield
    assert moe.moe_check_op_status() == 0


def _normal(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)


def _check(got, ref, mag, C, dt):
    bound = torch.finfo(dt).eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (C / 16 + 1) * mag + torch.finfo(dt).tiny
    off = (got.double() - ref).abs()
    assert not bool((off > bound).any()), f"{int((off > bound).sum())} of {off.numel()} values off, worst {float((off / bound).max()):.3g} bounds"


@pytest.mark.parametrize("how", ["16", "fp32", "accumulate"])
@pytest.mark.parametrize("K", [8, 72, 80, 200, 288, 336, 800])
def test_weights_gradient_of_odd_widths_over_many_tiles(K, how):
    """Every pair of SMs takes several tiles, whose last ones have an odd number of blocks; every other group is empty,
    so that a tile of zeros, which waits for nothing, follows a filled one.  Repeated back to back, bit for bit."""
    E, N = 256, 512  # 512 tiles and more for 74 pairs
    sizes = [0 if e % 2 else 1 + 37 * e % 50 for e in range(E)]
    off = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    M = int(off[-1])
    dy, x = _normal((M, N), torch.bfloat16, 21), _normal((M, K), torch.bfloat16, 22)
    odt = torch.bfloat16 if how == "16" else torch.float32
    before = _normal((E, N, K), torch.float32, 23) if how == "accumulate" else None

    def call():
        out = before.clone() if before is not None else torch.full((E, N, K), 7.0, dtype=odt, device="cuda")
        return moe.grouped_matmul_wgrad(dy, x, off, out=out, accumulate=before is not None)

    outs = [call() for _ in range(4)]
    o = off.tolist()
    for e in range(E):
        a, b = dy[o[e]:o[e + 1]].double().T, x[o[e]:o[e + 1]].double()
        ref, mag = a @ b, a.abs() @ b.abs()
        if before is not None:
            ref, mag = ref + before[e].double(), mag + before[e].double().abs()
        _check(outs[0][e], ref, mag, max(sizes[e], 1), odt)
    for other in outs[1:]:
        assert torch.equal(outs[0], other)
