"""Products of few rows (the warp-MMA kernel): every row count from 1 to 64, groups split and joined, against the
formula in 64 bits; tolerances as in the grouped products' tests (half a step, plus two fp32 steps per 16-wide step)."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("E,N,K", [(1, 40, 8), (3, 136, 328), (40, 64, 2056), (2, 1608, 264)])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_few_rows(M, E, N, K, dtype, out_dtype):
    g = torch.Generator(device="cuda").manual_seed(M * 100 + E)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 0.05).to(dtype)
    cuts = torch.randint(0, M + 1, (E + 1,), generator=torch.Generator().manual_seed(M)).sort().values
    if M > 3:
        x[:int(cuts[0])] = float("nan")
    out = torch.full((M, N), 7.0, dtype=out_dtype or dtype, device="cuda")
    moe.grouped_matmul(x, w, cuts.to(torch.int32).cuda(), out=out)
    f = torch.finfo(out.dtype)
    assert bool((out[:int(cuts[0])] == 7).all()) and bool((out[int(cuts[-1]):] == 7).all())
    for e in range(E):
        lo, hi = int(cuts[e]), int(cuts[e + 1])
        a, b = x[lo:hi].double(), w[e].double().T
        ref, mag = a @ b, a.abs() @ b.abs()
        bound = f.eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (K / 16 + 1) * mag + f.tiny
        assert bool(((out[lo:hi].double() - ref).abs() <= bound).all())
