"""Adapters of runs of tokens: what other runs, tokens without an adapter and old memory hold reaches no token."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu


def _poison():
    """Freed blocks that the next workspaces and results come from hold NaN."""
    for size in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
        torch.full((size,), float("nan"), device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,run", [(70, 33), (300, 60), (300, 300), (2000, 45), (2000, 700)])
@pytest.mark.parametrize("r", [8, 24, 72])
@pytest.mark.parametrize("form", ["projection", "added", "delta", "projection fp32"])
def test_runs(T, run, r, form, dtype):
    L, N, K = 4, 136, 264
    g = torch.Generator(device="cuda").manual_seed(T + r)
    normal = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(dtype)
    x, a, b = normal(T, K), normal(L, r, K, scale=K ** -0.5), normal(L, N, r, scale=0.2)
    w = normal(N, K, scale=0.05) if "projection" in form else None
    before = normal(T, N) if form == "added" else None
    ids = (torch.arange(T, device="cuda") // run % (L + 1)).int()  # 4: none
    flags = moe.MOE_OUT_FP32 if "fp32" in form else moe.MOE_ACCUMULATE if before is not None else 0

    def call(x, a, b):
        _poison()
        return moe.adapter_project(x, a, b, ids, w=w, out=before.clone() if before is not None else None, flags=flags)

    clean = call(x, a, b)
    assert bool(clean.isfinite().all())
    bad_a, bad_b, bad_x = a.clone(), b.clone(), x.clone()
    bad_a[1], bad_b[1] = float("nan"), float("inf")
    bad_x[T // 2] = float("inf")
    got = call(bad_x, bad_a, bad_b)
    keep = ids != 1
    keep[T // 2] = False
    assert torch.equal(got[keep], clean[keep])
    assert not bool(got[ids == 1].isfinite().any())
