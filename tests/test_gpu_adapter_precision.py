"""The adapters' inner values are held to fp32's precision in every form of the operator."""
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


def _digits(v):
    """v (integers below 2^22) as three exact 8-bit values for x = 2^14, 2^7, 1."""
    s, v = torch.sign(v), v.abs()
    return torch.stack([s * (v >> 14), s * ((v >> 7) & 127), s * (v & 127)], -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,ids", [(1, "one"), (40, "mixed"), (64, "one"), (65, "one"), (65, "mixed"), (300, "runs"), (300, "mixed"),
                                   (1500, "runs"), (1500, "mixed")])
@pytest.mark.parametrize("form", ["projection", "delta", "added"])
@pytest.mark.parametrize("out32", [False, True])
def test_a_delta_that_cancels(T, ids, form, out32, dtype):
    """Integers below 2^22, and sums of them below 2^24, are exact in fp32, and so are products of 8-bit parts.  The
    rank's values (and W x, or the old y) cancel to an integer of at most 7 bits, which any of the result's types holds:
    the results are equal to the last bit, at every batch size, if the inner values keep their 22 bits."""
    L, r, K, N = 3, 16, 64, 136
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, K)
    x[:, 8], x[:, 17], x[:, 42] = 2.0 ** 14, 2.0 ** 7, 1.0
    v0 = torch.randint(1 << 21, 1 << 22, (L,), generator=g) | 1
    small = torch.arange(N) % 100 + 1
    a, b = torch.zeros(L, r, K), torch.zeros(L, N, r)
    w, before = None, None
    b[:, :, 3] = 1.0
    if form == "projection":  # W x = small - v0: one adapter's value, so that the others' results are left out below
        w = torch.zeros(N, K)
        w[:, [8, 17, 42]] = _digits(small - v0[0]).float()
        a[0, 3][[8, 17, 42]] = _digits(v0[0]).float()
    else:  # the rank's values cancel each other: v0 - v1 - v2 = small of the feature's parity
        v2 = torch.randint(1 << 18, 1 << 20, (L,), generator=g)
        for i in range(L):
            a[i, 3][[8, 17, 42]] = _digits(v0[i]).float()
            a[i, 9][[8, 17, 42]] = _digits(v2[i]).float()
            a[i, 14][[8, 17, 42]] = _digits(v0[i] - v2[i] - 77).float()
        b[:, :, 9], b[:, :, 14] = -1.0, -1.0
    at = {"one": torch.zeros(T), "mixed": torch.arange(T) % (L + 1), "runs": torch.arange(T) * L // T}[ids].long()
    dev = lambda t: t.to(dtype).cuda()
    odt = torch.float32 if out32 else dtype
    if form == "added":
        before = (torch.arange(N) % 50).to(odt).cuda().expand(T, N).contiguous()
    got = moe.adapter_project(dev(x), dev(a), dev(b), at.int().cuda(), w=dev(w) if w is not None else None,
                              out=before.clone() if before is not None else None,
                              flags=(moe.MOE_OUT_FP32 if out32 else 0) | (moe.MOE_ACCUMULATE if before is not None else 0)).cpu()
    mine = at == 0 if form == "projection" else at < L
    want = small.expand(T, N) if form == "projection" else torch.full((T, N), 77) + (torch.arange(N) % 50 if before is not None else 0)
    assert bool(mine.any()) and torch.equal(got[mine].double(), want[mine].double())
