"""fp32 sums of the warp-MMA kernels (few rows; the adapters' inner values) over long contractions, of one sign.

A warp MMA costs at most two fp32 steps of a partial sum each 16 values; a part has at most 768 of them.  The parts, and
the warps' and slices' sums, are added in fp32, half a step each."""
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


def _positive(shape, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") * 0.1 + 0.1).to(dt)


def _bound(K):
    return 2 * 2.0 ** -23 * (768 / 16 + 1) + 2.0 ** -24 * (K / 512 + 24)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [1 << 17, 40008, 4104])
@pytest.mark.parametrize("M", [1, 8, 13, 30, 64])
@pytest.mark.parametrize("N", [40, 2400])
def test_few_rows(M, N, K, dtype):
    x, w = _positive((M, K), dtype, 1), _positive((1, N, K), dtype, 2)
    got = moe.grouped_matmul(x, w, torch.tensor([0, M], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    ref = torch.cat([x.double() @ p.double().T for p in w[0].split(256)], 1)
    assert float(((got.double() - ref) / ref).abs().max()) <= _bound(K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 5, 40, 48, 64])
def test_projection_of_few_tokens(T, dtype):
    K, N, L, r = 1 << 17, 136, 2, 8
    x, w = _positive((T, K), dtype, 3), _positive((N, K), dtype, 4)
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    got = moe.adapter_project(x, torch.zeros(L, r, K, dtype=dtype, device="cuda"), torch.zeros(L, N, r, dtype=dtype, device="cuda"),
                              ids, w=w, flags=moe.MOE_OUT_FP32)
    ref = x.double() @ w.double().T
    assert float(((got.double() - ref) / ref).abs().max()) <= _bound(K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,ids", [(1, 1 << 17, "one"), (9, 1 << 17, "one"), (9, 1 << 17, "mixed"), (100, 40008, "mixed"),
                                     (100, 40008, "one"), (1300, 16392, "one"), (1300, 16392, "mixed"), (8200, 4104, "mixed"),
                                     (8200, 4104, "one")])
@pytest.mark.parametrize("r", [8, 32, 72])
def test_inner_values(r, T, K, ids, dtype):
    """v itself, by a B that is the identity: every token's own values, at each window, rank pass and share of K."""
    L = 9
    x, a = _positive((T, K), dtype, 5), _positive((L, r, K), dtype, 6)
    b = torch.eye(r, device="cuda").to(dtype).expand(L, r, r).contiguous()
    at = (torch.arange(T, device="cuda") % L if ids == "mixed" else torch.full((T,), 4, device="cuda")).int()
    scale = torch.full((L,), 2.0 ** -6, device="cuda")  # (v below 2^15: fp16 keeps 22 bits of it)
    got = moe.adapter_project(x, a, b, at, scale=scale, flags=moe.MOE_OUT_FP32)
    ref = torch.zeros(T, r, dtype=torch.float64, device="cuda")
    for i in range(L):
        m = (at == i).nonzero()[:, 0]
        ref[m] = 2.0 ** -6 * x[m].double() @ a[i].double().T
    # fp16: two terms hold 2^-23 of the token's largest value, at most four times the smallest here
    assert float(((got.double() - ref) / ref).abs().max()) <= _bound(K) + (2.0 ** -21 if dtype == torch.float16 else 2.0 ** -24)
