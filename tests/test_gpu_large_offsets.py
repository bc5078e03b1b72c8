"""Operands and results of more than 2^31 values: rows at the start, at the 2^31st value and at the end, against the
formulas in 64 bits (half a step of the result's type, two fp32 steps per 16-wide step of the sums)."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROWS, D = 1_200_016, 2048  # 2.46e9 values


@pytest.fixture(autouse=True)
def _fresh():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()
    assert moe.moe_check_op_status() == 0


def _normal(*shape, seed, scale=1.0):
    return torch.empty(shape, dtype=BF, device="cuda").normal_(0.0, scale, generator=torch.Generator(device="cuda").manual_seed(seed))


def _probe(rows):
    at = (1 << 31) // D
    return torch.tensor([0, 1, 255, 256, at - 1, at, at + 1, rows // 2, rows - 257, rows - 2, rows - 1], device="cuda")


def _close(got, ref, mag, C):
    bound = torch.finfo(got.dtype).eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (C / 16 + 40) * mag + 1e-37
    off = (got.double() - ref).abs()
    assert not bool((off > bound).any()), f"worst {float((off / bound).max()):.3g} bounds"


@pytest.mark.parametrize("mode", ["forward", "rows"])
def test_product(mode):
    x, w = _normal(ROWS, D, seed=1), _normal(3, D, D, seed=2, scale=0.02)
    off = torch.tensor([0, 300, ROWS - 1000, ROWS], dtype=torch.int32, device="cuda")
    y = moe.grouped_matmul(x, w, off, transpose=mode == "rows")
    at = _probe(ROWS)
    e = torch.bucketize(at, off[1:].long(), right=True)
    for r, g in zip(at.tolist(), e.tolist()):
        a, b = x[r:r + 1].double(), w[g].double() if mode == "rows" else w[g].double().T
        _close(y[r:r + 1], a @ b, a.abs() @ b.abs(), D)


def test_weights_gradient():
    """The second group begins behind the 2^31st value of both operands."""
    n = 3000
    dy, x = _normal(ROWS, D, seed=3), _normal(ROWS, D, seed=4)
    off = torch.tensor([ROWS - n, ROWS - 100, ROWS], dtype=torch.int32, device="cuda")
    dw = moe.grouped_matmul_wgrad(dy, x, off)
    for e, (lo, hi) in enumerate(((ROWS - n, ROWS - 100), (ROWS - 100, ROWS))):
        a, b = dy[lo:hi].double().T, x[lo:hi].double()
        _close(dw[e], a @ b, a.abs() @ b.abs(), hi - lo)


def test_many_matrices():
    """Weights, and their gradient, of more than 2^31 values."""
    E, N, K = 1024, 1536, 1400
    w = _normal(E, N, K, seed=5, scale=0.02)
    sizes = torch.zeros(E, dtype=torch.long)
    sizes[[0, 7, 998, 999, 1000, E - 1]] = torch.tensor([3, 40, 5, 20, 33, 64])
    off = torch.cat([torch.zeros(1).long(), sizes.cumsum(0)])
    M = int(off[-1])
    x, dy, dev = _normal(M, K, seed=6), _normal(M, N, seed=7), off.int().cuda()
    y, dx, dw = moe.grouped_matmul(x, w, dev), moe.grouped_matmul(dy, w, dev, transpose=True), moe.grouped_matmul_wgrad(dy, x, dev)
    few = moe.grouped_matmul(x[:43], w, dev.clamp(max=43))  # (the few-row kernel's sizes)
    for e in (0, 7, 500, 998, 999, 1000, E - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        a, d, b = x[lo:hi].double(), dy[lo:hi].double(), w[e].double()
        _close(y[lo:hi], a @ b.T, a.abs() @ b.abs().T, K)
        _close(dx[lo:hi], d @ b, d.abs() @ b.abs(), N)
        _close(dw[e], d.T @ a, d.abs().T @ a.abs(), max(hi - lo, 1))
        if hi <= 43:
            _close(few[lo:hi], a @ b.T, a.abs() @ b.abs().T, K)


def test_swiglu():
    f = D // 2
    gu, rw = _normal(ROWS, D, seed=8), torch.rand(ROWS, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    dh = _normal(ROWS, f, seed=10)
    h = moe.swiglu(gu, rw)
    dgu, h2, drw = moe.swiglu_backward(gu, dh, rw, with_h=True)
    at = _probe(ROWS)
    assert torch.equal(h[at], h2[at])
    g, u, d, w = gu[at, :f].double(), gu[at, f:].double(), dh[at].double(), rw[at].double()[:, None]
    s = torch.sigmoid(g)
    _close(h[at], w * g * s * u, (g * u).abs(), 16)
    _close(dgu[at], torch.cat([w * d * u * s * (1 + g * (1 - s)), w * d * g * s], 1), torch.cat([(d * u).abs() * (1 + g.abs()), (d * g).abs()], 1), 16)
    _close(drw[at], (d * g * s * u).sum(1), (d * g * u).abs().sum(1), f)


@pytest.mark.parametrize("projection", [False, True])
def test_adapters_of_many_tokens(projection):
    L, r = 5, 16
    x, a, b = _normal(ROWS, D, seed=11), _normal(L, r, D, seed=12, scale=0.02), _normal(L, D, r, seed=13)
    w = _normal(D, D, seed=14, scale=0.02) if projection else None
    ids = (torch.arange(ROWS, device="cuda") // 70_001 % (L + 1)).int()
    y = moe.adapter_project(x, a, b, ids, w=w)
    for t in _probe(ROWS).tolist():
        v, i = x[t].double(), int(ids[t])
        ref, mag = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
        if projection:
            ref, mag = w.double() @ v, w.double().abs() @ v.abs()
        if i < L:
            ref, mag = ref + b[i].double() @ (a[i].double() @ v), mag + b[i].double().abs() @ (a[i].double().abs() @ v.abs())
        _close(y[t], ref, mag, D)


@pytest.mark.parametrize("T", [3, 40, 100, 2000])
@pytest.mark.parametrize("projection", [False, True])
def test_many_adapters(T, projection):
    """More than 2^31 values in A and in B, the last adapters used."""
    L, r, K, N = 70_000, 16, 2048, 2048
    x, a, b = _normal(T, K, seed=15), _normal(L, r, K, seed=16, scale=0.02), _normal(L, N, r, seed=17)
    w = _normal(N, K, seed=18, scale=0.02) if projection else None
    ids = (L - 1 - torch.arange(T, device="cuda") // 7 % 40).int()
    ids[::5] = 3
    y = moe.adapter_project(x, a, b, ids, w=w)
    for t in {0, 1, 2, T // 2, T - 2, T - 1}:
        v, i = x[t].double(), int(ids[t])
        ref, mag = b[i].double() @ (a[i].double() @ v), b[i].double().abs() @ (a[i].double().abs() @ v.abs())
        if projection:
            ref, mag = ref + w.double() @ v, mag + w.double().abs() @ v.abs()
        _close(y[t], ref, mag, K)
