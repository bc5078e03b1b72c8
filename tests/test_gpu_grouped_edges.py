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


def _few_rows(M, N, K, seed):
    return _normal((M, K), torch.bfloat16, seed), torch.full((M + 64, N), 5.0, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("E", [256, 257, 512, 513, 1024])
@pytest.mark.parametrize("M", [1, 10, 33, 59, 64])  # (64: 69 rows, the tensor-core kernel)
def test_few_rows_of_many_groups(E, M):
    """The few-row kernel's search for its group where a thread looks at several offsets: used groups anywhere in the
    table, the first and the last among them, several rows in some, and unused rows before and behind."""
    N, K = 40, 72
    x, buf = _few_rows(M + 5, N, K, 31)
    x[:2], x[2 + M:] = float("nan"), float("inf")
    w = _normal((E, N, K), torch.bfloat16, 32, 0.05)
    g = torch.Generator().manual_seed(M * E)
    ids = torch.randint(0, E, (M,), generator=g)
    ids[0] = E - 1
    if M > 1:
        ids[1] = 0
    off = (torch.cat([torch.zeros(1).long(), torch.bincount(ids, minlength=E).cumsum(0)]) + 2).tolist()
    out = buf[32:32 + M + 5]
    moe.grouped_matmul(x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            a, b = x[lo:hi].double(), w[e].double().T
            _check(out[lo:hi], a @ b, a.abs() @ b.abs(), K, torch.bfloat16)
    assert bool((buf[:34] == 5).all()) and bool((buf[34 + M:] == 5).all())


TABLES = [[0, -5, 4000, 20], [50, 20, 90, 10], [90, 90, 90, 90], [-9, -3, -1, 0], [0, 5, 2, 4], [7, 0, 0, 30, 12, 40],
          [0, 40, 10, 40, 20, 40, 30, 40]]


@pytest.mark.parametrize("table", TABLES, ids=str)
@pytest.mark.parametrize("M", [3, 40, 64, 65, 300])
@pytest.mark.parametrize("behind", [0, 600])
def test_a_bad_table_is_made_ascending(table, M, behind):
    """Whatever the table, and whichever kernel its size selects: offsets are clamped into [0, rows], an offset below an
    earlier one counts as that one, and every row of the result is its group's product, or left as it was."""
    N, K = 64, 72
    x, buf = _few_rows(M, N, K, 33)
    table = table + [table[-1]] * behind
    E = len(table) - 1
    w = _normal((E, N, K), torch.bfloat16, 34, 0.05)
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    out = buf[32:32 + M]
    moe.grouped_matmul(x, w, off, out=out)
    first = out.clone()
    for _ in range(3):
        assert torch.equal(first, moe.grouped_matmul(x, w, off, out=out))
    o = torch.tensor(table).clamp(0, M).cummax(0).values.tolist()
    seen = 0
    for e in range(E):
        a, b = x[o[e]:o[e + 1]].double(), w[e].double().T
        if o[e + 1] > o[e]:
            _check(out[o[e]:o[e + 1]], a @ b, a.abs() @ b.abs(), K, torch.bfloat16)
            seen += o[e + 1] - o[e]
    assert bool((buf[:32 + o[0]] == 5).all()) and bool((buf[32 + o[-1]:] == 5).all()) and seen == o[-1] - o[0]
    dy = _normal((M, N), torch.bfloat16, 35)
    dw = moe.grouped_matmul_wgrad(dy, x, off)
    for e in range(min(E, 8)):
        a, b = dy[o[e]:o[e + 1]].double().T, x[o[e]:o[e + 1]].double()
        _check(dw[e], a @ b, a.abs() @ b.abs(), max(o[e + 1] - o[e], 1), torch.bfloat16)
