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


# Long contractions into 16 bits.  Up to 8192 values are summed by the tensor core, which rounds its accumulator towards
# zero at each 16-wide step (at most two fp32 steps of it); longer ones in parts of 8192, added in fp32, half a step each.
def _check_long(got, ref, mag, C, more=0.0):
    f = torch.finfo(got.dtype)
    steps = min(C, 8192) / 16 + 1 + C / 8192
    bound = f.eps / 2 * ref.abs() + 2 * 2.0 ** -23 * steps * mag + more + f.tiny
    off = got.double() - ref
    assert not bool((off.abs() > bound).any()), f"worst {float((off.abs() / bound).max()):.3g} bounds, {int((off.abs() > bound).sum())} values"
    return off


def _positive(shape, dt, seed, lo, hi):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo).to(dt)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mode,C", [("weights", 300_008), ("weights", 8193), ("weights", 1_500_000), ("forward", 1 << 17),
                                    ("forward", 8200), ("rows", 1 << 17), ("rows", 16392)])
def test_long_sums_of_one_sign(mode, C, dtype):
    """Nothing cancels, so rounding towards zero would add up: no value is further off than the parts allow."""
    scale = 30000 / C / 0.75
    if mode == "weights":
        dy, x = _positive((C, 64), dtype, 41, 0.1, 0.2), _positive((C, 72), dtype, 42, scale * 3, scale * 7)
        off = torch.tensor([0, C], dtype=torch.int32, device="cuda")
        got = moe.grouped_matmul_wgrad(dy, x, off)[0]
        ref = sum(p.double().T @ q.double() for p, q in zip(dy.split(1 << 18), x.split(1 << 18)))
    else:
        M, F = 300, 72
        x, off = _positive((M, C), dtype, 43, 0.1, 0.2), torch.tensor([0, M], dtype=torch.int32, device="cuda")
        w = _positive((1, F, C) if mode == "forward" else (1, C, F), dtype, 44, scale * 3, scale * 7)
        got = moe.grouped_matmul(x, w, off, transpose=mode == "rows")
        ref = x.double() @ (w[0].double().T if mode == "forward" else w[0].double())
    _check_long(got, ref, ref, C)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_sums_have_no_bias(dtype):
    """Results spread over an octave and more, so that their roundings to 16 bits are of either sign: the mean of n of
    them is within five standard deviations, half a step over sqrt(3 n), and the sums' own part as above.  (In the test
    before, the results lie within 30 of 30000 and a bf16 step is 128: there all roundings share a sign.)"""
    C = 300_008
    dy = (_positive((C, 64), torch.float32, 54, 0.1, 0.2) * torch.linspace(1, 2, 64, device="cuda")).to(dtype)
    x = (_positive((C, 72), torch.float32, 55, 0.1, 0.2) * torch.linspace(1, 1.4, 72, device="cuda")).to(dtype)
    got = moe.grouped_matmul_wgrad(dy, x, torch.tensor([0, C], dtype=torch.int32, device="cuda"))[0]
    ref = dy.double().T @ x.double()
    off = _check_long(got, ref, ref, C)
    noise = 5 * torch.finfo(dtype).eps / 2 / (3 * off.numel()) ** 0.5
    assert float((off / ref).mean().abs()) <= 2 * 2.0 ** -23 * (8192 / 16 + 1 + C / 8192) + noise


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_and_short_tiles_follow_each_other(dtype):
    """Groups above and below the length of a part, and empty ones, over several tiles a pair of SMs."""
    sizes = [9000, 100, 0, 20000, 8192, 8193, 64, 8200, 1, 16385, 0, 500]
    o = torch.tensor([0] + sizes).cumsum(0).tolist()
    dy, x = _normal((o[-1], 1024), dtype, 45, 0.1), _normal((o[-1], 1096), dtype, 46, 0.1)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    got = [moe.grouped_matmul_wgrad(dy, x, off) for _ in range(3)]
    for e, n in enumerate(sizes):
        a, b = dy[o[e]:o[e + 1]].double().T, x[o[e]:o[e + 1]].double()
        _check_long(got[0][e], a @ b, a.abs() @ b.abs(), max(n, 1))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mode", ["forward", "rows"])
def test_long_products_over_many_tiles(mode, dtype):
    M, F, C = 2600, 2056, 16456  # three parts; 11 blocks by 9 tiles of features
    x = _normal((M, C), dtype, 47)
    w = _normal((3, F, C) if mode == "forward" else (3, C, F), dtype, 48, 0.02)
    off = torch.tensor([3, 1500, 1600, M], dtype=torch.int32, device="cuda")
    got = [moe.grouped_matmul(x, w, off, transpose=mode == "rows") for _ in range(2)]
    for e, (lo, hi) in enumerate(((3, 1500), (1500, 1600), (1600, M))):
        a, b = x[lo:hi].double(), w[e].double().T if mode == "forward" else w[e].double()
        _check_long(got[0][lo:hi], a @ b, a.abs() @ b.abs(), C)
        assert torch.equal(got[0][lo:hi], got[1][lo:hi])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("how", ["runs", "mixed"])
@pytest.mark.parametrize("added", [False, True])
def test_long_projection_with_adapters(how, added, dtype):
    """A projection of a long contraction takes its deltas and its old values once, in the last part."""
    T, N, K, r, L = 400, 264, 20008, 16, 3
    x, w = _positive((T, K), dtype, 49, 0.1, 0.2), _positive((N, K), dtype, 50, 0.1, 0.2)
    a, b = _normal((L, r, K), dtype, 51, K ** -0.5), _normal((L, N, r), dtype, 52, 5.0)
    ids = torch.arange(T, device="cuda") // 150 if how == "runs" else torch.arange(T, device="cuda") % (L + 1)
    before = _normal((T, N), dtype, 53, 100.0) if added else None
    got = moe.adapter_project(x, a, b, ids.int(), w=w, out=before.clone() if added else None,
                              flags=moe.MOE_ACCUMULATE if added else 0)
    ref = x.double() @ w.double().T
    mag, delta_mag = ref.clone(), torch.zeros_like(ref)
    for i in range(L):
        m = (ids == i).nonzero()[:, 0]
        ref[m] += (x[m].double() @ a[i].double().T) @ b[i].double().T
        delta_mag[m] = (x[m].double() @ a[i].double().abs().T) @ b[i].double().abs().T
    if added:
        ref, mag = ref + before.double(), mag + before.double().abs()
    # v is held to 2^-16 (bf16, two terms) or 2^-22 of its value's terms, its sum takes K / 16 steps
    v_terms = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22
    _check_long(got, ref, mag, K, more=(2 * 2.0 ** -23 * (K / 16 + r + 16) + v_terms) * delta_mag)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_the_longest_group(out_dtype):
    """As many rows as a call takes, in one group that ends inside a 16-row step: no wait runs out on the way (two
    million steps take longer than a wait's basic limit), and the sums hold."""
    M = (1 << 27) - 1
    g = torch.Generator(device="cuda").manual_seed(61)
    dy = torch.empty(M, 8, dtype=torch.bfloat16, device="cuda").uniform_(-1.0, 1.0, generator=g)
    x = torch.empty(M, 8, dtype=torch.bfloat16, device="cuda").uniform_(-1.0, 1.0, generator=g)
    x += dy  # (the diagonal grows with the rows)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    got = moe.grouped_matmul_wgrad(dy, x, off, out_dtype=out_dtype)[0]
    assert moe.moe_check_op_status() == 0
    ref, mag = torch.zeros(8, 8, dtype=torch.float64, device="cuda"), torch.zeros(8, 8, dtype=torch.float64, device="cuda")
    for p, q in zip(dy.split(1 << 22), x.split(1 << 22)):
        ref += p.double().T @ q.double()
        mag += p.double().abs().T @ q.double().abs()
    part = 8192 if out_dtype == torch.bfloat16 else 512
    # the parts' own steps, then one fp32 rounding of the sum so far for each part
    bound = (torch.finfo(out_dtype).eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (part / 16 + 1) * mag
             + M / part * 2.0 ** -24 * ref.abs().clamp(min=float(mag.max()) * 2.0 ** -8))
    off = (got.double() - ref).abs()
    print("relative error", float((off / ref.abs().clamp(min=1e-9)).diag().max()))
    assert not bool((off > bound).any()), f"worst {float((off / bound).max()):.3g} bounds"
