"""Grouped products of ragged row groups, and their gradients, against the formulas in 64 bits.

Tolerances, per value: one rounding to the result's type (half a step: eps / 2 relative) plus the fp32 sum.  The
tensor core adds 16 exact products to its accumulator at a time; aligning and adding them costs at most two fp32
steps (2 * 2^-23) of a partial sum, which is at most sum |a||b|: 2 * 2^-23 * (C / 16 + 1) * sum |a||b| over C terms.
"""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_expert_ffn_gemv_b200 import build
    build.build()
    yield
    assert moe.moe_check_op_status() == 0


def _offsets(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def _normal(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)


def _check(got, ref, mag, C, dt):
    """|got - ref| within the bound above; mag = sum |a||b|."""
    got, eps = got.double(), torch.finfo(dt).eps
    bound = eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (C / 16 + 1) * mag + torch.finfo(dt).tiny
    bad = (got - ref).abs() > bound
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values off, worst {float(((got - ref).abs() / bound).max()):.3g} bounds"


SHAPES = [
    # sizes, first, behind, N, K
    ([1], 0, 0, 8, 8),
    ([1], 0, 0, 256, 64),
    ([5, 0, 1, 40], 0, 0, 72, 136),
    ([0, 0, 300, 0], 3, 7, 200, 328),
    ([257, 16, 31, 33, 0, 65], 0, 5, 264, 520),
    ([64, 128, 256, 512], 0, 0, 512, 256),
    ([1000, 3, 0, 771], 1, 60, 640, 192),
    ([0, 0, 0], 0, 4, 128, 128),
    ([100] * 37, 0, 0, 1536, 256),
    ([2] * 1024, 0, 0, 64, 72),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["forward", "rows"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{sum(s[0])}+{s[1]}+{s[2]}-{s[3]}x{s[4]}")
@pytest.mark.parametrize("out32", [False, True])
def test_products(shape, mode, dtype, out32):
    sizes, first, behind, N, K = shape
    dt = TYPES[dtype]
    o = _offsets(sizes, first)
    M, E = o[-1] + behind, len(sizes)
    tr = mode == "rows"
    x = _normal((M, N if tr else K), dt, 1)
    x[:first] = float("nan")  # rows of no group must not reach any result
    x[o[-1]:] = float("inf")
    w = _normal((E, N, K), dt, 2, 0.05)
    odt = torch.float32 if out32 else dt
    out = torch.full((M, K if tr else N), 7.0, dtype=odt, device="cuda")
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    got = moe.grouped_matmul(x, w, off, out=out, transpose=tr)
    assert got is out
    assert bool((out[:first] == 7).all()) and bool((out[o[-1]:] == 7).all())
    for e in range(E):
        a, b = x[o[e]:o[e + 1]].double(), w[e].double() if tr else w[e].double().T
        _check(out[o[e]:o[e + 1]], a @ b, a.abs() @ b.abs(), N if tr else K, odt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{sum(s[0])}+{s[1]}+{s[2]}-{s[3]}x{s[4]}")
@pytest.mark.parametrize("how", ["16", "fp32", "accumulate"])
def test_weights_gradient(shape, dtype, how):
    sizes, first, behind, N, K = shape
    dt = TYPES[dtype]
    o = _offsets(sizes, first)
    M, E = o[-1] + behind, len(sizes)
    dy, x = _normal((M, N), dt, 3), _normal((M, K), dt, 4)
    for t in (dy, x):
        t[:first] = float("inf")
        t[o[-1]:] = float("nan")
    odt = dt if how == "16" else torch.float32
    before = _normal((E, N, K), torch.float32, 5) if how == "accumulate" else None
    out = before.clone() if before is not None else torch.full((E, N, K), 7.0, dtype=odt, device="cuda")
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    moe.grouped_matmul_wgrad(dy, x, off, out=out, accumulate=before is not None)
    for e in range(E):
        a, b = dy[o[e]:o[e + 1]].double().T, x[o[e]:o[e + 1]].double()
        ref, mag = a @ b, a.abs() @ b.abs()
        if before is not None:
            ref = ref + before[e].double()
            # one more fp32 rounding: the sum before it is added
            mag = mag + before[e].double().abs()
        _check(out[e], ref, mag, max(sizes[e], 1), odt)


def test_neighbour_groups_do_not_mix():
    """A group whose rows hold NaN and infinities leaves the groups beside it (same 16-row step) exact."""
    sizes = [3, 4, 5, 50]
    o = _offsets(sizes)
    dy, x = _normal((o[-1], 64), torch.bfloat16, 6), _normal((o[-1], 64), torch.bfloat16, 7)
    clean = moe.grouped_matmul_wgrad(dy, x, torch.tensor(o, dtype=torch.int32, device="cuda"))
    dy2, x2 = dy.clone(), x.clone()
    dy2[3:7] = float("nan")
    x2[3:7] = float("inf")
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    got = moe.grouped_matmul_wgrad(dy2, x2, off)
    for e in (0, 2, 3):
        assert torch.equal(got[e], clean[e])
    assert bool(got[1].isnan().all())
    w = _normal((4, 64, 64), torch.bfloat16, 8)
    y, y2 = moe.grouped_matmul(x, w, off), moe.grouped_matmul(x2, w, off)
    keep = torch.tensor([r for r in range(o[-1]) if not 3 <= r < 7], device="cuda")
    assert torch.equal(y[keep], y2[keep])


@pytest.mark.parametrize("mode", ["forward", "rows", "weights"])
def test_strided_rows(mode):
    """Row pitches above the row length, results into a slice of a wider buffer, results bit for bit as contiguous."""
    sizes = [100, 0, 45, 300]
    o = _offsets(sizes)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    wide = _normal((o[-1], 512), torch.bfloat16, 9)
    w = _normal((4, 136, 136), torch.bfloat16, 10)
    a, b = wide[:, 8:144], wide[:, 256:392]
    if mode == "weights":
        assert torch.equal(moe.grouped_matmul_wgrad(a, b, off), moe.grouped_matmul_wgrad(a.contiguous(), b.contiguous(), off))
        return
    buf = torch.full((o[-1], 400), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_matmul(a, w, off, out=buf[:, 16:152], transpose=mode == "rows")
    assert torch.equal(buf[:, 16:152], moe.grouped_matmul(a.contiguous(), w, off, transpose=mode == "rows"))
    assert bool((buf[:, :16] == 3).all()) and bool((buf[:, 152:] == 3).all())


@pytest.mark.parametrize("table", [[0, -5, 4000, 20], [50, 20, 90, 10], [90, 90, 90, 90], [-9, -3, -1, 0]])
def test_a_bad_offset_table_stays_in_range(table):
    """Offsets outside [0, rows] or descending: clamped, nothing outside the result is touched, and the groups that
    are well formed after clamping hold their product."""
    M, N, K = 80, 64, 72
    x, w = _normal((M, K), torch.bfloat16, 11), _normal((3, N, K), torch.bfloat16, 12)
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    buf = torch.full((M + 64, N), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_matmul(x, w, off, out=buf[32:32 + M])
    dw = moe.grouped_matmul_wgrad(_normal((M, N), torch.bfloat16, 13), x, off)
    torch.cuda.synchronize()
    assert bool((buf[:32] == 5).all()) and bool((buf[32 + M:] == 5).all())
    c = [min(max(v, 0), M) for v in table]
    covered = [0] * M
    for e in range(3):
        for r in range(c[e], max(c[e], c[e + 1])):
            covered[r] += 1
    for r in range(M):
        if covered[r] == 0:
            assert bool((buf[32 + r] == 5).all())
    for e in range(3):
        if c[e + 1] <= c[e]:
            assert bool((dw[e] == 0).all())


def test_long_group_fp32_gradient():
    """A weight gradient over many rows in fp32 keeps fp32 accuracy: relative 2-norm error below 2^-19 over 30001
    rows (each of the up to 30001 / 16 steps rounds a partial sum once; the sums are spread over bounded chunks)."""
    M, N, K = 30001, 256, 264
    dy, x = _normal((M, N), torch.bfloat16, 14), _normal((M, K), torch.bfloat16, 15)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    got = moe.grouped_matmul_wgrad(dy, x, off, out_dtype=torch.float32)[0].double()
    ref = dy.double().T @ x.double()
    err = float((got - ref).norm() / ref.norm())
    print("relative error", err)
    assert err < 2.0 ** -19


@pytest.mark.parametrize("mode", ["forward", "rows", "weights"])
def test_repeats_are_bit_identical(mode):
    sizes = [700, 13, 0, 256, 90]
    o = _offsets(sizes)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    x, dy = _normal((o[-1], 320), torch.bfloat16, 16), _normal((o[-1], 320), torch.bfloat16, 17)
    w = _normal((5, 320, 320), torch.bfloat16, 18)
    def call():
        if mode == "weights":
            return moe.grouped_matmul_wgrad(dy, x, off)
        return moe.grouped_matmul(x, w, off, transpose=mode == "rows")
    a = call()
    for _ in range(5):
        assert torch.equal(a, call())
