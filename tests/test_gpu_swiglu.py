"""SwiGLU between an expert's products and its gradient, against the formulas in 64 bits.

Tolerances, per value: half a step of the result's type, plus the fp32 arithmetic.  The sigmoid is within 16 fp32
steps (exp within 2 + |x| of them, |x| <= 8 here, then an add and a quotient of two), and each of at most six further
operations rounds once: 24 * 2^-23 of the term's magnitude, where a sum counts the magnitudes of its parts.
"""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ARITH = 24 * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_expert_ffn_gemv_b200 import build
    build.build()


def _near(got, ref, mag):
    """fp16's smallest values round at an absolute step."""
    f = torch.finfo(got.dtype)
    bound = f.eps / 2 * ref.abs() + ARITH * mag + (f.smallest_normal * f.eps if got.dtype == torch.float16 else 1e-37)
    bad = (got.double() - ref).abs() > bound
    assert not bool(bad.any()), f"{int(bad.sum())} off"


def _inputs(rows, f, dt, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gu = (torch.randn(rows, 2 * f, generator=g, device="cuda") * 2).clamp_(-8, 8).to(dt)
    dh = torch.randn(rows, f, generator=g, device="cuda").to(dt)
    rw = torch.rand(rows, generator=g, device="cuda")
    return gu, dh, rw


def _formulas(gu, dh, rw):
    f = gu.shape[1] // 2
    g, u, d = gu[:, :f].double(), gu[:, f:].double(), dh.double()
    w = rw.double()[:, None] if rw is not None else torch.ones_like(g[:, :1])
    s = torch.sigmoid(g)
    h = w * g * s * u
    dg = w * d * u * s * (1 + g * (1 - s))
    du = w * d * g * s
    mag = (w * d * u * s).abs() * (1 + g.abs() * (1 - s))
    return h, torch.cat([dg, du], 1), torch.cat([mag, du.abs()], 1), (d * g * s * u)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,f", [(1, 8), (1, 2048), (7, 264), (640, 768), (5000, 136), (4736, 64), (4735, 64)])
@pytest.mark.parametrize("weighted", [False, True])
def test_forward_and_gradient(rows, f, dtype, weighted):
    dt = TYPES[dtype]
    gu, dh, rw = _inputs(rows, f, dt)
    rw = rw if weighted else None
    h64, dgu64, mag, dots = _formulas(gu, dh, rw)
    _near(moe.swiglu(gu, rw), h64, h64.abs())
    dgu, h, drw = moe.swiglu_backward(gu, dh, rw, with_h=True)
    _near(h, h64, h64.abs())
    _near(dgu, dgu64, mag)
    assert torch.equal(h, moe.swiglu(gu, rw))
    if weighted:
        # a sum of f terms in fp32: f / 256 + 13 roundings of partial sums at most
        bound = (ARITH + (f / 256 + 13) * 2.0 ** -23) * dots.abs().sum(1)
        assert bool(((drw.double() - dots.sum(1)).abs() <= bound).all())
    else:
        assert drw is None


def test_gradient_against_differences():
    """dgu and drw predict the change of sum(dh * h) for a small change of gu and of the weights (in 64 bits)."""
    gu, dh, rw = _inputs(16, 64, torch.float16, 3)
    dgu, _, drw = moe.swiglu_backward(gu, dh, rw)
    step = 1e-4
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.randn(gu.shape, generator=g, device="cuda").double()
    q = torch.randn(rw.shape, generator=g, device="cuda").double()

    def loss(gu64, rw64):
        a, b = gu64[:, :64], gu64[:, 64:]
        return (dh.double() * rw64[:, None] * a * torch.sigmoid(a) * b).sum()

    fd = (loss(gu.double() + step * p, rw.double() + step * q) - loss(gu.double() - step * p, rw.double() - step * q)) / (2 * step)
    an = (dgu.double() * p).sum() + (drw.double() * q).sum()
    # fp16 results: each of the terms is off by at most half a step; the differences by step^2 times third derivatives
    bound = 2.0 ** -11 * (dgu.double() * p).abs().sum() + 1e-6 * gu.numel()
    assert float((fd - an).abs()) <= float(bound)


@pytest.mark.parametrize("rows,used", [(10, 0), (10, 4), (6000, 5990), (6000, 7000)])
def test_rows_behind_are_left(rows, used):
    f = 72
    gu, dh, rw = _inputs(rows, f, torch.bfloat16, 5)
    n = torch.tensor([used], dtype=torch.int32, device="cuda")
    used = min(used, rows)
    gu[used:] = float("nan")
    h = torch.full((rows, f), 3.0, dtype=gu.dtype, device="cuda")
    dgu = torch.full((rows, 2 * f), 3.0, dtype=gu.dtype, device="cuda")
    drw = torch.full((rows,), 3.0, device="cuda")
    moe.swiglu(gu, rw, out=h, n_rows=n)
    assert bool((h[used:] == 3).all()) and bool(h[:used].isfinite().all())
    h2 = torch.full_like(h, 3.0)
    moe.swiglu_backward(gu, dh, rw, dgu=dgu, h=h2, drw=drw, n_rows=n)
    assert torch.equal(h, h2)
    assert bool((dgu[used:] == 3).all()) and bool((drw[used:] == 3).all())
    assert bool(dgu[:used].isfinite().all())


def test_extremes():
    """Large negative and positive gates saturate without NaN; a NaN or an infinity stays in its own value."""
    gu = torch.tensor([[-500.0, 500.0, 0.0, -80.0, 3.0, 1.0, 2.0, 4.0] + [1.0] * 8], dtype=torch.bfloat16, device="cuda")
    dh = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    h = moe.swiglu(gu)
    assert bool(h.isfinite().all()) and float(h[0, 0]) == 0 and float(h[0, 1]) == 500
    dgu, _, _ = moe.swiglu_backward(gu, dh)
    assert bool(dgu.isfinite().all()) and float(dgu[0, 0]) == 0 and float(dgu[0, 1]) == 1
    gu[0, 2], gu[0, 12] = float("nan"), float("inf")
    h = moe.swiglu(gu)
    assert bool(h[0, 2].isnan()) and bool(h[0, 4].isinf())
    assert bool(h[0, [0, 1, 3, 5, 6, 7]].isfinite().all())


def test_strided_and_in_place_slices():
    gu, dh, rw = _inputs(300, 96, torch.bfloat16, 6)
    wide = torch.zeros(300, 400, dtype=gu.dtype, device="cuda")
    wide[:, 8:200] = gu
    out = torch.full((300, 200), 2.0, dtype=gu.dtype, device="cuda")
    moe.swiglu(wide[:, 8:200], rw, out=out[:, 24:120])
    assert torch.equal(out[:, 24:120], moe.swiglu(gu, rw))
    assert bool((out[:, :24] == 2).all()) and bool((out[:, 120:] == 2).all())
