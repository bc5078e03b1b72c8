"""Low-rank adapters of many requests beside a shared projection, against the formula in 64 bits.

Tolerance, per value: half a step of the result's type, plus the fp32 sums.  Each 16-wide step of a tensor-core sum
costs at most two fp32 steps of a partial sum, each of the rank additions of the delta one more; slices, the scale and
the join of the terms at most 16: 2 * 2^-23 * (K / 16 + rank + 16) * (sum |w||x| + |scale| sum |b| sum |a||x| + |y before|).
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


def _inputs(T, N, K, r, L, dt, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(dt)

    return dict(x=normal(T, K), a=normal(L, r, K, s=K ** -0.5), b=normal(L, N, r, s=0.2), w=normal(N, K, s=0.05),
                scale=torch.rand(L, generator=g, device="cuda") * 2 - 1)


def _ids(T, L, how, seed=2):
    g = torch.Generator().manual_seed(seed)
    if how == "mixed":
        ids = torch.randint(-1, L, (T,), generator=g)
    elif how == "one":
        ids = torch.full((T,), L - 1)
    elif how == "none":
        ids = torch.full((T,), -1)
    else:  # requests of uneven lengths, cuts anywhere
        cuts = torch.randint(0, T + 1, (max(1, T // 40),), generator=g).sort().values
        ids = torch.randint(-1, L, (cuts.numel() + 1,), generator=g)[torch.searchsorted(cuts, torch.arange(T), right=True)]
    return ids.to(torch.int32).cuda()


def _reference(p, ids, w, before):
    d = torch.float64
    T, N = p["x"].shape[0], p["b"].shape[1]
    x = p["x"].to(d)
    y, mag = torch.zeros(T, N, dtype=d, device="cuda"), torch.zeros(T, N, dtype=d, device="cuda")
    if w is not None:
        y += x @ w.to(d).T
        mag += x.abs() @ w.to(d).abs().T
    for i in range(p["a"].shape[0]):
        m = (ids == i).nonzero()[:, 0]
        s = float(p["scale"][i]) if p["scale"] is not None else 1.0
        a, b = p["a"][i].to(d), p["b"][i].to(d)
        y[m] += s * ((x[m] @ a.T) @ b.T)
        mag[m] += abs(s) * ((x[m].abs() @ a.abs().T) @ b.abs().T)
    if before is not None:
        y += before.to(d)
        mag += before.to(d).abs()
    return y, mag


def _check(got, ref, mag, K, r):
    f = torch.finfo(got.dtype)
    bound = f.eps / 2 * ref.abs() + 2 * 2.0 ** -23 * (K / 16 + r + 16) * mag + f.tiny
    off = (got.double() - ref).abs()
    assert not bool((off > bound).any()), f"worst {float((off / bound).max()):.3g} bounds, {int((off > bound).sum())} values"


CASES = [
    # T, N, K, r, L, ids
    (1, 8, 8, 8, 1, "one"), (1, 2048, 2048, 16, 4, "one"), (3, 72, 136, 24, 2, "mixed"), (8, 256, 512, 8, 3, "mixed"),
    (33, 264, 1032, 16, 40, "mixed"), (64, 512, 256, 64, 5, "requests"), (64, 128, 128, 16, 3, "none"),
    (65, 136, 200, 16, 3, "mixed"), (100, 264, 520, 40, 7, "requests"), (257, 512, 256, 72, 2, "mixed"),
    (700, 384, 328, 32, 9, "requests"), (700, 384, 328, 128, 3, "one"), (300, 256, 64, 256, 2, "mixed"),
    (2100, 640, 768, 16, 64, "requests"), (2100, 136, 768, 16, 64, "mixed"), (5000, 128, 128, 8, 3, "requests"),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("form", ["projection", "projection fp32", "delta", "delta fp32", "added", "projection added fp32",
                                  "projection added"])
def test_against_the_formula(case, form, dtype):
    T, N, K, r, L, how = case
    dt = TYPES[dtype]
    p = _inputs(T, N, K, r, L, dt)
    ids = _ids(T, L, how)
    if T > 5:
        ids[T // 2] = L + 3  # an id that names no adapter
    if form == "delta":
        p["scale"] = None
    w = p["w"] if "projection" in form else None
    odt = torch.float32 if "fp32" in form else dt
    before = (torch.randn(T, N, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(odt)
              if "added" in form else None)
    out = before.clone() if before is not None else None
    flags = (moe.MOE_OUT_FP32 if odt == torch.float32 else 0) | (moe.MOE_ACCUMULATE if before is not None else 0)
    got = moe.adapter_project(p["x"], p["a"], p["b"], ids, w=w, scale=p["scale"], out=out, flags=flags)
    ref, mag = _reference(p, ids, w, before)
    assert got.dtype == odt
    _check(got, ref, mag, K, r)


@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("projection", [False, True])
def test_a_bad_adapter_or_token_stays_its_own(T, projection):
    """NaN and infinities of one adapter, or of one token, reach no other token."""
    p = _inputs(T, 136, 264, 16, 3, torch.bfloat16, 3)
    ids = _ids(T, 3, "mixed", 4)
    ids[0], ids[1], ids[2] = -1, 1, 2
    w = p["w"] if projection else None
    clean = moe.adapter_project(p["x"], p["a"], p["b"], ids, w=w, scale=p["scale"])
    p["a"][1] = float("nan")
    p["b"][1] = float("inf")
    x = p["x"].clone()
    x[2] = float("inf")
    got = moe.adapter_project(x, p["a"], p["b"], ids, w=w, scale=p["scale"])
    keep = (ids != 1)
    keep[2] = False
    assert torch.equal(got[keep], clean[keep])
    assert not bool(got[ids == 1].isfinite().any())
    # the same with every token of one adapter but one without
    ids[:] = 1
    ids[0] = -1
    got = moe.adapter_project(p["x"], p["a"], p["b"], ids, w=w, scale=p["scale"])
    assert torch.equal(got[0], clean[0])


@pytest.mark.parametrize("T,projection", [(7, True), (70, True), (70, False)])
def test_strided(T, projection):
    p = _inputs(T, 136, 200, 16, 3, torch.float16, 5)
    ids = _ids(T, 3, "mixed", 6)
    w = p["w"] if projection else None
    wide = torch.zeros(T, 512, dtype=torch.float16, device="cuda")
    wide[:, 16:216] = p["x"]
    out = torch.full((T, 300 + 4), 2.0, dtype=torch.float16, device="cuda")
    moe.adapter_project(wide[:, 16:216], p["a"], p["b"], ids, w=w, scale=p["scale"], out=out[:, 8:144])
    assert torch.equal(out[:, 8:144], moe.adapter_project(p["x"], p["a"], p["b"], ids, w=w, scale=p["scale"]))
    assert bool((out[:, :8] == 2).all()) and bool((out[:, 144:] == 2).all())


@pytest.mark.parametrize("T", [4, 48, 500])
@pytest.mark.parametrize("projection", [False, True])
def test_captured_and_replayed(T, projection):
    """Captured calls read new inputs and ids at each replay; two graphs that share nothing may run together."""
    p = _inputs(T, 256, 512, 16, 6, torch.bfloat16, 7)
    w = p["w"] if projection else None
    ids = _ids(T, 6, "requests", 8)
    x = p["x"].clone()
    moe.adapter_project(x, p["a"], p["b"], ids, w=w, scale=p["scale"])
    torch.cuda.synchronize()
    outs = [torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.adapter_project(x, p["a"], p["b"], ids, w=w, scale=p["scale"], out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for k in range(3):
        x.copy_(_inputs(T, 256, 512, 16, 6, torch.bfloat16, 20 + k)["x"])
        ids.copy_(_ids(T, 6, "mixed", 30 + k))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ref = moe.adapter_project(x, p["a"], p["b"], ids, w=w, scale=p["scale"])
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    del graphs


def test_on_another_stream():
    """A call on a side stream while the caller's stream is busy: inputs made before, workspace kept until it ran."""
    p = _inputs(128, 256, 512, 16, 6, torch.bfloat16, 11)
    ids = _ids(128, 6, "mixed", 12)
    ref = moe.adapter_project(p["x"], p["a"], p["b"], ids, w=p["w"], scale=p["scale"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [torch.empty_like(ref) for _ in range(20)]
    for o in outs:
        moe.adapter_project(p["x"], p["a"], p["b"], ids, w=p["w"], scale=p["scale"], out=o, stream=s)
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # reuses freed blocks at once
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
