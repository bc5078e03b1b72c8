"""The 16-bit expert operators as they are used together: an expert FFN behind the library's router, its gradient, and
adapters beside the layer.

Tolerances of chained bf16 / fp16 steps are sums of half steps (eps / 2 of the value rounded), carried through the
following products by the magnitudes they are multiplied with; the fp32 sums between them are far below.
"""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe
from synth.layer import MoeShape

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_expert_ffn_gemv_b200 import build
    build.build()
    yield
    assert moe.moe_check_op_status() == 0


def _layer(sh, T):
    from synth import gpu
    codes, scales, wr, bias = gpu.layer_device(sh, 0x5EED_0016, 0, True)
    h = moe.MoeLayer(sh.d, sh.f, sh.E, sh.k, sh.n_shared, 1, sh.bits, T)
    h.load_layer(0, codes, scales, wr, bias)
    return h, gpu.x_device(sh, 0x5EED_0016, 5, T)


def _groups(h, x):
    """(token of each row in group order, routing weights in group order, offsets)"""
    ids, w = h.route(0, x)
    offsets, pairs, _, _, wsorted = h.bucket(ids, w)
    return (pairs // h.cfg.top_k).long(), wsorted, offsets


def _rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def test_dequantised_experts_give_the_quantised_layer():
    """The layer's experts as fp16 matrices (2-bit values times an fp16 scale are exact in fp16) through route,
    grouping, product, SwiGLU and product equal moe_forward: both round h and the weighted outputs to fp16."""
    sh, T = MoeShape(d=256, f=128, E=16, k=2, n_shared=0, bits=2), 300
    h, x = _layer(sh, T)
    try:
        ref = h.forward(0, x, flags=moe.MOE_OUT_FP32)
        w1 = torch.stack([torch.cat([h.debug_dequant(0, e, 0), h.debug_dequant(0, e, 1)]) for e in range(sh.E)]).half()
        w2 = torch.stack([h.debug_dequant(0, e, 2) for e in range(sh.E)]).half()
        tok, rw, off = _groups(h, x)
        gu = moe.grouped_matmul(x.half()[tok], w1, off, out_dtype=torch.float32)
        gu16 = moe.grouped_matmul(x.half()[tok], w1, off)
        hh = moe.swiglu(gu16, rw)
        o = moe.grouped_matmul(hh, w2, off, out_dtype=torch.float32)
        y = torch.zeros(T, sh.d, device="cuda").index_add_(0, tok, o)
        # gate, up and h rounded to fp16 here (3 half steps of 2^-11), h and the outputs there (2): in the 2-norm at
        # most their sum, and SwiGLU's slope is below 1.1 of its value's scale
        assert _rel(y, ref) < 6 * 2.0 ** -11
        assert _rel(gu16, gu) < 2.0 ** -11
    finally:
        h.close()


def _ffn_grad(x, w1, w2, rw, tok, off, dy, cast):
    """The FFN and its gradient by the operators; cast: the gradient's 16-bit type."""
    xr = x[tok]
    gu = moe.grouped_matmul(xr, w1, off)
    h = moe.swiglu(gu, rw)
    o = moe.grouped_matmul(h, w2, off, out_dtype=torch.float32)
    y = torch.zeros(x.shape[0], w2.shape[1], device="cuda").index_add_(0, tok, o)
    do = dy[tok].to(cast)
    dh = moe.grouped_matmul(do, w2, off, transpose=True)
    dgu, h2, drw = moe.swiglu_backward(gu, dh, rw, with_h=True)
    assert torch.equal(h, h2)
    dxr = moe.grouped_matmul(dgu, w1, off, transpose=True, out_dtype=torch.float32)
    dx = torch.zeros(x.shape, device="cuda").index_add_(0, tok, dxr)
    dw1 = moe.grouped_matmul_wgrad(dgu, xr, off, out_dtype=torch.float32)
    dw2 = moe.grouped_matmul_wgrad(do, h, off, out_dtype=torch.float32)
    return y, dx, dw1, dw2, drw


def _ffn_formula(x, w1, w2, rw, tok, off, dy):
    x, w1, w2, rw, dy = (t.double().detach().requires_grad_(True) if i < 4 else t.double() for i, t in enumerate((x, w1, w2, rw, dy)))
    y = torch.zeros(x.shape[0], w2.shape[1], dtype=torch.float64, device="cuda")
    o, f = off.tolist(), w2.shape[2]
    parts = []
    for e in range(w1.shape[0]):
        r = slice(o[e], o[e + 1])
        gu = x[tok[r]] @ w1[e].T
        h = rw[r, None] * torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
        parts.append(h @ w2[e].T)
    y = y.index_add(0, tok, torch.cat(parts))
    return (y,) + torch.autograd.grad((y * dy).sum(), (x, w1, w2, rw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_expert_ffn_and_gradient_against_the_formula(dtype):
    """Forward and all gradients of a routed 16-bit FFN against 64-bit autograd of the formula.  Each result passes at
    most six roundings to 16 bits (gu, h, dy, dh, dgu and its own), each half a step of a value that enters it linearly
    with relative weight at most about one: 2-norm error below 6 * eps / 2, and eps / 2 more for the slope's argument."""
    sh, T = MoeShape(d=256, f=128, E=16, k=2, n_shared=0, bits=2), 500
    h, x = _layer(sh, T)
    g = torch.Generator(device="cuda").manual_seed(1)
    try:
        tok, rw, off = _groups(h, x)
        x = x.to(dtype)
        w1 = (torch.randn(sh.E, 2 * sh.f, sh.d, generator=g, device="cuda") * sh.d ** -0.5).to(dtype)
        w2 = (torch.randn(sh.E, sh.d, sh.f, generator=g, device="cuda") * sh.f ** -0.5).to(dtype)
        dy = torch.randn(T, sh.d, generator=g, device="cuda").to(dtype)
        got = _ffn_grad(x, w1, w2, rw, tok, off, dy, dtype)
        ref = _ffn_formula(x, w1, w2, rw, tok, off, dy)
        for name, a, b in zip(("y", "dx", "dw1", "dw2", "drw"), got, ref):
            assert _rel(a, b) < 7 * torch.finfo(dtype).eps / 2, name
    finally:
        h.close()


def test_adapter_gradients_are_grouped_products():
    """Gradients of A and B of many adapters, from rows sorted by adapter: dB = dy^T v, dA = (dy B)^T x per group,
    against 64-bit autograd; each passes two 16-bit roundings (v or dy B, and the bf16 operands are exact)."""
    g = torch.Generator(device="cuda").manual_seed(2)
    L, r, d, T = 5, 16, 256, 400
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    a = (torch.randn(L, r, d, generator=g, device="cuda") / 16).bfloat16()
    b = (torch.randn(L, d, r, generator=g, device="cuda") / 4).bfloat16()
    off = torch.tensor([0, 100, 100, 250, 390, 400], dtype=torch.int32, device="cuda")
    ids = torch.bucketize(torch.arange(T, device="cuda"), off[1:].long(), right=True).int()
    v = moe.grouped_matmul(x, a, off)
    db = moe.grouped_matmul_wgrad(dy, v, off, out_dtype=torch.float32)
    dv = moe.grouped_matmul(dy, b, off, transpose=True)
    da = moe.grouped_matmul_wgrad(dv, x, off, out_dtype=torch.float32)
    A, B = a.double().requires_grad_(True), b.double().requires_grad_(True)
    y = torch.einsum("tr,tnr->tn", torch.einsum("td,trd->tr", x.double(), A[ids.long()]), B[ids.long()])
    rA, rB = torch.autograd.grad((y * dy.double()).sum(), (A, B))
    assert _rel(da, rA) < 2.0 ** -8 and _rel(db, rB) < 2.0 ** -8
    # and the forward of the same adapters
    got = moe.adapter_project(x, a, b, ids, flags=moe.MOE_OUT_FP32)
    assert _rel(got, y.detach()) < 1e-5


def test_a_training_step_in_a_graph():
    """The FFN and its gradient captured once and replayed on new rows and a new grouping (the row count stays, the
    offsets change on the device), while an eager step runs on another stream between the replays."""
    sh, T = MoeShape(d=256, f=128, E=16, k=2, n_shared=0, bits=2), 256
    h, x = _layer(sh, T)
    g = torch.Generator(device="cuda").manual_seed(3)
    try:
        w1 = (torch.randn(sh.E, 2 * sh.f, sh.d, generator=g, device="cuda") / 16).bfloat16()
        w2 = (torch.randn(sh.E, sh.d, sh.f, generator=g, device="cuda") / 11).bfloat16()
        tok, rw, off = _groups(h, x)
        dy = torch.randn(T, sh.d, generator=g, device="cuda").bfloat16()
        xr, do = x[tok].contiguous(), dy[tok].contiguous()

        def step(xr, do, rw, off):
            gu = moe.grouped_matmul(xr, w1, off)
            hh = moe.swiglu(gu, rw)
            o = moe.grouped_matmul(hh, w2, off)
            dh = moe.grouped_matmul(do, w2, off, transpose=True)
            dgu, h2, drw = moe.swiglu_backward(gu, dh, rw, with_h=True)
            return (o, moe.grouped_matmul(dgu, w1, off, transpose=True), moe.grouped_matmul_wgrad(dgu, xr, off),
                    moe.grouped_matmul_wgrad(do, h2, off, out_dtype=torch.float32), drw)

        step(xr, do, rw, off)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(xr, do, rw, off)
        side = torch.cuda.Stream()
        for k in range(3):
            from synth import gpu
            x2 = gpu.x_device(sh, 0x5EED_0016, 50 + k, T)
            tok2, rw2, off2 = _groups(h, x2)
            xr.copy_(x2[tok2]), do.copy_(dy[tok2]), rw.copy_(rw2), off.copy_(off2)
            torch.cuda.synchronize()
            graph.replay()
            with torch.cuda.stream(side):
                eager = step(xr, do, rw, off)
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                assert torch.equal(a, b)
        del graph
    finally:
        h.close()


@pytest.mark.parametrize("T", [1, 8, 100])
@pytest.mark.parametrize("flags", [0, moe.MOE_OUT_FP32, moe.MOE_NORM_INPUT, moe.MOE_ACCUMULATE | moe.MOE_OUT_FP32])
def test_adapters_beside_the_layer(T, flags):
    """MoeLayer.forward_adapted = forward, then the formula of the adapters on the same (normalised) input."""
    sh = MoeShape(d=256, f=128, E=16, k=2, n_shared=1, bits=2)
    h, x = _layer(sh, T)
    g = torch.Generator(device="cuda").manual_seed(4)
    try:
        L, r = 3, 8
        a = (torch.randn(L, r, sh.d, generator=g, device="cuda") / 16).bfloat16()
        b = (torch.randn(L, sh.d, r, generator=g, device="cuda") / 4).bfloat16()
        scale = torch.rand(L, generator=g, device="cuda") + 0.5
        ids = torch.randint(-1, L, (T,), generator=g, device="cuda").int()
        u = moe.rms_normalize(x) if flags & moe.MOE_NORM_INPUT else x
        f32 = bool(flags & moe.MOE_OUT_FP32)
        y0 = torch.randn(T, sh.d, generator=g, device="cuda").to(torch.float32 if f32 else torch.bfloat16)
        base = h.forward(0, x, y0.clone(), flags=flags)
        got = h.forward_adapted(0, x, a, b, ids, scale, y0.clone(), flags=flags)
        v = torch.einsum("td,trd->tr", u.double(), a.double()[ids.clamp(min=0).long()])
        d = torch.einsum("tr,tnr->tn", v, b.double()[ids.clamp(min=0).long()]) * (scale[ids.clamp(min=0).long()] * (ids >= 0))[:, None]
        ref = base.double() + d
        # one more rounding of y (half a step), the inner fp32 sums below 2^-18 of the terms' magnitude
        mag = base.double().abs() + d.abs().amax(1, keepdim=True) * 8
        bound = torch.finfo(got.dtype).eps / 2 * ref.abs() + 2.0 ** -18 * mag
        assert bool(((got.double() - ref).abs() <= bound).all())
        if flags & moe.MOE_NORM_INPUT:  # the residual step in place
            xi = x.clone()
            h.forward_adapted(0, xi, a, b, ids, scale, xi, flags=flags | moe.MOE_ACCUMULATE)
            two = h.forward(0, u, x.clone(), flags=moe.MOE_ACCUMULATE)
            assert torch.equal(xi, moe.adapter_project(u, a, b, ids, scale=scale, out=two, flags=moe.MOE_ACCUMULATE))
        else:
            with pytest.raises(ValueError):
                h.forward_adapted(0, x, a, b, ids, scale, x, flags=flags)
    finally:
        h.close()


def test_wrappers_refuse():
    """Shapes, types, strides and devices that do not match raise before anything is enqueued."""
    bf, dev = torch.bfloat16, "cuda"
    x, w = torch.zeros(6, 64, dtype=bf, device=dev), torch.zeros(2, 32, 64, dtype=bf, device=dev)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device=dev)
    a, b = torch.zeros(2, 8, 64, dtype=bf, device=dev), torch.zeros(2, 32, 8, dtype=bf, device=dev)
    ids = torch.zeros(6, dtype=torch.int32, device=dev)
    gu, dh = torch.zeros(6, 64, dtype=bf, device=dev), torch.zeros(6, 32, dtype=bf, device=dev)
    bad = [
        lambda: moe.grouped_matmul(x.float(), w, off), lambda: moe.grouped_matmul(x.half(), w, off),
        lambda: moe.grouped_matmul(x[:, :32], w, off), lambda: moe.grouped_matmul(x, w, off[:2]),
        lambda: moe.grouped_matmul(x, w, off.long()), lambda: moe.grouped_matmul(x, w.transpose(1, 2), off),
        lambda: moe.grouped_matmul(x, w, off, transpose=True), lambda: moe.grouped_matmul(x.t(), w, off),
        lambda: moe.grouped_matmul(x, w, off, out=torch.zeros(6, 32, dtype=torch.float16, device=dev)),
        lambda: moe.grouped_matmul(x, w, off, out=torch.zeros(5, 32, dtype=bf, device=dev)),
        lambda: moe.grouped_matmul(x, w, off.cpu()), lambda: moe.grouped_matmul(x, w, off, out_dtype=torch.float64),
        lambda: moe.grouped_matmul_wgrad(dh, x[:5], off), lambda: moe.grouped_matmul_wgrad(dh, x, off, accumulate=True),
        lambda: moe.grouped_matmul_wgrad(dh, x, off, out=torch.zeros(2, 64, 32, dtype=bf, device=dev)),
        lambda: moe.swiglu(gu[:, :63]), lambda: moe.swiglu(gu, torch.zeros(5, device=dev)),
        lambda: moe.swiglu(gu, torch.zeros(6, dtype=bf, device=dev)), lambda: moe.swiglu(gu, out=gu),
        lambda: moe.swiglu_backward(gu, gu), lambda: moe.swiglu_backward(gu, dh, drw=torch.zeros(6, device=dev)),
        lambda: moe.adapter_project(x, a, b[:1], ids), lambda: moe.adapter_project(x, a, b, ids[:5]),
        lambda: moe.adapter_project(x, a, b, ids.long()), lambda: moe.adapter_project(x, a.half(), b.half(), ids),
        lambda: moe.adapter_project(x, a, b, ids, w=w), lambda: moe.adapter_project(x, a, b, ids, flags=moe.MOE_ACCUMULATE),
        lambda: moe.adapter_project(x, a, b, ids, scale=torch.zeros(3, device=dev)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(moe.MoeError):  # ranks are multiples of 8
        moe.adapter_project(x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ids)
    with pytest.raises(moe.MoeError):  # rows that start off a 16-byte boundary
        moe.grouped_matmul(torch.zeros(6, 80, dtype=bf, device=dev)[:, 4:68], w, off)
    with pytest.raises(moe.MoeError):  # a result that is also the input
        moe.adapter_project(dh, torch.zeros(2, 8, 32, dtype=bf, device=dev), b, ids, out=dh)


@pytest.mark.parametrize("rows", [40, 300, 3000])
def test_back_to_back_calls_are_ordered(rows):
    """Kernels of these calls may start before the one before them has finished: a chain in which every call reads what
    the one before wrote, and overwrites what it read, gives the same bits as with a synchronisation after each call."""
    E, d, f, L, r = 6, 256, 128, 4, 16
    g = torch.Generator(device="cuda").manual_seed(7)

    def normal(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

    w1, w2, w = normal(E, 2 * f, d, s=d ** -0.5), normal(E, d, f, s=f ** -0.5), normal(d, d, s=d ** -0.5)
    a, b, rw = normal(L, r, d, s=d ** -0.5), normal(L, d, r, s=0.2), torch.rand(rows, generator=g, device="cuda")
    cuts = torch.randint(0, rows + 1, (E - 1,), generator=g, device="cuda").sort().values
    off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows)]).int()
    ids = torch.randint(-1, L, (rows,), generator=g, device="cuda").sort().values.int()
    x0 = normal(rows, d)

    def chain(wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        x, gu, h = x0.clone(), torch.empty(rows, 2 * f, dtype=x0.dtype, device="cuda"), torch.empty(rows, f, dtype=x0.dtype, device="cuda")
        y, dw = torch.empty_like(x), torch.zeros(E, 2 * f, d, device="cuda")
        done()
        for k in range(12):
            moe.grouped_matmul(x, w1, off, out=gu), done()
            moe.swiglu(gu, rw, out=h), done()
            moe.grouped_matmul(h, w2, off, out=y), done()
            moe.adapter_project(y, a, b, ids, w=w, out=x), done()
            moe.adapter_project(y, a, b, ids, out=x, flags=moe.MOE_ACCUMULATE), done()
            moe.swiglu_backward(gu, h, rw, dgu=gu.clone() if k % 2 else gu), done()
            moe.grouped_matmul_wgrad(gu, x, off, out=dw, accumulate=True), done()
            moe.grouped_matmul(y, w2, off, out=h, transpose=True), done()
            x.add_(moe.rms_normalize(y)), done()
            x.copy_(moe.rms_normalize(x)), done()
        return x, y, h, gu, dw

    plain = chain(True)
    for _ in range(4):
        for p, q in zip(plain, chain(False)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("op", ["grouped_matmul", "grouped_matmul_wgrad", "swiglu", "swiglu_backward", "adapter_project",
                                "forward_adapted"])
def test_a_result_allocated_for_a_given_stream(op):
    """A result that a call on another stream allocates is no block that the caller's stream still writes."""
    g = torch.Generator(device="cuda").manual_seed(12)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    sh = MoeShape(d=256, f=128, E=16, k=2, n_shared=0, bits=2)
    h, x = _layer(sh, 64)
    try:
        rows, E = 64, 4
        off = torch.arange(0, rows + 1, rows // E, device="cuda").int()
        w, gu, dy = rnd(E, 256, sh.d), rnd(rows, 512), rnd(rows, 256)
        a, b, ids = rnd(3, 8, sh.d), rnd(3, sh.d, 8), torch.arange(rows, device="cuda").int() % 3
        call = {"grouped_matmul": lambda s: moe.grouped_matmul(x, w, off, stream=s),
                "grouped_matmul_wgrad": lambda s: moe.grouped_matmul_wgrad(dy, x, off, stream=s),
                "swiglu": lambda s: moe.swiglu(gu, stream=s),
                "swiglu_backward": lambda s: moe.swiglu_backward(gu, dy, stream=s)[0],
                "adapter_project": lambda s: moe.adapter_project(x, a, b, ids, stream=s),
                "forward_adapted": lambda s: h.forward_adapted(0, x, a, b, ids, flags=moe.MOE_NORM_INPUT, stream=s)}[op]
        ref = call(None).clone()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        torch.cuda._sleep(50_000_000)  # the caller's stream is busy for some 25 ms
        busy = [torch.empty_like(ref).fill_(7) for _ in range(8)]  # written after that
        del busy
        got = call(s)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
    finally:
        h.close()


def test_a_stream_of_another_device_is_refused():
    class Other:  # (what the wrappers read of a torch.cuda.Stream)
        device_index, cuda_stream = torch.cuda.current_device() + 1, 0

    gu = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.swiglu(gu, stream=Other())
    with pytest.raises(AttributeError):
        moe.swiglu(gu, stream=3)
