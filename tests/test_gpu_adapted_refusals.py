"""MoeLayer.forward_adapted refuses what does not fit before the layer writes its result."""
import pytest
import torch

import bit_expert_ffn_gemv_b200 as moe
from synth.layer import MoeShape

pytestmark = pytest.mark.gpu

T, L, R = 6, 3, 8


@pytest.fixture(scope="module")
def layer():
    from bit_expert_ffn_gemv_b200 import build
    from synth import gpu
    build.build()
    sh = MoeShape(d=256, f=128, E=16, k=2, n_shared=1, bits=2)
    codes, scales, wr, bias = gpu.layer_device(sh, 0x5EED_0017, 0, True)
    h = moe.MoeLayer(sh.d, sh.f, sh.E, sh.k, sh.n_shared, 1, sh.bits, T)
    h.load_layer(0, codes, scales, wr, bias)
    yield h, gpu.x_device(sh, 0x5EED_0017, 5, T)
    h.close()


class OtherDevice:  # (what is read of a torch.cuda.Stream)
    device_index, cuda_stream = 7, 0


def _shifted(t):  # the same values off a 16-byte boundary
    s = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[1:1 + t.numel()].view(t.shape)
    return s.copy_(t)


BAD = {
    "a of another width": dict(a=lambda a, **_: a[:, :, :128].contiguous()),
    "a of another type": dict(a=lambda a, **_: a.half()),
    "b of fewer features": dict(b=lambda b, **_: b[:, :128].contiguous()),
    "b of fewer adapters": dict(b=lambda b, **_: b[:2]),
    "a, b of rank 4": dict(a=lambda a, **_: a[:, :4].contiguous(), b=lambda b, **_: b[:, :, :4].contiguous()),
    "a misaligned": dict(a=lambda a, **_: _shifted(a)),
    "b misaligned": dict(b=lambda b, **_: _shifted(b)),
    "ids of 64 bits": dict(ids=lambda ids, **_: ids.long()),
    "ids too few": dict(ids=lambda ids, **_: ids[:-1]),
    "ids on the host": dict(ids=lambda ids, **_: ids.cpu()),
    "scale too short": dict(scale=lambda scale, **_: scale[:2]),
    "b requires a gradient": dict(b=lambda b, **_: b.clone().requires_grad_(True)),
    "stream of another device": dict(stream=lambda **_: OtherDevice()),
}


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("in_place", [False, True])
def test_a_refused_call_leaves_y(layer, bad, in_place):
    h, x = layer
    g = torch.Generator(device="cuda").manual_seed(1)
    x = x.clone()
    args = dict(a=torch.randn(L, R, 256, generator=g, device="cuda").bfloat16(),
                b=torch.randn(L, 256, R, generator=g, device="cuda").bfloat16(),
                ids=torch.zeros(T, dtype=torch.int32, device="cuda"), scale=torch.rand(L, generator=g, device="cuda"), stream=None)
    y = x if in_place else torch.full_like(x, 3.0)
    flags = moe.MOE_NORM_INPUT | moe.MOE_ACCUMULATE if in_place else 0
    before = y.clone()
    changed = {k: fn(**args) for k, fn in BAD[bad].items()}
    with pytest.raises((ValueError, moe.MoeError)):
        h.forward_adapted(0, x, y=y, flags=flags, **{**args, **changed})
    torch.cuda.synchronize()
    assert torch.equal(y, before)
    h.forward_adapted(0, x, y=y, flags=flags, **args)
    torch.cuda.synchronize()
    assert not torch.equal(y, before)


def test_x_and_y_that_the_layer_cannot_take(layer):
    h, x = layer
    a, b = torch.zeros(L, R, 256, dtype=x.dtype, device="cuda"), torch.zeros(L, 256, R, dtype=x.dtype, device="cuda")
    ids, wide = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, 512, dtype=x.dtype, device="cuda")
    new = lambda *s, dtype=x.dtype: torch.zeros(s, dtype=dtype, device="cuda")
    for bad_x in (wide[:, :256], x.half(), x.float(), x[:, :128].contiguous(), x.cpu(), x[None]):
        with pytest.raises(ValueError):
            h.forward_adapted(0, bad_x, a, b, ids)
    for flags, y in ((0, wide[:, :256]), (0, new(T, 256, dtype=torch.float32)), (moe.MOE_OUT_FP32, new(T, 256)), (0, new(T - 1, 256)),
                     (0, new(T, 128)), (0, torch.zeros_like(x, device="cpu"))):
        with pytest.raises(ValueError):
            h.forward_adapted(0, x, a, b, ids, y=y, flags=flags)
    with pytest.raises(ValueError):
        h.forward_adapted(0, x, a, b, ids, flags=moe.MOE_ACCUMULATE)
    with pytest.raises(moe.MoeError):  # a result that starts off a 16-byte boundary
        h.forward_adapted(0, x, a, b, ids, y=_shifted(x))
