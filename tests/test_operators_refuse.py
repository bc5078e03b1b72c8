"""Refusals of the 16-bit expert operators: every argument error is returned before any CUDA call, so these run
without a GPU (the pointers are never read)."""
import ctypes

import pytest

import bit_expert_ffn_gemv_b200 as moe
from bit_expert_ffn_gemv_b200 import build

P = 1 << 20  # a 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


GOOD_MATMUL = dict(x=P, ldx=64, rows=10, w=3 * P, offsets=P, groups=4, n=32, k=64, y=2 * P, ldy=32, flags=0)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 27) + 1), dict(groups=0), dict(groups=1025), dict(n=0), dict(n=12), dict(k=4), dict(k=-8),
    dict(n=1 << 18), dict(ldx=56), dict(ldx=68), dict(ldy=24), dict(ldy=36), dict(x=0), dict(x=P + 8), dict(w=0), dict(w=P + 2),
    dict(y=0), dict(y=P + 4), dict(y=P), dict(y=3 * P), dict(offsets=0), dict(offsets=P + 2), dict(flags=0x2), dict(flags=0x4), dict(flags=1 << 31),
    dict(flags=0x200),  # transposed: x needs n columns a row, y needs k
], ids=str)
def test_grouped_matmul(L, bad):
    a = dict(GOOD_MATMUL, **bad)
    if bad == dict(flags=0x200):
        a["ldx"] = 24
    assert L.moe_grouped_matmul(a["x"], a["ldx"], a["rows"], a["w"], a["offsets"], a["groups"], a["n"], a["k"], a["y"],
                                a["ldy"], a["flags"], None) == 1


GOOD_WGRAD = dict(dy=P, lddy=32, x=3 * P, ldx=64, rows=10, offsets=P, groups=4, n=32, k=64, dw=2 * P, flags=0)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(groups=0), dict(groups=2000), dict(n=9), dict(k=0), dict(lddy=31), dict(ldx=8), dict(dy=0),
    dict(dy=P + 8), dict(x=0), dict(x=P + 1), dict(offsets=0), dict(dw=0), dict(dw=P + 8), dict(dw=P), dict(dw=3 * P),
    dict(flags=0x2),  # accumulate into 16 bits
    dict(flags=0x200), dict(flags=0x40)], ids=str)
def test_grouped_wgrad(L, bad):
    a = dict(GOOD_WGRAD, **bad)
    assert L.moe_grouped_wgrad(a["dy"], a["lddy"], a["x"], a["ldx"], a["rows"], a["offsets"], a["groups"], a["n"], a["k"],
                               a["dw"], a["flags"], None) == 1


GOOD_SWIGLU = dict(gu=P, ldgu=128, dh=P, lddh=64, rows=5, f=64, rw=0, n_rows=0, dgu=P, lddgu=128, h=P, ldh=64, drw=0, flags=0)


@pytest.mark.parametrize("bad", [dict(rows=-3), dict(f=4), dict(f=20), dict(ldgu=120), dict(ldgu=132), dict(ldh=56), dict(gu=0),
                                 dict(gu=P + 4), dict(h=P + 8), dict(flags=1), dict(flags=2), dict(rw=P + 2),
                                 dict(n_rows=P + 1)], ids=str)
def test_swiglu(L, bad):
    a = dict(GOOD_SWIGLU, **bad)
    assert L.moe_swiglu(a["gu"], a["ldgu"], a["rows"], a["f"], a["rw"], a["n_rows"], a["h"], a["ldh"], a["flags"], None) == 1


@pytest.mark.parametrize("bad", [dict(rows=-3), dict(f=12), dict(ldgu=120), dict(lddh=56), dict(lddgu=64), dict(ldh=8),
                                 dict(gu=0), dict(dh=0), dict(dh=P + 2), dict(dgu=0), dict(h=P + 8), dict(flags=1),
                                 dict(drw=P + 2)], ids=str)
def test_swiglu_backward(L, bad):
    a = dict(GOOD_SWIGLU, **bad)
    assert L.moe_swiglu_backward(a["gu"], a["ldgu"], a["dh"], a["lddh"], a["rows"], a["f"], a["rw"], a["n_rows"], a["dgu"],
                                 a["lddgu"], a["h"], a["ldh"], a["drw"], a["flags"], None) == 1


GOOD_ADAPTER = dict(x=P, ldx=64, tokens=10, n=32, k=64, w=P, a=P, b=P, scale=P, ids=P, n_adapters=3, rank=16, y=2 * P, ldy=32,
                    workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=(1 << 27) + 1), dict(n=4), dict(n=33), dict(k=60), dict(ldx=32), dict(ldx=70), dict(ldy=24),
    dict(rank=0), dict(rank=4), dict(rank=20), dict(rank=264), dict(n_adapters=0), dict(x=0), dict(x=P + 2), dict(a=0),
    dict(a=P + 8), dict(b=0), dict(b=P + 8), dict(w=P + 8), dict(y=0), dict(y=2 * P + 8), dict(ids=0), dict(ids=P + 1),
    dict(scale=P + 2), dict(workspace=0), dict(workspace=P + 8), dict(workspace_bytes=100), dict(y=P)], ids=str)
def test_adapter_project(L, bad):
    args = moe.MoeAdapterArgs(**dict(GOOD_ADAPTER, **bad))
    assert L.moe_adapter_project(ctypes.byref(args), 0, None) == 1


def test_adapter_flags_and_null(L):
    args = moe.MoeAdapterArgs(**GOOD_ADAPTER)
    assert L.moe_adapter_project(None, 0, None) == 1
    for flags in (0x4, 0x200, 0x40):
        assert L.moe_adapter_project(ctypes.byref(args), flags, None) == 1


def test_zero_rows_are_valid(L):
    a, s = GOOD_MATMUL, GOOD_SWIGLU
    assert L.moe_grouped_matmul(0, a["ldx"], 0, 0, 0, a["groups"], a["n"], a["k"], 0, a["ldy"], 0, None) == 0
    assert L.moe_grouped_wgrad(0, 32, 0, 64, 0, 0, 4, 32, 64, P, 0x3, None) == 0  # accumulating: nothing to add
    assert L.moe_swiglu(0, s["ldgu"], 0, s["f"], 0, 0, 0, s["ldh"], 0, None) == 0
    args = moe.MoeAdapterArgs(**dict(GOOD_ADAPTER, tokens=0, x=0, y=0, workspace=0))
    assert L.moe_adapter_project(ctypes.byref(args), 0, None) == 0


def test_workspace_size(L):
    assert L.moe_adapter_workspace(0, 16) == 0 and L.moe_adapter_workspace(10, 0) == 0
    assert L.moe_adapter_workspace(10, 264) == 0 and L.moe_adapter_workspace(-1, 16) == 0
    # three 16-bit terms a value and a factor a token; fp32 values of the single-token path fit too
    assert L.moe_adapter_workspace(1000, 64) >= 1000 * 64 * 6 + 1000 * 4
    assert L.moe_adapter_workspace(1 << 27, 256) > 1 << 32


def test_wrappers_refuse_tensors_they_cannot_take():
    import torch
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: moe.grouped_matmul(x, w, off), lambda: moe.grouped_matmul_wgrad(x, x, off), lambda: moe.swiglu(x),
                 lambda: moe.swiglu_backward(x, x[:, :32]),
                 lambda: moe.adapter_project(x, torch.zeros(1, 8, 64, dtype=x.dtype), torch.zeros(1, 32, 8, dtype=x.dtype),
                                             torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):  # CPU tensors: there is no CPU path
            call()
