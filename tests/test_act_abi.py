"""Refusals of the layer with its epilogue, the routing plan, the experts' layers and the combination: every check of
the C ABI runs before any HIP call, so these need no GPU.  The pointers are never read."""

from __future__ import annotations

import ctypes
import os

import pytest

from rank_augmented_quantized_amd import tq as tqb

NULL, SHAPE, DTYPE, BITS, ALIGN, WS, ACT = -1, -2, -3, -4, -5, -6, -8
PTR = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tqb.LIB):
        pytest.skip("libtq.so not built (run __graft_entry__.build())")
    return tqb.load()


def _act(lib, **kw):
    a = dict(X=PTR, x_dt=1, n=4, d=64, m=32, r=8, wc=PTR, sw=PTR, lr=PTR, bias=None, act=0, gated=0, res=None, res_dt=1, Y=PTR,
             y_dt=1, ws=PTR, wb=0, stream=None)
    a.update(kw)
    return lib.tq_linear_act(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), ACT), (dict(act=-1), ACT), (dict(x_dt=2), DTYPE), (dict(y_dt=7), DTYPE), (dict(res=PTR, res_dt=9), DTYPE),
    (dict(gated=1, m=31), SHAPE), (dict(d=48), SHAPE), (dict(d=0), SHAPE), (dict(d=65568), SHAPE), (dict(m=0), SHAPE),
    (dict(n=-1), SHAPE), (dict(r=257), SHAPE), (dict(X=None), NULL), (dict(wc=None), NULL), (dict(sw=None), NULL),
    (dict(lr=None), NULL), (dict(Y=None), NULL), (dict(ws=None), NULL), (dict(X=ODD), ALIGN), (dict(bias=ODD), ALIGN),
    (dict(res=ODD), ALIGN), (dict(Y=ODD), ALIGN), (dict(lr=ODD), ALIGN), (dict(wb=0), WS), (dict(n=0), 0),
])
def test_linear_act_refusals(lib, kw, status):
    assert _act(lib, **kw) == status


def _plan(lib, **kw):
    a = dict(ids=PTR, bits=32, n=4, k=2, E=8, off=PTR, order=PTR, pos=PTR, ws=None, wb=0, stream=None)
    a.update(kw)
    return lib.tq_expert_plan(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(bits=16), BITS), (dict(n=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(n=1 << 24), SHAPE), (dict(off=None), NULL), (dict(ids=None), NULL), (dict(order=None), NULL),
    (dict(pos=None), NULL), (dict(ids=ODD), ALIGN), (dict(off=ODD), ALIGN), (dict(order=ODD), ALIGN), (dict(pos=ODD), ALIGN),
    (dict(n=100000, ws=None), NULL), (dict(n=100000, ws=PTR, wb=15), WS),
])
def test_expert_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status


def _experts(lib, **kw):
    a = dict(X=PTR, x_dt=1, n=4, k=2, d=64, m=32, r=8, E=4, off=PTR, order=PTR, wc=PTR, sw=PTR, lr=PTR, bias=None, act=0, gated=0,
             Y=PTR, y_dt=1, ws=PTR, wb=0, stream=None)
    a.update(kw)
    return lib.tq_linear_experts(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(act=9), ACT), (dict(gated=1, m=33), SHAPE), (dict(order=None), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(n=(1 << 23) + 1), SHAPE), (dict(n=1 << 20, k=2, d=2048), SHAPE),
    (dict(d=40), SHAPE), (dict(r=300), SHAPE), (dict(off=None), NULL), (dict(lr=None), NULL), (dict(wc=None), NULL),
    (dict(off=ODD), ALIGN), (dict(order=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(wb=0), WS), (dict(x_dt=3), DTYPE),
    (dict(n=0), 0), (dict(E=1024, m=1 << 21), SHAPE),
])
def test_linear_experts_refusals(lib, kw, status):
    assert _experts(lib, **kw) == status


def _combine(lib, **kw):
    a = dict(Z=PTR, z_dt=1, rows=8, n=4, k=2, m=64, pos=PTR, w=PTR, w_dt=0, res=None, res_dt=1, Y=PTR, y_dt=1, stream=None)
    a.update(kw)
    return lib.tq_expert_combine(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(z_dt=2), DTYPE), (dict(w_dt=2), DTYPE), (dict(y_dt=2), DTYPE), (dict(res=PTR, res_dt=2), DTYPE), (dict(rows=-1), SHAPE),
    (dict(rows=(1 << 24) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE),
    (dict(n=-1), SHAPE), (dict(Z=None), NULL), (dict(pos=None), NULL), (dict(w=None), NULL), (dict(Y=None), NULL),
    (dict(Z=ODD), ALIGN), (dict(pos=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(res=ODD), ALIGN), (dict(Y=ODD), ALIGN),
    (dict(n=0), 0),
])
def test_expert_combine_refusals(lib, kw, status):
    assert _combine(lib, **kw) == status


def test_size_queries(lib):
    assert lib.tq_linear_act_workspace_bytes(4, 48, 32, 8) == 0
    assert lib.tq_linear_act_workspace_bytes(4, 64, 32, 257) == 0
    # the counter region, then scales, codes and the low-rank stage: grows with n, with r, never with m
    base = lib.tq_linear_act_workspace_bytes(0, 64, 32, 8)
    assert base >= 8192
    assert lib.tq_linear_act_workspace_bytes(100, 64, 32, 8) > lib.tq_linear_act_workspace_bytes(100, 64, 32, 0) > base
    assert lib.tq_linear_act_workspace_bytes(100, 64, 32, 8) == lib.tq_linear_act_workspace_bytes(100, 64, 4096, 8)
    assert lib.tq_linear_experts_workspace_bytes(4, 2, 64, 32, 8, 0) == 0
    assert lib.tq_linear_experts_workspace_bytes(4, 65, 64, 32, 8, 4) == 0
    assert lib.tq_linear_experts_workspace_bytes(100, 2, 64, 32, 8, 4) > 8192
    assert lib.tq_expert_plan_workspace_bytes(4, 2, 8) == 0
    assert lib.tq_expert_plan_workspace_bytes(1 << 20, 2, 8) > 0
    assert lib.tq_expert_plan_workspace_bytes(4, 2, 1025) == 0
    sizes = [lib.tq_expert_plan_workspace_bytes(1 << b, 1, 64) for b in range(25)]  # for the most tokens: enough for fewer
    assert sizes == sorted(sizes) and lib.tq_expert_plan_workspace_bytes((1 << 19) + 1, 1, 64) >= sizes[19]
    assert lib.tq_expert_plan_workspace_bytes((1 << 20) + 1, 1, 64) >= sizes[20]
    assert lib.tq_status_string(-8).startswith(b"TQ_ERR_ACT")
