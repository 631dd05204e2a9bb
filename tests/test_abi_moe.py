"""The second part of the C ABI (include/mxq_moe.h): the library exports every
entry point, and bad arguments are refused on the host before any HIP call (no
GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from nvfp4_quantization_grouped_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x1000000 * (i + 1) for i in range(8)]    # disjoint, aligned, never dereferenced
NULL, SHAPE, DTYPE, FORMAT, ALIGN, ALIAS = -1, -2, -3, -4, -6, -7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmxq.so is not built (python -m nvfp4_quantization_grouped_amd.build)")
    return _lib.moe_lib()


def test_header_declares_the_entry_points(L):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxq_moe.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(_lib.MOE_EXPORTS) == sorted(_lib._MOE_SIGS)
    for n in names:
        assert isinstance(getattr(L, n), ctypes._CFuncPtr)


def caller(f, names, good):
    def call(**kw):
        args = dict(zip(names.split(), good))
        assert set(kw) <= set(args)
        args.update(kw)
        return f(*args.values())
    return call


def test_route(L):
    call = caller(L.moe_route, "logits t tokens experts top_k score bias groups top_groups best renorm scale mask "
                  "weights index stream", (A[0], 0, 16, 64, 8, 1, A[1], 8, 4, 2, 1, 1.0, A[2], A[3], A[4], None))
    for kw in (dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=33), dict(top_k=65),
               dict(experts=8, groups=1, top_groups=1, top_k=9), dict(groups=0), dict(groups=7), dict(groups=65),
               dict(experts=1024, groups=128), dict(top_groups=0), dict(top_groups=9), dict(best=0), dict(best=3),
               dict(tokens=1 << 40)):
        assert call(**kw) == SHAPE, kw
    assert call(t=3) == DTYPE and call(score=2) == FORMAT
    assert call(logits=None) == call(weights=None) == call(index=None) == NULL
    assert call(bias=A[1] + 2) == call(weights=A[3] + 1) == call(index=A[4] + 2) == ALIGN
    assert call(weights=A[0] + 64) == call(index=A[3] + 4) == call(weights=A[1]) == call(index=A[2]) == ALIAS
    assert call(tokens=0) == 0
    b = caller(L.moe_route_bwd, "logits t tokens experts top_k score renorm scale index gw grad stream",
               (A[0], 1, 16, 64, 8, 0, 1, 1.0, A[1], A[2], A[3], None))
    assert b(experts=2000) == b(top_k=40) == SHAPE and b(t=7) == DTYPE and b(score=-1) == FORMAT
    assert b(gw=None) == b(index=None) == b(grad=None) == NULL
    assert b(index=A[1] + 1) == ALIGN and b(grad=A[0]) == b(grad=A[2]) == ALIAS
    assert b(tokens=0) == 0


def test_plan(L):
    W = L.moe_plan_workspace
    assert W(-1, 8, 32) == W(4, 0, 32) == W(4, 8, 0) == W(4, 8, 1025) == W(1 << 31, 1, 8) == W(1 << 60, 1 << 60, 8) == SHAPE
    assert W(0, 8, 32) == 0 and W(4, 8, 32) == 0
    need = W(65536, 8, 256)
    assert need > 0 and need % 4 == 0
    call = caller(L.moe_plan, "index tokens top_k first local offs rows slots work bytes stream",
                  (A[0], 16, 8, 0, 32, A[1], A[2], A[3], None, 0, None))
    assert call(tokens=-1) == call(top_k=0) == call(local=0) == call(first=-1) == call(first=(1 << 31) - 32) == SHAPE
    assert call(tokens=65536, bytes=0, work=A[4]) == SHAPE          # too small a workspace
    assert call(tokens=65536, bytes=1 << 20, work=None) == NULL
    assert call(tokens=65536, bytes=1 << 20, work=A[4] + 2) == ALIGN
    assert call(index=None) == call(offs=None) == call(rows=None) == call(slots=None) == NULL
    assert call(tokens=0, offs=None) == NULL
    assert call(rows=A[2] + 2) == ALIGN
    assert call(rows=A[0]) == call(slots=A[2] + 4) == call(offs=A[0] + 8) == ALIAS


def test_row_streams(L):
    names, good = "x t tokens hidden top_k rows out stream", (A[0], 1, 16, 64, 8, A[1], A[2], None)
    for f in (L.moe_dispatch, L.moe_dispatch_bwd):
        call = caller(f, names, good)
        assert call(tokens=-1) == call(hidden=-1) == call(hidden=(1 << 20) + 1) == call(top_k=0) == SHAPE
        assert call(tokens=1 << 31, top_k=1) == SHAPE
        assert call(t=4) == DTYPE
        assert call(x=None) == call(rows=None) == call(out=None) == NULL
        assert call(rows=A[1] + 1) == ALIGN
        assert call(out=A[0] + 64) == call(out=A[1]) == ALIAS
        assert call(tokens=0) == call(hidden=0) == 0
    call = caller(L.moe_combine, "y t tokens hidden top_k rows weights out stream",
                  (A[0], 1, 16, 64, 8, A[1], A[2], A[3], None))
    assert call(weights=None) == NULL and call(out=A[2]) == ALIAS and call(weights=A[2] + 2) == ALIGN
    assert call(top_k=0) == SHAPE and call(tokens=0) == 0
    call = caller(L.moe_dispatch_quantized, "x t tokens hidden top_k rows fmt codes scales stream",
                  (A[0], 1, 16, 64, 8, A[1], 0, A[2], A[3], None))
    assert call(hidden=48) == SHAPE and call(fmt=2) == FORMAT and call(t=9) == DTYPE
    assert call(codes=None) == call(scales=None) == NULL
    assert call(codes=A[0]) == call(scales=A[2] + 8) == ALIAS
    call = caller(L.moe_combine_bwd, "go y t tokens hidden top_k rows weights gy gw stream",
                  (A[0], A[1], 1, 16, 64, 8, A[2], A[3], A[4], A[5], None))
    assert call(y=None) == call(weights=None) == call(go=None) == call(rows=None) == NULL
    assert call(gy=A[1]) == call(gw=A[4] + 4) == call(gy=A[0]) == ALIAS
    assert call(gw=A[5] + 2) == ALIGN and call(hidden=-2) == SHAPE
    assert call(gy=None, gw=None) == call(tokens=0) == 0


def test_swiglu(L):
    call = caller(L.swiglu_fwd, "x t rows inter offs experts h codes scales stream",
                  (A[0], 1, 16, 64, A[1], 8, A[2], A[3], A[4], None))
    assert call(rows=-1) == call(inter=40) == call(inter=-32) == call(experts=0) == call(inter=1 << 21) == SHAPE
    assert call(rows=1 << 40) == SHAPE and call(t=5) == DTYPE
    assert call(x=None) == call(h=None) == call(codes=None) == call(scales=None) == NULL
    assert call(offs=A[1] + 2) == ALIGN
    assert call(h=A[0] + 32) == call(codes=A[2]) == call(scales=A[3]) == ALIAS
    assert call(rows=0) == call(inter=0) == 0
    call = caller(L.swiglu_bwd, "gh x codes scales t rows inter offs experts grad stream",
                  (A[0], None, A[1], A[2], 1, 16, 64, A[3], 8, A[4], None))
    assert call(gh=None) == call(grad=None) == call(codes=None) == call(x=A[5]) == NULL
    assert call(codes=None, scales=None) == NULL                      # neither the input nor what was kept of it
    assert call(grad=A[1]) == call(grad=A[0]) == ALIAS and call(inter=33) == SHAPE
    assert call(rows=0) == 0


def test_swiglu_quantized(L):
    call = caller(L.swiglu_quantized, "x t rows inter offs experts fmt codes scales stream",
                  (A[0], 1, 16, 64, A[1], 8, 1, A[2], A[3], None))
    assert call(rows=-1) == call(inter=40) == call(experts=0) == SHAPE and call(t=5) == DTYPE
    assert call(fmt=2) == call(fmt=-1) == FORMAT
    assert call(x=None) == call(codes=None) == call(scales=None) == NULL and call(offs=A[1] + 1) == ALIGN
    assert call(codes=A[0] + 32) == call(scales=A[2] + 8) == call(codes=A[1]) == ALIAS
    assert call(rows=0) == call(inter=0) == 0


def test_operators_refuse_cpu_tensors():
    x, e = torch.zeros(2, 64), torch.zeros(2, 1, dtype=torch.int32)
    plan = mxq.MoEPlan(torch.zeros(1, dtype=torch.int32), e, torch.zeros(2, dtype=torch.int32))
    for call in (lambda: mxq.moe_route(x, 1), lambda: mxq.moe_plan(e, 1), lambda: mxq.moe_dispatch(x, plan),
                 lambda: mxq.moe_dispatch_quantized(x, plan, "fp8"), lambda: mxq.moe_combine(x, x, plan),
                 lambda: mxq.swiglu(x), lambda: mxq.swiglu_quantized(x, "fp8")):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    with pytest.raises(ValueError):
        mxq.moe_route(x, 1, score="tanh")
    with pytest.raises(ValueError):
        mxq.mxfp4_moe(x, x, e, x, x, x, x, activations="int8")
    with pytest.raises(TypeError):
        mxq.mxfp4_moe(x, x, e, x, x, x, x)
