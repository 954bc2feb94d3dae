"""Host-side checks of moe_linear, moe_route and moe_rmsnorm_quantize: refused
arguments come back with the documented status before anything is launched, and
calls on no rows succeed without a device.

Fake device addresses as in test_capi_host: only where no GPU is present."""
import ctypes

import pytest
import torch

from routed_shared_experts_b200 import build, capi

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: CPU-only check")
P = 0x10000  # 16-byte aligned fake address, never dereferenced on the host
ARG, DTYPE, ALIGN, SHAPE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def _linear(lib, **kw):
    a = dict(dt=capi.MOE_DT_BF16, x=P, ldx=64, xs=None, w=P, ldw=64, ws=None, wsr=1, b=None, bdt=capi.MOE_DT_F32,
             act=0, r=None, ldr=0, o=P, odt=capi.MOE_DT_BF16, ldo=32, T=4, N=32, K=64)
    a.update(kw)
    return lib.moe_linear(a["dt"], a["x"], a["ldx"], a["xs"], a["w"], a["ldw"], a["ws"], a["wsr"], a["b"], a["bdt"],
                          a["act"], a["r"], a["ldr"], a["o"], a["odt"], a["ldo"], a["T"], a["N"], a["K"], None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dt=capi.MOE_DT_F32), DTYPE), (dict(dt=capi.MOE_DT_MXFP8_E4M3), DTYPE),
    (dict(odt=capi.MOE_DT_FP8_E4M3), DTYPE), (dict(b=P, bdt=capi.MOE_DT_FP8_E4M3), DTYPE),
    (dict(T=-1), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(act=6), ARG), (dict(act=-1), ARG),
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(o=None), ARG),
    (dict(xs=P), ARG), (dict(ws=P), ARG),                                  # scales with 16-bit operands
    (dict(dt=capi.MOE_DT_FP8_E4M3), ARG), (dict(dt=capi.MOE_DT_FP8_E4M3, xs=P, ws=P, wsr=2), ARG),
    (dict(ldx=56), ARG), (dict(ldw=56), ARG), (dict(ldo=31), ARG), (dict(r=P, ldr=31), ARG),
    (dict(x=P + 8), ALIGN), (dict(w=P + 2), ALIGN), (dict(ldx=68), ALIGN), (dict(ldw=65), ALIGN),
    (dict(dt=capi.MOE_DT_FP8_E4M3, xs=P, ws=P, ldx=72), ALIGN), (dict(o=P + 1), ALIGN), (dict(r=P + 1, ldr=32), ALIGN),
    (dict(odt=capi.MOE_DT_F32, o=P + 2), ALIGN), (dict(b=P + 2), ALIGN),
    (dict(dt=capi.MOE_DT_FP8_E4M3, xs=P + 1, ws=P), ALIGN), (dict(dt=capi.MOE_DT_FP8_E4M3, xs=P, ws=P + 2), ALIGN),
    (dict(T=(1 << 30) + 1), SHAPE), (dict(N=(1 << 30) + 1, ldo=1 << 31), SHAPE),
    (dict(K=(1 << 30) + 8, ldx=1 << 31, ldw=1 << 31), SHAPE), (dict(ldx=1 << 37), SHAPE), (dict(ldo=(1 << 36) + 1), SHAPE), (dict(r=P, ldr=1 << 40), SHAPE),
    (dict(T=0), 0), (dict(T=0, x=None, o=None), 0),
])
def test_linear_refusals(lib, kw, want):
    assert _linear(lib, **kw) == want


def _route(lib, **kw):
    a = dict(l=P, dt=capi.MOE_DT_F32, ld=8, b=None, m=None, nv=None, T=4, E=8, k=2, score=0, ng=1, tg=1, gs=0, ids=P,
             w=P)
    a.update(kw)
    return lib.moe_route(a["l"], a["dt"], a["ld"], a["b"], a["m"], a["nv"], a["T"], a["E"], a["k"], a["score"],
                         a["ng"], a["tg"], a["gs"], 1, 1.0, a["ids"], a["w"], None)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dt=capi.MOE_DT_FP8_E4M3), DTYPE), (dict(T=-1), ARG), (dict(E=0), ARG), (dict(E=513, ld=513), ARG),
    (dict(k=0), ARG), (dict(k=9), ARG), (dict(E=64, ld=64, k=33), ARG), (dict(score=2), ARG), (dict(gs=2), ARG),
    (dict(ng=3), ARG), (dict(ng=0), ARG), (dict(E=64, ld=64, ng=64), ARG), (dict(ng=4, tg=5), ARG),
    (dict(ng=4, tg=0), ARG), (dict(ng=4, tg=1, k=3), ARG), (dict(l=None), ARG), (dict(ids=None), ARG),
    (dict(w=None), ARG), (dict(ld=7), ARG), (dict(l=P + 2), ALIGN), (dict(dt=capi.MOE_DT_BF16, l=P + 1), ALIGN),
    (dict(b=P + 1), ALIGN), (dict(nv=P + 2), ALIGN), (dict(ids=P + 1), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(T=0), 0), (dict(T=0, l=None), 0),
])
def test_route_refusals(lib, kw, want):
    assert _route(lib, **kw) == want


def _norm(lib, **kw):
    a = dict(dt=capi.MOE_DT_BF16, q=capi.MOE_DT_NONE, x=P, r=None, g=P, gdt=capi.MOE_DT_BF16, eps=1e-6, T=4, H=64,
             ro=None, y=P, c=None, s=None)
    a.update(kw)
    return lib.moe_rmsnorm_quantize(a["dt"], a["q"], a["x"], a["r"], a["g"], a["gdt"], ctypes.c_float(a["eps"]), a["T"],
                                    a["H"], a["ro"], a["y"], a["c"], a["s"], None)


FP8, MX8 = capi.MOE_DT_FP8_E4M3, capi.MOE_DT_MXFP8_E4M3


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dt=capi.MOE_DT_F32), DTYPE), (dict(gdt=capi.MOE_DT_FP16), DTYPE), (dict(q=capi.MOE_DT_MXFP4_E2M1), DTYPE),
    (dict(q=capi.MOE_DT_BF16), DTYPE), (dict(T=-1), ARG), (dict(H=0), ARG), (dict(eps=0.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(H=60), SHAPE), (dict(q=MX8, c=P, s=P, H=48), SHAPE), (dict(H=16392), SHAPE),
    (dict(x=None), ARG), (dict(g=None), ARG), (dict(y=None), ARG), (dict(c=P), ARG), (dict(s=P), ARG),
    (dict(q=FP8), ARG), (dict(q=FP8, c=P), ARG), (dict(q=MX8, s=P), ARG),
    (dict(x=P + 8), ALIGN), (dict(r=P + 8), ALIGN), (dict(g=P + 8), ALIGN), (dict(ro=P + 8), ALIGN),
    (dict(y=P + 2), ALIGN), (dict(q=FP8, c=P + 4, s=P), ALIGN), (dict(q=FP8, c=P, s=P + 2), ALIGN),
    (dict(T=0), 0), (dict(T=0, x=None), 0),
])
def test_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def test_wrapper_refuses_cpu_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        capi.moe_linear(capi.MOE_DT_BF16, x, None, x, None, None, 0, None, torch.zeros((4, 4), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        capi.moe_route(x, None, None, None, 2, 0, 1, 1, 0, True, 1.0, torch.zeros((4, 2), dtype=torch.int32),
                       torch.zeros((4, 2)))


def test_constants_match_the_header():
    import re
    import os
    src = open(os.path.join(os.path.dirname(__file__), "..", "include", "moe_b200.h")).read()
    val = {m.group(1): m.group(2) for m in re.finditer(r"#define (MOE_[A-Z0-9_]+) (\S+)", src)}
    assert val["MOE_NO_EXPERT"] == "INT32_MIN" and capi.MOE_NO_EXPERT == -(2 ** 31)
    assert val["MOE_DT_NONE"] == "(-1)" and capi.MOE_DT_NONE == -1
    for name, v in capi.ACTS.items():
        assert int(val["MOE_ACT_" + name.upper()]) == v
    for name in ("MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_GROUP_TOP2", "MOE_GROUP_MAX"):
        assert int(val[name]) == getattr(capi, name)


def test_binding_leaves_malformed_calls_alone(lib):
    """The binding answers None, without an exception and without keeping a
    reference, to whatever is not a well-formed call."""
    import sys
    b = capi._binding()
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    objs = [x, None, 3, "text", object(), (1, 2)]
    counts = [sys.getrefcount(v) for v in objs]
    for _ in range(50):
        for o in objs:
            assert b.linear(0, o, None, x, None, None, 0, None, o, None) is None
            assert b.route(o, None, None, None, 2, 0, 1, 1, 0, True, 1.0, o, o, None) is None
            assert b.rmsnorm_quantize(-1, o, None, x, 1e-6, None, o, None, None, None) is None
        assert b.linear() is None and b.route(1) is None and b.rmsnorm_quantize(*range(10)) is None
        assert b.linear("bf16", x, None, x, None, None, "relu", None, x, None) is None
    del o  # the loop's own reference to the last one
    assert [sys.getrefcount(v) for v in objs] == counts


def test_kernels_that_start_early_use_no_read_only_loads():
    """A kernel launched while its predecessor drains (launch_early) may read what
    that one still writes: loads through the read-only path, which is defined for
    data that stays as it is for the kernel's whole life, have no place in it."""
    import os
    import re
    for name in ("linear.cuh", "route.cuh", "norm.cuh"):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        assert "grid_dependency_wait()" in src
        for word in ("__ldg", ".nc.", "__restrict__"):
            assert word not in src, (name, word)


def test_remote_shared_memory_is_read_under_a_predicate():
    """A read of a peer CTA's shared memory whose value nothing uses is not waited
    for by the relaxed cluster barrier that ends moe_linear's kernels: each takes a
    predicate, and the calls give the condition under which the value is used."""
    import os
    import re
    src = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, "linear.cuh")).read())
    loads = re.findall(r'"([^"]*)ld\.shared::cluster', src)
    assert loads and all(head.startswith("@p ") for head in loads), loads
    calls = re.findall(r"ld_shared_cluster_f32(?:x4)?_if\(\s*(peer[^;]*);", src)
    assert len(calls) == 2 and "in && c0 + i < c_hi" in calls[0] and "t0 + r0 + j < g.T" in calls[1], calls
