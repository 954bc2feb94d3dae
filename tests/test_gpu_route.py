"""moe_route against a per-token statement of the definition in 64 bits: ids
equal, weights within the one rounding to fp32 (2^-24 relative, doubled for the
double arithmetic's own noise)."""
import math

import numpy as np
import pytest
import torch

from routed_shared_experts_b200 import capi

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _oracle(logits, bias, mask, k, score, G, tg, gscore, renorm, rsf):
    T, E = logits.shape
    ids, wts = np.zeros((T, k), np.int32), np.zeros((T, k), np.float64)
    size = E // G
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = ~np.isnan(l) & (l != -np.inf)
        if mask is not None:
            live &= mask != 0
        s = np.zeros(E)
        if score == "softmax":
            if live.any():
                mx = l[live].max()
                with np.errstate(invalid="ignore"):
                    e = np.where(l == mx, 1.0, np.exp(l - mx))
                e = np.where(live, e, 0.0)
                s = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s = np.where(live, 1 / (1 + np.exp(-l)), 0.0)
        c = s.astype(np.float32)
        if bias is not None:
            c = (c + bias).astype(np.float32)
        live &= ~np.isnan(c) & (c != -np.inf)
        gs = []
        for g in range(G):
            v = sorted((float(x) for x, ok in zip(c[g * size:(g + 1) * size], live[g * size:(g + 1) * size]) if ok),
                       reverse=True)
            gs.append(-math.inf if not v else v[0] if gscore == "max" or len(v) == 1 else
                      float(np.float32(v[0]) + np.float32(v[1])))
        kept = sorted(range(G), key=lambda g: (-gs[g], g))[:tg]
        cand = [e for e in range(E) if e // size in kept]
        pick = sorted(cand, key=lambda e: (not live[e], -float(c[e]) if live[e] else 0.0, e))[:k]
        w = np.array([s[e] if live[e] else 0.0 for e in pick])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        ids[t], wts[t] = pick, w * np.float64(np.float32(rsf))
    return ids, wts


def _check(logits, bias, mask, k, score, G=1, tg=1, gscore="top2", renorm=True, rsf=1.0, valid=None):
    """logits: a CPU tensor, possibly strided."""
    T, E = logits.shape
    dev = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device="cuda")
    dev.copy_(logits)
    ids = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    wts = torch.full((T, k), 9.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    m = None if mask is None else torch.from_numpy(mask).cuda()
    nv = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    capi.moe_route(dev, b, m, nv, k, capi.SCORES[score], G, tg, capi.GROUP_SCORES[gscore], renorm, rsf, ids, wts)
    torch.cuda.synchronize()
    n = T if valid is None else max(0, min(T, valid))
    rid, rw = _oracle(logits[:n].float().numpy(), bias, mask, k, score, G, tg, gscore, renorm, rsf)
    got_i, got_w = ids.cpu().numpy(), wts.cpu().numpy()
    assert np.array_equal(got_i[:n], rid)
    assert np.all(np.abs(got_w[:n].astype(np.float64) - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149)
    assert np.all(got_i[n:] == capi.MOE_NO_EXPERT) and np.all(got_w[n:] == 0)
    return got_i, got_w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm,rsf", [(True, 1.0), (False, 2.5)])
@pytest.mark.parametrize("T,E,k,G,tg,gscore,dt,use_bias,use_mask", [
    (1, 1, 1, 1, 1, "top2", "f32", True, False), (1, 2, 2, 2, 2, "top2", "f32", True, False),
    (5, 31, 4, 1, 1, "top2", "bf16", False, False), (33, 33, 6, 3, 2, "max", "fp16", True, True),
    (64, 64, 6, 8, 4, "top2", "f32", False, True), (32, 128, 8, 1, 1, "top2", "f32", True, False),
    (130, 160, 6, 8, 3, "max", "bf16", False, False), (300, 256, 8, 8, 4, "top2", "f32", True, False),
    (40, 257, 10, 1, 1, "top2", "f32", True, True), (9, 512, 32, 32, 7, "top2", "bf16", True, True),
    (7, 480, 16, 5, 1, "max", "f32", True, True), (3, 62, 9, 31, 30, "top2", "f32", True, True),
    (4, 32, 32, 1, 1, "top2", "f32", False, True)])
def test_route_matches_definition(cuda_lib, score, renorm, rsf, T, E, k, G, tg, gscore, dt, use_bias, use_mask):
    rng = np.random.default_rng(T * 1000 + E + k)
    logits = torch.from_numpy(rng.normal(0, 2, (T, E)).astype(np.float32)).to(DT[dt])
    bias = rng.normal(0, 0.2, E).astype(np.float32) if use_bias else None
    mask = (rng.random(E) > 0.3).astype(np.uint8) if use_mask else None
    _check(logits, bias, mask, k, score, G, tg, gscore, renorm, rsf)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_take_the_lower_index(cuda_lib, score):
    """16-bit logits on a coarse grid: most rows hold many equal values."""
    rng = np.random.default_rng(4)
    logits = torch.from_numpy(rng.integers(-2, 3, (200, 96)).astype(np.float32)).to(torch.bfloat16)
    for G, tg, gs in ((1, 1, "max"), (8, 3, "top2"), (12, 5, "max")):
        _check(logits, None, None, 12, score, G, tg, gs)
        _check(logits, np.zeros(96, np.float32), None, 12, score, G, tg, gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,gscore", [(1, 1, "top2"), (4, 2, "top2"), (4, 3, "max")])
def test_route_dead_experts(cuda_lib, score, G, tg, gscore):
    """Masks that leave a row fewer experts than k or none; the type's lowest
    value, infinities and NaN among the logits; infinite and NaN biases."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    E, k = 32, 6
    rng = np.random.default_rng(6)
    l = rng.normal(0, 1, (12, E)).astype(np.float32)
    l[0] = -inf                       # nothing lives
    l[1] = nan
    l[2, :] = -inf
    l[2, 9] = 0.5                     # one lives
    l[3, ::2] = -inf
    l[4, 3], l[4, 20] = inf, inf      # share the softmax
    l[5] = low                        # masked by value: alive, all equal
    l[6, 1:] = low
    l[7, 5] = nan
    l[8] = inf
    l[9, :16] = -inf
    l[10, 4], l[10, 5] = -200.0, 200.0
    l[11, 8:] = nan
    lt = torch.from_numpy(l)
    _check(lt, None, None, k, score, G, tg, gscore)
    _check(lt, None, None, k, score, G, tg, gscore, renorm=False, rsf=0.5)
    bias = rng.normal(0, 0.3, E).astype(np.float32)
    bias[3], bias[4], bias[5] = -inf, nan, inf
    _check(lt, bias, None, k, score, G, tg, gscore)
    _check(lt, bias, np.zeros(E, np.uint8), k, score, G, tg, gscore)
    one = np.zeros(E, np.uint8)
    one[30] = 200                     # any non-zero byte is on
    ids, w = _check(lt, None, one, k, score, G, tg, gscore)
    assert ids[9, 0] == 30


@pytest.mark.parametrize("valid", [0, 1, 37, 64, 100, -3])
def test_route_padding_rows(cuda_lib, valid):
    rng = np.random.default_rng(8)
    _check(torch.from_numpy(rng.normal(0, 1, (64, 40)).astype(np.float32)), None, None, 5, "sigmoid", valid=valid)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_strided_logits(cuda_lib, dt):
    rng = np.random.default_rng(9)
    wide = torch.from_numpy(rng.normal(0, 1, (50, 77)).astype(np.float32)).to(DT[dt])
    _check(wide[:, 5:5 + 48], None, None, 4, "softmax")
    _check(wide[::2, 1:65], None, None, 4, "sigmoid")


def test_route_offsets_past_32_bits(cuda_lib):
    """Logit rows far apart, the last one past 2^32 elements."""
    T, E, gap = 3000, 40, 1_600_000
    big = torch.empty((T - 1) * gap + E, dtype=torch.bfloat16, device="cuda")
    logits = torch.as_strided(big, (T, E), (gap, 1))
    logits.copy_(torch.randn((T, E), generator=torch.Generator().manual_seed(3)).bfloat16())
    out = []
    for l in (logits, logits.contiguous()):
        ids = torch.empty((T, 4), dtype=torch.int32, device="cuda")
        w = torch.empty((T, 4), device="cuda")
        capi.moe_route(l, None, None, None, 4, capi.MOE_SCORE_SIGMOID, 4, 2, capi.MOE_GROUP_TOP2, True, 1.0, ids, w)
        out.append((ids, w))
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_route_softmax_agrees_with_the_plain_top_k(cuda_lib):
    """No bias, no groups: the same experts and weights as moe_router_topk."""
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((500, 128), generator=g).cuda()
    out = []
    for route in (0, 1):
        ids = torch.empty((500, 8), dtype=torch.int32, device="cuda")
        w = torch.empty((500, 8), device="cuda")
        if route:
            capi.moe_route(logits, None, None, None, 8, capi.MOE_SCORE_SOFTMAX, 1, 1, 0, True, 2.5, ids, w)
        else:
            capi.moe_router_topk(logits, None, 8, capi.MOE_ROUTE_SOFTMAX, 1, 1, True, 2.5, ids, w)
        out.append((ids.cpu(), w.cpu()))
    assert torch.equal(out[0][0], out[1][0])
    assert torch.allclose(out[0][1], out[1][1], rtol=2.0 ** -22, atol=0)


def test_route_no_rows_and_graph(cuda_lib):
    e = torch.empty((0, 16), device="cuda")
    capi.moe_route(e, None, None, None, 2, 0, 1, 1, 0, True, 1.0, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                   torch.empty((0, 2), device="cuda"))
    # a captured call follows num_valid and the logits of the replay
    logits = torch.zeros((8, 16), device="cuda")
    nv = torch.tensor([8], dtype=torch.int32, device="cuda")
    ids = torch.empty((8, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((8, 2), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.moe_route(logits, None, None, nv, 2, 0, 1, 1, 0, True, 1.0, ids, w)
    rng = np.random.default_rng(1)
    for n in (3, 8, 0):
        new = rng.normal(0, 1, (8, 16)).astype(np.float32)
        logits.copy_(torch.from_numpy(new))
        nv.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        rid, _ = _oracle(new[:n], None, None, 2, "softmax", 1, 1, "top2", True, 1.0)
        assert np.array_equal(ids.cpu().numpy()[:n], rid)
        assert np.all(ids.cpu().numpy()[n:] == capi.MOE_NO_EXPERT)


def test_route_wrapper_refusals(cuda_lib):
    l = torch.zeros((4, 16), device="cuda")
    i, w = torch.empty((4, 2), dtype=torch.int32, device="cuda"), torch.empty((4, 2), device="cuda")
    with pytest.raises(TypeError):
        capi.moe_route(l.double(), None, None, None, 2, 0, 1, 1, 0, True, 1.0, i, w)
    with pytest.raises(ValueError):
        capi.moe_route(l, torch.zeros(15, device="cuda"), None, None, 2, 0, 1, 1, 0, True, 1.0, i, w)
    with pytest.raises(ValueError):
        capi.moe_route(l, None, None, None, 3, 0, 1, 1, 0, True, 1.0, i, w)
    with pytest.raises(TypeError):
        capi.moe_route(l, None, None, None, 2, 0, 1, 1, 0, True, 1.0, i.long(), w)
    with pytest.raises(capi.MoEError):
        capi.moe_route(l, None, None, None, 2, 0, 3, 1, 0, True, 1.0, i, w)


@pytest.mark.parametrize("cluster", [False, True])
def test_padding_rows_pass_the_sort(cuda_lib, cluster):
    """MOE_NO_EXPERT slots are dropped without a device error, by both sorts."""
    T, k, E, bm = (1024, 8, 16, 32) if cluster else (40, 3, 8, 16)
    rng = np.random.default_rng(3)
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    ids[T - T // 4:] = capi.MOE_NO_EXPERT
    cap = capi.sorted_capacity(T, k, E, bm)
    i32 = dict(dtype=torch.int32, device="cuda")
    s, be = torch.full((cap,), -7, **i32), torch.empty(cap // bm, **i32)
    c, o, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32)
    capi.device_error()
    capi.moe_align_sort(torch.from_numpy(ids).cuda(), E, bm, s, be, c, o, n)
    torch.cuda.synchronize()
    assert capi.device_error() == 0
    flat = ids.reshape(-1)
    s, c, o = s.cpu().numpy(), c.cpu().numpy(), o.cpu().numpy()
    for e in range(E):
        want = np.nonzero(flat == e)[0]
        assert c[e] == len(want) and np.array_equal(s[o[e]:o[e] + c[e]], want)
        assert np.all(s[o[e] + c[e]:o[e + 1]] == T * k)


def test_padding_rows_take_no_shared_slots(cuda_lib):
    T, k, E, m = 6, 2, 8, 3
    ids = torch.tensor([[1, 2]] * 4 + [[capi.MOE_NO_EXPERT] * 2] * 2, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    gate = torch.full((T,), 0.25, dtype=torch.bfloat16, device="cuda")
    oi, ow = torch.empty((T, k + m), dtype=torch.int32, device="cuda"), torch.empty((T, k + m), device="cuda")
    capi.moe_append_shared_slots(ids, w, E, m, gate, oi, ow)
    torch.cuda.synchronize()
    assert oi[:4, k:].cpu().tolist() == [[8, 9, 10]] * 4 and torch.all(ow[:4, k:] == 0.25)
    assert torch.all(oi[4:] == capi.MOE_NO_EXPERT) and torch.all(ow[4:, k:] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_live_group_below_the_fp32_range(cuda_lib, score):
    """A bias of the type's lowest value masks experts without switching them
    off. Two of them add up below the fp32 range: their group still counts more
    than one in which nothing lives, whatever the order of the groups."""
    low = torch.finfo(torch.float32).min
    E, G = 32, 4
    logits = torch.from_numpy(np.random.default_rng(8).normal(0, 1, (5, E)).astype(np.float32))
    for dead, alive in ((0, 2), (3, 1)):
        bias = np.full(E, low, np.float32)
        mask = np.ones(E, np.uint8)
        mask[dead * 8:dead * 8 + 8] = 0
        others = [g for g in range(G) if g not in (dead, alive)]
        for g in others:
            bias[g * 8:g * 8 + 8] = 0.0
        dev = logits.cuda()
        ids = torch.empty((5, 20), dtype=torch.int32, device="cuda")
        w = torch.empty((5, 20), device="cuda")
        capi.moe_route(dev, torch.from_numpy(bias).cuda(), torch.from_numpy(mask).cuda(), None, 20, capi.SCORES[score],
                       G, 3, capi.MOE_GROUP_TOP2, False, 1.0, ids, w)
        got = ids.cpu() // 8
        assert set(got.unique().tolist()) == set(others + [alive])
        assert torch.all(w > 0)  # all twenty picks live


def test_route_most_rows_there_are(cuda_lib):
    """T = 2^31 - 1, the largest that the call takes."""
    T = (1 << 31) - 1
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.zeros((T, 1), device="cuda")
    capi.moe_route(logits, None, None, None, 1, 0, 1, 1, 0, True, 1.0, ids, w)
    torch.cuda.synchronize()
    for lo in range(0, T, 1 << 28):
        assert torch.all(ids[lo:lo + (1 << 28)] == 0) and torch.all(w[lo:lo + (1 << 28)] == 1)
