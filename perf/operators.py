"""Measured cases of the operators around the expert layer.

Three operators that a decoder block runs next to ``MoELayer``:

* ``linear``: ``moe_linear``, a dense matrix product whose epilogue applies operand scales, bias,
  activation and residual before the one rounding (attention output projection, router logits,
  dense feed-forward projections);
* ``route``: ``moe_route``, expert routing from softmax or sigmoid scores with a balance bias, expert
  groups, masked experts and padded batches;
* ``norm``: ``moe_rmsnorm_quantize``, residual add, RMS norm and the quantisation of the normalised
  activations to the layer's operand formats in one pass.

``run`` computes an operator in plain torch operations, or, with ``own`` set, through the package.
"""
import math

import torch

own = False

NO_EXPERT = -(1 << 31)  # routing id of a row behind the last token
TORCH_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
EPS = 1e-6


def listed():
    return [
        # linear ---------------------------------------------------------------------------------
        # one generated token: attention output projection onto the residual stream of the decode layer
        _lin("linear_token_bf16", 1, 2048, 2048, "bf16", residual=True),
        # a decode batch of the widest layer: 103 MB of weights read for 32 tokens
        _lin("linear_decode_bf16", 32, 7168, 7168, "bf16", residual=True),
        # router logits of a decode batch, in 32 bits for the routing that follows
        _lin("linear_router_decode", 32, 128, 2048, "bf16", out="f32", bias=True),
        # router logits of a prefill
        _lin("linear_router_prefill", 4096, 256, 7168, "bf16", out="f32", bias=True),
        # a ragged batch against an odd number of outputs, operands and output cut from wider buffers
        _lin("linear_ragged_fp16", 777, 2815, 4096, "fp16", bias=True, act="gelu", strided=True),
        # the dense feed-forward projection of the fp8 layer: gate_up width, one scale per token and output
        _lin("linear_up_fp8", 1024, 5632, 4096, "fp8", bias=True, act="silu"),
        # a prefill through the widest square projection, residual added
        _lin("linear_prefill_bf16", 4096, 7168, 7168, "bf16", residual=True),
        # route ----------------------------------------------------------------------------------
        # a decode batch, plain softmax routing with a balance bias
        _rt("route_decode_softmax", 32, 128, 8, "softmax", bias=True),
        # a prefill over 256 experts in 8 groups, 4 kept, sigmoid scores and balance bias
        _rt("route_prefill_groups", 4096, 256, 8, "sigmoid", n_group=8, topk_group=4, bias=True, rsf=2.5),
        # a batch padded for a captured graph, 16-bit logits, some experts switched off
        _rt("route_padded_bf16", 1000, 64, 6, "softmax", n_group=8, topk_group=4, group_score="max",
            renormalize=False, dtype="bf16", mask=True, padded=True),
        # norm -----------------------------------------------------------------------------------
        # a decode batch: residual add and norm in front of the bf16 layer
        _nm("norm_decode_bf16", 32, 2048, "bf16", "none"),
        # a prefill in front of the MXFP8 layer: 16-bit activations for router and gate, codes for the experts
        _nm("norm_prefill_mxfp8", 4096, 7168, "bf16", "mxfp8"),
    ]


def _lin(name, T, N, K, dtype, out=None, bias=False, act="none", residual=False, strided=False):
    return dict(name=name, op="linear", T=T, N=N, K=K, dtype=dtype, out=out or ("bf16" if dtype == "fp8" else dtype),
                bias=bias, act=act, residual=residual, strided=strided)


def _rt(name, T, E, k, score, n_group=1, topk_group=1, group_score="top2", bias=False, renormalize=True, rsf=1.0,
        dtype="f32", mask=False, padded=False):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, n_group=n_group, topk_group=topk_group,
                group_score=group_score, bias=bias, renormalize=renormalize, rsf=rsf, dtype=dtype, mask=mask,
                padded=padded)


def _nm(name, T, H, dtype, quant, residual=True, y=True):
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, quant=quant, residual=residual, y=y)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "norm"])
    if op == "linear":
        dtype = rng.choice(["bf16", "fp16", "fp8"])
        return dict(_lin("", _log_int(rng, 1, 4096), _log_int(rng, 8, 7168), 16 * _log_int(rng, 4, 448), dtype,
                         out=rng.choice(["f32", None, None]), bias=rng.random() < 0.6,
                         act=rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]),
                         residual=rng.random() < 0.5, strided=rng.random() < 0.3))
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log_int(rng, 2, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        return _rt("", _log_int(rng, 1, 4096), E, rng.randint(1, min(16, topk_group * E // n_group)),
                   rng.choice(["softmax", "sigmoid"]), n_group, topk_group, rng.choice(["top2", "max"]),
                   rng.random() < 0.6, rng.random() < 0.7, rng.choice([1.0, 2.5]),
                   rng.choice(["f32", "bf16", "fp16"]), rng.random() < 0.3, rng.random() < 0.3)
    H = 32 * _log_int(rng, 2, 512)
    return _nm("", _log_int(rng, 1, min(4096, 4096 * 7168 // H)), H, rng.choice(["bf16", "fp16"]),
               *rng.choice([("none", True, True), ("none", False, True), ("fp8", True, True), ("fp8", False, False),
                            ("mxfp8", True, True), ("mxfp8", True, False)]))


# ------------------------------------------------------------------------------------------ inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _rows(v, strided):
    """``v`` [R, C] as a view into a wider buffer: rows further apart than they are long."""
    if not strided:
        return v
    wide = torch.zeros((v.shape[0], v.shape[1] + 48), dtype=v.dtype, device=v.device)
    view = wide[:, 16:16 + v.shape[1]]
    view.copy_(v)
    return view


def _e4m3_rows(v):
    """Codes and one 32-bit scale per row."""
    scale = v.abs().amax(1).clamp_min(1e-12) / 448.0
    return (v / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    T = case["T"]
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    st = dict(case)
    if op == "linear":
        N, K, dt = case["N"], case["K"], case["dtype"]
        x, w = rand(T, K), rand(N, K) * 0.02
        st["x_scale"] = st["w_scale"] = st["b"] = st["r"] = None
        if dt == "fp8":
            x, st["x_scale"] = _e4m3_rows(x)
            w, st["w_scale"] = _e4m3_rows(w)
        st["x"] = _rows(x.to(TORCH_DT[dt]), case["strided"])
        st["w"] = _rows(w.to(TORCH_DT[dt]), case["strided"])
        if case["bias"]:
            st["b"] = rand(N) * 0.5
        if case["residual"]:
            st["r"] = _rows(rand(T, N).to(TORCH_DT[case["out"]]), case["strided"])
        st["y"] = _rows(torch.zeros((T, N), dtype=TORCH_DT[case["out"]], device="cuda"), case["strided"])
    elif op == "route":
        E, k = case["E"], case["k"]
        st["logits"] = rand(T, E).mul_(1.5).to(TORCH_DT[case["dtype"]])
        st["b"] = rand(E) * 0.1 if case["bias"] else None
        st["m"] = None
        if case["mask"]:  # about one expert in eight switched off
            st["m"] = (torch.rand(E, generator=g, device="cuda") >= 0.125).to(torch.uint8)
        st["valid"] = None
        if case["padded"]:  # tokens of the batch, the rest of the rows is padding
            st["valid"] = torch.randint(T // 2, T + 1, (1,), generator=g, device="cuda", dtype=torch.int32)
        st["ids"] = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        st["wts"] = torch.zeros((T, k), dtype=torch.float32, device="cuda")
    else:
        H, dt = case["H"], TORCH_DT[case["dtype"]]
        st["x"] = rand(T, H).to(dt)
        st["r"] = (rand(T, H) * 3).to(dt) if case["residual"] else None
        st["gamma"] = (1 + 0.2 * rand(H)).to(dt)
        st["sum"] = torch.empty((T, H), dtype=dt, device="cuda") if case["residual"] else None
        st["out"] = torch.empty((T, H), dtype=dt, device="cuda") if case["y"] else None
        st["codes"] = st["scale"] = None
        if case["quant"] != "none":
            st["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
            st["scale"] = (torch.empty(T, dtype=torch.float32, device="cuda") if case["quant"] == "fp8" else
                           torch.empty((T, H // 32), dtype=torch.uint8, device="cuda"))
    return st


# ------------------------------------------------------------------------------------- the operators


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "route": _plain_route, "norm": _plain_norm}[state["op"]](state)


def _own(st):
    from routed_shared_experts_b200 import capi

    if st["op"] == "linear":
        capi.moe_linear(capi.DTYPES[st["dtype"]], st["x"], st["x_scale"], st["w"], st["w_scale"], st["b"],
                        capi.ACTS[st["act"]], st["r"], st["y"])
        return st["y"]
    if st["op"] == "route":
        capi.moe_route(st["logits"], st["b"], st["m"], st["valid"], st["k"], capi.SCORES[st["score"]], st["n_group"],
                       st["topk_group"], capi.GROUP_SCORES[st["group_score"]], st["renormalize"], st["rsf"],
                       st["ids"], st["wts"])
        return {"ids": st["ids"], "weights": st["wts"]}
    qdt = None if st["quant"] == "none" else capi.DTYPES[st["quant"]]
    capi.moe_rmsnorm_quantize(qdt, st["x"], st["r"], st["gamma"], EPS, st["sum"], st["out"], st["codes"],
                              st["scale"])
    return _norm_outputs(st["sum"], st["out"], st["codes"], st["scale"])


def _norm_outputs(total, y, codes, scale):
    """The codes and shared exponents as the 8-bit floating-point values they are."""
    out = {"sum": total, "y": y, "codes": codes, "scale": scale}
    if scale is not None and scale.dtype == torch.uint8:
        out["scale"] = scale.view(torch.float8_e8m0fnu)
    return {name: v for name, v in out.items() if v is not None}


def _activation(v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def _plain_linear(st):
    v = st["x"].float() @ st["w"].float().t()
    if st["x_scale"] is not None:
        v = v * st["x_scale"][:, None] * st["w_scale"]
    if st["b"] is not None:
        v = v + st["b"]
    v = _activation(v, st["act"])
    if st["r"] is not None:
        v = v + st["r"].float()
    return v.to(TORCH_DT[st["out"]])


def _plain_route(st):
    """Scores in 64 bits and rounded once, because a choice between neighbours hangs on them."""
    T, E, k, G = st["T"], st["E"], st["k"], st["n_group"]
    l = st["logits"].double()
    off = torch.isnan(l) | (l == -math.inf)
    if st["m"] is not None:
        off = off | (st["m"] == 0)
    if st["score"] == "softmax":
        top = l.masked_fill(off, -math.inf).amax(1, keepdim=True)
        e = torch.exp(torch.where(l == top, 0.0, l - top)).masked_fill(off, 0.0)
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1 / (1 + torch.exp(-l))
    c = s.float()
    if st["b"] is not None:
        c = c + st["b"]
    c = c.masked_fill(off | torch.isnan(c), -math.inf)
    order = torch.sort(c, dim=1, descending=True, stable=True).indices  # ties: lower index
    if G > 1:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values
        gs = best[..., 0]
        if st["group_score"] == "top2" and E // G > 1:
            gs = gs + best[..., 1].masked_fill(best[..., 1] == -math.inf, 0.0)
        groups = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :st["topk_group"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, groups, True)
        in_kept = kept.repeat_interleave(E // G, 1).gather(1, order)
        order = order.gather(1, torch.sort(in_kept.int(), dim=1, descending=True, stable=True).indices)
    ids = order[:, :k]
    w = s.gather(1, ids).masked_fill(c.gather(1, ids) == -math.inf, 0.0)
    if st["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    w = (w * st["rsf"]).float()
    ids = ids.int()
    if st["valid"] is not None:
        pad = (torch.arange(T, device=l.device) >= st["valid"])[:, None]
        ids, w = ids.masked_fill(pad, NO_EXPERT), w.masked_fill(pad, 0.0)
    return {"ids": ids, "weights": w}


def _plain_norm(st):
    dt = st["x"].dtype
    z = st["x"].float()
    total = None
    if st["r"] is not None:
        z = z + st["r"].float()
        total = z.to(dt)  # the residual stream as it is kept; the norm reads the unrounded sum
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * st["gamma"].float()
    codes = scale = None
    if st["quant"] == "fp8":
        amax = y.abs().amax(1)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        codes = (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    elif st["quant"] == "mxfp8":
        b = y.view(y.shape[0], -1, 32)
        amax = b.abs().amax(2)
        e = (torch.frexp(amax).exponent - 9).clamp(-127, 127)
        e = torch.where(amax > 0, e, -127)
        codes = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(y.shape)
        scale = (e + 127).to(torch.uint8)
    return _norm_outputs(total, y.to(dt) if st["y"] else None, codes, scale)


# ------------------------------------------------------------------------------------ in 64 bits


def work(case):
    """Bytes: every operand once, every output once."""
    T = case["T"]
    size = {"bf16": 2, "fp16": 2, "f32": 4, "fp8": 1}
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        es, os_ = size[case["dtype"]], size[case["out"]]
        b = (T + N) * K * es + T * N * os_ * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        if case["dtype"] == "fp8":
            b += 4 * (T + N)
        return {"bytes": b, "flops": 2 * T * N * K}
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    H, es = case["H"], size[case["dtype"]]
    b = T * H * es * (1 + (2 if case["residual"] else 0) + (1 if case["y"] else 0)) + H * es
    if case["quant"] == "fp8":
        b += T * H + 4 * T
    elif case["quant"] == "mxfp8":
        b += T * H + T * H // 32
    return {"bytes": b, "flops": 6 * T * H}


def exact(case, seed):
    """The definitions in 64 bits; routing by successive maxima instead of sorts."""
    st = prepare(case, seed)
    if case["op"] == "linear":
        a = torch.einsum("tk,nk->tn", st["x"].double(), st["w"].double())
        if st["x_scale"] is not None:
            a = torch.einsum("tn,t,n->tn", a, st["x_scale"].double(), st["w_scale"].double())
        if st["b"] is not None:
            a += st["b"].double()
        act = case["act"]
        if act == "relu":
            a = torch.where(a > 0, a, 0.0)
        elif act == "silu":
            a = a * torch.special.expit(a)
        elif act == "gelu":
            a = a * torch.special.ndtr(a)
        elif act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
            a = a * torch.special.expit(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
        elif act == "sigmoid":
            a = torch.special.expit(a)
        return a + st["r"].double() if st["r"] is not None else a
    if case["op"] == "norm":
        z = st["x"].double()
        out = {}
        if st["r"] is not None:
            z = z + st["r"].double()
            out["sum"] = z
        rms = (torch.einsum("th,th->t", z, z) / case["H"] + EPS).sqrt()
        y = torch.einsum("th,t,h->th", z, 1 / rms, st["gamma"].double())
        if case["y"]:
            out["y"] = y
        if case["quant"] == "fp8":
            out["scale"] = y.abs().max(1).values / 448
            out["codes"] = y / out["scale"][:, None]
        elif case["quant"] == "mxfp8":
            blocks = y.reshape(case["T"], -1, 32)
            out["scale"] = torch.exp2(torch.floor(torch.log2(blocks.abs().max(2).values)) - 8)
            out["codes"] = (blocks / out["scale"][..., None]).reshape(y.shape)
        return out
    T, E, G = case["T"], case["E"], case["n_group"]
    l = st["logits"].double()
    live = torch.ones_like(l, dtype=torch.bool) if st["m"] is None else (st["m"] != 0).expand(T, E)
    if case["score"] == "softmax":
        s = torch.softmax(l.masked_fill(~live, -math.inf), 1)
        s = torch.where(live.any(1, keepdim=True), s, 0.0)
    else:
        s = torch.special.expit(l)
    c = s.float() if st["b"] is None else s.float() + st["b"]
    c = torch.where(live, c, -math.inf)
    allowed = torch.ones((T, E), dtype=torch.bool, device=l.device)
    if G > 1:
        size = E // G
        cg = c.reshape(T, G, size)
        first = cg.max(2)
        gs = first.values
        if case["group_score"] == "top2" and size > 1:
            rest = cg.scatter(2, first.indices[..., None], -math.inf).max(2).values
            gs = gs + torch.where(rest == -math.inf, 0.0, rest)
        open_ = torch.zeros((T, G), dtype=torch.bool, device=l.device)
        number = torch.arange(G, device=l.device)
        for _ in range(case["topk_group"]):
            left = ~open_
            m = gs.masked_fill(open_, -math.inf).max(1, keepdim=True).values
            pick = torch.where(left & (gs == m), number, G).min(1).values
            open_[torch.arange(T, device=l.device), pick] = True
        allowed = open_.repeat_interleave(size, 1)
    number = torch.arange(E, device=l.device)
    picked = []
    for _ in range(case["k"]):
        m = c.masked_fill(~allowed, -math.inf).max(1, keepdim=True).values
        pick = torch.where(allowed & (c == m), number, E).min(1).values
        allowed[torch.arange(T, device=l.device), pick] = False
        picked.append(pick)
    ids = torch.stack(picked, 1)
    w = torch.where(live.gather(1, ids), s.gather(1, ids), 0.0)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * case["rsf"]
    if st["valid"] is not None:
        w = torch.where(torch.arange(T, device=l.device)[:, None] < st["valid"], w, 0.0)
    return {"ids": None, "weights": w}
