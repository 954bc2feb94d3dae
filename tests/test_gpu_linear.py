"""moe_linear against the formula in 64 bits.

Two kinds of cases. With small whole numbers every partial sum is exact in
fp32 whatever its order, so the result is the formula's value rounded once: the
comparison is for equality, over the shapes and strides where tiles, K splits
and tails can go wrong. With random values the tolerance is

    u |y|                 the store's rounding (u = eps / 2 of the output type)
  + 1.2 * dpre            the accumulator's error through the activation
                          (every activation's slope is below 1.2)
  + 2^-19 |act|           the fast exponential and division
  + 2^-23 (|act| + |res|) the residual add

with dpre = 2^-23 (K / 8 + 8) sum|x w| scales + 2^-23 |bias|: an MMA adds 16
(or 32) products to the accumulator, each of those K / 16 additions and the few
of the K split off by at most two units of the last place of a partial sum that
sum|x w| bounds, plus the scale products.
"""
import math

import pytest
import torch

from routed_shared_experts_b200 import capi

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
GUARD = 77.0


def _wide(v, pad, dtype):
    """v as a view into a wider buffer filled with GUARD, and the buffer."""
    R, C = v.shape
    if pad == 0:
        b = v.to(dtype).cuda().contiguous()
        return b, None
    off = 16
    b = torch.full((R, C + off + pad), GUARD, dtype=torch.float32).to(dtype).cuda()
    b[:, off:off + C] = v.to(dtype).cuda()
    return b[:, off:off + C], b


def _act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def _reference(x, w, xs, ws, b, act, r):
    """(value, dpre, act) in float64 on the host."""
    x, w = x.double().cpu(), w.double().cpu()
    pre = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if xs is not None:
        s = xs.double().cpu()[:, None] * ws.double().cpu()[None, :]
        pre, mag = pre * s, mag * s
    d = 2.0 ** -23 * (x.shape[1] / 8 + 8) * mag
    if b is not None:
        pre = pre + b.double().cpu()
        d = d + 2.0 ** -23 * b.double().cpu().abs()
    a = _act64(pre, act)
    return (a if r is None else a + r.double().cpu()), d, a


def _run(T, N, K, dt, odt, bias=None, act="none", residual=False, pad=0, ints=False, seed=0, one_scale=False,
         in_place=False, stream=None):
    g = torch.Generator().manual_seed(1000 * T + 10 * N + K + seed)
    if ints:
        x = torch.randint(-3, 4, (T, K), generator=g).float()
        w = torch.randint(-3, 4, (N, K), generator=g).float()
    else:
        x, w = torch.randn((T, K), generator=g), torch.randn((N, K), generator=g) * 0.05
    xs = ws = None
    if dt == "fp8":
        xs = (2.0 ** torch.randint(-2, 3, (T,), generator=g)).float() if ints else torch.rand(T, generator=g) + 0.5
        n_ws = 1 if one_scale else N
        ws = (2.0 ** torch.randint(-2, 3, (n_ws,), generator=g)).float() if ints else torch.rand(n_ws, generator=g) + 0.5
    xv, _ = _wide(x, pad, DT[dt])
    wv, _ = _wide(w, pad, DT[dt])
    b = r = rv = None
    if bias:
        b = (torch.randint(-8, 9, (N,), generator=g).float() if ints else torch.randn(N, generator=g)).to(DT[bias]).cuda()
    if residual:
        r = torch.randint(-9, 10, (T, N), generator=g).float() if ints else torch.randn((T, N), generator=g)
        rv, _ = _wide(r, pad, DT[odt])
    ov, ob = _wide(torch.full((T, N), -55.0), pad, DT[odt])
    if in_place:
        ov.copy_(rv)
        rv_call = ov
        r_ref = rv.clone()
    else:
        rv_call, r_ref = rv, rv
    xs_d = None if xs is None else xs.cuda()
    ws_d = None if ws is None else ws.cuda()
    capi.moe_linear(capi.DTYPES[dt], xv, xs_d, wv, ws_d, b, capi.ACTS[act], rv_call, ov, stream)
    torch.cuda.synchronize()
    assert capi.device_error() == 0
    ref, d, a = _reference(xv, wv, xs, None if ws is None else ws.expand(N), b, act, r_ref)
    if ob is not None:  # nothing between the rows is written
        assert torch.all(ob[:, :16].float() == GUARD) and torch.all(ob[:, 16 + N:].float() == GUARD)
    return ov, ref, d, a, r_ref


def _check(T, N, K, dt, odt, **kw):
    out, ref, d, a, r = _run(T, N, K, dt, odt, **kw)
    if kw.get("ints"):
        want = ref.to(DT[odt]) if odt != "f32" else ref.float()
        assert torch.equal(out.cpu(), want), (T, N, K, (out.cpu().double() - ref).abs().max())
        return
    u = torch.finfo(DT[odt]).eps / 2
    tol = u * ref.abs() + 1.2 * d + 2.0 ** -19 * a.abs() + 2.0 ** -23 * (a.abs() + (0 if r is None else r.double().cpu().abs()))
    tol = tol + torch.finfo(DT[odt]).smallest_normal * u  # half a subnormal step
    err = (out.double().cpu() - ref).abs()
    assert torch.all(err <= tol), (T, N, K, (err / tol).max())


# every token tile width with one row, a row short, full and one over; outputs below, at and past a
# 128-row tile and odd; K of less than an atom, one atom, ragged atoms and long enough for each K split
SHAPES = [(1, 1, 8), (1, 128, 64), (1, 2048, 2048), (2, 129, 72), (15, 127, 136), (16, 128, 512), (17, 256, 1024),
          (31, 33, 520), (32, 7168, 256), (33, 640, 2048), (63, 65, 4096), (64, 1000, 264), (65, 384, 1032),
          (127, 255, 128), (128, 128, 7168), (129, 257, 192), (255, 1409, 320), (256, 512, 2816), (257, 130, 640),
          (300, 2815, 408), (511, 768, 1408), (513, 77, 2056), (1000, 1000, 1000), (1024, 512, 16), (2049, 384, 200),
          (4096, 256, 512), (1, 20000, 64), (4097, 8, 64),
          # more than 64 tokens: K over 4 and 2 pairs of a cluster, with one and two accumulations, tails of every
          # kind, and tiles of every width on the way to whole waves
          (66, 256, 7168), (129, 512, 4096), (200, 250, 4104), (257, 97, 3600), (700, 150, 6664), (1000, 256, 7168),
          (100, 2048, 7168), (400, 1030, 5000), (512, 512, 4096), (300, 7168, 520), (2000, 1500, 264),
          (1500, 2300, 72), (3000, 1700, 136), (4096, 2048, 96), (2304, 4400, 64)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear_exact_bf16(cuda_lib, T, N, K):
    _check(T, N, K, "bf16", "f32", ints=True)


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "f32")])
def test_linear_exact_epilogue(cuda_lib, T, N, K, dt, odt):
    """Bias, residual, ReLU and strides; whole numbers, so one rounding."""
    _check(T, N, K, dt, odt, ints=True, bias="f32", act="relu", residual=True, pad=24 if N % 2 else 0)


@pytest.mark.parametrize("T,N,K", [(t, n, -(-k // 16) * 16) for t, n, k in SHAPES])
@pytest.mark.parametrize("odt", ["f32", "bf16", "fp16"])
def test_linear_exact_fp8(cuda_lib, T, N, K, odt):
    _check(T, N, K, "fp8", odt, ints=True, bias="bf16", residual=T % 2 == 1, pad=16 if T % 3 == 0 else 0,
           one_scale=N % 2 == 0)


@pytest.mark.parametrize("act", sorted(capi.ACTS))
@pytest.mark.parametrize("T,N,K,dt,odt", [(3, 200, 512, "bf16", "f32"), (70, 333, 2048, "fp16", "fp16"),
                                          (515, 1100, 1024, "bf16", "bf16"), (40, 96, 4096, "fp8", "f32"),
                                          (600, 514, 640, "fp8", "bf16")])
def test_linear_random(cuda_lib, act, T, N, K, dt, odt):
    _check(T, N, K, dt, odt, bias="f32", act=act, residual=True)


@pytest.mark.parametrize("T,N,K,dt,odt", [(1, 2048, 7168, "bf16", "f32"), (4096, 256, 7168, "bf16", "f32"),
                                          (40, 1000, 7168, "fp16", "f32"), (100, 256, 7168, "bf16", "f32"),
                                          (900, 512, 7168, "fp8", "f32"), (2000, 2816, 4096, "bf16", "f32"),
                                          (777, 2815, 4096, "fp16", "fp16"), (1024, 5632, 4096, "fp8", "bf16")])
def test_linear_long_k(cuda_lib, T, N, K, dt, odt):
    _check(T, N, K, dt, odt, bias="bf16", pad=8 if dt != "fp8" else 16)


@pytest.mark.parametrize("T", [1, 20, 100, 300, 2000])
def test_linear_residual_in_place(cuda_lib, T):
    for odt in ("bf16", "f32"):
        _check(T, 640, 512, "bf16", odt, ints=True, residual=True, in_place=True, pad=8)
        _check(T, 333, 512, "bf16", odt, ints=True, residual=True, in_place=True)


@pytest.mark.parametrize("T,N,K", [(5, 300, 256), (600, 520, 256)])
def test_linear_infinities_and_nan(cuda_lib, T, N, K):
    """Infinities and NaN of an operand reach exactly the outputs they belong
    to, through every activation as the formula has it."""
    for act in sorted(capi.ACTS):
        g = torch.Generator().manual_seed(3)
        x, w = torch.randn((T, K), generator=g).to(torch.bfloat16), torch.randn((N, K), generator=g).to(torch.bfloat16)
        x[1, 3], x[2, 200], w[7, 9] = float("inf"), float("nan"), float("-inf")
        out = torch.zeros((T, N), dtype=torch.float32, device="cuda")
        capi.moe_linear(capi.MOE_DT_BF16, x.cuda(), None, w.cuda(), None, None, capi.ACTS[act], None, out)
        torch.cuda.synchronize()
        v = x.float() @ w.float().t()
        ref = _act64(v, act)  # fp32 has the same infinities and NaN
        got = out.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), act
        assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), act


@pytest.mark.parametrize("T,N,K", [(1, 256, 7168), (40, 1000, 7168), (100, 256, 7168), (300, 2048, 7168),
                                   (4096, 256, 7168), (2000, 2816, 4096)])
def test_linear_fp32_results_keep_precision(cuda_lib, T, N, K):
    """fp32 results sum pieces of at most 14 K atoms (896 values) of the tensor
    core's accumulation in fp32: an accumulation over L values, each addition
    cutting the sum to 24 bits (an error below 2^-23 of it, of one sign), is off
    by less than 2^-23 (L / 16) / 2 of its size on average, pieces add with
    independent signs like their values do, so the 2-norm error stays below
    2^-23 * 28 = 3.4e-6 relative; in fact it is below 1e-6."""
    g = torch.Generator().manual_seed(T + N)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((N, K), generator=g) * 0.05).to(torch.bfloat16).cuda()
    out = torch.empty((T, N), device="cuda")
    capi.moe_linear(capi.MOE_DT_BF16, x, None, w, None, None, 0, None, out)
    ref = x.double() @ w.double().t()
    assert (out.double() - ref).norm() <= 3.4e-6 * ref.norm()


def test_linear_no_rows(cuda_lib):
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((0, 8), dtype=torch.bfloat16, device="cuda")
    capi.moe_linear(capi.MOE_DT_BF16, x, None, w, None, None, 0, None, out)
    torch.cuda.synchronize()


def test_linear_wrapper_refusals(cuda_lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    bf = capi.MOE_DT_BF16
    with pytest.raises(TypeError):
        capi.moe_linear(capi.MOE_DT_FP16, x, None, w, None, None, 0, None, out)
    with pytest.raises(ValueError):
        capi.moe_linear(bf, x, None, w[:, :32], None, None, 0, None, out)
    with pytest.raises(ValueError):
        capi.moe_linear(bf, x, None, w, None, None, 0, None, out.t())
    with pytest.raises(TypeError):
        capi.moe_linear(bf, x, None, w, None, None, 0, out.float(), out)
    with pytest.raises(ValueError):  # an expanded operand's rows overlap
        capi.moe_linear(bf, x[:1].expand(4, 64), None, w, None, None, 0, None, out)
    with pytest.raises(capi.MoEError):  # rows of 66 values are not 16-byte aligned
        y = torch.zeros((4, 66), dtype=torch.bfloat16, device="cuda")[:, :64]
        capi.moe_linear(bf, y, None, w, None, None, 0, None, out)
    with pytest.raises(capi.MoEError):
        capi.moe_linear(bf, x, None, w, None, None, 17, None, out)


@pytest.mark.parametrize("T,N,K", [(8, 512, 2048), (40, 4000, 512), (200, 512, 4096), (700, 1100, 512)])
def test_linear_repeatable_and_concurrent(cuda_lib, T, N, K):
    """The same bits every time, two calls at once on two streams included, and
    from a captured graph replayed on new inputs."""
    g = torch.Generator().manual_seed(9)
    xs = [torch.randn((T, K), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    w = (torch.randn((N, K), generator=g) * 0.05).to(torch.bfloat16).cuda()
    call = lambda x, o, s=None: capi.moe_linear(capi.MOE_DT_BF16, x, None, w, None, None, 2, None, o, s)  # noqa: E731
    want = [torch.empty((T, N), dtype=torch.float32, device="cuda") for _ in range(2)]
    for x, o in zip(xs, want):
        call(x, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(want[0]) for _ in range(2)]
    for _ in range(20):
        for x, o, s in zip(xs, got, streams):
            call(x, o, s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x, o = xs[0].clone(), torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, o)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i])


@pytest.mark.parametrize("T,gap", [(64, 70_000_000), (120, 40_000_000), (3000, 1_600_000)])
def test_linear_offsets_past_32_bits(cuda_lib, T, gap):
    """Rows far apart: operands, residual and result reach past 2^32 elements."""
    N, K = 333, 136
    big = torch.empty((T - 1) * gap + 4096, dtype=torch.bfloat16, device="cuda")
    view = lambda cols, at: torch.as_strided(big, (T, cols), (gap, 1), at)  # noqa: E731
    x, r, out = view(K, 0), view(N, 512), view(N, 1024)
    g = torch.Generator().manual_seed(T)
    x.copy_(torch.randint(-3, 4, (T, K), generator=g).to(torch.bfloat16))
    r.copy_(torch.randint(-9, 10, (T, N), generator=g).to(torch.bfloat16))
    w = torch.randint(-3, 4, (N, K), generator=g).to(torch.bfloat16).cuda()
    capi.moe_linear(capi.MOE_DT_BF16, x, None, w, None, None, 0, r, out)
    torch.cuda.synchronize()
    assert capi.device_error() == 0
    ref = (x.double() @ w.double().t() + r.double()).to(torch.bfloat16)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("T,N,K", [(3, 40, 256), (40, 300, 2048), (130, 96, 7168), (300, 520, 256), (1024, 1024, 512)])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_linear_scales_far_apart(cuda_lib, T, N, K, odt):
    """The sum is scaled by token and then by output, as the formula has it: a
    pair of scales whose own product leaves the fp32 range costs nothing where
    the result does not. Powers of two and whole numbers, so one rounding."""
    g = torch.Generator().manual_seed(T)
    x, w = (torch.randint(-3, 4, (n, K), generator=g).float().to(DT["fp8"]) for n in (T, N))
    ref = x.double() @ w.double().t()
    for ex, ew in ((-100, -40), (-100, -60), (-90, -58), (90, -100), (100, 60)):
        xs, ws = torch.full((T,), 2.0 ** ex), torch.full((N,), 2.0 ** ew)
        if ex + ew > 127:  # only zeros stay in range: 0 * scale is 0
            xz = torch.zeros((T, K)).to(DT["fp8"])
            want, xv = torch.zeros((T, N), dtype=torch.float64), xz
        else:
            want, xv = ref * 2.0 ** (ex + ew), x
        out = torch.full((T, N), 7.0, dtype=DT[odt], device="cuda")
        capi.moe_linear(capi.MOE_DT_FP8_E4M3, xv.cuda(), xs.cuda(), w.cuda(), ws.cuda(), None, 0, None, out)
        if odt == "f32":
            assert torch.equal(out.cpu(), want.float()), (ex, ew)
        else:  # fp32 first (exact down to its subnormal step), then the result type
            assert torch.equal(out.cpu(), want.float().to(DT[odt])), (ex, ew)


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu_tanh"])
@pytest.mark.parametrize("T,N,K", [(4, 1024, 64), (40, 1024, 64), (300, 1024, 64), (66, 1024, 4096)])
def test_linear_activations_over_the_exponentials_range(cuda_lib, act, T, N, K):
    """Pre-activations from -80 to 80 that the sum gives exactly (one product of
    a power of two and a bf16 value per output), fp32 results.

    The exponential of an exact argument is within 2 units of the last place
    (2^-22), the sum 1 + e and the quotient within 2^-24 and 2^-23, a product with
    v 2^-24: 2^-20 in all. GELU's exponent is rounded itself: v^2, the cubic
    term, the sum and two products leave 6 roundings of 2^-24 relative, that is
    6 * 2^-24 |u| in the exponential, u = 2 sqrt(2/pi) (v + 0.044715 v^3); the
    constant's own rounding is one of them more. Results below 2^-126 are off by
    that of the subnormal steps of e (2^-149) times |v|, at most 2^-142."""
    v = torch.linspace(-80, 80, N).bfloat16()
    if act == "gelu_tanh":
        v = torch.linspace(-9, 9, N).bfloat16()
    x = torch.zeros((T, K), dtype=torch.bfloat16)
    w = torch.zeros((N, K), dtype=torch.bfloat16)
    p = torch.arange(T) % 4
    x[torch.arange(T), torch.arange(T) % K] = torch.exp2(-p.float()).bfloat16()
    w[:, :min(T, K)] = v[:, None]
    out = torch.empty((T, N), device="cuda")
    capi.moe_linear(capi.MOE_DT_BF16, x.cuda(), None, w.cuda(), None, None, capi.ACTS[act], None, out)
    pre = x.double().sum(1, keepdim=True) * v.double()
    if act == "silu":
        ref = pre * torch.special.expit(pre)
    elif act == "sigmoid":
        ref = torch.special.expit(pre)
    else:
        ref = pre * torch.special.expit(2 * math.sqrt(2 / math.pi) * (pre + 0.044715 * pre ** 3))
    rel = 2.0 ** -20
    if act == "gelu_tanh":
        rel = rel + 7 * 2.0 ** -24 * (2 * math.sqrt(2 / math.pi) * (pre + 0.044715 * pre ** 3)).abs()
    err = (out.cpu().double() - ref).abs()
    tol = rel * ref.abs() + 2.0 ** -142
    assert torch.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("T", [4, 300])
def test_linear_activations_tails_in_bf16(cuda_lib, act, T):
    """bf16 results far down the left tail: the fast exponential's error, (4 + 1.2
    |v|) 2^-23 or below 2^-16 here, is far below the store's half step 2^-8. The
    fast division gives zero where its divisor 1 + exp(-v) passes 2^126, that is for
    v < -87.3: what it drops there is below 88.8 / 2^126 < 2^-119."""
    v = torch.linspace(-84, 20, 512).bfloat16()
    x = torch.zeros((T, 64), dtype=torch.bfloat16)
    x[:, 0] = 1.0
    w = torch.zeros((512, 64), dtype=torch.bfloat16)
    w[:, 0] = v
    b = torch.full((512,), -4.5, device="cuda")
    out = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
    capi.moe_linear(capi.MOE_DT_BF16, x.cuda(), None, w.cuda(), None, b, capi.ACTS[act], None, out)
    pre = v.double() - 4.5
    ref = torch.special.expit(pre) * (pre if act == "silu" else 1.0)
    tol = (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 2.0 ** -119
    assert torch.all((out.cpu().double() - ref).abs() <= tol)


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(257, 640, 520), (300, 2815, 136), (384, 4400, 64), (2100, 1500, 264), (66, 256, 7168)])
def test_linear_back_to_back(cuda_lib, T, N, K, odt):
    """Launches that start while the one before them ends, rows of the last tile's
    second half missing (its CTA then releases the accumulators last of all): forty
    in a row on alternating operands, each result as the first time."""
    g = torch.Generator().manual_seed(T + N)
    xs = [torch.randint(-3, 4, (T, K), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    w = torch.randint(-3, 4, (N, K), generator=g).to(torch.bfloat16).cuda()
    want = [(x.double() @ w.double().t()).to(DT[odt]) for x in xs]
    outs = [torch.empty((T, N), dtype=DT[odt], device="cuda") for _ in range(40)]
    for i, o in enumerate(outs):
        capi.moe_linear(capi.MOE_DT_BF16, xs[i % 2], None, w, None, None, 0, None, o)
    torch.cuda.synchronize()
    assert capi.device_error() == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2]), i


@pytest.mark.parametrize("T,N,K", [(1, 140, 2048), (3, 8, 4096), (33, 200, 2048), (64, 1025, 7168), (66, 130, 7168),
                                   (130, 250, 4104), (401, 97, 3600)])
def test_linear_joins_of_partly_filled_tiles(cuda_lib, T, N, K):
    """Warps and rows of a K split that have nothing to finish, in launches that
    follow one another without a gap."""
    g = torch.Generator().manual_seed(N)
    x = torch.randint(-3, 4, (T, K), generator=g).to(torch.bfloat16).cuda()
    w = torch.randint(-3, 4, (N, K), generator=g).to(torch.bfloat16).cuda()
    want = x.double() @ w.double().t()
    outs = [torch.empty((T, N), dtype=torch.bfloat16 if i % 2 else torch.float32, device="cuda") for i in range(40)]
    for o in outs:
        capi.moe_linear(capi.MOE_DT_BF16, x, None, w, None, None, 0, None, o)
    torch.cuda.synchronize()
    assert capi.device_error() == 0
    for o in outs:
        assert torch.equal(o, want.to(o.dtype))


@pytest.mark.parametrize("T,N,K,dt", [(1, 300, 16384, "bf16"), (20, 1000, 28672, "fp16"), (64, 256, 16384, "bf16"),
                                      (64, 256, 57344, "bf16"), (5, 130, 32768, "fp8"), (33, 20000, 7168, "bf16"),
                                      (64, 256, 32768, "fp8")])
def test_linear_fp32_results_keep_precision_at_any_length(cuda_lib, T, N, K, dt):
    """A piece of 14 atoms is the longest accumulation of an fp32 result whatever
    K: eight of them are K = 7168 (fp8: 14336). With positive values nothing cancels
    and every cut of the tensor core's additions goes one way, so a sum of pieces is
    off by the mean of their relative errors, which is the same for two full pieces
    of one distribution and less for a short one: the relative error at K is that
    at eight pieces, half of it again for the draw, and the roundings of the sums of
    pieces (2^-24 each, fifteen at most). Accumulations as long as K / 8 would make
    it grow with K."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    short = 14336 if dt == "fp8" else 7168
    L = max(K, short)
    x = torch.rand((T, L), generator=g, device="cuda").to(DT[dt])
    w = (torch.rand((N, L), generator=g, device="cuda") * 0.05).to(DT[dt])
    xs, ws = (torch.ones(n, device="cuda") for n in (T, N)) if dt == "fp8" else (None, None)
    out = torch.empty((T, N), device="cuda")

    def error(k):
        capi.moe_linear(capi.DTYPES[dt], x[:, :k], xs, w[:, :k], ws, None, 0, None, out)
        ref = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        for i in range(0, k, 1024):  # in slices: w in 64 bits is eight times its size
            ref += x[:, i:min(i + 1024, k)].double() @ w[:, i:min(i + 1024, k)].double().t()
        return ((out.double() - ref).norm() / ref.norm()).item()

    e, e0 = error(K), error(short)
    assert e <= 1.5 * e0 + 15 * 2.0 ** -24, (e, e0)


@pytest.mark.parametrize("T,N,K", [(1, 300, 16384), (16, 128, 7304), (17, 96, 8200), (33, 130, 28680), (64, 256, 57344),
                                   (2, 20000, 14352), (40, 1025, 14336)])
@pytest.mark.parametrize("dt", ["bf16", "fp8"])
def test_linear_exact_long_k_fp32(cuda_lib, T, N, K, dt):
    """Whole numbers (sums below 2^24), so equality, where a CTA adds several pieces
    of K: one, two, three and more, the last one short, bias and residual."""
    _check(T, N, -(-K // 16) * 16, dt, "f32", ints=True, bias="f32", residual=True, pad=16 if T % 2 else 0)


@pytest.mark.parametrize("T", [1, 5, 70, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (2, 3), (3, 7), (1, 9), (130, 1), (33, 63), (7, 65), (5, 127), (3, 129)])
def test_linear_smallest_and_odd_k(cuda_lib, T, N, K):
    """K of any length, in rows whose stride is a multiple of 16 bytes; what lies
    between K and the next row (NaN here) is not read as part of the sum."""
    g = torch.Generator().manual_seed(T + 10 * N + K)
    for dt, odt in (("bf16", "f32"), ("fp16", "fp16"), ("fp8", "bf16")):
        ld = -(-K // 16) * 16 + 16
        xb, wb = (torch.full((n, ld), float("nan")).to(DT[dt]).cuda() for n in (T, N))
        x, w = (torch.randint(-3, 4, (n, K), generator=g).float() for n in (T, N))
        xb[:, :K], wb[:, :K] = x.to(DT[dt]).cuda(), w.to(DT[dt]).cuda()
        s = [torch.ones(n, device="cuda") for n in (T, N)] if dt == "fp8" else (None, None)
        out = torch.empty((T, N), dtype=DT[odt], device="cuda")
        capi.moe_linear(capi.DTYPES[dt], xb[:, :K], s[0], wb[:, :K], s[1], None, 0, None, out)
        torch.cuda.synchronize()
        assert capi.device_error() == 0
        assert torch.equal(out.cpu(), (x.double() @ w.double().t()).to(DT[odt])), (dt, odt)


def test_first_calls_of_a_process_inside_a_capture(cuda_lib):
    """A process whose first call of each operator is a captured one, every kernel
    choice of the product among them."""
    import subprocess
    import sys
    from routed_shared_experts_b200 import build
    code = """
import torch
from routed_shared_experts_b200 import capi
w = torch.ones((512, 4096), dtype=torch.bfloat16, device="cuda")
xs = [torch.ones((t, 4096), dtype=torch.bfloat16, device="cuda") for t in (1, 40, 100, 500, 3000)]
outs = [torch.zeros((x.shape[0], 512), dtype=d, device="cuda") for x in xs for d in (torch.bfloat16, torch.float32)]
ids, wt = torch.zeros((500, 4), dtype=torch.int32, device="cuda"), torch.zeros((500, 4), device="cuda")
gamma, y = torch.ones(512, device="cuda"), torch.zeros((500, 512), dtype=torch.bfloat16, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for i, o in enumerate(outs):
        capi.moe_linear(capi.MOE_DT_BF16, xs[i // 2], None, w, None, None, 0, None, o)
    capi.moe_rmsnorm_quantize(None, outs[6], None, gamma, 1e-6, None, y, None, None)
    capi.moe_route(outs[7], None, None, None, 4, 0, 8, 2, 0, True, 1.0, ids, wt)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
assert capi.device_error() == 0
assert all(torch.all(o == 4096) for o in outs)
assert torch.all(y == 1) and torch.all(ids == torch.arange(4, device="cuda")) and torch.all(wt == 0.25)
print("ok")
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stderr


def test_linear_from_two_threads(cuda_lib):
    """Calls of two Python threads on streams of their own (the binding lets the
    other thread run during the launch)."""
    import threading
    g = torch.Generator().manual_seed(2)
    w = torch.randint(-3, 4, (640, 512), generator=g).to(torch.bfloat16).cuda()
    xs = [torch.randint(-3, 4, (t, 512), generator=g).to(torch.bfloat16).cuda() for t in (3, 300)]
    want = [(x.double() @ w.double().t()).float() for x in xs]
    outs = [[torch.zeros((x.shape[0], 640), device="cuda") for _ in range(50)] for x in xs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for o in outs[i]:
                    capi.moe_linear(capi.MOE_DT_BF16, xs[i], None, w, None, None, 0, None, o)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_first_call_of_a_thread(cuda_lib):
    """A thread whose first use of CUDA is this call: no context is current yet."""
    import threading
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((4, 4), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            capi.moe_linear(capi.MOE_DT_BF16, x, None, x, None, None, 0, None, out, s)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    s.synchronize()
    assert not failed and torch.all(out == 64)
