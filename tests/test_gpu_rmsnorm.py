"""moe_rmsnorm_quantize against the formula in 64 bits.

Tolerances: the sum of squares is off by at most 50 units of 2^-24 (up to 32
fused additions per thread, ten in the reductions, the division), half of which
reach 1/rms; the square root, two products and z's own rounding add a few, so
the unrounded y is within 2^-18 of the formula, relative to |y| plus the
cancellation of z: 2^-24 (|x| + |residual|) through the same factor. The 16-bit
store adds half a step of its type, a code half a step of e4m3 (2^-4, or 2^-10
in its subnormal range), measured in units of the scale; values past 448 units
saturate."""
import math

import pytest
import torch

from routed_shared_experts_b200 import capi

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
QUANT = {"none": None, "fp8": capi.MOE_DT_FP8_E4M3, "mxfp8": capi.MOE_DT_MXFP8_E4M3}


def _inputs(T, H, dt, seed=0):
    g = torch.Generator().manual_seed(100 * T + H + seed)
    x, r = torch.randn((T, H), generator=g), 3 * torch.randn((T, H), generator=g)
    gamma = 1 + 0.3 * torch.randn(H, generator=g)
    if T > 3:
        x[1], r[1] = 0, 0             # a row of zeros
        x[2, 7 % H] = 300.0           # an outlier
        x[3, :32], r[3, :32] = 0, 0   # a block of zeros
    return x.to(DT[dt]), r.to(DT[dt]), gamma.to(DT[dt])


def _check(T, H, dt, quant, residual=True, y=True, gamma_f32=False, eps=1e-6):
    x, r, gamma = _inputs(T, H, dt)
    if gamma_f32:
        gamma = gamma.float() * 1.001
    dev = dict(device="cuda")
    res = r.cuda() if residual else None
    ro = torch.empty((T, H), dtype=DT[dt], **dev) if residual else None
    yo = torch.empty((T, H), dtype=DT[dt], **dev) if y else None
    codes = scale = None
    if quant != "none":
        codes = torch.empty((T, H), dtype=torch.uint8, **dev)
        scale = torch.empty(T, **dev) if quant == "fp8" else torch.empty((T, H // 32), dtype=torch.uint8, **dev)
    capi.moe_rmsnorm_quantize(QUANT[quant], x.cuda(), res, gamma.cuda(), eps, ro, yo, codes, scale)
    torch.cuda.synchronize()
    z = x.double() + (r.double() if residual else 0)
    if residual:  # one rounding of the fp32 sum
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(DT[dt]))
    rms = torch.sqrt((z * z).mean(1, keepdim=True) + eps)
    ref = z / rms * gamma.double()
    slack = 2.0 ** -18 * ref.abs()
    if residual:
        slack = slack + 2.0 ** -24 * (x.double().abs() + r.double().abs()) / rms * gamma.double().abs()
    if y:
        fi = torch.finfo(DT[dt])
        tol = slack + fi.eps / 2 * (ref.abs() + slack) + fi.smallest_normal * fi.eps / 2
        assert torch.all((yo.cpu().double() - ref).abs() <= tol)
    if quant == "none":
        return
    c = codes.cpu().view(torch.float8_e4m3fn).double()
    if quant == "fp8":
        s = scale.cpu().double()[:, None]
        amax = ref.abs().amax(1, keepdim=True)
        want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        # the amax's own slack, and two fp32 roundings
        assert torch.all((s - want).abs() <= slack.amax(1, keepdim=True) / 448 + 2.0 ** -22 * want)
        unit = s
    else:
        sb = scale.cpu().int()
        b = ref.view(T, -1, 32)
        hi = (b.abs() + slack.view(T, -1, 32)).amax(2)
        lo = (b.abs() - slack.view(T, -1, 32)).amax(2)
        byte = lambda a: torch.where(a > 0, (torch.floor(torch.log2(a.clamp_min(1e-300))) - 8).clamp(-127, 127), -127.0).int() + 127  # noqa: E731
        assert torch.all((sb >= byte(lo)) & (sb <= byte(hi)))
        unit = torch.exp2(sb.double() - 127).repeat_interleave(32, 1)
    v = (ref / unit).clamp(-448, 448)
    tol = slack / unit + 2.0 ** -4 * (v.abs() + slack / unit) + 2.0 ** -10 + 2.0 ** -20
    assert torch.all((c - v).abs() <= tol)


# one chunk, every threads-per-row and chunks-per-thread variant with ragged ends, and the widest row
WIDTHS = [8, 32, 64, 200, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 14656, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm(cuda_lib, H, dt):
    _check(5, H, dt, "none")
    _check(1, H, dt, "none", residual=False, gamma_f32=True)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm_fp8(cuda_lib, H, dt):
    _check(9, H, dt, "fp8")
    _check(4, H, dt, "fp8", residual=False, y=False)


@pytest.mark.parametrize("H", [h // 32 * 32 for h in WIDTHS if h >= 32])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm_mxfp8(cuda_lib, H, dt):
    _check(9, H, dt, "mxfp8")
    _check(4, H, dt, "mxfp8", residual=False, y=False, gamma_f32=True)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 1000, 4097])
@pytest.mark.parametrize("quant", ["none", "fp8", "mxfp8"])
def test_norm_rows(cuda_lib, T, quant):
    _check(T, 96, "bf16", quant)


def test_norm_in_place_and_guards(cuda_lib):
    """residual_out = residual and y = x give the same bits, and nothing behind
    the rows is written."""
    T, H = 13, 520
    x, r, gamma = _inputs(T, H, "bf16")
    xs, rs = (torch.full((T + 2, H), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    xs[:T], rs[:T] = x.cuda(), r.cuda()
    yo, ro = torch.empty_like(xs[:T]), torch.empty_like(xs[:T])
    capi.moe_rmsnorm_quantize(None, xs[:T], rs[:T], gamma.cuda(), 1e-5, ro, yo, None, None)
    capi.moe_rmsnorm_quantize(None, xs[:T], rs[:T], gamma.cuda(), 1e-5, rs[:T], xs[:T], None, None)
    torch.cuda.synchronize()
    assert torch.equal(xs[:T], yo) and torch.equal(rs[:T], ro)
    assert torch.all(xs[T:] == 5) and torch.all(rs[T:] == 5)


def test_norm_infinities_and_nan(cuda_lib):
    """A NaN spoils its own row only; an infinity gives zeros beside it and a
    NaN in its place, as the formula does; codes of NaN are NaN codes."""
    T, H = 4, 256
    x, _, gamma = _inputs(T, H, "bf16", seed=1)
    x[0, 3], x[1, 200] = float("nan"), float("inf")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    c, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    capi.moe_rmsnorm_quantize(QUANT["fp8"], x.cuda(), None, gamma.cuda(), 1e-6, None, y, c, s)
    torch.cuda.synchronize()
    y, c = y.cpu().float(), c.cpu().view(torch.float8_e4m3fn).float()
    assert torch.isnan(y[0]).all() and torch.isnan(c[0]).all()
    assert torch.isnan(y[1, 200]) and torch.isnan(c[1, 200])
    keep = torch.arange(H) != 200
    assert torch.all(y[1][keep] == 0) and torch.all(c[1][keep] == 0)
    assert torch.isfinite(y[2:]).all() and torch.isfinite(c[2:]).all()


def test_norm_fp8_tiny_scale(cuda_lib):
    """A row whose scale is subnormal still gets finite codes: 448 for its
    amax (the quotient amax / (amax / 448) with the subnormal scale's own
    rounding, half a step of 2^-149 in about 2^-129) and 0 for zeros."""
    H = 64
    x = torch.ones((2, H), dtype=torch.bfloat16, device="cuda")
    x[:, 1] = 0
    gamma = torch.full((H,), 1e-36, dtype=torch.float32, device="cuda")
    c, s = torch.empty((2, H), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    capi.moe_rmsnorm_quantize(QUANT["fp8"], x, None, gamma, 1e-6, None, None, c, s)
    torch.cuda.synchronize()
    v = c.cpu().view(torch.float8_e4m3fn).float()
    assert torch.all(v[:, 1] == 0) and torch.all(v[:, 2:] == 448) and torch.all(s > 0)


def test_norm_matches_the_quantiser(cuda_lib):
    """With gamma such that y is exactly representable the codes and scales are
    those of moe_quantize_activations on the stored y."""
    T, H = 6, 512
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    gamma = (torch.arange(H) % 31 + 1).to(torch.bfloat16).cuda()
    for name, sshape, sdt in (("fp8", (T,), torch.float32), ("mxfp8", (T, H // 32), torch.uint8)):
        y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        c, c2 = (torch.empty((T, H), dtype=torch.uint8, device="cuda") for _ in range(2))
        s, s2 = (torch.empty(sshape, dtype=sdt, device="cuda") for _ in range(2))
        capi.moe_rmsnorm_quantize(QUANT[name], x, None, gamma, 2.0 ** -40, None, y, c, s)  # rms rounds to 1
        capi.moe_quantize_activations(QUANT[name], y, c2, s2)
        torch.cuda.synchronize()
        assert torch.equal(y.float(), gamma.float().expand(T, H))
        assert torch.equal(c, c2) and torch.equal(s, s2)


def test_norm_no_rows_graph_and_refusals(cuda_lib):
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    capi.moe_rmsnorm_quantize(None, z, None, g, 1e-6, None, z, None, None)
    x, y = torch.randn((4, 64), device="cuda").bfloat16(), torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.moe_rmsnorm_quantize(None, x, None, g, 1e-6, None, y, None, None)
    for _ in range(2):
        new = torch.randn((4, 64), device="cuda").bfloat16()
        x.copy_(new)
        graph.replay()
        want = torch.empty_like(y)
        capi.moe_rmsnorm_quantize(None, new, None, g, 1e-6, None, want, None, None)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    with pytest.raises(TypeError):
        capi.moe_rmsnorm_quantize(None, x, x.float(), g, 1e-6, None, y, None, None)
    with pytest.raises(ValueError):
        capi.moe_rmsnorm_quantize(None, x, None, g[:32], 1e-6, None, y, None, None)
    with pytest.raises(ValueError):
        capi.moe_rmsnorm_quantize(None, x.t(), None, g[:4], 1e-6, None, y.t(), None, None)
    with pytest.raises(capi.MoEError):
        capi.moe_rmsnorm_quantize(None, x.float(), None, g.float(), 1e-6, None, y.float(), None, None)
    with pytest.raises(capi.MoEError):
        capi.moe_rmsnorm_quantize(None, x, None, g, 0.0, None, y, None, None)


def test_norm_offsets_past_32_bits(cuda_lib):
    """In place over more than 2^32 values: the last rows like the first."""
    T, H = 530_000, 8192
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    rows = torch.randn((4, H), generator=g).bfloat16().cuda()
    at = [0, 1, T - 2, T - 1]
    for i, t in enumerate(at):
        x[t] = rows[i]
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    want = torch.empty_like(rows)
    capi.moe_rmsnorm_quantize(None, rows, None, gamma, 1e-6, None, want, None, None)
    capi.moe_rmsnorm_quantize(None, x, None, gamma, 1e-6, None, x, None, None)
    torch.cuda.synchronize()
    for i, t in enumerate(at):
        assert torch.equal(x[t], want[i])
    assert torch.count_nonzero(x[2:T - 2][::997]).item() == 0


def _norm_of_gamma(gamma, quant):
    """Codes, scales and rows of a row of ones: rms rounds to 1, so the unrounded y is gamma itself."""
    H = gamma.numel()
    x = torch.ones((1, H), dtype=torch.bfloat16, device="cuda")
    codes = torch.empty((1, H), dtype=torch.uint8, device="cuda")
    scale = torch.empty(1, device="cuda") if quant == "fp8" else torch.empty((1, H // 32), dtype=torch.uint8, device="cuda")
    capi.moe_rmsnorm_quantize(QUANT[quant], x, None, gamma, 2.0 ** -40, None, None, codes, scale)
    return codes, scale


def test_norm_fp8_codes_match_the_quantiser_at_ties(cuda_lib):
    """The quotient behind a code is the IEEE one, as moe_quantize_activations
    has it: 39 / (52 / 448) is 336 exactly, a tie that goes to the even code 320.
    Whole numbers up to every amax that bf16 holds exactly, both signs and zeros."""
    H = 512
    for amax in range(1, 257):
        gamma = (torch.arange(H, device="cuda") % (2 * amax + 1) - amax).to(torch.bfloat16)
        gamma[0], gamma[1], gamma[2] = amax, 0.0, -0.0
        codes, scale = _norm_of_gamma(gamma, "fp8")
        want, ws = torch.empty_like(codes), torch.empty_like(scale)
        capi.moe_quantize_activations(QUANT["fp8"], gamma[None], want, ws)
        assert torch.equal(scale, ws) and torch.equal(codes, want), amax


@pytest.mark.parametrize("H", [512, 2048, 7168, 16384])
def test_norm_fp8_codes_are_of_the_ieee_quotient(cuda_lib, H):
    """fp32 gamma: y takes any value. Codes equal e4m3(y / s) with the fp32
    division rounded to nearest, over scales from the subnormal to the largest,
    values next to ties of the codes, and infinities beside finite values."""
    g = torch.Generator(device="cuda").manual_seed(H)
    rand = lambda: torch.rand(H, generator=g, device="cuda")  # noqa: E731
    mid = torch.tensor([(a + b) / 2 for a, b in zip(_E4M3, _E4M3[1:])], device="cuda")
    for i in range(60):
        unit = torch.exp2(torch.tensor(-126.0 + 4.28 * i, device="cuda")) * (1 + rand()[0])
        s = unit / 448
        if i % 2:  # ties of the codes times the scale, and their neighbours
            y = mid[torch.randint(0, mid.numel(), (H,), generator=g, device="cuda")] * s
            y = y.view(torch.int32).add(torch.randint(-2, 3, (H,), generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
        else:
            y = (rand() * 2 - 1) * unit
        y[0] = unit
        if i == 59:
            y[5] = float("inf")
        codes, scale = _norm_of_gamma(y, "fp8")
        amax = y.abs().max()
        want_s = amax / torch.full_like(amax, 448.0)  # by a tensor: by a number torch multiplies by its reciprocal
        assert torch.equal(scale[0], want_s), i
        want = (y / want_s).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = codes[0].view(torch.float8_e4m3fn)
        if i == 59:
            assert torch.isnan(got.float()[5])
            y[5], want = 0.0, want.float().nan_to_num(0.0).to(torch.float8_e4m3fn)
            got = got.float().nan_to_num(0.0).to(torch.float8_e4m3fn)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), i


_E4M3 = sorted({float(v) for v in torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()})


def test_norm_mxfp8_infinities_and_nan(cuda_lib):
    """A NaN spoils its own row; an infinity gives zeros beside it in the whole
    row and NaN in its place. A block's exponent goes by its values that are not
    NaN: those are zeros here, so its byte is 0."""
    T, H = 4, 256
    x, _, gamma = _inputs(T, H, "bf16", seed=1)
    x[0, 3], x[1, 200] = float("nan"), float("-inf")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    c, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    capi.moe_rmsnorm_quantize(QUANT["mxfp8"], x.cuda(), None, gamma.cuda(), 1e-6, None, y, c, s)
    torch.cuda.synchronize()
    y, c, s = y.cpu().float(), c.cpu().view(torch.float8_e4m3fn).float(), s.cpu()
    assert torch.isnan(y[0]).all() and torch.isnan(c[0]).all() and torch.all(s[0] == 0)
    assert torch.isnan(y[1, 200]) and torch.isnan(c[1, 200]) and torch.all(s[1] == 0)
    keep = torch.arange(H) != 200
    assert torch.all(y[1][keep] == 0) and torch.all(c[1][keep] == 0)
    assert torch.isfinite(y[2:]).all() and torch.isfinite(c[2:]).all()


def test_norm_mxfp8_gamma_infinities(cuda_lib):
    """An infinite y that no infinite row made (an infinite gamma): its block
    takes the largest exponent, 128 - 8, the infinity the largest code and its
    finite neighbours vanish; other blocks do not notice."""
    gamma = torch.linspace(-3, 3, 128, device="cuda")
    gamma[40], gamma[50] = float("inf"), float("nan")
    codes, scale = _norm_of_gamma(gamma, "mxfp8")
    c, s = codes[0].cpu().view(torch.float8_e4m3fn).float(), scale[0].cpu()
    assert c[40] == 448 and torch.isnan(c[50]) and s[1] == 127 + 120
    rest = torch.arange(32, 64)
    rest = rest[(rest != 40) & (rest != 50)]
    assert torch.all(c[rest] == 0)
    b = gamma.cpu().double().view(4, 32)
    for i in (0, 2, 3):
        e = math.floor(math.log2(b[i].abs().max())) - 8
        assert s[i] == e + 127
        want = (b[i] / 2.0 ** e).float().to(torch.float8_e4m3fn).float()
        assert torch.equal(c[32 * i:32 * i + 32], want)
