"""What the shared gate of a layer reads, without a GPU: the calls of a layer
with every operand format are recorded in place of being launched."""
import pytest
import torch

from routed_shared_experts_b200 import block, build, capi, configs, layer, synth

CFG = dict(T=6, H=256, E=8, top_k=2, I=128, Is=128, block_m=16, n_group=1, topk_group=1, shared_gate=True)
BASES = {"bf16": configs.DECODE_BF16, "fp8": configs.FP8_A8W8, "mxfp8": configs.MXFP8_PREFILL,
         "mxfp4": configs.MXFP4_DECODE}


class _Stream:
    def __init__(self, *a, **k):
        pass

    def __getattr__(self, name):
        return lambda *a, **k: None


@pytest.fixture
def calls(monkeypatch):
    build.build()
    seen = []
    for name in [n for n in dir(capi) if n.startswith("moe_") or n == "shared_expert_gate_dot"]:
        monkeypatch.setattr(capi, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "Event", _Stream)
    return seen


def _layer(kind, dtype, **kw):
    cfg = configs.small(BASES[dtype], name=f"gate_{dtype}", seed=3, **CFG)
    inp = synth.make_layer_inputs(cfg)
    return cfg, inp, kind(cfg, inp, device="cpu", **kw)


def _gate_call(calls):
    (args,) = [a for n, a in calls if n == "shared_expert_gate_dot"]
    return args


@pytest.mark.parametrize("dtype", sorted(BASES))
@pytest.mark.parametrize("kind", [layer.MoELayer, layer.FusedSharedMoELayer])
def test_gate_reads_16_bit_rows(calls, kind, dtype):
    """The gate's dot reads T * H values of 16 bits: never the codes of an 8-bit
    layer, which are half as many bytes."""
    cfg, inp, lay = _layer(kind, dtype)
    calls.clear()
    lay.forward(_Stream())
    dt, x, w, sigmoid, out = _gate_call(calls)[:5]
    assert dt == capi.MOE_DT_BF16 and x.dtype == w.dtype == out.dtype == torch.bfloat16
    assert tuple(x.shape) == (cfg.T, cfg.H) and out.numel() == cfg.T
    assert x is inp["x" if dtype == "bf16" else "x_r"]


@pytest.mark.parametrize("dtype", ["fp8", "mxfp8"])
def test_gate_reads_the_rows_that_are_quantised(calls, dtype):
    cfg, inp, lay = _layer(layer.MoELayer, dtype, quantize_x=True)
    calls.clear()
    lay.forward(_Stream())
    assert _gate_call(calls)[1] is inp["x_r"]


@pytest.mark.parametrize("dtype", sorted(BASES))
@pytest.mark.parametrize("kind", [layer.MoELayer, layer.FusedSharedMoELayer])
def test_block_feeds_the_gate(calls, kind, dtype):
    """The rows that the block's norm writes are the ones the gate reads."""
    cfg, inp, lay = _layer(kind, dtype)
    b = block.MoEBlock(lay, {"gamma": None, "w_r": None, "w_o": None}, None, None)
    calls.clear()
    b.forward(_Stream())
    (norm,) = [a for n, a in calls if n == "moe_rmsnorm_quantize"]
    assert norm[6] is b.y and _gate_call(calls)[1] is b.y
    assert norm[7] is (None if dtype == "bf16" else inp["x"])


@pytest.mark.parametrize("kind", [layer.MoELayer, layer.FusedSharedMoELayer])
def test_gated_8_bit_layer_without_16_bit_rows_is_refused(calls, kind):
    cfg = configs.small(BASES["fp8"], name="gate_refused", seed=3, **CFG)
    inp = synth.make_layer_inputs(cfg)
    for bad in (None, inp["x"], inp["x_r"][:3], inp["x_r"].float()):
        with pytest.raises(ValueError, match="x_r"):
            kind(cfg, dict(inp, x_r=bad), device="cpu")
    ungated = configs.small(cfg, shared_gate=False)
    kind(ungated, dict(inp, x_r=None), device="cpu")
