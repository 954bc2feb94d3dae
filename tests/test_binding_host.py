"""The CPython binding and the checked path beside it without a GPU: fake
tensors, and a recording function in place of each entry point."""
import ctypes

import pytest
import torch

from routed_shared_experts_b200 import build, capi

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
NAMES = ("moe_linear", "moe_route", "moe_rmsnorm_quantize")


class T:
    """What the wrappers read of a tensor; an empty one has no address."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, device
        self.device = f"cuda:{device}"

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 0x10000 if self.numel() else 0


@pytest.fixture(params=["binding", "checked"])
def calls(request, monkeypatch):
    """Records the calls that reach the library, by either path."""
    build.build()
    real = capi.lib()
    seen = []

    def recorder(name):
        restype, argtypes = capi.SIGNATURES[name]
        return ctypes.CFUNCTYPE(restype, *argtypes)(lambda *a: (seen.append((name, a)), 0)[1])

    fakes = {n: recorder(n) for n in NAMES}
    if request.param == "binding":
        binding = capi._binding()
        binding.init(tuple(ctypes.cast(fakes[n], ctypes.c_void_p).value for n in NAMES),
                     (torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.bool,
                      torch.int32), lambda: 0, lambda dev: 0)
    else:
        class Nothing:
            def __getattr__(self, name):
                return lambda *a: None
        monkeypatch.setattr(capi, "_BINDING", Nothing())

    class Lib:
        def __getattr__(self, name):
            return fakes[name] if name in fakes else getattr(real, name)

    monkeypatch.setattr(capi, "_LIB", Lib())
    monkeypatch.setattr(capi, "_current_device", lambda: 0)
    monkeypatch.setattr(capi, "_current_stream", lambda dev: 0)
    yield seen
    monkeypatch.undo()
    if request.param == "binding":
        capi._load_binding(real)  # its own functions again


def _linear(x=None, xs=None, ws=None, b=None, r=None, dtype=capi.MOE_DT_BF16, act=0):
    t = {capi.MOE_DT_BF16: BF, capi.MOE_DT_FP8_E4M3: U8}[dtype]
    capi.moe_linear(dtype, T((4, 64), t), xs, T((32, 64), t), ws, b, act, r, T((4, 32), BF))


def _route(b=None, m=None, nv=None, k=2, score=0, n_group=1, topk_group=1, gs=0, ids=None):
    capi.moe_route(T((4, 8), F32), b, m, nv, k, score, n_group, topk_group, gs, True, 1.0,
                   ids or T((4, 2), I32), T((4, 2), F32))


def _norm(quant=None, r=None, ro=None, y=None, c=None, s=None):
    capi.moe_rmsnorm_quantize(quant, T((4, 64), BF), r, T((64,), BF), 1e-6, ro, y, c, s)


def test_well_formed_calls_arrive(calls):
    _linear(b=T((32,), F32), r=T((4, 32), BF))
    _linear(dtype=capi.MOE_DT_FP8_E4M3, xs=T((4,), F32), ws=T((1,), F32))
    _route(b=T((8,), F32), m=T((8,), U8), nv=T((1,), I32))
    _norm(r=T((4, 64), BF), ro=T((4, 64), BF), y=T((4, 64), BF))
    assert [n for n, _ in calls] == ["moe_linear", "moe_linear", "moe_route", "moe_rmsnorm_quantize"]
    assert calls[0][1][8] == calls[0][1][11] == 0x10000  # bias and residual


@pytest.mark.parametrize("call", [
    lambda e: _linear(b=e(F32)), lambda e: _linear(b=e(BF)), lambda e: _linear(xs=e(F32)), lambda e: _linear(ws=e(F32)),
    lambda e: _linear(dtype=capi.MOE_DT_FP8_E4M3, xs=T((4,), F32), ws=e(F32)),
    lambda e: _linear(dtype=capi.MOE_DT_FP8_E4M3, xs=e(F32), ws=T((1,), F32)),
    lambda e: _route(b=e(F32)), lambda e: _route(m=e(U8)), lambda e: _route(nv=e(I32)),
    lambda e: _norm(y=T((4, 64), BF), r=e(BF)), lambda e: _norm(y=T((4, 64), BF), ro=e(BF)),
    lambda e: _norm(ro=T((4, 64), BF), y=e(BF)), lambda e: _norm(y=T((4, 64), BF), c=e(U8)),
    lambda e: _norm(quant=capi.MOE_DT_FP8_E4M3, y=T((4, 64), BF), c=e(U8), s=e(F32)),
])
def test_an_empty_tensor_is_not_an_absent_one(calls, call):
    """An empty bias, mask or output has no address, and the library takes a null
    pointer for an operand that was not given: such a call is refused."""
    with pytest.raises(ValueError):
        call(lambda dtype: T((0,), dtype))
    assert not calls


def test_the_library_does_not_need_the_binding():
    """Without a binding the library loads, and the operators' calls go through the
    checked path: refused arguments come back as before, no rows are no error."""
    import subprocess
    import sys
    code = """
import sys
sys.modules["routed_shared_experts_b200._binding"] = None  # its import raises
import torch
from routed_shared_experts_b200 import capi
assert capi.sorted_capacity(32, 8, 128, 16) > 0
capi._current_device, capi._current_stream = (lambda: 0), (lambda dev: 0)
class T:
    dtype, shape, device = torch.bfloat16, torch.Size((0, 64)), "cuda:0"
    stride = lambda s: (64, 1)
    get_device = lambda s: 0
    data_ptr = lambda s: 0
    numel = lambda s: 0
    is_contiguous = lambda s: True
class W(T):
    shape = torch.Size((8, 64))
    data_ptr = lambda s: 0x10000
class O(T):
    shape = torch.Size((0, 8))
    stride = lambda s: (8, 1)
capi.moe_linear(0, T(), None, W(), None, None, 0, None, O())
try:
    capi.moe_linear(0, T(), None, W(), None, None, 17, None, O())
except capi.MoEError as e:
    print("refused", e.status)
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert res.returncode == 0, res.stderr
    assert res.stdout.split() == ["refused", "-1"]


def test_the_binding_is_optional_and_of_one_abi(monkeypatch, tmp_path, capsys):
    """Its file name carries Python's ABI, and neither a missing compiler nor
    missing headers stop the build."""
    import sysconfig
    assert build.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert ".cpython-" in build.BINDING_PATH
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "b.so"))
    with monkeypatch.context() as m:
        m.setattr(build.shutil, "which", lambda name: None)
        assert build.build_binding(force=True) is None
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        assert build.build_binding(force=True) is None
    assert "checked path" in capsys.readouterr().err and not (tmp_path / "b.so").exists()
    assert build.build_binding() == str(tmp_path / "b.so")


@pytest.mark.parametrize("call", [
    lambda: _route(k=2 + (1 << 32)), lambda: _route(score=1 << 32), lambda: _route(n_group=1 + (1 << 32)),
    lambda: _route(topk_group=1 - (1 << 32)), lambda: _route(gs=1 << 33), lambda: _linear(act=1 << 32),
    lambda: _linear(act=(1 << 32) + 2), lambda: _norm(quant=(1 << 32) - 1, y=T((4, 64), BF)),
    lambda: _norm(quant=1 << 70, y=T((4, 64), BF)), lambda: _linear(act=-(1 << 64)),
    lambda: _linear(dtype=capi.MOE_DT_FP8_E4M3, xs=T((4,), F32), ws=T(((1 << 32) + 1,), F32)),
])
def test_numbers_past_32_bits_are_refused(calls, call):
    """Not taken for their low 32 bits, which may well be valid."""
    with pytest.raises(ValueError):
        call()
    assert not calls


@pytest.mark.parametrize("rows", [1 << 31, (1 << 32) + 4])
def test_rows_past_32_bits_are_refused(calls, rows):
    """2^32 + 4 rows of 16 bits fit a GPU; a call on 4 of them is not the one that
    was made."""
    with pytest.raises(ValueError):
        capi.moe_route(T((rows, 1), BF), None, None, None, 1, 0, 1, 1, 0, True, 1.0, T((rows, 1), I32), T((rows, 1), F32))
    with pytest.raises(ValueError):
        capi.moe_rmsnorm_quantize(None, T((rows, 8), BF), None, T((8,), BF), 1e-6, None, T((rows, 8), BF), None, None)
    with pytest.raises(ValueError):
        capi.moe_linear(capi.MOE_DT_BF16, T((rows, 8), BF), None, T((4, 8), BF), None, None, 0, None, T((rows, 4), BF))
    with pytest.raises(ValueError):
        capi.moe_linear(capi.MOE_DT_BF16, T((4, 8), BF), None, T((rows, 8), BF), None, None, 0, None, T((4, rows), BF))
    assert not calls


def test_import_with_a_torch_built_without_cuda():
    """The size queries and refusals of capi need no CUDA in torch."""
    import subprocess
    import sys
    code = """
import torch
del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
from routed_shared_experts_b200 import capi
assert capi.sorted_capacity(32, 8, 128, 16) > 0
x = torch.zeros((4, 64), dtype=torch.bfloat16)
try:
    capi.moe_linear(capi.MOE_DT_BF16, x, None, x, None, None, 0, None, torch.zeros((4, 4), dtype=torch.bfloat16))
except ValueError:
    print("refused")
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert res.returncode == 0, res.stderr
    assert res.stdout.split() == ["refused"]
