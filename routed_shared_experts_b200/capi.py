"""ctypes binding of ``libmoe_b200.so`` (C ABI in ``include/moe_b200.h``).

Argument marshalling only: each function takes torch tensors (device memory)
and plain numbers, checks device and contiguity, and calls the C entry point of
the same name on the current (or given) CUDA stream. A non-zero status raises
``MoEError``. There is no fallback: if the library is not built, the first call
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

MOE_OK = 0
MOE_DT_BF16, MOE_DT_FP16, MOE_DT_FP8_E4M3, MOE_DT_MXFP8_E4M3, MOE_DT_F32, MOE_DT_MXFP4_E2M1 = 0, 1, 2, 3, 4, 5
MOE_ROUTE_SOFTMAX, MOE_ROUTE_GROUPED_SIGMOID = 0, 1
# block-scaled layer formats (MXFP4 layers keep MXFP8 activations)
MX_FORMATS = ("mxfp8", "mxfp4")
DTYPES = {"bf16": MOE_DT_BF16, "fp16": MOE_DT_FP16, "fp8": MOE_DT_FP8_E4M3, "mxfp8": MOE_DT_MXFP8_E4M3,
          "mxfp4": MOE_DT_MXFP4_E2M1,
          "f32": MOE_DT_F32}
MOE_DT_NONE = -1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_TOP2, MOE_GROUP_MAX = 0, 1
MOE_NO_EXPERT = -(1 << 31)  # expert id of a padding row
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
GROUP_SCORES = {"top2": MOE_GROUP_TOP2, "max": MOE_GROUP_MAX}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_b200.so")

# name -> (restype, argtypes)
_P, _I, _F, _SZ, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_version": (ctypes.c_char_p, []),
    "moe_last_cuda_error": (ctypes.c_char_p, []),
    "moe_supports_output_addend": (_I, []),
    "moe_device_error": (_I, [ctypes.POINTER(ctypes.c_int), _P]),
    "moe_selftest_wait_timeout": (_I, [_P]),
    "moe_sorted_capacity": (_SZ, [_I, _I, _I, _I]),
    "moe_stage2_workspace_bytes": (_SZ, [_I, _I]),
    "moe_stage1_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_mx_weight_scale_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_mx_h_scale_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_mx_pack_weight_scales": (_I, [_I, _P, _P, _I, _I, _I, _P]),
    "moe_router_topk": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "moe_router_gemm_topk": (_I, [_I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
    "moe_align_sort": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_stage1_gemm": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_stage2_gemm_accumulate": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P,
                                        _P, _P, _P]),
    "moe_stage2_gemm_accumulate_static_ws": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                                  _P, _P, _P, _P]),
    "shared_expert_gate_dot": (_I, [_I, _P, _P, _I, _I, _I, _P, _P]),
    "moe_quantize_activations": (_I, [_I, _P, _I, _I, _P, _P, _P]),
    "moe_linear": (_I, [_I, _P, _L, _P, _P, _L, _P, _I, _P, _I, _I, _P, _L, _P, _I, _L, _I, _I, _I, _P]),
    "moe_route": (_I, [_P, _I, _L, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "moe_rmsnorm_quantize": (_I, [_I, _I, _P, _P, _P, _I, _F, _I, _I, _P, _P, _P, _P, _P]),
    "moe_append_shared_slots": (_I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
}

_LIB = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib_ = lib()
        msg = lib_.moe_status_string(status).decode()
        cuda = lib_.moe_last_cuda_error().decode()
        super().__init__(f"{fn}: {msg}" + (f" ({cuda})" if status in (-5, -7) and cuda else ""))
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m routed_shared_experts_b200.build")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _load_binding(handle)
        _LIB = handle
    return _LIB


# None in a torch built without CUDA, which has no tensors that a call could take
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_BINDING = None  # csrc/binding.c: well-formed calls of the small operators without ctypes


class _CheckedPath:
    """Stands in for a binding that is not built: it makes no call, so that every
    one takes the checked path."""

    @staticmethod
    def linear(*args):
        return None

    route = rmsnorm_quantize = linear


def _load_binding(handle):
    global _BINDING
    try:
        from . import _binding
    except ImportError:
        _binding = None
    if _binding is None or _current_device is None:
        _BINDING = _CheckedPath
        return
    address = lambda name: ctypes.cast(getattr(handle, name), ctypes.c_void_p).value  # noqa: E731
    _binding.init((address("moe_linear"), address("moe_route"), address("moe_rmsnorm_quantize")),
                  (torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.bool,
                   torch.int32), _current_device, _current_stream)
    _BINDING = _binding


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _event(ev):
    if ev is None:
        return None
    return ev.cuda_event or None


def _check(name: str, status: int):
    if status != MOE_OK:
        raise MoEError(name, status)


def sorted_capacity(T: int, top_k: int, E: int, block_m: int) -> int:
    return lib().moe_sorted_capacity(T, top_k, E, block_m)


def stage2_workspace_bytes(T: int, H: int) -> int:
    return lib().moe_stage2_workspace_bytes(T, H)


def stage1_workspace_bytes(dtype: int, T: int, top_k: int, E: int, H: int, I: int, block_m: int) -> int:
    return lib().moe_stage1_workspace_bytes(dtype, T, top_k, E, H, I, block_m)


def mx_weight_scale_bytes(which: int, E: int, H: int, I: int) -> int:
    return lib().moe_mx_weight_scale_bytes(which, E, H, I)


def mx_h_scale_bytes(T: int, top_k: int, E: int, I: int, block_m: int) -> int:
    return lib().moe_mx_h_scale_bytes(T, top_k, E, I, block_m)


def moe_mx_pack_weight_scales(which, src, dst, E, H, I, stream=None):
    _check("moe_mx_pack_weight_scales", lib().moe_mx_pack_weight_scales(
        which, _ptr(src), _ptr(dst), E, H, I, _stream(stream)))


def device_error(stream=None) -> int:
    code = ctypes.c_int(0)
    _check("moe_device_error", lib().moe_device_error(ctypes.byref(code), _stream(stream)))
    return code.value


def moe_selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self-test (device error 1 after ~4 s)."""
    _check("moe_selftest_wait_timeout", lib().moe_selftest_wait_timeout(_stream(stream)))


def moe_router_topk(logits, correction_bias, top_k, mode, n_group, topk_group, renormalize,
                    routed_scaling_factor, topk_ids, topk_weights, stream=None):
    T, E = logits.shape
    _check("moe_router_topk", lib().moe_router_topk(
        _ptr(logits), _ptr(correction_bias), T, E, top_k, mode, n_group, topk_group, int(renormalize),
        float(routed_scaling_factor), _ptr(topk_ids), _ptr(topk_weights), _stream(stream)))


def moe_router_gemm_topk(x, w_r, logit_bias, correction_bias, top_k, mode, n_group, topk_group, renormalize,
                         routed_scaling_factor, logits, topk_ids, topk_weights, stream=None):
    T, H = x.shape
    E = w_r.shape[1]
    dtype = MOE_DT_BF16 if x.dtype == torch.bfloat16 else MOE_DT_FP16
    _check("moe_router_gemm_topk", lib().moe_router_gemm_topk(
        dtype, _ptr(x), _ptr(w_r), _ptr(logit_bias), _ptr(correction_bias), T, H, E, top_k, mode, n_group,
        topk_group, int(renormalize), float(routed_scaling_factor), _ptr(logits), _ptr(topk_ids),
        _ptr(topk_weights), _stream(stream)))


def moe_align_sort(topk_ids, E, block_m, sorted_ids, block_expert, expert_counts, expert_offsets, num_padded,
                   stream=None):
    T, k = topk_ids.shape
    _check("moe_align_sort", lib().moe_align_sort(
        _ptr(topk_ids), T, k, E, block_m, _ptr(sorted_ids), _ptr(block_expert), _ptr(expert_counts),
        _ptr(expert_offsets), _ptr(num_padded), _stream(stream)))


def moe_stage1_gemm(dtype, x, x_scale, w13, w13_scale, sorted_ids, block_expert, num_padded, T, top_k, H, I, E,
                    block_m, h, h_scale, ws, stream=None):
    _check("moe_stage1_gemm", lib().moe_stage1_gemm(
        dtype, _ptr(x), _ptr(x_scale), _ptr(w13), _ptr(w13_scale), _ptr(sorted_ids), _ptr(block_expert),
        _ptr(num_padded), T, top_k, H, I, E, block_m, _ptr(h), _ptr(h_scale), _ptr(ws), _stream(stream)))


def moe_stage2_gemm_accumulate(dtype, h, h_scale, w2, w2_scale, weights, weights_dtype, sorted_ids, block_expert,
                               num_padded, T, top_k, H, I, E, block_m, addend, addend_ready, acc_ws, out,
                               stream=None):
    _check("moe_stage2_gemm_accumulate", lib().moe_stage2_gemm_accumulate(
        dtype, _ptr(h), _ptr(h_scale), _ptr(w2), _ptr(w2_scale), _ptr(weights), weights_dtype,
        _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded), T, top_k, H, I, E, block_m, _ptr(addend),
        _event(addend_ready), _ptr(acc_ws), _ptr(out), _stream(stream)))


def moe_stage2_gemm_accumulate_static_ws(dtype, h, h_scale, w2, w2_scale, weights, weights_dtype, sorted_ids,
                                         block_expert, num_padded, T, top_k, H, I, E, block_m, addend,
                                         addend_ready, out, stream=None):
    """Stage 2 with the library's own static workspace (no device allocation
    by the caller or the library); see include/moe_b200.h for its limit."""
    _check("moe_stage2_gemm_accumulate_static_ws", lib().moe_stage2_gemm_accumulate_static_ws(
        dtype, _ptr(h), _ptr(h_scale), _ptr(w2), _ptr(w2_scale), _ptr(weights), weights_dtype,
        _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded), T, top_k, H, I, E, block_m, _ptr(addend),
        _event(addend_ready), _ptr(out), _stream(stream)))


def moe_append_shared_slots(topk_ids, topk_weights, E, m, gate, out_ids, out_weights, stream=None):
    T, k = topk_ids.shape
    gdt = MOE_DT_FP16 if (gate is not None and gate.dtype == torch.float16) else MOE_DT_BF16
    _check("moe_append_shared_slots", lib().moe_append_shared_slots(
        _ptr(topk_ids), _ptr(topk_weights), T, k, E, m, _ptr(gate), gdt, _ptr(out_ids), _ptr(out_weights),
        _stream(stream)))


def moe_quantize_activations(dtype, x, codes, scale, stream=None):
    T, H = x.shape
    _check("moe_quantize_activations", lib().moe_quantize_activations(
        dtype, _ptr(x), T, H, _ptr(codes), _ptr(scale), _stream(stream)))


def shared_expert_gate_dot(dtype, x, w, apply_sigmoid, out, stream=None):
    T, K = x.shape
    _check("shared_expert_gate_dot", lib().shared_expert_gate_dot(
        dtype, _ptr(x), _ptr(w), T, K, int(apply_sigmoid), _ptr(out), _stream(stream)))


_FLOAT_DT = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_FP16, torch.float32: MOE_DT_F32}
_OPERAND_DT = {MOE_DT_BF16: (torch.bfloat16,), MOE_DT_FP16: (torch.float16,),
               MOE_DT_FP8_E4M3: (torch.uint8, torch.float8_e4m3fn)}
_F32, _I32, _BYTES = (torch.float32,), (torch.int32,), (torch.uint8, torch.bool)
_CODES = (torch.uint8, torch.float8_e4m3fn)

# The wrappers below are called once per operator of a decode step, whose kernels
# take a few microseconds. The binding makes a well-formed call (None: it is not
# one); the checks here name what is wrong with the others, and make the calls
# that the binding leaves alone (no rows).


def _binding():
    lib()
    return _BINDING


def _refuse_device(first, others):
    for t in others:
        if t is not None and t.get_device() != first.get_device():
            raise ValueError("tensors must live on one CUDA device")
    raise ValueError(f"tensors on {first.device}: they must live on the current CUDA device")


def _device(first, *others):
    """Index of the one device that every tensor lives on, the current one (the
    calls launch on its stream)."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            _refuse_device(first, others)
    if dev < 0 or dev != _current_device():
        _refuse_device(first, others)
    return dev


def _rows(t, name, rows, cols, types):
    """Row stride in elements of a [rows, cols] tensor whose rows are dense."""
    if t.dtype in types and t.shape == (rows, cols):
        ld, step = t.stride()
        if step == 1 or cols == 1:
            if rows < 2:
                return -(-cols // 16) * 16  # the stride of a single row says nothing
            if ld >= cols:
                return ld
        elif rows == 0:
            return -(-cols // 16) * 16
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    _check_type(t, name, types)
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")


def _check_type(t, name, types):
    if t.dtype not in types:
        raise TypeError(f"{name} has type {t.dtype}")


def _int(v, name):
    """A number that the entry point takes in 32 bits (ctypes would cut it to them)."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} is {v}, past 32 bits")
    return v


def _vec(t, name, n, types):
    """Address of a dense tensor of n elements (None: NULL)."""
    if t is None:
        return None
    if t.dtype in types and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    _check_type(t, name, types)
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    raise ValueError(f"{name} must be contiguous")


def moe_linear(dtype, x, x_scale, w, w_scale, bias, act, residual, out, stream=None):
    """out = act((x . w^T) * x_scale * w_scale + bias) + residual; x [T,K], w
    [N,K], residual and out [T,N] may be views with any row stride."""
    status = (_BINDING or _binding()).linear(dtype, x, x_scale, w, w_scale, bias, act, residual, out, stream)
    if status is not None:
        if status:
            raise MoEError("moe_linear", status)
        return
    types = _OPERAND_DT.get(dtype)
    if types is None:
        raise MoEError("moe_linear", -2)
    T, K = x.shape
    N = w.shape[0]
    out_type = out.dtype
    ldx = _rows(x, "x", T, K, types)
    ldw = _rows(w, "w", N, K, types)
    ldo = _rows(out, "out", T, N, _FLOAT_DT)
    dev = _device(x, w, out, residual, bias, x_scale, w_scale)
    ldr, pr, pb, bias_dt, ws_rows = 0, None, None, MOE_DT_F32, 1
    if residual is not None:
        ldr = _rows(residual, "residual", T, N, (out_type,))
        pr = residual.data_ptr()
    if bias is not None:
        pb = _vec(bias, "bias", N, _FLOAT_DT)
        bias_dt = _FLOAT_DT[bias.dtype]
    if w_scale is not None:
        ws_rows = w_scale.numel()
        if not ws_rows:  # its null address would read as no scale
            raise ValueError("w_scale has no elements")
    status = (_LIB or lib()).moe_linear(
        dtype, x.data_ptr(), ldx, _vec(x_scale, "x_scale", T, _F32), w.data_ptr(), ldw,
        _vec(w_scale, "w_scale", ws_rows, _F32), _int(ws_rows, "w_scale's length"), pb, bias_dt, _int(act, "act"), pr,
        ldr, out.data_ptr(), _FLOAT_DT[out_type], ldo, _int(T, "T"), _int(N, "N"), _int(K, "K"), _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise MoEError("moe_linear", status)


def moe_route(logits, bias, expert_mask, num_valid, top_k, score, n_group, topk_group, group_score, renormalize,
              routed_scaling_factor, topk_ids, topk_weights, stream=None):
    """Routing from softmax or sigmoid scores; logits [T,E] may be a view with
    any row stride."""
    status = (_BINDING or _binding()).route(logits, bias, expert_mask, num_valid, top_k, score, n_group, topk_group,
                                            group_score, renormalize, routed_scaling_factor, topk_ids, topk_weights,
                                            stream)
    if status is not None:
        if status:
            raise MoEError("moe_route", status)
        return
    T, E = logits.shape
    ld = _rows(logits, "logits", T, E, _FLOAT_DT)
    dev = _device(logits, topk_ids, topk_weights, bias, expert_mask, num_valid)
    n = T * top_k
    status = (_LIB or lib()).moe_route(
        logits.data_ptr(), _FLOAT_DT[logits.dtype], ld, bias if bias is None else _vec(bias, "bias", E, _F32),
        expert_mask if expert_mask is None else _vec(expert_mask, "expert_mask", E, _BYTES),
        num_valid if num_valid is None else _vec(num_valid, "num_valid", 1, _I32), _int(T, "T"), _int(E, "E"),
        _int(top_k, "top_k"), _int(score, "score"), _int(n_group, "n_group"), _int(topk_group, "topk_group"),
        _int(group_score, "group_score"), renormalize, routed_scaling_factor, _vec(topk_ids, "topk_ids", n, _I32),
        _vec(topk_weights, "topk_weights", n, _F32), _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise MoEError("moe_route", status)


def moe_rmsnorm_quantize(quant, x, residual, gamma, eps, residual_out, y, codes, scale, stream=None):
    """z = x + residual -> residual_out; RMS norm of z -> y and / or codes with
    scale. ``quant``: MOE_DT_FP8_E4M3, MOE_DT_MXFP8_E4M3, or None."""
    status = (_BINDING or _binding()).rmsnorm_quantize(MOE_DT_NONE if quant is None else quant, x, residual, gamma, eps,
                                                       residual_out, y, codes, scale, stream)
    if status is not None:
        if status:
            raise MoEError("moe_rmsnorm_quantize", status)
        return
    T, H = x.shape
    n = T * H
    xt = x.dtype
    same = (xt,)
    mx = quant == MOE_DT_MXFP8_E4M3
    dev = _device(x, gamma, y, residual, residual_out, codes, scale)
    status = (_LIB or lib()).moe_rmsnorm_quantize(
        _FLOAT_DT.get(xt, MOE_DT_F32), MOE_DT_NONE if quant is None else _int(quant, "quant"), _vec(x, "x", n, same),
        residual if residual is None else _vec(residual, "residual", n, same),
        _vec(gamma, "gamma", H, (xt, torch.float32)), _FLOAT_DT.get(gamma.dtype, MOE_DT_F32), eps, _int(T, "T"),
        _int(H, "H"),
        residual_out if residual_out is None else _vec(residual_out, "residual_out", n, same),
        y if y is None else _vec(y, "y", n, same), codes if codes is None else _vec(codes, "codes", n, _CODES),
        scale if scale is None else _vec(scale, "scale", n // 32 if mx else T, (torch.uint8,) if mx else _F32),
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise MoEError("moe_rmsnorm_quantize", status)
