"""ctypes binding of libm3.so (argument marshalling only).

Each function has the name of the C entry point it calls and takes torch
tensors (CUDA, float32, contiguous) in the C argument order; it passes their
device pointers and the current CUDA stream, and raises M3Error on a nonzero
status. No step of the computation runs here: if libm3.so is missing the call
fails loudly, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libm3.so")

M3_OK = 0
M3_ERR_INVALID_ARGUMENT = 1
M3_ERR_UNALIGNED = 2
M3_ERR_WORKSPACE = 3
M3_ERR_CUDA = 4
M3_ERR_TIMEOUT = 5
M3_ERR_DEVICE_STATE = 6
M3_MATH_FP32 = 0
M3_MATH_TF32 = 1
M3_DTYPE_FP32 = 0
M3_DTYPE_BF16 = 1

EXPORTED = ("m3_preprocess", "m3_preprocess_backward_workspace", "m3_preprocess_backward",
            "m3_siso_forward_workspace", "m3_siso_forward",
            "m3_siso_forward_static", "m3_siso_forward_static_status",
            "m3_siso_forward_packed_workspace", "m3_siso_forward_packed",
            "m3_mimo_forward_packed_workspace", "m3_mimo_forward_packed", "m3_siso_prefill_workspace", "m3_siso_prefill",
            "m3_mimo_prefill_workspace", "m3_mimo_prefill",
            "m3_siso_backward_workspace", "m3_siso_backward",
            "m3_mimo_backward_workspace", "m3_mimo_backward",
            "m3_mimo_forward_workspace", "m3_mimo_forward", "m3_siso_step", "m3_mimo_step",
            "m3_qk_norm_rope", "m3_qk_norm_rope_backward_workspace", "m3_qk_norm_rope_backward",
            "m3_linear_attention_forward_workspace", "m3_linear_attention_forward",
            "m3_linear_attention_step", "m3_linear_attention_backward_workspace",
            "m3_linear_attention_backward",
            "m3_workspace_status", "m3_selftest_wait_timeout", "m3_status_string",
            "m3_launch_count")


class M3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class PreprocessConfig(ctypes.Structure):
    """m3_preprocess_config (mirrors Mamba3PreprocessConfig)."""
    _fields_ = [("inner_size", ctypes.c_int64), ("state_size", ctypes.c_int64),
                ("num_heads", ctypes.c_int64), ("num_rope_angles", ctypes.c_int64),
                ("num_groups", ctypes.c_int64), ("mimo_rank", ctypes.c_int64),
                ("epsilon", ctypes.c_float), ("dt_min", ctypes.c_float),
                ("dt_max", ctypes.c_float), ("a_floor", ctypes.c_float)]


class SsmConfig(ctypes.Structure):
    """m3_ssm_config (mirrors SsmConfig, plus math_mode)."""
    _fields_ = [("batch_size", ctypes.c_int64), ("sequence_length", ctypes.c_int64),
                ("num_heads", ctypes.c_int64), ("num_groups", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("state_size", ctypes.c_int64),
                ("num_rope_angles", ctypes.c_int64), ("mimo_rank", ctypes.c_int64),
                ("has_z", ctypes.c_int32), ("has_d", ctypes.c_int32),
                ("has_output_norm", ctypes.c_int32), ("math_mode", ctypes.c_int32)]


class QkNormRopeConfig(ctypes.Structure):
    """m3_qk_norm_rope_config."""
    _fields_ = [("rows", ctypes.c_int64), ("num_q_heads", ctypes.c_int64),
                ("num_k_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("num_rope_angles", ctypes.c_int64), ("max_positions", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
                ("epsilon", ctypes.c_float), ("dtype", ctypes.c_int32)]


class LinearAttentionConfig(ctypes.Structure):
    """m3_linear_attention_config."""
    _fields_ = [("batch_size", ctypes.c_int64), ("sequence_length", ctypes.c_int64),
                ("total_rows", ctypes.c_int64), ("num_heads", ctypes.c_int64),
                ("num_groups", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("state_size", ctypes.c_int64), ("num_slots", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


def ssm_config(d: dict, math_mode: int = M3_MATH_FP32) -> SsmConfig:
    return SsmConfig(d["batch_size"], d["sequence_length"], d["num_heads"], d["num_groups"],
                     d["head_dim"], d["state_size"], d["num_rope_angles"], d.get("mimo_rank", 1),
                     int(d.get("has_z", 1)), int(d.get("has_d", 1)),
                     int(d.get("has_output_norm", 0)), int(d.get("math_mode", math_mode)))


def preprocess_config(**kw) -> PreprocessConfig:
    return PreprocessConfig(kw["inner_size"], kw["state_size"], kw["num_heads"],
                            kw["num_rope_angles"], kw["num_groups"], kw["mimo_rank"],
                            kw["epsilon"], kw["dt_min"], kw["dt_max"], kw["a_floor"])


_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p


def load_library():
    """Loads libm3.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libm3.so not built ({LIB_PATH}); run "
                               "selective_state_space_mamba3_gb300.build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        cfgp = ctypes.POINTER(SsmConfig)
        lib.m3_preprocess.argtypes = [ctypes.POINTER(PreprocessConfig), ctypes.c_int64] + [_vp] * 11
        lib.m3_preprocess_backward_workspace.argtypes = [ctypes.POINTER(PreprocessConfig),
                                                         ctypes.c_int64,
                                                         ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_preprocess_backward.argtypes = ([ctypes.POINTER(PreprocessConfig), ctypes.c_int64] +
                                               [_vp] * 13 + [ctypes.c_size_t, _vp])
        lib.m3_siso_forward_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_mimo_forward_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_siso_forward.argtypes = [cfgp] + [_vp] * 13 + [ctypes.c_size_t, _vp]
        lib.m3_mimo_forward.argtypes = [cfgp] + [_vp] * 17 + [ctypes.c_size_t, _vp]
        lib.m3_siso_forward_static.argtypes = [cfgp] + [_vp] * 12 + [_vp]
        lib.m3_siso_forward_static_status.argtypes = [_vp]
        pcfgp = ctypes.POINTER(PreprocessConfig)
        lib.m3_siso_forward_packed_workspace.argtypes = [cfgp, pcfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_siso_forward_packed.argtypes = [cfgp, pcfgp] + [_vp] * 7 + [ctypes.c_size_t, _vp]
        lib.m3_mimo_forward_packed_workspace.argtypes = [cfgp, pcfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_mimo_forward_packed.argtypes = [cfgp, pcfgp] + [_vp] * 11 + [ctypes.c_size_t, _vp]
        lib.m3_siso_prefill_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_mimo_prefill_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_siso_prefill.argtypes = [cfgp] + [_vp] * 17 + [ctypes.c_size_t, _vp]
        lib.m3_mimo_prefill.argtypes = [cfgp] + [_vp] * 21 + [ctypes.c_size_t, _vp]
        lib.m3_siso_step.argtypes = [cfgp] + [_vp] * 16 + [_vp]
        lib.m3_siso_backward_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_siso_backward.argtypes = [cfgp] + [_vp] * 24 + [ctypes.c_size_t, _vp]
        lib.m3_mimo_backward_workspace.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        lib.m3_mimo_backward.argtypes = [cfgp] + [_vp] * 32 + [ctypes.c_size_t, _vp]
        lib.m3_mimo_step.argtypes = [cfgp] + [_vp] * 20 + [_vp]
        rope, la = ctypes.POINTER(QkNormRopeConfig), ctypes.POINTER(LinearAttentionConfig)
        szp = ctypes.POINTER(ctypes.c_size_t)
        lib.m3_qk_norm_rope.argtypes = [rope] + [_vp] * 10
        lib.m3_qk_norm_rope_backward_workspace.argtypes = [rope, szp]
        lib.m3_qk_norm_rope_backward.argtypes = [rope] + [_vp] * 14 + [ctypes.c_size_t, _vp]
        lib.m3_linear_attention_forward_workspace.argtypes = [la, szp]
        lib.m3_linear_attention_forward.argtypes = [la] + [_vp] * 9 + [ctypes.c_size_t, _vp]
        lib.m3_linear_attention_step.argtypes = [la] + [_vp] * 8
        lib.m3_linear_attention_backward_workspace.argtypes = [la, szp]
        lib.m3_linear_attention_backward.argtypes = [la] + [_vp] * 13 + [ctypes.c_size_t, _vp]
        lib.m3_workspace_status.argtypes = [_vp, ctypes.c_size_t, _vp]
        lib.m3_selftest_wait_timeout.argtypes = [_vp, ctypes.c_size_t, ctypes.c_int64, _vp]
        lib.m3_status_string.argtypes = [ctypes.c_int]
        lib.m3_status_string.restype = ctypes.c_char_p
        lib.m3_launch_count.restype = ctypes.c_uint64
        for name in EXPORTED:
            if name not in ("m3_status_string", "m3_launch_count"):
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().m3_status_string(int(status)).decode()


def launch_count() -> int:
    return int(load_library().m3_launch_count())


def _ptr(t):
    """Device pointer of a CUDA float32 contiguous tensor (None passes NULL)."""
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.device.type != "cuda" or t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError("operands must be contiguous float32 CUDA tensors")
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(status, where):
    if status != M3_OK:
        raise M3Error(status, where)


def m3_preprocess(cfg: PreprocessConfig, rows, projected, dt_bias, x, z, bh, ch, dt, adt, trap,
                  angle, stream=None):
    lib = load_library()
    _check(lib.m3_preprocess(ctypes.byref(cfg), int(rows), *[_ptr(t) for t in (
        projected, dt_bias, x, z, bh, ch, dt, adt, trap, angle)], _stream(stream)), "m3_preprocess")


def m3_preprocess_backward_workspace(cfg: PreprocessConfig, rows) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_preprocess_backward_workspace(ctypes.byref(cfg), int(rows),
                                                           ctypes.byref(n)),
           "m3_preprocess_backward_workspace")
    return n.value


def m3_preprocess_backward(cfg: PreprocessConfig, rows, projected, dt_bias, grad_x, grad_z,
                           grad_bh, grad_ch, grad_dt, grad_adt, grad_trap, grad_angle,
                           grad_projected, grad_dt_bias, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_preprocess_backward(ctypes.byref(cfg), int(rows), *[_ptr(t) for t in (
        projected, dt_bias, grad_x, grad_z, grad_bh, grad_ch, grad_dt, grad_adt, grad_trap,
        grad_angle, grad_projected, grad_dt_bias)], wp, wn, _stream(stream)),
        "m3_preprocess_backward")


def m3_siso_forward_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_siso_forward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_siso_forward_workspace")
    return n.value


def m3_mimo_forward_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_mimo_forward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_mimo_forward_workspace")
    return n.value


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def m3_siso_forward(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, out,
                    workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_siso_forward(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, out)], wp, wn, _stream(stream)),
        "m3_siso_forward")


def m3_siso_forward_static(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                           out, stream=None):
    """m3_siso_forward without a workspace: the library's fixed device scratch
    array is used instead (for callers that cannot allocate device memory)."""
    _check(load_library().m3_siso_forward_static(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, out)], _stream(stream)),
        "m3_siso_forward_static")


def m3_siso_forward_packed_workspace(cfg: SsmConfig, pcfg: PreprocessConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_siso_forward_packed_workspace(ctypes.byref(cfg), ctypes.byref(pcfg),
                                                            ctypes.byref(n)),
           "m3_siso_forward_packed_workspace")
    return n.value


def m3_siso_forward_packed(cfg: SsmConfig, pcfg: PreprocessConfig, projected, dt_bias, c_bias,
                           b_bias, d, out, workspace=None, stream=None):
    """m3_preprocess and m3_siso_forward in one call (packed projection in,
    scan output out)."""
    wp, wn = _ws(workspace)
    _check(load_library().m3_siso_forward_packed(ctypes.byref(cfg), ctypes.byref(pcfg), *[
        _ptr(t) for t in (projected, dt_bias, c_bias, b_bias, d, out)], wp, wn, _stream(stream)),
        "m3_siso_forward_packed")


def m3_mimo_forward_packed_workspace(cfg: SsmConfig, pcfg: PreprocessConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_mimo_forward_packed_workspace(ctypes.byref(cfg), ctypes.byref(pcfg),
                                                            ctypes.byref(n)),
           "m3_mimo_forward_packed_workspace")
    return n.value


def m3_mimo_forward_packed(cfg: SsmConfig, pcfg: PreprocessConfig, projected, dt_bias, c_bias,
                           b_bias, d, mimo_x, mimo_z, mimo_o, norm_weight, out, workspace=None,
                           stream=None):
    """m3_preprocess and m3_mimo_forward in one call."""
    wp, wn = _ws(workspace)
    _check(load_library().m3_mimo_forward_packed(ctypes.byref(cfg), ctypes.byref(pcfg), *[
        _ptr(t) for t in (projected, dt_bias, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
                          norm_weight, out)], wp, wn, _stream(stream)), "m3_mimo_forward_packed")


def m3_siso_forward_static_status(stream=None) -> int:
    """Status word of the last m3_siso_forward_static call on the current
    device (waits for the stream): M3_OK, M3_ERR_TIMEOUT or M3_ERR_DEVICE_STATE."""
    return int(load_library().m3_siso_forward_static_status(_stream(stream)))


def m3_siso_prefill_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_siso_prefill_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_siso_prefill_workspace")
    return n.value


def m3_mimo_prefill_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_mimo_prefill_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_mimo_prefill_workspace")
    return n.value


def m3_siso_prefill(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                    ssm_state, angle_state, k_state, v_state, out, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_siso_prefill(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, ssm_state, angle_state, k_state,
        v_state, out)], wp, wn, _stream(stream)), "m3_siso_prefill")


def m3_siso_backward_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_siso_backward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_siso_backward_workspace")
    return n.value


def m3_siso_backward(cfg: SsmConfig, grad_out, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias,
                     d, grad_c, grad_b, grad_x, grad_z, grad_adt, grad_dt, grad_trap, grad_angle,
                     grad_c_bias, grad_b_bias, grad_d, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_siso_backward(ctypes.byref(cfg), *[_ptr(t) for t in (
        grad_out, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, grad_c, grad_b, grad_x,
        grad_z, grad_adt, grad_dt, grad_trap, grad_angle, grad_c_bias, grad_b_bias, grad_d)],
        wp, wn, _stream(stream)), "m3_siso_backward")


def m3_mimo_backward_workspace(cfg: SsmConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_mimo_backward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_mimo_backward_workspace")
    return n.value


def m3_mimo_backward(cfg: SsmConfig, grad_out, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias,
                     d, mimo_x, mimo_z, mimo_o, norm_weight, grad_c, grad_b, grad_x, grad_z,
                     grad_adt, grad_dt, grad_trap, grad_angle, grad_c_bias, grad_b_bias, grad_d,
                     grad_mimo_x, grad_mimo_z, grad_mimo_o, grad_norm_weight, workspace=None,
                     stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_mimo_backward(ctypes.byref(cfg), *[_ptr(t) for t in (
        grad_out, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
        norm_weight, grad_c, grad_b, grad_x, grad_z, grad_adt, grad_dt, grad_trap, grad_angle,
        grad_c_bias, grad_b_bias, grad_d, grad_mimo_x, grad_mimo_z, grad_mimo_o,
        grad_norm_weight)], wp, wn, _stream(stream)), "m3_mimo_backward")


def m3_mimo_prefill(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x,
                    mimo_z, mimo_o, norm_weight, ssm_state, angle_state, k_state, v_state, out,
                    workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_mimo_prefill(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
        norm_weight, ssm_state, angle_state, k_state, v_state, out)], wp, wn, _stream(stream)),
        "m3_mimo_prefill")


def m3_mimo_forward(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x,
                    mimo_z, mimo_o, norm_weight, out, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_mimo_forward(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
        norm_weight, out)], wp, wn, _stream(stream)), "m3_mimo_forward")


def m3_siso_step(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, ssm_state,
                 angle_state, k_state, v_state, out, stream=None):
    _check(load_library().m3_siso_step(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, ssm_state, angle_state, k_state,
        v_state, out)], _stream(stream)), "m3_siso_step")


def m3_mimo_step(cfg: SsmConfig, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x,
                 mimo_z, mimo_o, norm_weight, ssm_state, angle_state, k_state, v_state, out,
                 stream=None):
    _check(load_library().m3_mimo_step(ctypes.byref(cfg), *[_ptr(t) for t in (
        c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
        norm_weight, ssm_state, angle_state, k_state, v_state, out)], _stream(stream)),
        "m3_mimo_step")


def m3_workspace_status(workspace, stream=None) -> int:
    wp, wn = _ws(workspace)
    return int(load_library().m3_workspace_status(wp, wn, _stream(stream)))


def m3_selftest_wait_timeout(workspace, budget_cycles, stream=None):
    wp, wn = _ws(workspace)
    _check(load_library().m3_selftest_wait_timeout(wp, wn, int(budget_cycles), _stream(stream)),
           "m3_selftest_wait_timeout")


# --- linear-attention operators --------------------------------------------------
# Activations are CUDA tensors of float32 or bfloat16 shaped [..., heads, width]
# whose heads are adjacent; the leading dimensions are the rows, any uniform
# stride apart (views into packed rows are fine). The calls for single tokens
# take a few microseconds on the GPU, so every check has a short form for the
# tensor that is as expected: no import, no attribute twice.

_types = None


def _torch_types():
    """(float32, bfloat16, int32, the raw handle of a device's current stream, the current device)."""
    global _types
    if _types is None:
        import torch
        _types = (torch.float32, torch.bfloat16, torch.int32,
                  getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                  (lambda i: torch.cuda.current_stream(i).cuda_stream),
                  getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device)
    return _types


def _device_of(t):
    """The device of a call, from one of its operands: the library launches on the calling
    thread's current device, so it has to be that one."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError("activations must be CUDA tensors")
    current = _torch_types()[4]()
    if dev != current:
        raise ValueError(f"operands on cuda:{dev}, but the current device is cuda:{current}")
    return dev


def _other_device(t, dev):
    return ValueError(f"operands on different devices: cuda:{t.get_device()} and cuda:{dev}")


def _stream_of(stream, dev):
    """The given stream, or the device's current one."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _torch_types()[3](dev)


def _ws_on(workspace, dev):
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev:
        if workspace.get_device() < 0:
            raise TypeError("the workspace must be a CUDA tensor")
        raise _other_device(workspace, dev)
    return _ws(workspace)


def _row_stride(t):
    """Elements from one row of [..., heads, width] to the next."""
    if t.dim() < 3:
        raise TypeError("expected a tensor [..., heads, width]")
    shape, st = t.shape, t.stride()
    heads, width = shape[-2], shape[-1]
    if t.numel() == 0:
        return heads * width
    if (width > 1 and st[-1] != 1) or (heads > 1 and st[-2] != width):
        raise TypeError("the heads of a row must be adjacent in memory")
    step, run = None, 1
    for size, stride in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if size > 1:
            if step is None:
                step = stride
            elif stride != step * run:
                raise TypeError("the rows of an operand must be evenly spaced")
        run *= size
    return heads * width if step is None else step


def _dtype(t):
    types = _torch_types()
    if t.dtype == types[0]:
        return M3_DTYPE_FP32
    if t.dtype == types[1]:
        return M3_DTYPE_BF16
    raise TypeError("activations must be float32 or bfloat16")


def _act(t, dtype, rows, heads, width, stride, dev):
    """Device pointer of an activation; its shape and stride must be the config's."""
    stride = stride or heads * width
    if (t.dtype is dtype and t.get_device() == dev and rows and t.shape == (rows, heads, width) and
            t.stride() == (stride, width, 1)):
        return t.data_ptr()
    if not t.is_cuda or t.dtype != dtype:
        raise TypeError("activations must be CUDA tensors of the config's type")
    if t.get_device() != dev:
        raise _other_device(t, dev)
    n = t.numel()
    if tuple(t.shape[-2:]) != (heads, width) or n != rows * heads * width:
        raise ValueError(f"expected {rows} rows of [{heads}, {width}], got {tuple(t.shape)}")
    if _row_stride(t) != stride and rows > 1:
        raise ValueError("row stride differs from the config's")
    return t.data_ptr() if n > 0 else None


def _ends(shape):
    out, run = [], 1
    for size in reversed(shape):
        run *= size
        out.append(run)
    return out


def _same_memory(shape, want):
    """Whether a dense tensor of `shape` lies in memory as one of `want`: it may merge
    dimensions, split the first one and have others of one value."""
    mine, ends = _ends(shape) or [1], _ends(want)
    inner = ends[-2] if len(ends) > 1 else 1
    return mine[-1:] == ends[-1:] and all(
        x == 1 or x in ends or (x > inner and (inner == 1 or inner in mine)) for x in mine)


def _dense(t, dtype, shape, dev):
    """Device pointer of a dense operand of one type and shape (None passes NULL)."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"expected a contiguous {dtype} CUDA tensor")
        raise _other_device(t, dev)
    if t.shape != shape:
        if t.numel() == 0 and 0 in shape:
            return None
        if not _same_memory(t.shape, shape):
            raise ValueError(f"expected a tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def qk_norm_rope_config(q, k, *, num_rope_angles, max_positions=0, epsilon=1e-6, q_out=None,
                        k_out=None) -> QkNormRopeConfig:
    """The config of q [..., heads, head_dim] and k (either may be None); outputs
    are dense unless q_out / k_out say otherwise."""
    some = q if q is not None else k
    heads = [0 if t is None else t.shape[-2] for t in (q, k)]
    strides = [0 if t is None else _row_stride(t) for t in (q, k, q_out, k_out)]
    width = some.shape[-1]
    return QkNormRopeConfig(some.numel() // max(1, some.shape[-2] * width), *heads, width,
                            num_rope_angles, max_positions, *strides, epsilon, _dtype(some))


def _rope_tables(cfg, types, rows, d, q_weight, k_weight, cos_table, sin_table, positions, dev):
    f32, a = types[0], cfg.num_rope_angles
    table = (cfg.max_positions, a) if a else (0,)
    return (_dense(q_weight, f32, (d,), dev), _dense(k_weight, f32, (d,), dev),
            _dense(cos_table, f32, table, dev), _dense(sin_table, f32, table, dev),
            _dense(positions, types[2], (rows,), dev))


def _rope_shapes(cfg, some):
    """(types, activations' type, device, rows, query heads, key heads, width) of a call."""
    types = _torch_types()
    return (types, types[cfg.dtype], _device_of(some), cfg.rows, cfg.num_q_heads, cfg.num_k_heads,
            cfg.head_dim)


def m3_qk_norm_rope(cfg: QkNormRopeConfig, q, k, q_weight, k_weight, cos_table, sin_table,
                    positions, q_out, k_out, stream=None):
    types, dt, dev, rows, hq, hk, d = _rope_shapes(cfg, k if q is None else q)
    _check(load_library().m3_qk_norm_rope(
        ctypes.byref(cfg), _act(q, dt, rows, hq, d, cfg.q_stride, dev) if hq else None,
        _act(k, dt, rows, hk, d, cfg.k_stride, dev) if hk else None,
        *_rope_tables(cfg, types, rows, d, q_weight, k_weight, cos_table, sin_table, positions, dev),
        _act(q_out, dt, rows, hq, d, cfg.q_out_stride, dev) if hq else None,
        _act(k_out, dt, rows, hk, d, cfg.k_out_stride, dev) if hk else None,
        _stream_of(stream, dev)), "m3_qk_norm_rope")


def m3_qk_norm_rope_backward_workspace(cfg: QkNormRopeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_qk_norm_rope_backward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_qk_norm_rope_backward_workspace")
    return n.value


def m3_qk_norm_rope_backward(cfg: QkNormRopeConfig, q, k, q_weight, k_weight, cos_table, sin_table,
                             positions, grad_q_out, grad_k_out, grad_q, grad_k, grad_q_weight,
                             grad_k_weight, workspace=None, stream=None):
    types, dt, dev, rows, hq, hk, d = _rope_shapes(cfg, k if q is None else q)
    wp, wn = _ws_on(workspace, dev)
    side = lambda t, heads, stride: _act(t, dt, rows, heads, d, stride, dev) if heads else None  # noqa: E731
    _check(load_library().m3_qk_norm_rope_backward(
        ctypes.byref(cfg), side(q, hq, cfg.q_stride), side(k, hk, cfg.k_stride),
        *_rope_tables(cfg, types, rows, d, q_weight, k_weight, cos_table, sin_table, positions, dev),
        side(grad_q_out, hq, cfg.q_out_stride), side(grad_k_out, hk, cfg.k_out_stride),
        side(grad_q, hq, 0), side(grad_k, hk, 0), _dense(grad_q_weight, types[0], (d,), dev),
        _dense(grad_k_weight, types[0], (d,), dev), wp, wn, _stream_of(stream, dev)),
        "m3_qk_norm_rope_backward")


def linear_attention_config(q, k, v, *, batch_size, sequence_length, num_heads=None, num_groups=0,
                            scale=1.0, num_slots=0, out=None) -> LinearAttentionConfig:
    """The config of q, k [..., groups, state_size] and v [..., heads, head_dim];
    out is dense unless given."""
    heads = v.shape[-2] if num_heads is None else num_heads
    strides = [0 if t is None else _row_stride(t) for t in (q, k, v, out)]
    return LinearAttentionConfig(batch_size, sequence_length,
                                 v.numel() // max(1, v.shape[-2] * v.shape[-1]), heads, num_groups,
                                 v.shape[-1], q.shape[-1], num_slots, *strides, scale, _dtype(v))


def _la_shapes(cfg, v):
    """(types, activations' type, device, B, rows, H, G, N, P) of a call."""
    types, heads = _torch_types(), cfg.num_heads
    return (types, types[cfg.dtype], _device_of(v), cfg.batch_size, cfg.total_rows, heads,
            cfg.num_groups or heads, cfg.state_size, cfg.head_dim)


def m3_linear_attention_forward_workspace(cfg: LinearAttentionConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_linear_attention_forward_workspace(ctypes.byref(cfg), ctypes.byref(n)),
           "m3_linear_attention_forward_workspace")
    return n.value


def m3_linear_attention_forward(cfg: LinearAttentionConfig, q, k, v, log_decay, offsets,
                                initial_state, out, final_state, workspace=None, stream=None):
    types, dt, dev, b, r, h, g, n, p = _la_shapes(cfg, v)
    f32, state = types[0], (b, h, p, n)
    wp, wn = _ws_on(workspace, dev)
    _check(load_library().m3_linear_attention_forward(
        ctypes.byref(cfg), _act(q, dt, r, g, n, cfg.q_stride, dev),
        _act(k, dt, r, g, n, cfg.k_stride, dev), _act(v, dt, r, h, p, cfg.v_stride, dev),
        _dense(log_decay, f32, (h,), dev), _dense(offsets, types[2], (b + 1,), dev),
        _dense(initial_state, f32, state, dev), _act(out, dt, r, h, p, cfg.out_stride, dev),
        _dense(final_state, f32, state, dev), wp, wn, _stream_of(stream, dev)),
        "m3_linear_attention_forward")


def m3_linear_attention_step(cfg: LinearAttentionConfig, q, k, v, log_decay, slots, state, out,
                             stream=None):
    types, dt, dev, b, r, h, g, n, p = _la_shapes(cfg, v)
    f32 = types[0]
    _check(load_library().m3_linear_attention_step(
        ctypes.byref(cfg), _act(q, dt, r, g, n, cfg.q_stride, dev),
        _act(k, dt, r, g, n, cfg.k_stride, dev), _act(v, dt, r, h, p, cfg.v_stride, dev),
        _dense(log_decay, f32, (h,), dev), _dense(slots, types[2], (b,), dev),
        _dense(state, f32, (cfg.num_slots or b, h, p, n), dev),
        _act(out, dt, r, h, p, cfg.out_stride, dev), _stream_of(stream, dev)),
        "m3_linear_attention_step")


def m3_linear_attention_backward_workspace(cfg: LinearAttentionConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().m3_linear_attention_backward_workspace(ctypes.byref(cfg),
                                                                 ctypes.byref(n)),
           "m3_linear_attention_backward_workspace")
    return n.value


def m3_linear_attention_backward(cfg: LinearAttentionConfig, grad_out, q, k, v, log_decay, offsets,
                                 initial_state, grad_final_state, grad_q, grad_k, grad_v,
                                 grad_initial_state, workspace=None, stream=None):
    types, dt, dev, b, r, h, g, n, p = _la_shapes(cfg, v)
    f32, state = types[0], (b, h, p, n)
    wp, wn = _ws_on(workspace, dev)
    _check(load_library().m3_linear_attention_backward(
        ctypes.byref(cfg), _act(grad_out, dt, r, h, p, cfg.out_stride, dev),
        _act(q, dt, r, g, n, cfg.q_stride, dev), _act(k, dt, r, g, n, cfg.k_stride, dev),
        _act(v, dt, r, h, p, cfg.v_stride, dev), _dense(log_decay, f32, (h,), dev),
        _dense(offsets, types[2], (b + 1,), dev), _dense(initial_state, f32, state, dev),
        _dense(grad_final_state, f32, state, dev), _act(grad_q, dt, r, g, n, 0, dev),
        _act(grad_k, dt, r, g, n, 0, dev), _act(grad_v, dt, r, h, p, 0, dev),
        _dense(grad_initial_state, f32, state, dev), wp, wn, _stream_of(stream, dev)),
        "m3_linear_attention_backward")
