"""ctypes binding of libradamw.so -- argument marshalling only.

Every function here has the name of the C entry point it calls.  Torch is
used for device memory and streams: the binding checks what raw pointers
cannot express (tensor device, dtype, contiguity, element count; FA-zh
"增加的实际能力": non-contiguous, broadcast and mismatched device/queue
inputs are errors), passes ``data_ptr()`` and the current HIP stream, and
raises ``RadamwError`` on a non-zero status.  No arithmetic of the method
happens here, and there is no fallback: without the built library every call
raises.

Page abbreviation: FA-zh = RUDA docs page "实验性融合 AdamW / AMSGrad".
"""
from __future__ import annotations

import ctypes
import os
import sys
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libradamw.so")

RADAMW_OK = 0
F32, F16, BF16 = 0, 1, 2
_DTYPE_CODE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_INDEX_CODE = {torch.int32: 0, torch.int64: 1}


class RadamwError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = status_string(status) if _lib is not None else str(status)
        extra = ""
        if status == -6 and _lib is not None:
            extra = f" (hipError {_lib.radamw_last_hip_error()})"
        super().__init__(f"{where}: {msg} [{status}]{extra}")


RADAMW_ERR_DECISION = -7


class DecisionMismatch(RadamwError):
    """RADAMW_ERR_DECISION from a fused step: the host's decision differed
    from the device's, and the step ran as the device decided.  ``result``
    and ``step`` (or ``steps``) are what the call reported, so the caller's
    step counts can follow the state that was written."""

    def __init__(self, where: str, result, step=None, steps=None):
        super().__init__(RADAMW_ERR_DECISION, where)
        self.result, self.step, self.steps = result, step, steps


# ----------------------------------------------------------------- structs --

class Options(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("amsgrad", ctypes.c_int32), ("maximize", ctypes.c_int32)]


class Control(ctypes.Structure):
    _fields_ = [("gradient_scale", ctypes.c_double), ("skip_update", ctypes.c_int32)]


class _State(ctypes.Structure):
    _fields_ = [("step", ctypes.c_uint64), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("max_exp_avg_sq", ctypes.c_void_p)]


class _Segment(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("max_exp_avg_sq", ctypes.c_void_p),
                ("n", ctypes.c_int64)]


class PolicyOptions(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double), ("kl_coef", ctypes.c_double)]


class PreferenceOptions(ctypes.Structure):
    _fields_ = [("beta", ctypes.c_double), ("label_smoothing", ctypes.c_double)]


class DropoutOptions(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("first_row", ctypes.c_int64)]


class ResidualOptions(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_double), ("weight_offset", ctypes.c_double), ("residual_scale", ctypes.c_double),
                ("dropout", DropoutOptions)]


class _ResidualBlock(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("dim", ctypes.c_int64), ("stream_dtype", ctypes.c_int32),
                ("branch_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("branch", ctypes.c_void_p), ("branch_stride", ctypes.c_int64), ("gate", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("rows_per_gate", ctypes.c_int64), ("post_weight", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p)]


class BalanceOptions(ctypes.Structure):
    _fields_ = [("balance_coef", ctypes.c_double), ("z_coef", ctypes.c_double), ("score", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [("w", ctypes.c_uint32 * 3)]

    @property
    def sumsq(self) -> float:
        return ctypes.c_double.from_buffer_copy(
            (ctypes.c_uint32 * 2)(self.w[0], self.w[1])).value

    @property
    def nonfinite(self) -> int:
        return int(self.w[2])


class FusedResult(ctypes.Structure):
    _fields_ = [("updated", ctypes.c_int32), ("found_inf", ctypes.c_int32),
                ("nonfinite", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("sumsq", ctypes.c_double), ("total_norm", ctypes.c_double),
                ("clip_coef", ctypes.c_double)]


def options(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-5, weight_decay=1e-4, amsgrad=False,
            maximize=False) -> Options:
    return Options(lr, beta1, beta2, eps, weight_decay, int(amsgrad), int(maximize))


def policy_options(clip_low=0.2, clip_high=0.2, kl_coef=0.0) -> PolicyOptions:
    return PolicyOptions(float(clip_low), float(clip_high), float(kl_coef))


def preference_options(beta=0.1, label_smoothing=0.0) -> PreferenceOptions:
    return PreferenceOptions(float(beta), float(label_smoothing))


def _word64(v: int, what: str) -> int:
    if not 0 <= int(v) < 1 << 64:
        raise ValueError(f"{what} must be within 0 .. 2^64 - 1 (got {v})")
    return int(v)


def dropout_options(p=0.0, seed=0, offset=0, first_row=0) -> DropoutOptions:
    return DropoutOptions(float(p), _word64(seed, "seed"), _word64(offset, "offset"), int(first_row))


def residual_options(eps=1e-6, weight_offset=0.0, residual_scale=1.0, p=0.0, seed=0, offset=0,
                     first_row=0) -> ResidualOptions:
    return ResidualOptions(float(eps), float(weight_offset), float(residual_scale),
                           dropout_options(p, seed, offset, first_row))


_SCORES = {"softmax": 0, "sigmoid": 1}


def balance_options(balance_coef=0.01, z_coef=0.0, score="softmax") -> BalanceOptions:
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)} (got {score!r})")
    return BalanceOptions(float(balance_coef), float(z_coef), _SCORES[score])


def control(gradient_scale=1.0, skip_update=False) -> Control:
    return Control(float(gradient_scale), int(bool(skip_update)))


@dataclass
class AdamWState:
    """Host step count + device moment tensors (the exposed parts of the
    pages' optimizer state).  step == 0 means "no state yet"."""
    step: int = 0
    exp_avg: Optional[torch.Tensor] = None
    exp_avg_sq: Optional[torch.Tensor] = None
    max_exp_avg_sq: Optional[torch.Tensor] = None

    def _c(self) -> _State:
        return _State(self.step, _ptr_or_none(self.exp_avg), _ptr_or_none(self.exp_avg_sq),
                      _ptr_or_none(self.max_exp_avg_sq))


@dataclass
class Segment:
    """One tensor of a multi-tensor in-place update."""
    param: torch.Tensor
    grad: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    max_exp_avg_sq: Optional[torch.Tensor] = None


# ----------------------------------------------------------------- loading --

_lib = None


def load(path: str = LIB_PATH):
    """Load libradamw.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m optimizer_step_dl_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u64, dbl = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double
    P = ctypes.POINTER
    sig = {
        "radamw_options_default": ([], Options),
        "radamw_step": ([vp, vp, i32, i64, P(_State), vp, P(_State), P(Options), P(Control), vp, P(i32)], ctypes.c_int),
        "radamw_step_inplace": ([vp, vp, i32, i64, P(_State), P(Options), P(Control), vp, P(i32)], ctypes.c_int),
        "radamw_step_multi": ([P(_Segment), i32, i32, P(u64), P(Options), P(Control), vp, P(i32)], ctypes.c_int),
        "radamw_step_staged_inplace": ([vp, vp, i32, i64, P(_State), vp, P(Options), P(Control), vp, P(i32)],
                                       ctypes.c_int),
        "radamw_stream_probe": ([P(vp), i32, P(vp), i32, i64, i32, vp], ctypes.c_int),
        "radamw_bucket_layout": ([i64, P(i32), i32, P(i64), P(i64)], ctypes.c_int),
        "radamw_step_multi_writeback": ([P(_Segment), P(vp), i32, i32, i32, P(u64), P(Options), P(Control), vp,
                                         P(i32)], ctypes.c_int),
        "radamw_stats_plan": ([i64, P(i64), P(i32)], ctypes.c_int),
        "radamw_grad_stats_rows": ([i64, i32], i64),
        "radamw_grad_stats": ([vp, i32, i64, vp, i64, P(i64), vp], ctypes.c_int),
        "radamw_merge_stats": ([vp, i64, vp, i64, vp, i32, vp], ctypes.c_int),
        "radamw_read_report": ([vp, P(Stats), vp], ctypes.c_int),
        "radamw_decide": ([P(Stats), dbl, dbl, P(Control), P(FusedResult)], ctypes.c_int),
        "radamw_check_decision": ([P(Stats), P(ctypes.c_uint32), dbl, dbl, P(FusedResult)], ctypes.c_int),
        "radamw_fused_workspace_bytes": ([P(_Segment), i32, i32], i64),
        "radamw_fused_step_multi": ([P(_Segment), i32, i32, P(u64), P(Options), dbl, dbl, i32, vp, i64, vp,
                                     P(FusedResult)], ctypes.c_int),
        "radamw_fused_step_multi_noalloc": ([P(_Segment), i32, i32, P(u64), P(Options), dbl, dbl, i32, vp,
                                             P(FusedResult)], ctypes.c_int),
        "radamw_host_coefficients": ([P(Options), u64, dbl, P(ctypes.c_float)], ctypes.c_int),
        "radamw_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "radamw_last_hip_error": ([], ctypes.c_int),
        "radamw_launch_count": ([], u64),
        "radamw_time_next_update": ([vp, vp], ctypes.c_int),
        "radamw_list_create": ([P(_Segment), i32, i32, i32, P(vp), i32, vp, P(vp)], ctypes.c_int),
        "radamw_list_step": ([vp, P(u64), P(Options), P(Control), vp, P(i32)], ctypes.c_int),
        "radamw_list_fused_step": ([vp, P(u64), P(Options), dbl, dbl, i32, vp, P(FusedResult)], ctypes.c_int),
        "radamw_list_destroy": ([vp], ctypes.c_int),
        "radamw_lists_fused_step": ([P(vp), i32, P(u64), P(Options), dbl, dbl, i32, vp, P(FusedResult)],
                                    ctypes.c_int),
        "radamw_embedding_lookup": ([vp, i32, i64, i64, i64, vp, i32, i64, dbl, vp, i32, i64, vp], ctypes.c_int),
        "radamw_embedding_grad_workspace_bytes": ([i64, i64, i64], i64),
        "radamw_embedding_grad": ([vp, i32, i64, vp, i32, i64, i64, i64, dbl, i64, i32, vp, i32, i64, vp, i64, vp],
                                  ctypes.c_int),
        "radamw_policy_options_default": ([], PolicyOptions),
        "radamw_policy_loss": ([vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, P(PolicyOptions), dbl, vp, vp, vp, vp,
                                vp, i64, vp], ctypes.c_int),
        "radamw_preference_options_default": ([], PreferenceOptions),
        "radamw_preference_loss": ([vp, i32, i64, i64, i64, vp, i32, vp, i64, vp, vp, P(PreferenceOptions), dbl, vp, vp,
                                    vp, vp, vp, vp, i64, vp], ctypes.c_int),
        "radamw_logits_grad": ([vp, i32, i64, i64, i64, vp, i32, vp, vp, dbl, vp, i64, vp], ctypes.c_int),
        "radamw_dropout_options_default": ([], DropoutOptions),
        "radamw_dropout": ([vp, i32, i64, i64, i64, P(DropoutOptions), vp, i64, vp], ctypes.c_int),
        "radamw_residual_options_default": ([], ResidualOptions),
        "radamw_residual_norm": ([P(_ResidualBlock), vp, i64, P(ResidualOptions), vp, i64, vp, i64, vp, vp],
                                 ctypes.c_int),
        "radamw_residual_grad_workspace_bytes": ([i64, i64, i64], i64),
        "radamw_residual_norm_grad": ([P(_ResidualBlock), vp, i64, vp, P(ResidualOptions), vp, i64, vp, i64, vp, i64, vp,
                                       i64, vp, i64, vp, vp, vp, i64, vp], ctypes.c_int),
        "radamw_balance_options_default": ([], BalanceOptions),
        "radamw_balance_workspace_bytes": ([i64, i64, i64], i64),
        "radamw_balance_loss": ([vp, i32, i64, i64, i64, vp, i32, i64, vp, vp, i64, vp, P(BalanceOptions), dbl, vp, vp,
                                 vp, vp, vp, vp, i64, vp, i64, vp], ctypes.c_int),
        "radamw_balance_grad": ([vp, i32, i64, i64, i64, i64, vp, vp, i32, i64, vp, P(BalanceOptions), vp, vp, vp, dbl,
                                 vp, i64, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


EXPORTS = ("radamw_options_default", "radamw_step", "radamw_step_inplace", "radamw_step_multi",
           "radamw_step_staged_inplace", "radamw_stream_probe", "radamw_bucket_layout", "radamw_step_multi_writeback",
           "radamw_stats_plan", "radamw_grad_stats_rows", "radamw_grad_stats", "radamw_merge_stats",
           "radamw_read_report", "radamw_decide", "radamw_check_decision", "radamw_fused_workspace_bytes",
           "radamw_fused_step_multi", "radamw_fused_step_multi_noalloc", "radamw_host_coefficients", "radamw_status_string",
           "radamw_last_hip_error", "radamw_launch_count", "radamw_time_next_update",
           "radamw_list_create", "radamw_list_step", "radamw_list_fused_step", "radamw_list_destroy",
           "radamw_lists_fused_step", "radamw_embedding_lookup", "radamw_embedding_grad_workspace_bytes",
           "radamw_embedding_grad", "radamw_policy_options_default", "radamw_policy_loss",
           "radamw_preference_options_default", "radamw_preference_loss", "radamw_logits_grad",
           "radamw_dropout_options_default", "radamw_dropout", "radamw_residual_options_default", "radamw_residual_norm",
           "radamw_residual_grad_workspace_bytes", "radamw_residual_norm_grad", "radamw_balance_options_default",
           "radamw_balance_workspace_bytes", "radamw_balance_loss", "radamw_balance_grad")


# ----------------------------------------------------------------- helpers --

def _ptr_or_none(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(rc: int, where: str):
    if rc != RADAMW_OK:
        raise RadamwError(rc, where)


def _stream(device: torch.device):
    return torch.cuda.current_stream(device).cuda_stream


def _dense(t: torch.Tensor, what: str, dtype=None, numel=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a device tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} (got {t.dtype})")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, expected {numel}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return t


def _grad_code(g: torch.Tensor) -> int:
    if g.dtype not in _DTYPE_CODE:
        raise ValueError(f"gradient dtype {g.dtype} is not float32/float16/bfloat16")
    return _DTYPE_CODE[g.dtype]


def _check_fast(t: torch.Tensor, what: str, dev_index: int, numel: int, dtype=None):
    """Cheap form of _dense for long tensor lists (same checks)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if t.get_device() != dev_index:
        raise ValueError(f"{what} is on device {t.get_device()}, expected {dev_index}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, expected {numel}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} (got {t.dtype})")


def _segments(segs: Sequence[Segment], amsgrad: bool):
    arr = (_Segment * max(1, len(segs)))()
    code = None
    dev_index = None
    f32 = torch.float32
    for i, s in enumerate(segs):
        p = s.param
        if dev_index is None:
            if not isinstance(p, torch.Tensor) or not p.is_cuda:
                raise ValueError(f"segment {i} param must be a device tensor")
            dev_index = p.get_device()
        n = p.numel()
        _check_fast(p, f"segment {i} param", dev_index, n, f32)
        _check_fast(s.grad, f"segment {i} grad", dev_index, n)
        c = _grad_code(s.grad)
        if code is not None and c != code:
            raise ValueError("all gradients of one call must share a dtype")
        code = c
        _check_fast(s.exp_avg, f"segment {i} exp_avg", dev_index, n, f32)
        _check_fast(s.exp_avg_sq, f"segment {i} exp_avg_sq", dev_index, n, f32)
        if s.max_exp_avg_sq is not None:
            _check_fast(s.max_exp_avg_sq, f"segment {i} max_exp_avg_sq", dev_index, n, f32)
        arr[i] = _Segment(p.data_ptr(), s.grad.data_ptr(), s.exp_avg.data_ptr(),
                          s.exp_avg_sq.data_ptr(), _ptr_or_none(s.max_exp_avg_sq), n)
    device = torch.device("cuda", torch.cuda.current_device() if dev_index is None else dev_index)
    return arr, (F32 if code is None else code), device


class SegmentList:
    """A tensor list marshalled once, for repeated multi-tensor steps over
    the same tensors (optimizer state and parameters normally keep their
    storage for a whole run).  Holds references to the tensors; the C entry
    points still validate every pointer on each call."""

    def __init__(self, segments: Sequence[Segment]):
        self.segments = list(segments)
        self.array, self.code, self.device = _segments(self.segments, False)

    def __len__(self):
        return len(self.segments)


def _marshal(segments):
    if isinstance(segments, SegmentList):
        return segments.array, segments.code, segments.device, len(segments)
    arr, code, dev = _segments(segments, False)
    return arr, code, dev, len(segments)


# ------------------------------------------------------------- entry points --

def radamw_options_default() -> Options:
    return load().radamw_options_default()


def radamw_step(param: torch.Tensor, grad: torch.Tensor, state: AdamWState, opts: Options,
                ctrl: Control, out_param: torch.Tensor, out_state: AdamWState) -> bool:
    """Out-of-place update: writes out_param/out_state, never the inputs.
    Returns True when launched (then out_state.step = state.step + 1)."""
    lib = load()
    dev = param.device
    n = param.numel()
    _dense(param, "param", torch.float32)
    _dense(grad, "grad", numel=n, device=dev)
    _dense(out_param, "out_param", torch.float32, n, dev)
    for name in ("exp_avg", "exp_avg_sq", "max_exp_avg_sq"):
        t = getattr(out_state, name)
        if t is not None:
            _dense(t, f"out_state.{name}", torch.float32, n, dev)
        t = getattr(state, name)
        if t is not None and state.step > 0:
            _dense(t, f"state.{name}", torch.float32, n, dev)
    cin, cout = state._c(), out_state._c()
    updated = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_step(param.data_ptr(), grad.data_ptr(), _grad_code(grad), n, ctypes.byref(cin),
                             out_param.data_ptr(), ctypes.byref(cout), ctypes.byref(opts), ctypes.byref(ctrl),
                             _stream(dev), ctypes.byref(updated))
    _check(rc, "radamw_step")
    if updated.value:
        out_state.step = cout.step
    return bool(updated.value)


def radamw_step_inplace(param: torch.Tensor, grad: torch.Tensor, state: AdamWState, opts: Options,
                        ctrl: Control) -> bool:
    """In-place update of param and state; state.step advances on launch."""
    lib = load()
    dev = param.device
    n = param.numel()
    _dense(param, "param", torch.float32)
    _dense(grad, "grad", numel=n, device=dev)
    for name in ("exp_avg", "exp_avg_sq", "max_exp_avg_sq"):
        t = getattr(state, name)
        if t is not None:
            _dense(t, f"state.{name}", torch.float32, n, dev)
    cst = state._c()
    updated = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_step_inplace(param.data_ptr(), grad.data_ptr(), _grad_code(grad), n,
                                     ctypes.byref(cst), ctypes.byref(opts), ctypes.byref(ctrl),
                                     _stream(dev), ctypes.byref(updated))
    _check(rc, "radamw_step_inplace")
    state.step = cst.step
    return bool(updated.value)


def radamw_step_staged_inplace(param: torch.Tensor, grad: torch.Tensor, state: AdamWState, delta: torch.Tensor,
                               opts: Options, ctrl: Control) -> bool:
    """The staged (unfused, 4 or 5 launches) baseline, in place; delta is an
    FP32 scratch tensor of the same size.  For measurement."""
    lib = load()
    dev = param.device
    n = param.numel()
    _dense(param, "param", torch.float32)
    _dense(grad, "grad", numel=n, device=dev)
    _dense(delta, "delta", torch.float32, n, dev)
    for name in ("exp_avg", "exp_avg_sq", "max_exp_avg_sq"):
        t = getattr(state, name)
        if t is not None:
            _dense(t, f"state.{name}", torch.float32, n, dev)
    cst = state._c()
    updated = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_step_staged_inplace(param.data_ptr(), grad.data_ptr(), _grad_code(grad), n,
                                            ctypes.byref(cst), delta.data_ptr(), ctypes.byref(opts),
                                            ctypes.byref(ctrl), _stream(dev), ctypes.byref(updated))
    _check(rc, "radamw_step_staged_inplace")
    state.step = cst.step
    return bool(updated.value)


def radamw_stream_probe(ins: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], cap_per_cu: int = 0,
                        sink: Optional[torch.Tensor] = None) -> None:
    """Streaming ceiling (measurement only): len(ins) FP32 read streams and
    len(outs) write streams with the update kernel's geometry;
    outs[w] = sum(ins) + w.  With no output, ``sink`` (an FP32 tensor of the
    streams' size) is the never-written sink."""
    lib = load()
    tensors = list(ins) + list(outs) + ([] if sink is None else [sink])
    if not tensors:
        raise ValueError("at least one stream")
    dev = tensors[0].device
    n = tensors[0].numel()
    for i, t in enumerate(tensors):
        _dense(t, f"stream {i}", torch.float32, n, dev)
    # an output given as one of the inputs is updated in place
    if not outs and sink is None:
        raise ValueError("a read-only probe needs a sink tensor")
    pin = (ctypes.c_void_p * max(1, len(ins)))(*[t.data_ptr() for t in ins])
    wr = list(outs) if outs else [sink]
    pout = (ctypes.c_void_p * len(wr))(*[t.data_ptr() for t in wr])
    with torch.cuda.device(dev):
        rc = lib.radamw_stream_probe(pin, len(ins), pout, len(outs), n, int(cap_per_cu), _stream(dev))
    _check(rc, "radamw_stream_probe")


def radamw_bucket_layout(n: int, element_bytes: Sequence[int]):
    """(byte offsets, arena bytes) of the library's placement for the
    streams of one flattened bucket in a single allocation."""
    k = len(element_bytes)
    eb = (ctypes.c_int32 * max(1, k))(*[int(x) for x in element_bytes])
    offs = (ctypes.c_int64 * max(1, k))()
    total = ctypes.c_int64()
    _check(load().radamw_bucket_layout(int(n), eb, k, offs, ctypes.byref(total)), "radamw_bucket_layout")
    return [int(offs[i]) for i in range(k)], int(total.value)


_PITCH_ALIGN = 2 << 20


def bucket_arena(n: int, dtypes: Sequence[torch.dtype], device=None):
    """One device allocation holding len(dtypes) streams of n elements, placed
    by radamw_bucket_layout (from a 2 MiB-aligned start).  Returns the views,
    in order; each keeps the allocation alive."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    sizes = [torch.empty(0, dtype=d).element_size() for d in dtypes]
    offs, total = radamw_bucket_layout(n, sizes)
    raw = torch.empty(total + _PITCH_ALIGN, dtype=torch.uint8, device=device)
    lead = (-raw.data_ptr()) % _PITCH_ALIGN
    return [raw[lead + o:lead + o + n * es].view(d) for o, es, d in zip(offs, sizes, dtypes)]


def bucket_segment(n: int, grad_dtype: torch.dtype = torch.float32, amsgrad: bool = False, device=None) -> Segment:
    """A flattened bucket's p, gradient, m, v (and v_max) as one allocation
    in the library's placement (bucket_arena); contents uninitialised."""
    f32 = torch.float32
    dts = [f32, grad_dtype, f32, f32] + ([f32] if amsgrad else [])
    views = bucket_arena(n, dts, device)
    return Segment(views[0], views[1], views[2], views[3], views[4] if amsgrad else None)


def radamw_step_multi(segments, step: int, opts: Options, ctrl: Control):
    """In-place update of a tensor list (a sequence of Segment or a
    SegmentList) sharing options and step count.  Returns (updated, new_step)."""
    lib = load()
    arr, code, dev, count = _marshal(segments)
    st = ctypes.c_uint64(step)
    updated = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_step_multi(arr, count, code, ctypes.byref(st), ctypes.byref(opts),
                                   ctypes.byref(ctrl), _stream(dev), ctypes.byref(updated))
    _check(rc, "radamw_step_multi")
    return bool(updated.value), int(st.value)


def _models(models, segs, dev):
    """Host array of model-copy pointers (None entries stay NULL) and their
    shared dtype."""
    mdt = None
    ptrs = (ctypes.c_void_p * max(1, len(segs)))()
    for i, (m, s) in enumerate(zip(models, segs)):
        if m is None:
            continue
        _dense(m, f"model copy {i}", numel=s.param.numel(), device=dev)
        if m.dtype not in (torch.float16, torch.bfloat16) or (mdt is not None and m.dtype != mdt):
            raise ValueError("model copies must all be float16 or all bfloat16")
        mdt = m.dtype
        ptrs[i] = m.data_ptr()
    return ptrs, mdt


def radamw_step_multi_writeback(segments, models: Sequence[Optional[torch.Tensor]], step: int, opts: Options,
                                ctrl: Control):
    """radamw_step_multi plus a 16-bit model copy per tensor, written in the
    same pass.  models[i] is a float16 / bfloat16 tensor of segments[i]'s
    size, or None; all copies share one dtype.  Returns (updated, new_step)."""
    lib = load()
    arr, code, dev, count = _marshal(segments)
    if len(models) != count:
        raise ValueError("one model entry (tensor or None) per segment")
    segs = segments.segments if isinstance(segments, SegmentList) else segments
    ptrs, mdt = _models(models, segs, dev)
    st = ctypes.c_uint64(step)
    updated = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_step_multi_writeback(arr, ptrs, count, code, _DTYPE_CODE[mdt or torch.bfloat16],
                                             ctypes.byref(st), ctypes.byref(opts), ctypes.byref(ctrl), _stream(dev),
                                             ctypes.byref(updated))
    _check(rc, "radamw_step_multi_writeback")
    return bool(updated.value), int(st.value)


def radamw_stats_plan(rows: int):
    """(scratch_elements, extra_merge_kernels) for ``rows`` records."""
    se, ex = ctypes.c_int64(), ctypes.c_int32()
    _check(load().radamw_stats_plan(rows, ctypes.byref(se), ctypes.byref(ex)), "radamw_stats_plan")
    return se.value, ex.value


def radamw_grad_stats_rows(n: int, dtype: torch.dtype) -> int:
    r = load().radamw_grad_stats_rows(n, _DTYPE_CODE[dtype])
    if r < 0:
        raise RadamwError(int(r), "radamw_grad_stats_rows")
    return int(r)


def radamw_grad_stats(grad: torch.Tensor, rows: torch.Tensor, row_offset: int = 0) -> int:
    """Analyse ``grad`` into records rows[row_offset:]; ``rows`` is an int32
    tensor of 3 * capacity words.  Returns the number of records written."""
    lib = load()
    dev = grad.device
    _dense(grad, "grad")
    _dense(rows, "rows", torch.int32, device=dev)
    cap = rows.numel() // 3 - row_offset
    written = ctypes.c_int64(0)
    with torch.cuda.device(dev):
        rc = lib.radamw_grad_stats(grad.data_ptr(), _grad_code(grad), grad.numel(),
                                   rows.data_ptr() + 12 * row_offset, cap, ctypes.byref(written),
                                   _stream(dev))
    _check(rc, "radamw_grad_stats")
    return int(written.value)


def radamw_merge_stats(rows: torch.Tensor, nrows: int, scratch: Optional[torch.Tensor],
                       report: torch.Tensor, hierarchical: bool = True) -> None:
    lib = load()
    dev = rows.device
    _dense(rows, "rows", torch.int32)
    _dense(report, "report", torch.int32, 3, dev)
    if scratch is not None:
        _dense(scratch, "scratch", torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = lib.radamw_merge_stats(rows.data_ptr(), nrows, _ptr_or_none(scratch),
                                    0 if scratch is None else scratch.numel(), report.data_ptr(),
                                    int(bool(hierarchical)), _stream(dev))
    _check(rc, "radamw_merge_stats")


def radamw_read_report(report: torch.Tensor) -> Stats:
    lib = load()
    _dense(report, "report", torch.int32, 3)
    out = Stats()
    with torch.cuda.device(report.device):
        rc = lib.radamw_read_report(report.data_ptr(), ctypes.byref(out), _stream(report.device))
    _check(rc, "radamw_read_report")
    return out


def radamw_decide(host_report: Stats, gradient_scale: float, max_grad_norm: Optional[float]):
    """(Control, FusedResult) of the host decision for a read-back report."""
    ctrl, res = Control(), FusedResult()
    rc = load().radamw_decide(ctypes.byref(host_report), float(gradient_scale),
                              0.0 if max_grad_norm is None else float(max_grad_norm),
                              ctypes.byref(ctrl), ctypes.byref(res))
    _check(rc, "radamw_decide")
    return ctrl, res


def radamw_check_decision(host_report: Stats, device_skip: int, device_inv_scale_bits: int,
                          gradient_scale: float, max_grad_norm: Optional[float]):
    """(agree, FusedResult): the host's decision from ``host_report`` against
    a device decision {skip, bits of the FP32 unscale factor}; the result's
    ``updated`` follows the device's."""
    dec = (ctypes.c_uint32 * 2)(int(device_skip) & 0xffffffff, int(device_inv_scale_bits) & 0xffffffff)
    res = FusedResult()
    rc = load().radamw_check_decision(ctypes.byref(host_report), dec, float(gradient_scale),
                                      0.0 if max_grad_norm is None else float(max_grad_norm), ctypes.byref(res))
    if rc not in (RADAMW_OK, RADAMW_ERR_DECISION):
        _check(rc, "radamw_check_decision")
    return rc == RADAMW_OK, res


def radamw_fused_workspace_bytes(segments) -> int:
    arr, code, _, count = _marshal(segments)
    r = load().radamw_fused_workspace_bytes(arr, count, code)
    if r < 0:
        raise RadamwError(int(r), "radamw_fused_workspace_bytes")
    return int(r)


def radamw_fused_step_multi(segments, step: int, opts: Options,
                            gradient_scale: float, max_grad_norm: Optional[float],
                            hierarchical: bool, workspace: Optional[torch.Tensor]):
    """Statistics -> merge -> read-back -> decision -> one update launch.
    Returns (FusedResult, new_step)."""
    lib = load()
    arr, code, dev, count = _marshal(segments)
    if workspace is not None:
        _dense(workspace, "workspace", device=dev)
    st = ctypes.c_uint64(step)
    res = FusedResult()
    with torch.cuda.device(dev):
        rc = lib.radamw_fused_step_multi(
            arr, count, code, ctypes.byref(st), ctypes.byref(opts), float(gradient_scale),
            0.0 if max_grad_norm is None else float(max_grad_norm), int(bool(hierarchical)),
            _ptr_or_none(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(dev), ctypes.byref(res))
    if rc == RADAMW_ERR_DECISION:
        raise DecisionMismatch("radamw_fused_step_multi", res, step=int(st.value))
    _check(rc, "radamw_fused_step_multi")
    return res, int(st.value)


def radamw_fused_step_multi_noalloc(segments, step: int, opts: Options, gradient_scale: float,
                                    max_grad_norm: Optional[float], hierarchical: bool):
    """radamw_fused_step_multi over one flattened bucket (at most one
    segment) with no workspace: the library's static device scratch holds
    the statistics, so the call allocates nothing.  Returns when the step has
    completed.  Returns (FusedResult, new_step)."""
    lib = load()
    arr, code, dev, count = _marshal(segments)
    st = ctypes.c_uint64(step)
    res = FusedResult()
    with torch.cuda.device(dev):
        rc = lib.radamw_fused_step_multi_noalloc(
            arr, count, code, ctypes.byref(st), ctypes.byref(opts), float(gradient_scale),
            0.0 if max_grad_norm is None else float(max_grad_norm), int(bool(hierarchical)), _stream(dev),
            ctypes.byref(res))
    if rc == RADAMW_ERR_DECISION:
        raise DecisionMismatch("radamw_fused_step_multi_noalloc", res, step=int(st.value))
    _check(rc, "radamw_fused_step_multi_noalloc")
    return res, int(st.value)


class TensorList:
    """A persistent tensor list (radamw_list_create): the segments are
    validated once and their launch tables kept in device memory, so each
    step only launches.  The list holds a reference to every tensor it was
    built from, so their storage stays allocated while it lives; a gradient
    that moves to a new tensor needs a new list.  ``models`` optionally
    gives a float16 / bfloat16 model copy per segment (or None), rewritten
    by every update.  Free it with close() (or a ``with`` block)."""

    def __init__(self, segments, amsgrad: bool, models: Optional[Sequence[Optional[torch.Tensor]]] = None):
        lib = load()
        self.segments = list(segments.segments if isinstance(segments, SegmentList) else segments)
        arr, code, dev = _segments(self.segments, False)
        self.device, self.code, self.amsgrad = dev, code, bool(amsgrad)
        self.models = None if models is None else list(models)
        ptrs, mdt = None, None
        if self.models is not None:
            if len(self.models) != len(self.segments):
                raise ValueError("one model entry (tensor or None) per segment")
            ptrs, mdt = _models(self.models, self.segments, dev)
        handle = ctypes.c_void_p()
        with torch.cuda.device(dev):
            rc = lib.radamw_list_create(arr, len(self.segments), code, int(self.amsgrad), ptrs,
                                        _DTYPE_CODE[mdt or torch.bfloat16], _stream(dev), ctypes.byref(handle))
        _check(rc, "radamw_list_create")
        self._handle = handle

    def _live(self):
        if self._handle is None:
            raise RuntimeError("the tensor list was closed")
        return self._handle

    def step(self, step: int, opts: Options, ctrl: Control):
        """radamw_step_multi over the list.  Returns (updated, new_step)."""
        st = ctypes.c_uint64(step)
        updated = ctypes.c_int32(0)
        with torch.cuda.device(self.device):
            rc = load().radamw_list_step(self._live(), ctypes.byref(st), ctypes.byref(opts), ctypes.byref(ctrl),
                                         _stream(self.device), ctypes.byref(updated))
        _check(rc, "radamw_list_step")
        return bool(updated.value), int(st.value)

    def fused_step(self, step: int, opts: Options, gradient_scale: float, max_grad_norm: Optional[float],
                   hierarchical: bool):
        """radamw_fused_step_multi over the list.  Returns (FusedResult, new_step)."""
        st = ctypes.c_uint64(step)
        res = FusedResult()
        with torch.cuda.device(self.device):
            rc = load().radamw_list_fused_step(self._live(), ctypes.byref(st), ctypes.byref(opts),
                                               float(gradient_scale),
                                               0.0 if max_grad_norm is None else float(max_grad_norm),
                                               int(bool(hierarchical)), _stream(self.device), ctypes.byref(res))
        if rc == RADAMW_ERR_DECISION:
            raise DecisionMismatch("radamw_list_fused_step", res, step=int(st.value))
        _check(rc, "radamw_list_fused_step")
        return res, int(st.value)

    def close(self):
        if getattr(self, "_handle", None) is not None:
            h, self._handle = self._handle, None
            _check(load().radamw_list_destroy(h), "radamw_list_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        if getattr(self, "_handle", None) is not None and not sys.is_finalizing():
            try:
                self.close()
            except Exception:
                pass

    def __len__(self):
        return len(self.segments)


def radamw_list_create(segments, amsgrad: bool, models=None) -> TensorList:
    return TensorList(segments, amsgrad, models)


def radamw_list_step(lst: TensorList, step: int, opts: Options, ctrl: Control):
    return lst.step(step, opts, ctrl)


def radamw_list_fused_step(lst: TensorList, step: int, opts: Options, gradient_scale: float,
                           max_grad_norm: Optional[float], hierarchical: bool):
    return lst.fused_step(step, opts, gradient_scale, max_grad_norm, hierarchical)


def radamw_list_destroy(lst: TensorList) -> None:
    lst.close()


def radamw_lists_fused_step(lists: Sequence[TensorList], steps: Sequence[int], opts: Sequence[Options],
                            gradient_scale: float, max_grad_norm: Optional[float], hierarchical: bool):
    """One fused step over several lists (parameter groups): one statistics
    reduction and one decision, then each list's update with its own options
    and step count.  Returns (FusedResult, new_steps)."""
    k = len(lists)
    if len(steps) != k or len(opts) != k or k == 0:
        raise ValueError("one step count and one options struct per list")
    dev = lists[0].device
    handles = (ctypes.c_void_p * k)(*[lst._live().value for lst in lists])
    st = (ctypes.c_uint64 * k)(*[int(x) for x in steps])
    op = (Options * k)(*opts)
    res = FusedResult()
    with torch.cuda.device(dev):
        rc = load().radamw_lists_fused_step(handles, k, st, op, float(gradient_scale),
                                            0.0 if max_grad_norm is None else float(max_grad_norm),
                                            int(bool(hierarchical)), _stream(dev), ctypes.byref(res))
    if rc == RADAMW_ERR_DECISION:
        raise DecisionMismatch("radamw_lists_fused_step", res, steps=[int(x) for x in st])
    _check(rc, "radamw_lists_fused_step")
    return res, [int(x) for x in st]


# ------------------------------------------------------ vocabulary operators --

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _submit(where: str, entry, device: torch.device, *args) -> None:
    """Call a C entry point on the device's current stream, its last
    argument.  Device scope and stream object (3 us together) are left out
    where the device is the current one."""
    i = device.index
    if _raw_stream is not None and _current_device() == i:
        rc = entry(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            rc = entry(*args, _stream(device))
    if rc != RADAMW_OK:
        raise RadamwError(rc, where)


def _rows2d(t: torch.Tensor, what: str, device, n=None, width=None) -> int:
    """Check a [n, width] device tensor with unit column stride; its row
    stride in elements."""
    try:  # the usual case in few questions; what fails it is named below
        (rows, cols), (row, col) = t.shape, t.stride()
        if (col == 1 and rows > 1 and row >= cols and t.get_device() == device.index and t.dtype in _DTYPE_CODE
                and (n is None or rows == n) and (width is None or cols == width)):
            return row
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions (got {t.dim()})")
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"{what} dtype {t.dtype} is not float32/float16/bfloat16")
    rows, cols = t.shape
    if (n is not None and rows != n) or (width is not None and cols != width):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(n, width)}")
    row, col = t.stride()
    if rows <= 1:  # one row (or none): its stride is never used
        row = max(row, cols)
    if (cols > 1 and col != 1) or row < cols:
        raise ValueError(f"{what} must have unit column stride and rows that do not overlap (strides {t.stride()})")
    return row


def _index(t: torch.Tensor, what: str, n: int, device) -> int:
    """Check a contiguous index tensor of n entries; its type code."""
    code = _INDEX_CODE.get(getattr(t, "dtype", None))
    if code is not None and t.numel() == n and t.get_device() == device.index and t.is_contiguous():
        return code
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype not in _INDEX_CODE:
        raise ValueError(f"{what} dtype {t.dtype} is not int32/int64")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} entries (got {t.numel()})")
    return _INDEX_CODE[t.dtype]


def _row_values(t: Optional[torch.Tensor], what: str, n: int, dev_index: int):
    """Pointer of a contiguous FP32 tensor of n values, or None."""
    if t is None:
        return None
    try:
        good = t.dtype is torch.float32 and t.numel() == n and t.get_device() == dev_index and t.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        _check_fast(t, what, dev_index, n, torch.float32)  # says what is wrong
    return t.data_ptr()


def radamw_embedding_lookup(table: torch.Tensor, ids: torch.Tensor, out: torch.Tensor, scale: float = 1.0) -> None:
    """out[t] = scale * table[ids[t]] for table [rows, dim], ids of any shape
    (int32 / int64, contiguous) and out [ids.numel(), dim]; zeros where an
    id is outside the table."""
    lib = load()
    dev = table.device
    ts = _rows2d(table, "table", dev)
    rows, dim = table.shape
    n = ids.numel()
    idt = _index(ids, "ids", n, dev)
    os_ = _rows2d(out, "out", dev, n, dim)
    _submit("radamw_embedding_lookup", lib.radamw_embedding_lookup, dev, table.data_ptr(), _DTYPE_CODE[table.dtype],
            rows, dim, ts, ids.data_ptr(), idt, n, float(scale), out.data_ptr(), _DTYPE_CODE[out.dtype], os_)


def radamw_embedding_grad_workspace_bytes(n: int, rows: int, dim: int) -> int:
    r = load().radamw_embedding_grad_workspace_bytes(n, rows, dim)
    if r < 0:
        raise RadamwError(int(r), "radamw_embedding_grad_workspace_bytes")
    return int(r)


def radamw_embedding_grad(grad_out: torch.Tensor, ids: torch.Tensor, table_grad: torch.Tensor,
                          workspace: torch.Tensor, scale: float = 1.0, padding_id: Optional[int] = None,
                          accumulate: bool = False) -> None:
    """table_grad (+)= the lookup's gradient: every row, or with
    ``accumulate`` only the rows some token names.  grad_out is
    [ids.numel(), dim], table_grad [rows, dim]; ``workspace`` holds at least
    radamw_embedding_grad_workspace_bytes(ids.numel(), rows, dim) bytes."""
    lib = load()
    dev = table_grad.device
    ts = _rows2d(table_grad, "table_grad", dev)
    rows, dim = table_grad.shape
    n = ids.numel()
    idt = _index(ids, "ids", n, dev)
    gs = _rows2d(grad_out, "grad_out", dev, n, dim)
    _dense(workspace, "workspace", device=dev)
    _submit("radamw_embedding_grad", lib.radamw_embedding_grad, dev, grad_out.data_ptr(), _DTYPE_CODE[grad_out.dtype],
            gs, ids.data_ptr(), idt, n, rows, dim, float(scale), -1 if padding_id is None else int(padding_id),
            int(bool(accumulate)), table_grad.data_ptr(), _DTYPE_CODE[table_grad.dtype], ts, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())


def radamw_policy_options_default() -> PolicyOptions:
    return load().radamw_policy_options_default()


def radamw_preference_options_default() -> PreferenceOptions:
    return load().radamw_preference_options_default()


def _logits(logits, labels, grad):
    """(device, n, vocab, row stride, labels' type code, gradient pointer and
    row stride) of a loss's logits, labels and optional gradient."""
    dev = logits.device
    st = _rows2d(logits, "logits", dev)
    n, vocab = logits.shape
    idt = _index(labels, "labels", n, dev)
    if grad is None:
        return dev, n, vocab, st, idt, None, 0
    gs = _rows2d(grad, "grad", dev, n, vocab)
    if grad.dtype != logits.dtype:
        raise ValueError(f"grad must be {logits.dtype} (got {grad.dtype})")
    return dev, n, vocab, st, idt, grad.data_ptr(), gs


def radamw_policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: Optional[torch.Tensor],
                       advantages: torch.Tensor, opts: PolicyOptions, total: torch.Tensor, loss: torch.Tensor,
                       logp: torch.Tensor, *, ref_logp: Optional[torch.Tensor] = None,
                       weights: Optional[torch.Tensor] = None, row_stats: Optional[torch.Tensor] = None,
                       grad: Optional[torch.Tensor] = None, grad_scale: float = 1.0) -> None:
    """Clipped policy loss of the rows of logits [n, vocab]: writes total
    (1), loss and logp (n), row_stats (n x 4, when given) and, when ``grad``
    is given, grad_scale * d total / d logits (``grad`` may be ``logits``)."""
    lib = load()
    dev, n, vocab, st, idt, gp, gs = _logits(logits, labels, grad)
    di = dev.index
    old = _row_values(old_logp, "old_logp", n, di)
    ref = _row_values(ref_logp, "ref_logp", n, di)
    adv = _row_values(advantages, "advantages", n, di)
    wts = _row_values(weights, "weights", n, di)
    tot = _row_values(total, "total", 1, di)
    los = _row_values(loss, "loss", n, di)
    lgp = _row_values(logp, "logp", n, di)
    sta = _row_values(row_stats, "row_stats", 4 * n, di)
    _submit("radamw_policy_loss", lib.radamw_policy_loss, dev, logits.data_ptr(), _DTYPE_CODE[logits.dtype], n, vocab,
            st, labels.data_ptr(), idt, old, ref, adv, wts, ctypes.byref(opts), float(grad_scale), tot, los, lgp, sta,
            gp, gs)


def radamw_preference_loss(logits: torch.Tensor, labels: torch.Tensor, offsets: torch.Tensor, ref_logp: torch.Tensor,
                           opts: PreferenceOptions, total: torch.Tensor, loss: torch.Tensor, seq_logp: torch.Tensor,
                           logp: torch.Tensor, row_stats: torch.Tensor, *, weights: Optional[torch.Tensor] = None,
                           grad: Optional[torch.Tensor] = None, grad_scale: float = 1.0) -> None:
    """Preference loss of pairs of sequences packed along the rows of logits
    [n, vocab]; offsets (2 * pairs + 1, the labels' dtype) give the rows of
    the chosen sequences, then of the rejected ones.  Writes total (1), loss
    (pairs), seq_logp (2 * pairs), logp (n), row_stats (n x 4) and, when
    ``grad`` is given, grad_scale * d total / d logits."""
    lib = load()
    dev, n, vocab, st, idt, gp, gs = _logits(logits, labels, grad)
    di = dev.index
    pairs = loss.numel()
    if _index(offsets, "offsets", 2 * pairs + 1, dev) != idt:
        raise ValueError(f"offsets must be {labels.dtype}, as the labels (got {offsets.dtype})")
    ref = _row_values(ref_logp, "ref_logp", 2 * pairs, di)
    wts = _row_values(weights, "weights", pairs, di)
    tot = _row_values(total, "total", 1, di)
    los = _row_values(loss, "loss", pairs, di)
    seq = _row_values(seq_logp, "seq_logp", 2 * pairs, di)
    lgp = _row_values(logp, "logp", n, di)
    sta = _row_values(row_stats, "row_stats", 4 * n, di)
    _submit("radamw_preference_loss", lib.radamw_preference_loss, dev, logits.data_ptr(), _DTYPE_CODE[logits.dtype],
            n, vocab, st, labels.data_ptr(), idt, offsets.data_ptr(), pairs, ref, wts, ctypes.byref(opts),
            float(grad_scale), tot, los, seq, lgp, sta, gp, gs)


def radamw_logits_grad(logits: torch.Tensor, labels: torch.Tensor, row_stats: torch.Tensor, grad: torch.Tensor,
                       upstream: Optional[torch.Tensor] = None, grad_scale: float = 1.0) -> None:
    """grad = upstream * grad_scale * the gradient either loss's records
    (row_stats) stand for; upstream is one FP32 value on the device."""
    lib = load()
    if grad is None:
        raise ValueError("grad must be a device tensor")
    dev, n, vocab, st, idt, gp, gs = _logits(logits, labels, grad)
    sta = _row_values(row_stats, "row_stats", 4 * n, dev.index)
    ups = _row_values(upstream, "upstream", 1, dev.index)
    _submit("radamw_logits_grad", lib.radamw_logits_grad, dev, logits.data_ptr(), _DTYPE_CODE[logits.dtype], n, vocab,
            st, labels.data_ptr(), idt, sta, ups, float(grad_scale), gp, gs)


# ----------------------------------------------------------- block operators --

def radamw_dropout_options_default() -> DropoutOptions:
    return load().radamw_dropout_options_default()


def radamw_residual_options_default() -> ResidualOptions:
    return load().radamw_residual_options_default()


def radamw_balance_options_default() -> BalanceOptions:
    return load().radamw_balance_options_default()


def radamw_dropout(x: torch.Tensor, out: torch.Tensor, opts: DropoutOptions) -> None:
    """out = x / keep where the generator keeps an element, else 0, for x and
    out [n, dim] of one dtype (out may be x)."""
    lib = load()
    dev = x.device
    xs = _rows2d(x, "x", dev)
    n, dim = x.shape
    os_ = _rows2d(out, "out", dev, n, dim)
    if out.dtype != x.dtype:
        raise ValueError(f"out must be {x.dtype} (got {out.dtype})")
    _submit("radamw_dropout", lib.radamw_dropout, dev, x.data_ptr(), _DTYPE_CODE[x.dtype], n, dim, xs,
            ctypes.byref(opts), out.data_ptr(), os_)


def _typed_rows(t: Optional[torch.Tensor], what: str, device, n: int, dim: int, dtype: torch.dtype):
    """(pointer, row stride) of an optional [n, dim] tensor of a dtype."""
    if t is None:
        return None, 0
    stride = _rows2d(t, what, device, n, dim)
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} (got {t.dtype})")
    return t.data_ptr(), stride


def _column_values(t: Optional[torch.Tensor], what: str, dim: int, dev_index: int, dtype: torch.dtype):
    """Pointer of an optional contiguous [dim] tensor of a dtype."""
    if t is None:
        return None
    try:
        good = t.dtype is dtype and t.numel() == dim and t.get_device() == dev_index and t.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        _check_fast(t, what, dev_index, dim, dtype)  # says what is wrong
    return t.data_ptr()


def _residual_block(like: torch.Tensor, stream_dtype, branch_dtype, branch, gate, rows_per_gate, post_weight,
                    pre_weight) -> _ResidualBlock:
    """The shapes and inputs that both residual calls share; ``like`` has the
    stream's shape and device."""
    dev = like.device
    n, dim = like.shape
    b = _ResidualBlock(n=n, dim=dim, stream_dtype=_DTYPE_CODE[stream_dtype], branch_dtype=_DTYPE_CODE[branch_dtype],
                       rows_per_gate=1)
    if branch is not None:
        b.branch, b.branch_stride = branch.data_ptr(), _rows2d(branch, "branch", dev, n, dim)
    if gate is not None:
        if rows_per_gate is None:  # one gate row for equal numbers of rows
            rows_per_gate = -(-n // max(1, gate.shape[0])) or 1
        b.rows_per_gate = int(rows_per_gate)
        if b.rows_per_gate < 1:
            raise ValueError(f"rows_per_gate must be at least 1 (got {rows_per_gate})")
        b.gate_stride = _rows2d(gate, "gate", dev, -(-n // b.rows_per_gate), dim)
        b.gate, b.gate_dtype = gate.data_ptr(), _DTYPE_CODE[gate.dtype]
    weight = post_weight if post_weight is not None else pre_weight
    if weight is not None:
        if weight.dtype not in _DTYPE_CODE:
            raise ValueError(f"weight dtype {weight.dtype} is not float32/float16/bfloat16")
        b.weight_dtype = _DTYPE_CODE[weight.dtype]
        b.post_weight = _column_values(post_weight, "post_weight", dim, dev.index, weight.dtype)
        b.pre_weight = _column_values(pre_weight, "pre_weight", dim, dev.index, weight.dtype)
    return b


def radamw_residual_norm(x: torch.Tensor, branch: Optional[torch.Tensor], opts: ResidualOptions, *,
                         gate: Optional[torch.Tensor] = None, rows_per_gate: Optional[int] = None,
                         post_weight: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
                         h: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         rstd: Optional[torch.Tensor] = None) -> None:
    """h = x + residual_scale * gate * drop(norm(branch) * post_weight) and out
    = norm(h) * pre_weight, for x, branch, h, out [n, dim], gate [ceil(n /
    rows_per_gate), dim], weights [dim] and rstd (2 n FP32, the norms' records
    for the gradient).  Absent: no gate, no such norm; without a branch only
    out is written.  h may be x, out may be the branch."""
    lib = load()
    dev = x.device
    xs = _rows2d(x, "x", dev)
    n, dim = x.shape
    kind = branch if branch is not None else out if out is not None else x
    if not isinstance(kind, torch.Tensor) or kind.dtype not in _DTYPE_CODE:
        raise ValueError("branch and out must be float32/float16/bfloat16 device tensors")
    b = _residual_block(x, x.dtype, kind.dtype, branch, gate, rows_per_gate, post_weight, pre_weight)
    hp, hs = _typed_rows(h, "h", dev, n, dim, x.dtype)
    op, os_ = _typed_rows(out, "out", dev, n, dim, kind.dtype)
    rp = _row_values(rstd, "rstd", 2 * n, dev.index)
    _submit("radamw_residual_norm", lib.radamw_residual_norm, dev, ctypes.byref(b), x.data_ptr(), xs,
            ctypes.byref(opts), hp, hs, op, os_, rp)


def radamw_residual_grad_workspace_bytes(n: int, dim: int, rows_per_gate: int = 1) -> int:
    r = load().radamw_residual_grad_workspace_bytes(n, dim, rows_per_gate)
    if r < 0:
        raise RadamwError(int(r), "radamw_residual_grad_workspace_bytes")
    return int(r)


def radamw_residual_norm_grad(h: Optional[torch.Tensor], branch: Optional[torch.Tensor], opts: ResidualOptions,
                              rstd: Optional[torch.Tensor], workspace: Optional[torch.Tensor], *,
                              grad_x: torch.Tensor, gate: Optional[torch.Tensor] = None,
                              rows_per_gate: Optional[int] = None, post_weight: Optional[torch.Tensor] = None,
                              pre_weight: Optional[torch.Tensor] = None, grad_h: Optional[torch.Tensor] = None,
                              grad_out: Optional[torch.Tensor] = None, grad_branch: Optional[torch.Tensor] = None,
                              grad_gate: Optional[torch.Tensor] = None,
                              grad_post_weight: Optional[torch.Tensor] = None,
                              grad_pre_weight: Optional[torch.Tensor] = None) -> None:
    """The gradients of radamw_residual_norm from grad_h and grad_out: grad_x
    and grad_branch [n, dim] (which may be grad_h and grad_out), and those
    asked for of grad_gate, grad_post_weight and grad_pre_weight.
    ``workspace`` holds at least radamw_residual_grad_workspace_bytes(n, dim,
    rows_per_gate) bytes (None where no weight's or shared gate's gradient is
    asked for)."""
    lib = load()
    dev = grad_x.device
    gxs = _rows2d(grad_x, "grad_x", dev)
    n, dim = grad_x.shape
    kind = branch if branch is not None else grad_out if grad_out is not None else grad_x
    if not isinstance(kind, torch.Tensor) or kind.dtype not in _DTYPE_CODE:
        raise ValueError("branch and grad_out must be float32/float16/bfloat16 device tensors")
    b = _residual_block(grad_x, grad_x.dtype, kind.dtype, branch, gate, rows_per_gate, post_weight, pre_weight)
    hp, hs = _typed_rows(h if pre_weight is not None else None, "h", dev, n, dim, grad_x.dtype)
    rp = _row_values(rstd, "rstd", 2 * n, dev.index)
    ghp, ghs = _typed_rows(grad_h, "grad_h", dev, n, dim, grad_x.dtype)
    gop, gos = _typed_rows(grad_out, "grad_out", dev, n, dim, kind.dtype)
    gbp, gbs = _typed_rows(grad_branch, "grad_branch", dev, n, dim, kind.dtype)
    ggp, ggs = (None, 0) if grad_gate is None or gate is None else _typed_rows(grad_gate, "grad_gate", dev,
                                                                              gate.shape[0], dim, gate.dtype)
    if grad_gate is not None and gate is None:
        raise ValueError("grad_gate without a gate")
    for g, w, what in ((grad_post_weight, post_weight, "post_weight"), (grad_pre_weight, pre_weight, "pre_weight")):
        if g is not None and w is None:
            raise ValueError(f"grad_{what} without a {what}")
    gpost = None if post_weight is None else _column_values(grad_post_weight, "grad_post_weight", dim, dev.index,
                                                            post_weight.dtype)
    gpre = None if pre_weight is None else _column_values(grad_pre_weight, "grad_pre_weight", dim, dev.index,
                                                          pre_weight.dtype)
    if workspace is not None:
        _dense(workspace, "workspace", device=dev)
    _submit("radamw_residual_norm_grad", lib.radamw_residual_norm_grad, dev, ctypes.byref(b), hp, hs, rp,
            ctypes.byref(opts), ghp, ghs, gop, gos, grad_x.data_ptr(), gxs, gbp, gbs, ggp, ggs, gpost, gpre,
            _ptr_or_none(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())


def _whole(t: torch.Tensor, what: str, n: int, dev_index: int, dtype: torch.dtype):
    """Pointer of a contiguous tensor of n values of a dtype."""
    return _column_values(t, what, n, dev_index, dtype)


def _balance_inputs(logits, offsets, mask, weights, groups, index_code):
    """Checked pointers of offsets, mask and weights, and the index type."""
    dev = logits.device
    n = logits.shape[0]
    off = None
    if offsets is not None:
        code = _index(offsets, "offsets", groups + 1, dev)
        if index_code is not None and code != index_code:
            raise ValueError(f"offsets must have the ids' type (got {offsets.dtype})")
        index_code, off = code, offsets.data_ptr()
    elif groups != 1:
        raise ValueError(f"{groups} groups need offsets")
    msk = None
    if mask is not None:
        if getattr(mask, "dtype", None) not in (torch.bool, torch.uint8):
            raise ValueError("mask must be a bool or uint8 tensor")
        msk = _whole(mask, "mask", n, dev.index, mask.dtype)
    return off, msk, _row_values(weights, "weights", groups, dev.index), index_code or 0


def radamw_balance_workspace_bytes(n: int, experts: int, groups: int = 1) -> int:
    r = load().radamw_balance_workspace_bytes(n, experts, groups)
    if r < 0:
        raise RadamwError(int(r), "radamw_balance_workspace_bytes")
    return int(r)


def radamw_balance_loss(logits: torch.Tensor, ids: torch.Tensor, opts: BalanceOptions, total: torch.Tensor,
                        loss: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor, mean_prob: torch.Tensor,
                        workspace: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                        offsets: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                        grad: Optional[torch.Tensor] = None, grad_scale: float = 1.0) -> None:
    """Balance loss of a router's logits [n, experts] with the experts ids [n,
    top_k] that were chosen: writes total (1), loss (groups), counts [groups,
    experts] and tokens (groups) (int32), mean_prob [groups, experts] and, when
    ``grad`` is given, grad_scale * d total / d logits (``grad`` may be
    ``logits``).  ``offsets`` (groups + 1, of the ids' type) give the rows of
    each group; without them all rows are one group."""
    lib = load()
    dev = logits.device
    st = _rows2d(logits, "logits", dev)
    n, experts = logits.shape
    di = dev.index
    if ids.dim() != 2 or ids.shape[0] != n:
        raise ValueError(f"ids must be [{n}, top_k] (got {tuple(ids.shape)})")
    top_k = ids.shape[1]
    idt = _index(ids, "ids", n * top_k, dev)
    groups = loss.numel()
    off, msk, wts, _ = _balance_inputs(logits, offsets, mask, weights, groups, idt)
    tot = _row_values(total, "total", 1, di)
    los = _row_values(loss, "loss", groups, di)
    cnt = _whole(counts, "counts", groups * experts, di, torch.int32)
    tok = _whole(tokens, "tokens", groups, di, torch.int32)
    mpr = _row_values(mean_prob, "mean_prob", groups * experts, di)
    gp, gs = _typed_rows(grad, "grad", dev, n, experts, logits.dtype)
    _dense(workspace, "workspace", device=dev)
    _submit("radamw_balance_loss", lib.radamw_balance_loss, dev, logits.data_ptr(), _DTYPE_CODE[logits.dtype], n,
            experts, st, ids.data_ptr(), idt, top_k, msk, off, groups, wts, ctypes.byref(opts), float(grad_scale), tot,
            los, cnt, tok, mpr, gp, gs, workspace.data_ptr(), workspace.numel() * workspace.element_size())


def radamw_balance_grad(logits: torch.Tensor, top_k: int, opts: BalanceOptions, counts: torch.Tensor,
                        tokens: torch.Tensor, grad: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                        offsets: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                        upstream: Optional[torch.Tensor] = None, grad_scale: float = 1.0) -> None:
    """grad = upstream * grad_scale * d total / d logits from the counts and
    tokens that radamw_balance_loss left; upstream is one FP32 value on the
    device."""
    lib = load()
    dev = logits.device
    st = _rows2d(logits, "logits", dev)
    n, experts = logits.shape
    di = dev.index
    groups = tokens.numel()
    off, msk, wts, idt = _balance_inputs(logits, offsets, mask, weights, groups, None)
    cnt = _whole(counts, "counts", groups * experts, di, torch.int32)
    tok = _whole(tokens, "tokens", groups, di, torch.int32)
    ups = _row_values(upstream, "upstream", 1, di)
    if grad is None:
        raise ValueError("grad must be a device tensor")
    gp, gs = _typed_rows(grad, "grad", dev, n, experts, logits.dtype)
    _submit("radamw_balance_grad", lib.radamw_balance_grad, dev, logits.data_ptr(), _DTYPE_CODE[logits.dtype], n,
            experts, st, int(top_k), msk, off, idt, groups, wts, ctypes.byref(opts), cnt, tok, ups, float(grad_scale),
            gp, gs)


def radamw_host_coefficients(opts: Options, t: int, gradient_scale: float = 1.0) -> list[float]:
    out = (ctypes.c_float * 9)()
    _check(load().radamw_host_coefficients(ctypes.byref(opts), t, float(gradient_scale), out),
           "radamw_host_coefficients")
    return list(out)


def radamw_status_string(status: int) -> str:
    return load().radamw_status_string(status).decode()


status_string = radamw_status_string


def radamw_last_hip_error() -> int:
    return load().radamw_last_hip_error()


def radamw_launch_count() -> int:
    return int(load().radamw_launch_count())


def radamw_time_next_update(start: Optional["torch.cuda.Event"], stop: Optional["torch.cuda.Event"]) -> None:
    """Record torch events at the first update kernel's start and the last
    one's end in the next launching update call on this thread.  The events
    must already exist on the device (recorded once)."""
    load().radamw_time_next_update(None if start is None else start.cuda_event,
                                   None if stop is None else stop.cuda_event)
