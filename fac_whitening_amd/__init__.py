"""Python binding of libgift (GIFT encode/decode on MI355X).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libgift.so`` (built from ``csrc/`` by ``build.py``).  PyTorch provides the
device memory and the current stream; nothing here computes on the data.
Importing this module raises if the library has not been built: there is no
fallback.

Function names follow the C ABI in ``include/gift.h``.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgift.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libgift.so not built ({LIB_PATH}); run `python -m fac_whitening_amd.build` "
                      "or __graft_entry__.build()")

_lib = ctypes.CDLL(LIB_PATH)

# enums (include/gift.h)
EUCLID, DIAG, LOWRANK, CHOL_INPUT, CHOL_TWOSIDED = range(5)
E4M3, E5M2, E2M1 = 0, 1, 2
SCALE_TENSOR, SCALE_BLOCK128, SCALE_BLOCK16, SCALE_BLOCK512 = 0, 1, 2, 3
BF16, FP32, FP16 = 0, 1, 2   # FP16: activation operators only
NORM_LAYER, NORM_RMS = 0, 1
ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SIGMOID = range(5)
SIDE_A, SIDE_G = 0, 1
LAYER_TRANSIENT_STATS = 1   # statistics windows committed in one call, S in the workspace
FLAG_NONFINITE, FLAG_SPIN_TIMEOUT = 1, 2
TRANSFORMS = {"euclid": EUCLID, "diag": DIAG, "lowrank": LOWRANK, "chol": CHOL_INPUT, "twosided": CHOL_TWOSIDED}
FORMATS = {"e4m3": E4M3, "e5m2": E5M2}
NORMS = {"layer": NORM_LAYER, "rms": NORM_RMS}
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU, "sigmoid": ACT_SIGMOID}
DTYPES = {torch.bfloat16: BF16, torch.float32: FP32, torch.float16: FP16}
SCALINGS = {"tensor": SCALE_TENSOR, "block": SCALE_BLOCK128}
STATUS = {0: "GIFT_OK", 1: "GIFT_ERR_INVALID_ARG", 2: "GIFT_ERR_WORKSPACE", 3: "GIFT_ERR_NOT_READY",
          4: "GIFT_ERR_NUMERICAL", 5: "GIFT_ERR_UNSUPPORTED", 6: "GIFT_ERR_HIP"}

EXPORTS = [
    "gift_layer_state_bytes", "gift_layer_create", "gift_layer_destroy", "gift_layer_get_counters",
    "gift_layer_set_counters", "gift_layer_flags", "gift_layer_buffers", "gift_layer_mark_ready",
    "gift_accumulate_stats", "gift_commit_stats", "gift_refresh_factors", "gift_encode", "gift_encode_ef",
    "gift_decode_reduce", "gift_encode_fp4", "gift_decode_reduce_fp4", "gift_payload_bytes", "gift_profiler_create", "gift_profiler_destroy",
    "gift_profiler_workspace_bytes", "gift_profile_step", "gift_select_layers", "gift_status_string",
    "gift_last_hip_error", "gift_set_fused", "gift_bucket_table_bytes", "gift_bucket_create",
    "gift_bucket_destroy", "gift_bucket_sizes", "gift_bucket_flags", "gift_bucket_amax", "gift_bucket_encode",
    "gift_bucket_decode_reduce", "gift_scale_sync_due", "gift_set_max_resident", "gift_layer_route",
    "gift_bucket_encode_static", "gift_group_table_bytes", "gift_group_create", "gift_group_destroy",
    "gift_group_encode", "gift_group_decode_reduce",
    "gift_act_scale_bytes", "gift_act_save", "gift_act_restore", "gift_norm_forward", "gift_norm_workspace_bytes",
    "gift_norm_backward", "gift_weight_grad_workspace_bytes", "gift_weight_grad",
    "gift_weight_grad_x_workspace_bytes", "gift_weight_grad_x", "gift_dropout_apply", "gift_glu_workspace_bytes",
    "gift_glu_forward", "gift_glu_backward_workspace_bytes", "gift_glu_backward",
]


class GroupItem(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_void_p), ("d_W", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("d_codes", ctypes.c_void_p), ("d_scales", ctypes.c_void_p), ("d_rcodes", ctypes.c_void_p),
                ("code_stride", ctypes.c_int64), ("d_rscales", ctypes.c_void_p), ("scale_stride", ctypes.c_int64),
                ("d_out", ctypes.c_void_p), ("ldo", ctypes.c_int64)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int32), ("d_in", ctypes.c_int32), ("transform", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("oversample", ctypes.c_int32), ("power_iters", ctypes.c_int32),
                ("ema_decay", ctypes.c_float), ("damping_rel", ctypes.c_float), ("flags", ctypes.c_int32)]


class ActCkpt(ctypes.Structure):
    _fields_ = [("d_codes", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("d_bscales", ctypes.c_void_p),
                ("fmt", ctypes.c_int32)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("d_offset", ctypes.c_void_p)]


_vp, _sz, _i32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_P = ctypes.POINTER


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("gift_layer_state_bytes", _i32, _P(LayerDesc), _P(_sz), _P(_sz))
_sig("gift_layer_create", _i32, _P(LayerDesc), _vp, _sz, _vp, _P(_vp))
_sig("gift_layer_destroy", _i32, _vp)
_sig("gift_layer_get_counters", _i32, _vp, _P(_i64))
_sig("gift_layer_set_counters", _i32, _vp, _P(_i64))
_sig("gift_layer_flags", _i32, _vp, _vp, _P(ctypes.c_uint32))
_sig("gift_layer_buffers", _i32, _vp, *[_P(_vp)] * 8)
_sig("gift_layer_mark_ready", _i32, _vp, _vp)
_sig("gift_accumulate_stats", _i32, _vp, _i32, _vp, _i32, _i64, _i64, _i32, _vp, _sz, _vp)
_sig("gift_commit_stats", _i32, _vp, _i32, _vp)
_sig("gift_refresh_factors", _i32, _vp, _vp, _vp, _sz, _vp)
_sig("gift_encode", _i32, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("gift_encode_ef", _i32, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("gift_encode_fp4", _i32, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("gift_decode_reduce_fp4", _i32, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _sz, _vp)
_sig("gift_decode_reduce", _i32, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _sz, _vp)
_sig("gift_payload_bytes", _sz, _i32, _i32, _i32)
_sig("gift_profiler_create", _i32, _i32, _i32, _i32, _vp, _vp, _P(_vp))
_sig("gift_profiler_destroy", _i32, _vp)
_sig("gift_profiler_workspace_bytes", _sz, _i32, _i32, _i64)
_sig("gift_profile_step", _i32, _vp, _i32, _P(_vp), _P(_i64), _vp, _sz, _vp)
_sig("gift_select_layers", _i32, _vp, _i32, _P(ctypes.c_double), _P(_i32), _P(_i32), _P(_i32), _vp)
_sig("gift_status_string", ctypes.c_char_p, _i32)
_sig("gift_last_hip_error", _i32)
_sig("gift_set_fused", _i32, _i32)
_sig("gift_set_max_resident", _i32, _i32)
_sig("gift_layer_route", _i32, _vp, _i32, _i64, _i32, _P(_i32))
_sig("gift_bucket_table_bytes", _sz, _i32)
_sig("gift_bucket_create", _i32, _i32, _P(_i64), _i32, _vp, _sz, _vp, _P(_vp))
_sig("gift_bucket_destroy", _i32, _vp)
_sig("gift_bucket_sizes", _i32, _vp, _P(_i64), _P(_i64), _P(_sz))
_sig("gift_bucket_flags", _i32, _vp, _vp, _P(ctypes.c_uint32))
_sig("gift_bucket_amax", _i32, _vp, _vp, _vp, _vp)
_sig("gift_bucket_encode", _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("gift_bucket_encode_static", _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp)
_sig("gift_bucket_decode_reduce", _i32, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp)
_sig("gift_scale_sync_due", _i32, _i64, _i32)
_sig("gift_group_table_bytes", _sz, _i32)
_sig("gift_group_create", _i32, _i32, _P(GroupItem), _i32, _i32, _i32, _vp, _sz, _vp, _P(_vp))
_sig("gift_group_destroy", _i32, _vp)
_sig("gift_group_encode", _i32, _vp, _vp)
_sig("gift_group_decode_reduce", _i32, _vp, _vp)
_f32 = ctypes.c_float
_sig("gift_act_scale_bytes", _sz, _i64, _i32)
_sig("gift_act_save", _i32, _vp, _i32, _i64, _i64, _i32, _P(ActCkpt), _vp)
_sig("gift_act_restore", _i32, _P(ActCkpt), _i64, _i32, _vp, _i32, _i64, _vp)
_sig("gift_norm_forward", _i32, _i32, _vp, _i32, _i64, _i64, _i32, _vp, _vp, _i32, _f32, _vp, _i64, _vp, _vp,
     _P(ActCkpt), _vp)
_sig("gift_norm_workspace_bytes", _sz, _i64, _i32)
_sig("gift_norm_backward", _i32, _i32, _vp, _i32, _i64, _vp, _i64, _P(ActCkpt), _i64, _i32, _vp, _i32, _vp, _vp, _vp,
     _i64, _vp, _vp, _i32, _vp, _sz, _vp)
_sig("gift_weight_grad_workspace_bytes", _sz, _i64, _i32, _i32, _i32)
_sig("gift_weight_grad", _i32, _vp, _i32, _i64, _i32, _P(ActCkpt), _i64, _i32, _f32, _i32, _vp, _i64, _vp, _sz, _vp)
_sig("gift_weight_grad_x_workspace_bytes", _sz, _i64, _i32, _i32, _i32, _i32)
_sig("gift_weight_grad_x", _i32, _vp, _i32, _i64, _i32, _vp, _i64, _i64, _i32, _f32, _i32, _vp, _i64, _vp, _sz, _vp)
_sig("gift_dropout_apply", _i32, _P(DropoutDesc), _vp, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp)
_sig("gift_glu_workspace_bytes", _sz, _i64, _i32, _i32, _i32, _i32)
_sig("gift_glu_forward", _i32, _i32, _vp, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _P(DropoutDesc), _vp,
     _i64, _vp, _i64, _vp, _i64, _P(ActCkpt), _vp, _sz, _vp)
_sig("gift_glu_backward_workspace_bytes", _sz, _i64, _i32, _i32, _i32, _i32)
_sig("gift_glu_backward", _i32, _i32, _vp, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _P(DropoutDesc), _vp, _i64,
     _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _sz, _vp)


def set_fused(enable: bool) -> bool:
    """Select the persistent single-launch rank-k kernels (True, default) or
    the multi-kernel path (False); returns the previous setting."""
    return bool(_lib.gift_set_fused(1 if enable else 0))


def set_max_resident(max_groups: int) -> int:
    """Cap the workgroups persistent launches may count on being resident at
    once (0: the device's own limit); returns the previous cap."""
    return int(_lib.gift_set_max_resident(int(max_groups)))


class GiftError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = f"{where}: {STATUS.get(status, status)} ({_lib.gift_status_string(status).decode()})"
        if status == 6:
            msg += f", hipError {_lib.gift_last_hip_error()}"
        super().__init__(msg)
        self.status = status


def _check(status: int, where: str):
    if status != 0:
        raise GiftError(status, where)


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def nblocks(m: int, d: int, scaling: int) -> int:
    return 1 if scaling == SCALE_TENSOR else -(-m // 128) * -(-d // 128)


def payload_bytes(d_out: int, d_in: int, scaling: int) -> int:
    return int(_lib.gift_payload_bytes(d_out, d_in, scaling))


def _alloc(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class Layer:
    """One layer's state and calls (gift_layer_*)."""

    def __init__(self, d_out: int, d_in: int, transform="lowrank", rank: int = 32, oversample: int = 16,
                 power_iters: int = 4, ema_decay: float = 0.0, damping_rel: float = 1e-3, device="cuda",
                 stream=None, workspace=None, transient_stats: bool = False):
        tr = TRANSFORMS[transform] if isinstance(transform, str) else int(transform)
        self.desc = LayerDesc(d_out, d_in, tr, rank, oversample, power_iters, ema_decay, damping_rel,
                              LAYER_TRANSIENT_STATS if transient_stats else 0)
        sb, wb = _sz(), _sz()
        _check(_lib.gift_layer_state_bytes(ctypes.byref(self.desc), ctypes.byref(sb), ctypes.byref(wb)),
               "gift_layer_state_bytes")
        self.device = torch.device(device)
        self.state = _alloc(sb.value, self.device)
        self.work_bytes = wb.value
        self.work = workspace if workspace is not None else _alloc(wb.value, self.device)
        h = _vp()
        _check(_lib.gift_layer_create(ctypes.byref(self.desc), _ptr(self.state), sb.value, _stream(stream),
                                      ctypes.byref(h)), "gift_layer_create")
        self._h = h
        self.m, self.d, self.k = d_out, d_in, rank

    # -- lifecycle ---------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            _lib.gift_layer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def counters(self):
        arr = (_i64 * 8)()
        _check(_lib.gift_layer_get_counters(self._h, arr), "gift_layer_get_counters")
        return list(arr)

    def set_counters(self, vals):
        arr = (_i64 * 8)(*vals)
        _check(_lib.gift_layer_set_counters(self._h, arr), "gift_layer_set_counters")

    def flags(self, stream=None) -> int:
        f = ctypes.c_uint32()
        _check(_lib.gift_layer_flags(self._h, _stream(stream), ctypes.byref(f)), "gift_layer_flags")
        return f.value

    def buffers(self) -> dict:
        """Views into the state buffer (device tensors), by name."""
        ptrs = [_vp() for _ in range(8)]
        _check(_lib.gift_layer_buffers(self._h, *[ctypes.byref(p) for p in ptrs]), "gift_layer_buffers")
        names = ["A", "G", "U", "coef", "tinv_a", "t_a", "lg_inv", "lg"]
        m, d = self.m, self.d
        shapes = {"A": (d, d), "G": (m, m), "U": (d, 32), "tinv_a": (d, d), "t_a": (d, d), "lg_inv": (m, m),
                  "lg": (m, m), "coef": (68,) if self.desc.transform == LOWRANK else (2 * d,)}
        base = self.state.data_ptr()
        out = {}
        for n, p in zip(names, ptrs):
            if not p.value:
                continue
            off = p.value - base
            cnt = 1
            for s in shapes[n]:
                cnt *= s
            out[n] = self.state[off:off + 4 * cnt].view(torch.float32).view(*shapes[n])
        return out

    def route(self, op: str, ld=None, R: int = 1) -> str:
        """'fused' or 'multi': the route gift_encode (op='encode') or
        gift_decode_reduce (op='decode') takes for this layer now."""
        f = _i32()
        _check(_lib.gift_layer_route(self._h, 0 if op == "encode" else 1, self.d if ld is None else ld, R,
                                     ctypes.byref(f)), "gift_layer_route")
        return "fused" if f.value else "multi"

    def mark_ready(self, stream=None):
        _check(_lib.gift_layer_mark_ready(self._h, _stream(stream)), "gift_layer_mark_ready")

    # -- statistics / refresh --------------------------------------------
    def accumulate_stats(self, x: torch.Tensor, side: int = SIDE_A, commit: bool = False, stream=None):
        dtype = BF16 if x.dtype == torch.bfloat16 else FP32
        if x.dtype not in (torch.bfloat16, torch.float32) or x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("x must be a row-major [T][n] bf16 or fp32 tensor")
        _check(_lib.gift_accumulate_stats(self._h, side, _ptr(x), dtype, x.shape[0], x.stride(0), int(commit),
                                          _ptr(self.work), self.work_bytes, _stream(stream)), "gift_accumulate_stats")

    def commit_stats(self, side: int = SIDE_A, stream=None):
        _check(_lib.gift_commit_stats(self._h, side, _stream(stream)), "gift_commit_stats")

    def refresh(self, omega=None, stream=None):
        _check(_lib.gift_refresh_factors(self._h, _ptr(omega), _ptr(self.work), self.work_bytes, _stream(stream)),
               "gift_refresh_factors")

    # -- encode / decode --------------------------------------------------
    def encode(self, W: torch.Tensor, fmt=E4M3, scaling=SCALE_TENSOR, amax_in=None, codes=None, scales=None,
               amax_out=None, whitened=None, want_codes=True, resid=None, stream=None):
        fmt = FORMATS.get(fmt, fmt)
        scaling = SCALINGS.get(scaling, scaling)
        m, d = self.m, self.d
        nb = nblocks(m, d, scaling)
        if W.dtype != torch.float32 or W.shape != (m, d) or W.stride(1) != 1:
            raise ValueError("W must be fp32 [d_out][d_in] with unit column stride")
        if want_codes:
            if codes is None:
                codes = torch.empty(m, d, dtype=torch.uint8, device=W.device)
            if scales is None:
                scales = torch.empty(nb, dtype=torch.float32, device=W.device)
        if resid is None:
            _check(_lib.gift_encode(self._h, _ptr(W), W.stride(0), fmt, scaling, _ptr(amax_in), _ptr(amax_out),
                                    _ptr(codes) if want_codes else None, _ptr(scales) if want_codes else None,
                                    _ptr(whitened), _ptr(self.work), self.work_bytes, _stream(stream)), "gift_encode")
        else:
            if resid.dtype != torch.float32 or resid.shape != (m, d) or not resid.is_contiguous():
                raise ValueError("resid must be a contiguous fp32 [d_out][d_in] tensor")
            _check(_lib.gift_encode_ef(self._h, _ptr(W), W.stride(0), fmt, scaling, _ptr(amax_in), _ptr(amax_out),
                                       _ptr(codes) if want_codes else None, _ptr(scales) if want_codes else None,
                                       _ptr(whitened), _ptr(resid), _ptr(self.work), self.work_bytes,
                                       _stream(stream)), "gift_encode_ef")
        return codes, scales

    def decode_reduce(self, codes: torch.Tensor, scales: torch.Tensor, fmt=E4M3, scaling=SCALE_TENSOR, out=None,
                      R=None, stream=None):
        """codes [R][m][d] uint8, scales [R][nblk] fp32 (contiguous replicas)."""
        fmt = FORMATS.get(fmt, fmt)
        scaling = SCALINGS.get(scaling, scaling)
        m, d = self.m, self.d
        if codes.dim() == 2:
            codes = codes.unsqueeze(0)
            scales = scales.reshape(1, -1)
        R = codes.shape[0] if R is None else R
        if out is None:
            out = torch.empty(m, d, dtype=torch.float32, device=codes.device)
        cs = codes.stride(0) if R > 1 else m * d
        ss = scales.stride(0) if R > 1 else scales.shape[-1]
        _check(_lib.gift_decode_reduce(self._h, _ptr(codes), cs, _ptr(scales), ss, R, fmt, scaling, _ptr(out),
                                       out.stride(0), _ptr(self.work), self.work_bytes, _stream(stream)),
               "gift_decode_reduce")
        return out

    def encode_fp4(self, W: torch.Tensor, amax_in=None, codes=None, bscales=None, tscale=None, amax_out=None,
                   whitened=None, want_codes=True, resid=None, stream=None):
        """FP4 payload: codes [m][d/2] uint8 (two per byte, even column low),
        bscales [m][d/16] uint8 (E4M3), tscale [1] fp32."""
        m, d = self.m, self.d
        if W.dtype != torch.float32 or W.shape != (m, d) or W.stride(1) != 1:
            raise ValueError("W must be fp32 [d_out][d_in] with unit column stride")
        if resid is not None and (resid.dtype != torch.float32 or resid.shape != (m, d) or not resid.is_contiguous()):
            raise ValueError("resid must be a contiguous fp32 [d_out][d_in] tensor")
        if want_codes:
            if codes is None:
                codes = torch.empty(m, d // 2, dtype=torch.uint8, device=W.device)
            if bscales is None:
                bscales = torch.empty(m, d // 16, dtype=torch.uint8, device=W.device)
            if tscale is None:
                tscale = torch.empty(1, dtype=torch.float32, device=W.device)
        _check(_lib.gift_encode_fp4(self._h, _ptr(W), W.stride(0), _ptr(amax_in), _ptr(amax_out),
                                    _ptr(codes) if want_codes else None, _ptr(bscales) if want_codes else None,
                                    _ptr(tscale) if want_codes else None, _ptr(whitened), _ptr(resid),
                                    _ptr(self.work), self.work_bytes, _stream(stream)), "gift_encode_fp4")
        return codes, bscales, tscale

    def decode_reduce_fp4(self, codes: torch.Tensor, bscales: torch.Tensor, tscales: torch.Tensor, out=None,
                          stream=None):
        """codes [R][m][d/2], bscales [R][m][d/16] uint8, tscales [R] fp32."""
        m, d = self.m, self.d
        if codes.dim() == 2:
            codes, bscales = codes.unsqueeze(0), bscales.unsqueeze(0)
        R = codes.shape[0]
        tscales = tscales.reshape(-1)
        if tscales.numel() < R or tscales.dtype != torch.float32 or not tscales.is_contiguous():
            raise ValueError("tscales must be a contiguous fp32 tensor of R entries")
        if out is None:
            out = torch.empty(m, d, dtype=torch.float32, device=codes.device)
        cs = codes.stride(0) if R > 1 else m * d // 2
        bs = bscales.stride(0) if R > 1 else m * d // 16
        _check(_lib.gift_decode_reduce_fp4(self._h, _ptr(codes), cs, _ptr(bscales), bs, _ptr(tscales), R, _ptr(out),
                                           out.stride(0), _ptr(self.work), self.work_bytes, _stream(stream)),
               "gift_decode_reduce_fp4")
        return out


class Profiler:
    """FP8 boundary-hit profiler over a list of layers (gift_profiler_*)."""

    def __init__(self, n_layers: int, fmt=E4M3, scaling=SCALE_TENSOR, device="cuda", stream=None):
        self.n = n_layers
        self.counts = torch.zeros(n_layers, 2, dtype=torch.int64, device=device)
        self.work_bytes = int(_lib.gift_profiler_workspace_bytes(n_layers, scaling, 0))
        self.work = _alloc(self.work_bytes, device)
        h = _vp()
        _check(_lib.gift_profiler_create(n_layers, FORMATS.get(fmt, fmt), SCALINGS.get(scaling, scaling),
                                         _ptr(self.counts), _stream(stream), ctypes.byref(h)), "gift_profiler_create")
        self._h = h

    def step(self, grads, stream=None):
        ptrs = (_vp * self.n)(*[g.data_ptr() for g in grads])
        numel = (_i64 * self.n)(*[g.numel() for g in grads])
        for g in grads:
            if g.dtype != torch.float32 or not g.is_contiguous():
                raise ValueError("gradients must be contiguous fp32")
        _check(_lib.gift_profile_step(self._h, self.n, ptrs, numel, _ptr(self.work), self.work_bytes,
                                      _stream(stream)), "gift_profile_step")

    def select(self, max_select: int, stream=None):
        sc = (ctypes.c_double * self.n)()
        order = (_i32 * self.n)()
        sel = (_i32 * self.n)()
        nsel = _i32()
        _check(_lib.gift_select_layers(self._h, max_select, sc, order, sel, ctypes.byref(nsel), _stream(stream)),
               "gift_select_layers")
        return list(sc), list(order), list(sel[:nsel.value])

    def close(self):
        if getattr(self, "_h", None):
            _lib.gift_profiler_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def scale_sync_due(step: int, period: int) -> bool:
    """Whether `step` is a scale-sync step of a schedule syncing every
    `period` steps (gift_scale_sync_due)."""
    return bool(_lib.gift_scale_sync_due(step, period))


class Bucket:
    """Flat gradient bucket of Euclidean tensors (gift_bucket_*): the tensors
    of `sizes` elements lie one after another in one flat fp32 buffer."""

    def __init__(self, sizes, scaling=SCALE_TENSOR, device="cuda", stream=None):
        self.sizes = [int(n) for n in sizes]
        self.scaling = SCALINGS.get(scaling, scaling)
        n = len(self.sizes)
        tb = int(_lib.gift_bucket_table_bytes(n))
        self.table = _alloc(tb, device)
        arr = (_i64 * n)(*self.sizes)
        h = _vp()
        _check(_lib.gift_bucket_create(n, arr, self.scaling, _ptr(self.table), tb, _stream(stream), ctypes.byref(h)),
               "gift_bucket_create")
        self._h = h
        ne, ns, wb = _i64(), _i64(), _sz()
        _check(_lib.gift_bucket_sizes(h, ctypes.byref(ne), ctypes.byref(ns), ctypes.byref(wb)), "gift_bucket_sizes")
        self.numel, self.nscales, self.work_bytes = ne.value, ns.value, wb.value
        self.work = _alloc(max(self.work_bytes, 256), device)

    def _grad(self, g):
        if g.dtype != torch.float32 or not g.is_contiguous() or g.numel() < self.numel:
            raise ValueError("the bucket needs a contiguous fp32 buffer of all its elements")

    def amax(self, grad, amax_out=None, stream=None):
        self._grad(grad)
        if amax_out is None:
            amax_out = torch.empty(self.nscales, dtype=torch.float32, device=grad.device)
        _check(_lib.gift_bucket_amax(self._h, _ptr(grad), _ptr(amax_out), _stream(stream)), "gift_bucket_amax")
        return amax_out

    def encode(self, grad, fmt=E4M3, amax_in=None, amax_out=None, codes=None, scales=None, stream=None):
        self._grad(grad)
        if codes is None:
            codes = torch.empty(self.numel, dtype=torch.uint8, device=grad.device)
        if scales is None:
            scales = torch.empty(self.nscales, dtype=torch.float32, device=grad.device)
        _check(_lib.gift_bucket_encode(self._h, _ptr(grad), FORMATS.get(fmt, fmt), _ptr(amax_in), _ptr(amax_out),
                                       _ptr(codes), _ptr(scales), _ptr(self.work), self.work_bytes, _stream(stream)),
               "gift_bucket_encode")
        return codes, scales

    def encode_static(self, grad, fmt=E4M3, amax_in=None, amax_out=None, codes=None, scales=None, stream=None):
        """gift_bucket_encode_static: the encode without a workspace (the
        library's per-device scratch array holds the amax slots)."""
        self._grad(grad)
        if codes is None:
            codes = torch.empty(self.numel, dtype=torch.uint8, device=grad.device)
        if scales is None:
            scales = torch.empty(self.nscales, dtype=torch.float32, device=grad.device)
        _check(_lib.gift_bucket_encode_static(self._h, _ptr(grad), FORMATS.get(fmt, fmt), _ptr(amax_in),
                                              _ptr(amax_out), _ptr(codes), _ptr(scales), _stream(stream)),
               "gift_bucket_encode_static")
        return codes, scales

    def decode_reduce(self, codes, scales, fmt=E4M3, out=None, stream=None):
        """codes [R][numel] uint8, scales [R][nscales] fp32."""
        if codes.dim() == 1:
            codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
        R = codes.shape[0]
        if out is None:
            out = torch.empty(self.numel, dtype=torch.float32, device=codes.device)
        cs = codes.stride(0) if R > 1 else self.numel
        ss = scales.stride(0) if R > 1 else self.nscales
        _check(_lib.gift_bucket_decode_reduce(self._h, _ptr(codes), cs, _ptr(scales), ss, R, FORMATS.get(fmt, fmt),
                                              _ptr(out), _stream(stream)), "gift_bucket_decode_reduce")
        return out

    def flags(self, stream=None) -> int:
        f = ctypes.c_uint32()
        _check(_lib.gift_bucket_flags(self._h, _stream(stream), ctypes.byref(f)), "gift_bucket_flags")
        return f.value

    def close(self):
        if getattr(self, "_h", None):
            _lib.gift_bucket_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Group:
    """Grouped rank-k layers (gift_group_*): one launch encodes all of them,
    one launch decode-reduces all of them.  items: a list of dicts with the
    layer (a Layer), W, codes, scales (this worker's payload), rcodes
    [R][m][d], rscales [R][nblk] (the payloads to decode) and out."""

    def __init__(self, items, R, fmt=E4M3, scaling=SCALE_TENSOR, device="cuda", stream=None):
        n = len(items)
        arr = (GroupItem * n)()
        self._keep = items
        for k, it in enumerate(items):
            L = it["layer"]
            rc, rs = it["rcodes"], it["rscales"]
            arr[k] = GroupItem(L.handle, it["W"].data_ptr(), it["W"].stride(0), it["codes"].data_ptr(),
                               it["scales"].data_ptr(), rc.data_ptr(), rc.stride(0) if R > 1 else L.m * L.d,
                               rs.data_ptr(), rs.stride(0) if R > 1 else rs.shape[-1], it["out"].data_ptr(),
                               it["out"].stride(0))
        tb = int(_lib.gift_group_table_bytes(n))
        self.table = _alloc(tb, device)
        h = _vp()
        _check(_lib.gift_group_create(n, arr, R, FORMATS.get(fmt, fmt), SCALINGS.get(scaling, scaling),
                                      _ptr(self.table), tb, _stream(stream), ctypes.byref(h)), "gift_group_create")
        self._h = h

    def encode(self, stream=None):
        _check(_lib.gift_group_encode(self._h, _stream(stream)), "gift_group_encode")

    def decode_reduce(self, stream=None):
        _check(_lib.gift_group_decode_reduce(self._h, _stream(stream)), "gift_group_decode_reduce")

    def close(self):
        if getattr(self, "_h", None):
            _lib.gift_group_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# -- activation operators (gift_act_*, gift_norm_*, gift_weight_grad*) -----------
# What these functions allocate (outputs not given, workspaces) comes from the
# allocator's pool of the stream they launch on, so it may be dropped as soon
# as the call returns; tensors the caller passes are the caller's to order.
# All operands of a call are on one device, the current one.  The functions
# record no graph, also where an operand requires a gradient: a module of
# theirs calls the backward functions from its own torch.autograd.Function.

# Small calls cost what the host does (a launch is about 4 us, a current_stream
# object 3, an allocation 2), so these wrappers do each thing once.

def _rows(t, what, T=None, n=None, dtype=None, device=None):
    """Checks a [T][n] tensor with unit column stride (on `device`, or on any GPU); returns its leading dimension."""
    dt, shape = t.dtype, t.shape
    if dt not in DTYPES or len(shape) != 2 or (dtype is not None and dt != dtype):
        raise ValueError(f"{what} must be a [T][n] tensor of {dtype or 'bf16, fp16 or fp32'}")
    rows, cols = shape
    if (T is not None and rows != T) or (n is not None and cols != n):
        raise ValueError(f"{what} must have shape [{T}][{n}], not {tuple(shape)}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what} must have unit column stride")
    if not t.is_cuda if device is None else t.device != device:
        raise ValueError(f"{what} must be on {device or 'the GPU'}")
    return ld if rows > 1 else max(cols, 1)


def _vector(t, what, n, dtypes, device):
    """Checks a dense vector; returns its address (None for None)."""
    if t is None:
        return None
    if t.shape != (n,) or t.dtype not in dtypes or (n > 1 and t.stride(0) != 1) or t.device != device:
        raise ValueError(f"{what} must be a dense vector of {n} {' or '.join(map(str, dtypes))} on {device}")
    return t.data_ptr()


def _empty(stream, shape, dtype, device):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(stream, t):
    """A dense tensor of t's shape and type."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)      # a little quicker than torch.empty
    return _empty(stream, t.shape, t.dtype, t.device)


def _raw_stream(stream, device):
    """Handle of the stream, or of the current one, for a call whose operands are on `device`."""
    here = torch._C._cuda_getDevice()
    if device.index != here or (stream is not None and stream.device != device):
        raise ValueError(f"operands on {device} need that device to be the current one, and its streams")
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _on(device, t, what):
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")


def _bytes(device, t, what):
    """Bytes behind the address of a dense tensor of any type."""
    _on(device, t, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.numel() * t.element_size()


def _kind(kind):
    kind = NORMS.get(kind, kind)
    if kind not in (NORM_LAYER, NORM_RMS):
        raise ValueError(f"kind must be one of {', '.join(NORMS)}, not {kind!r}")
    return kind


_F32 = (torch.float32,)
_WEIGHTS = {t: (t, torch.float32) for t in DTYPES}


class ActCheckpoint:
    """8-bit checkpoint of a [T][d] activation (gift_act_*): codes [T][ldc]
    uint8 with ldc = d rounded up to 32, and bscales
    [ceil(T / 8)][ceil(d / 32)][8] uint8, the biased exponent of the scale of
    each token and 32 columns.  Buffers that are not given are allocated (on
    `stream`'s pool); given ones are used as they are, so a checkpoint kept
    elsewhere can be wrapped without a copy.  The buffers' addresses are taken
    here: other buffers need another checkpoint."""

    _FIXED = frozenset(("T", "d", "fmt", "codes", "bscales", "device"))

    def __init__(self, T: int, d: int, fmt=E4M3, codes=None, bscales=None, device="cuda", stream=None):
        T, d, fmt = int(T), int(d), FORMATS.get(fmt, fmt)
        if T < 0 or d < 1 or fmt not in (E4M3, E5M2):
            raise ValueError("a checkpoint needs T >= 0, d >= 1 and the format E4M3 or E5M2")
        nb, groups = -(-d // 32), -(-T // 8)
        if codes is None:
            codes = _empty(stream, (T, nb * 32), torch.uint8, device)
        elif codes.dtype != torch.uint8 or codes.dim() != 2 or codes.shape[0] != T or (
                codes.shape[1] < nb * 32) or codes.stride(1) != 1:
            raise ValueError(f"codes must be a uint8 [{T}][>= {nb * 32}] tensor on the GPU with unit column stride")
        if not codes.is_cuda:
            raise ValueError("a checkpoint must be on the GPU")
        if bscales is None:
            bscales = _empty(stream, (groups, nb, 8), torch.uint8, codes.device)
        elif bscales.dtype != torch.uint8 or bscales.numel() != groups * nb * 8 or not bscales.is_contiguous() or (
                bscales.device != codes.device):
            raise ValueError(f"bscales must be a contiguous uint8 [{groups}][{nb}][8] tensor beside the codes")
        c = ActCkpt(codes.data_ptr(), codes.stride(0) if T > 1 else codes.shape[1] // 32 * 32, bscales.data_ptr(), fmt)
        self.__dict__.update(T=T, d=d, fmt=fmt, codes=codes, bscales=bscales, device=codes.device, _c=c,
                             _ref=ctypes.byref(c))

    def __setattr__(self, name, value):
        if name in self._FIXED:
            raise AttributeError(f"a checkpoint's {name} cannot be replaced")
        super().__setattr__(name, value)

    def nbytes(self) -> int:
        return self.codes.numel() + self.bscales.numel()

    def save(self, x: torch.Tensor, stream=None):
        ld = _rows(x, "x", self.T, self.d, device=self.device)
        _check(_lib.gift_act_save(x.data_ptr(), DTYPES[x.dtype], ld, self.T, self.d, self._ref,
                                  _raw_stream(stream, self.device)), "gift_act_save")
        return self

    def restore(self, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
        raw = _raw_stream(stream, self.device)
        if out is None:
            if dtype not in DTYPES:
                raise ValueError(f"a checkpoint restores to bf16, fp16 or fp32, not to {dtype}")
            out, ld = _empty(stream, (self.T, self.d), dtype, self.device), self.d
        else:
            ld = _rows(out, "out", self.T, self.d, device=self.device)
        _check(_lib.gift_act_restore(self._ref, self.T, self.d, out.data_ptr(), DTYPES[out.dtype], ld, raw),
               "gift_act_restore")
        return out


def norm_forward(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5, kind="layer", ckpt=None, out=None,
                 stream=None):
    """Layer norm (kind "layer") or RMS norm ("rms") of the rows of x [T][d]:
    returns y (of x's type), mean (None for "rms") and rstd, fp32 [T].  With
    `ckpt` (an ActCheckpoint of the same T and d) x is also saved there.
    weight and bias: of x's type or both fp32."""
    kind = _kind(kind)
    ld = _rows(x, "x")
    (T, d), dev, dt = x.shape, x.device, x.dtype
    raw = _raw_stream(stream, dev)
    wt = weight.dtype if weight is not None else bias.dtype if bias is not None else dt
    wp = _vector(weight, "weight", d, _WEIGHTS[dt], dev)
    bp = _vector(bias, "bias", d, _WEIGHTS[dt] if weight is None else (wt,), dev)
    if ckpt is not None:
        if (ckpt.T, ckpt.d) != (T, d):
            raise ValueError("the checkpoint has another shape than x")
        _on(dev, ckpt, "the checkpoint")
    if out is None:
        y, ldy = _empty_like(stream, x), d
    else:
        y, ldy = out, _rows(out, "out", T, d, dt, dev)
    mean = _empty(stream, (T,), torch.float32, dev) if kind == NORM_LAYER else None
    rstd = _empty(stream, (T,), torch.float32, dev)
    _check(_lib.gift_norm_forward(kind, x.data_ptr(), DTYPES[dt], ld, T, d, wp, bp, DTYPES[wt], eps, y.data_ptr(), ldy,
                                  None if mean is None else mean.data_ptr(), rstd.data_ptr(),
                                  None if ckpt is None else ckpt._ref, raw), "gift_norm_forward")
    return y, mean, rstd


def norm_backward(dy: torch.Tensor, x, mean, rstd, weight=None, kind="layer", dx=None, dweight=None, dbias=None,
                  accumulate: bool = False, work=None, stream=None):
    """Backward of norm_forward.  x: the forward's input, or its ActCheckpoint.
    Returns dx (of dy's type), dweight and dbias (fp32 [d]; dbias None for
    "rms" unless given).  accumulate: added to the given dweight and dbias."""
    kind = _kind(kind)
    ld = _rows(dy, "dy")
    (T, d), dev, dt = dy.shape, dy.device, dy.dtype
    raw = _raw_stream(stream, dev)
    ck = x if isinstance(x, ActCheckpoint) else None
    if ck is not None:
        if (ck.T, ck.d) != (T, d):
            raise ValueError("the checkpoint has another shape than dy")
        _on(dev, ck, "the checkpoint")
        ldx, xp = 0, None
    else:
        ldx, xp = _rows(x, "x", T, d, dt, dev), x.data_ptr()
    wp = _vector(weight, "weight", d, _WEIGHTS[dt], dev)
    mp, rp = _vector(mean, "mean", T, _F32, dev), _vector(rstd, "rstd", T, _F32, dev)
    if accumulate and dweight is None and dbias is None:
        raise ValueError("accumulate needs the gradients to add to")
    if dweight is not None:
        dwp = _vector(dweight, "dweight", d, _F32, dev)
    elif not accumulate:
        dweight = _empty(stream, (d,), torch.float32, dev)
        dwp = dweight.data_ptr()
    else:
        dwp = None
    if dbias is not None:
        dbp = _vector(dbias, "dbias", d, _F32, dev)
    elif not accumulate and kind == NORM_LAYER:
        dbias = _empty(stream, (d,), torch.float32, dev)
        dbp = dbias.data_ptr()
    else:
        dbp = None
    if dx is None:
        dx, lddx = _empty_like(stream, dy), d
    else:
        lddx = _rows(dx, "dx", T, d, dt, dev)
    if work is None:
        work = _empty(stream, (_lib.gift_norm_workspace_bytes(T, d),), torch.uint8, dev)
        wbytes = work.numel()
    else:
        wbytes = _bytes(dev, work, "work")
    _check(_lib.gift_norm_backward(kind, dy.data_ptr(), DTYPES[dt], ld, xp, ldx, None if ck is None else ck._ref,
                                   T, d, wp, DTYPES[dt if weight is None else weight.dtype], mp, rp, dx.data_ptr(),
                                   lddx, dwp, dbp, int(accumulate), work.data_ptr(), wbytes, raw),
           "gift_norm_backward")
    return dx, dweight, dbias


def weight_grad(delta: torch.Tensor, ckpt, alpha: float = 1.0, out=None, accumulate: bool = False, work=None,
                stream=None) -> torch.Tensor:
    """alpha delta^T a [m][d] in fp32 (plus `out` when accumulate), from the
    output gradients delta [T][m] and the layer's input a [T][d], either its
    checkpoint or the tensor itself (of delta's type): the gradient
    Layer.encode takes."""
    whole = not isinstance(ckpt, ActCheckpoint)
    if whole:
        ldx = _rows(ckpt, "the activation", None, None, delta.dtype)
        T, d = ckpt.shape
    else:
        T, d = ckpt.T, ckpt.d
    ld = _rows(delta, "delta", T)
    m, dev, dt = delta.shape[1], delta.device, DTYPES[delta.dtype]
    raw = _raw_stream(stream, dev)
    _on(dev, ckpt, "the activation" if whole else "the checkpoint")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the tensor to add to")
        out, ldw = _empty(stream, (m, d), torch.float32, dev), d
    else:
        ldw = _rows(out, "out", m, d, torch.float32, dev)
    if whole:
        dp, xp = delta.data_ptr(), ckpt.data_ptr()
        work, wp, wbytes = _workspace(stream, work, dev, lambda: _lib.gift_weight_grad_x_workspace_bytes(
            T, m, d, dt, _rows16(dt, (dp, ld, T), (xp, ldx, T))))
        _check(_lib.gift_weight_grad_x(dp, dt, ld, m, xp, ldx, T, d, alpha, int(accumulate), out.data_ptr(), ldw, wp,
                                       wbytes, raw), "gift_weight_grad_x")
    else:
        work, wp, wbytes = _workspace(stream, work, dev, lambda: _lib.gift_weight_grad_workspace_bytes(T, m, d, dt))
        _check(_lib.gift_weight_grad(delta.data_ptr(), dt, ld, m, ckpt._ref, T, d, alpha, int(accumulate),
                                     out.data_ptr(), ldw, wp, wbytes, raw), "gift_weight_grad")
    return out


# -- gated feed-forward block and dropout (gift_glu_*, gift_dropout_apply) ------

def _rows16(dt, *rows):
    """Whether all matrices (address, leading dimension, rows) have 16-byte aligned rows, at most 4 MB apart."""
    size = 4 if dt == FP32 else 2
    for p, ld, n in rows:
        if p % 16 or (n > 1 and (ld * size % 16 or ld * size > 1 << 22)):
            return 0
    return 1


def _workspace(stream, work, device, size):
    """The given workspace, or a new one of size() bytes (none for 0; asked only then, it takes 1 to 2 us): tensor,
    address, bytes."""
    if work is not None:
        return work, work.data_ptr(), _bytes(device, work, "work")
    nbytes = size()
    if nbytes == 0:
        return None, None, 0
    work = _empty(stream, (nbytes,), torch.uint8, device)
    return work, work.data_ptr(), nbytes


def _act(act):
    code = ACTS.get(act, act)
    if code not in ACTS.values():
        raise ValueError(f"act must be one of {', '.join(ACTS)}, not {act!r}")
    return code


class Dropout:
    """Dropout of probability p (counted in steps of 2^-16) whose mask is a
    function of an element's place, `seed` and the offset: nothing is stored,
    the backward pass takes the same Dropout.  The offset is `offset` plus,
    when `counter` is given, the number in that one-element int64 GPU tensor,
    read when the kernel runs: a captured graph draws another mask at each
    replay if the counter is increased between them.  Uses that are to draw
    apart need different seeds or offsets."""

    _FIXED = frozenset(("p", "seed", "offset", "counter"))

    def __init__(self, p: float, seed: int, offset: int = 0, counter=None):
        p, seed, offset = float(p), int(seed), int(offset)
        if not 0.0 <= p <= 1.0 or not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
            raise ValueError("dropout needs 0 <= p <= 1 and a seed and an offset of 64 bits")
        if counter is not None and (counter.dtype != torch.int64 or counter.numel() != 1 or not counter.is_cuda):
            raise ValueError("counter must be an int64 tensor of one element on the GPU")
        c = DropoutDesc(p, seed, offset, None if counter is None else counter.data_ptr())
        self.__dict__.update(p=p, seed=seed, offset=offset, counter=counter, _c=c, _ref=ctypes.byref(c))

    def __setattr__(self, name, value):
        if name in self._FIXED:
            raise AttributeError(f"a dropout's {name} cannot be replaced")
        super().__setattr__(name, value)


def _drop(drop, device):
    if drop is None:
        return None
    if drop.counter is not None:
        _on(device, drop.counter, "the dropout's counter")
    return drop._ref


def dropout_forward(x: torch.Tensor, drop: Dropout, residual=None, out=None, stream=None) -> torch.Tensor:
    """Dropout of x [T][d], plus `residual` [T][d] when given.  `out` may be x or the residual."""
    ld = _rows(x, "x")
    (T, d), dev, dt = x.shape, x.device, x.dtype
    raw = _raw_stream(stream, dev)
    ref = _drop(drop, dev)
    ldr, rp = (0, None) if residual is None else (_rows(residual, "residual", T, d, dt, dev), residual.data_ptr())
    if out is None:
        out, ldo = _empty_like(stream, x), d
    else:
        ldo = _rows(out, "out", T, d, dt, dev)
    _check(_lib.gift_dropout_apply(ref, x.data_ptr(), DTYPES[dt], ld, T, d, rp, ldr, out.data_ptr(), ldo, raw),
           "gift_dropout_apply")
    return out


def dropout_backward(dy: torch.Tensor, drop: Dropout, dx=None, stream=None) -> torch.Tensor:
    """Gradient of dropout_forward's x from that of its output (the residual's is dy itself)."""
    return dropout_forward(dy, drop, out=dx, stream=stream)


def glu_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act="silu", keep: bool = False, drop=None,
                ckpt=None, out=None, gate=None, up=None, work=None, stream=None):
    """Gated feed-forward block: h = drop(act(x w_gate^T) (x w_up^T)) [T][f],
    for x [T][d] and weights [f][d] of its type (separate, or halves of one
    matrix).  Returns h, gate and up: with `keep` (or given tensors) the two
    products, for glu_backward, else None.  With `ckpt` (an ActCheckpoint
    [T][f]) h is also saved there."""
    act = _act(act)
    ld = _rows(x, "x")
    (T, d), dev, dt = x.shape, x.device, x.dtype
    raw = _raw_stream(stream, dev)
    ldg, f = _rows(w_gate, "w_gate", None, d, dt, dev), w_gate.shape[0]
    ldu = _rows(w_up, "w_up", f, d, dt, dev)
    ref = _drop(drop, dev)
    if ckpt is not None:
        if (ckpt.T, ckpt.d) != (T, f):
            raise ValueError("the checkpoint has another shape than h")
        _on(dev, ckpt, "the checkpoint")
    if out is None:
        out, ldh = _empty(stream, (T, f), dt, dev), f
    else:
        ldh = _rows(out, "out", T, f, dt, dev)
    if (gate is None) != (up is None):
        raise ValueError("gate and up are given together")
    if gate is not None:
        ldz, ldup = _rows(gate, "gate", T, f, dt, dev), _rows(up, "up", T, f, dt, dev)
    elif keep:
        gate, up, ldz, ldup = _empty(stream, (T, f), dt, dev), _empty(stream, (T, f), dt, dev), f, f
    else:
        ldz = ldup = 0
    t, xp, gp, wp = DTYPES[dt], x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    work, kp, wbytes = _workspace(stream, work, dev, lambda: _lib.gift_glu_workspace_bytes(
        T, d, f, t, _rows16(t, (xp, ld, T), (gp, ldg, f), (wp, ldu, f))))
    _check(_lib.gift_glu_forward(act, xp, t, ld, T, d, gp, ldg, wp, ldu, f, ref, out.data_ptr(), ldh,
                                 None if gate is None else gate.data_ptr(), ldz, None if up is None else up.data_ptr(),
                                 ldup, None if ckpt is None else ckpt._ref, kp, wbytes, raw), "gift_glu_forward")
    return out, gate, up


def glu_backward(dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, w_gate=None, w_up=None, act="silu", drop=None,
                 dx=None, dgate=None, dup=None, work=None, stream=None):
    """Backward of glu_forward from dh [T][f] and what it kept.  Returns dx
    [T][d] (None without the weights), and the gradients of both products,
    dgate and dup [T][f], which weight_grad takes (given as the halves of one
    [T][2 f] tensor, one weight_grad makes the gradient of both weights).
    dgate and dup may be gate, up or dh."""
    act = _act(act)
    ld = _rows(dh, "dh")
    (T, f), dev, dt = dh.shape, dh.device, dh.dtype
    raw = _raw_stream(stream, dev)
    ldz, ldup = _rows(gate, "gate", T, f, dt, dev), _rows(up, "up", T, f, dt, dev)
    ref = _drop(drop, dev)
    if (w_gate is None) != (w_up is None) or (w_gate is None and dx is not None):
        raise ValueError("dx needs both weights")
    if dgate is None:
        dgate, lddz = _empty(stream, (T, f), dt, dev), f
    else:
        lddz = _rows(dgate, "dgate", T, f, dt, dev)
    if dup is None:
        dup, lddup = _empty(stream, (T, f), dt, dev), f
    else:
        lddup = _rows(dup, "dup", T, f, dt, dev)
    t, zp, up_ = DTYPES[dt], dgate.data_ptr(), dup.data_ptr()
    if w_gate is None:
        d = ldg = ldu = lddx = 0
        gp = wp = xp = None
    else:
        ldg, d = _rows(w_gate, "w_gate", f, None, dt, dev), w_gate.shape[1]
        ldu = _rows(w_up, "w_up", f, d, dt, dev)
        if dx is None:
            dx, lddx = _empty(stream, (T, d), dt, dev), d
        else:
            lddx = _rows(dx, "dx", T, d, dt, dev)
        gp, wp, xp = w_gate.data_ptr(), w_up.data_ptr(), dx.data_ptr()
    work, kp, wbytes = _workspace(stream, work, dev, lambda: 0 if w_gate is None else (
        _lib.gift_glu_backward_workspace_bytes(
            T, d, f, t, int((lddz == lddup or T == 1) and (ldg == ldu or f == 1) and
                            _rows16(t, (zp, lddz, T), (up_, lddup, T), (gp, ldg, f), (wp, ldu, f))))))
    _check(_lib.gift_glu_backward(act, dh.data_ptr(), t, ld, T, f, gate.data_ptr(), ldz, up.data_ptr(), ldup, ref, zp,
                                  lddz, up_, lddup, gp, ldg, wp, ldu, d, xp, lddx, kp, wbytes, raw), "gift_glu_backward")
    return dx, dgate, dup
