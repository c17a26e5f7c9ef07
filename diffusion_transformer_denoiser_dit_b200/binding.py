"""ctypes binding of libdit_b200.so (include/dit.h).

Argument marshalling only: every step of the forward runs in the library's CUDA
kernels.  torch provides device memory and streams.  If the library is missing or
cannot be loaded, every call raises; there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int, c_longlong, c_uint16, c_void_p
from typing import Optional, Sequence

import numpy as np

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdit_b200.so")

DIT_OK, DIT_ERR_INVALID_ARG, DIT_ERR_UNSUPPORTED, DIT_ERR_OOM, DIT_ERR_CUDA = 0, 1, 2, 3, 4
DIT_ERR_DEVICE_TIMEOUT, DIT_ERR_BAD_LABEL, DIT_ERR_NO_DEVICE = 5, 6, 7
DIT_OPT_FORCE_GUIDANCE, DIT_OPT_USE_GRAPH, DIT_OPT_OVERLAP_LAUNCH, DIT_OPT_CFG_CHANNELS = 1, 2, 3, 4
DIT_OPT_REPEAT_KIND, DIT_OPT_SPLIT_K, DIT_OPT_PAIR_GEMM = 5, 6, 7
DIT_SAMPLER_DDIM, DIT_SAMPLER_EULER = 0, 1
DIT_DTYPE_F32, DIT_DTYPE_BF16, DIT_DTYPE_FP16 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu_tanh": 2, "gelu": 3, "silu": 4}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ROTARY_MAX_PAIRS = 256

# every exported symbol declared in include/dit.h
EXPORTS = [
    "dit_create", "dit_weight_count", "dit_forward", "dit_forward_host", "dit_sync_status", "dit_last_error",
    "dit_status_string", "dit_destroy", "dit_set_option", "dit_debug_residual", "dit_debug_condition",
    "dit_debug_wait_probe", "dit_op_linear_bf16", "dit_forward_launch_count", "dit_profile_enable",
    "dit_profile_read", "dit_condition_static", "dit_op_linear_bf16_pair", "dit_sampler_step", "dit_sample",
    "dit_op_attention_bf16", "dit_debug_attention_rescales", "dit_op_linear_e4m3", "dit_op_linear_fused",
    "dit_op_attention_packed", "dit_rotary_frequencies", "dit_rotary_init", "dit_op_rotary",
]

KERNEL_KINDS = ["cond", "adaln", "patch", "ln", "qkv", "attn", "proj", "fc1", "fc2", "decode", "sampler"]


class DitConfig(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("in_channels", c_int), ("frames", c_int), ("height", c_int), ("width", c_int),
                ("patch_t", c_int), ("patch_h", c_int), ("patch_w", c_int), ("hidden", c_int), ("depth", c_int),
                ("heads", c_int), ("mlp_hidden", c_int), ("learn_sigma", c_int), ("pos_kind", c_int),
                ("qk_norm", c_int), ("cond_kind", c_int), ("num_classes", c_int), ("freq_dim", c_int),
                ("max_batch", c_int), ("t_scale", c_float), ("block_kind", c_int), ("ffn_fp8", c_int),
                ("attn_fp8", c_int)]


class RotaryPlan(ctypes.Structure):
    """dit_rotary of include/dit.h."""
    _fields_ = [("pairs", c_int), ("axes", c_int), ("amplitude", c_float),
                ("turns", ctypes.c_uint64 * ROTARY_MAX_PAIRS)]


class DitError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


_LIB = None


def load() -> ctypes.CDLL:
    """Load the library (raises if it was not built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m diffusion_transformer_denoiser_dit_b200.build")
    lib = ctypes.CDLL(LIB_PATH)
    P, L = c_void_p, c_longlong
    sig = {
        "dit_create": (c_int, [POINTER(DitConfig), POINTER(c_void_p), c_int, POINTER(c_void_p)]),
        "dit_weight_count": (c_int, [POINTER(DitConfig)]),
        "dit_forward": (c_int, [P, P, P, P, c_int, c_float, P, P]),
        "dit_forward_host": (c_int, [P, P, P, P, c_int, c_float, P, P]),
        "dit_sampler_step": (c_int, [P, c_int, P, P, c_int, c_float, c_float, P, P]),
        "dit_sample": (c_int, [P, c_int, P, P, c_int, c_float, c_int, POINTER(c_float), POINTER(c_float), P]),
        "dit_sync_status": (c_int, [P]),
        "dit_last_error": (ctypes.c_char_p, [P]),
        "dit_status_string": (ctypes.c_char_p, [c_int]),
        "dit_destroy": (None, [P]),
        "dit_set_option": (c_int, [P, c_int, c_int]),
        "dit_debug_residual": (c_int, [P, P, P, P, c_int, c_float, c_int, P, P]),
        "dit_debug_condition": (c_int, [P, P, P, c_int, c_float, P, P]),
        "dit_debug_wait_probe": (c_int, [P, c_int, P]),
        "dit_op_linear_bf16": (c_int, [P, P, P, P, c_int, c_int, c_int, c_int, P]),
        "dit_op_linear_bf16_pair": (c_int, [P, P, P, P, c_int, c_int, c_int, c_int, P]),
        "dit_forward_launch_count": (c_int, [P, c_int, c_float]),
        "dit_profile_enable": (c_int, [P, c_int]),
        "dit_profile_read": (c_int, [P, POINTER(c_float), POINTER(c_int)]),
        "dit_condition_static": (c_int, [P, P, c_int, c_int, P, P, P, P, P, c_int, c_int, c_int, c_int, c_float,
                                         P, P, P]),
        "dit_op_attention_bf16": (c_int, [P, P, P, P, c_int, c_int, c_int, c_int, P, P]),
        "dit_debug_attention_rescales": (c_int, [P, POINTER(ctypes.c_longlong)]),
        "dit_op_linear_e4m3": (c_int, [P, P, P, P, P, P, c_int, c_int, c_int, c_int, P]),
        "dit_op_linear_fused": (c_int, [c_int, P, L, P, L, P, c_int, P, L, P, L, c_int, c_int, c_int, c_int, P, P]),
        "dit_op_attention_packed": (c_int, [c_int] + [P] * 7 + [c_int] * 8 + [POINTER(L), c_float, c_int, P, P]),
        "dit_rotary_frequencies": (c_int, [c_int, c_int, c_double, c_double, c_int, POINTER(c_double),
                                           POINTER(c_float)]),
        "dit_rotary_init": (c_int, [POINTER(RotaryPlan), POINTER(c_double), c_int, c_int, c_float]),
        "dit_op_rotary": (c_int, [POINTER(RotaryPlan), c_int, P, L, L, P, c_int, P, L, L] + [c_int] * 5 + [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def make_config(cfg, max_batch: Optional[int] = None) -> DitConfig:
    """dit_config from any object with the same field names (e.g. dit_synth.DiTConfig)."""
    mb = max_batch if max_batch is not None else cfg.batch
    return DitConfig(cfg.dtype, cfg.in_channels, cfg.frames, cfg.height, cfg.width, cfg.patch_t, cfg.patch_h,
                     cfg.patch_w, cfg.hidden, cfg.depth, cfg.heads, cfg.mlp_hidden, cfg.learn_sigma, cfg.pos_kind,
                     cfg.qk_norm, cfg.cond_kind, cfg.num_classes, cfg.freq_dim, mb, float(cfg.t_scale),
                     int(getattr(cfg, "block_kind", 0)), int(getattr(cfg, "ffn_fp8", 0)),
                     int(getattr(cfg, "attn_fp8", 0)))


def status_string(code: int) -> str:
    return load().dit_status_string(code).decode()


def _ptr(t) -> int:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


class DiT:
    """A created model: device weights + workspace owned by the library."""

    def __init__(self, cfg, weights: Sequence[np.ndarray], max_batch: Optional[int] = None):
        self.lib = load()
        self.cfg = cfg
        self._c = make_config(cfg, max_batch)
        arrs = [np.ascontiguousarray(w, dtype=np.float32) for w in weights]
        ptrs = (c_void_p * len(arrs))(*[a.ctypes.data for a in arrs])
        h = c_void_p()
        rc = self.lib.dit_create(ctypes.byref(self._c), ptrs, len(arrs), ctypes.byref(h))
        if rc != DIT_OK:
            raise DitError(rc, f"dit_create failed: {status_string(rc)}")
        self.h = h

    # ---- helpers
    def _check(self, rc: int, what: str):
        if rc != DIT_OK:
            msg = self.lib.dit_last_error(self.h).decode() if self.h else ""
            raise DitError(rc, f"{what}: {status_string(rc)} {msg}")

    def rows(self, B: int, cfg_scale: float) -> int:
        return 2 * B if (self.cfg.cond_kind == 0 and cfg_scale != 1.0) else B

    def out_shape(self, B: int):
        return self.cfg.out_shape(B)

    # ---- calls
    def forward(self, x, t, y, cfg_scale: float, out=None, stream=None):
        import torch
        B = x.shape[0]
        if out is None:
            out = torch.empty(self.out_shape(B), dtype=torch.float32, device=x.device)
        rc = self.lib.dit_forward(self.h, _ptr(x), _ptr(t), _ptr(y), B, float(cfg_scale), _ptr(out), _stream(stream))
        self._check(rc, "dit_forward")
        return out

    def forward_host(self, x: np.ndarray, t: np.ndarray, y: np.ndarray, cfg_scale: float, out: np.ndarray = None,
                     stream=None):
        B = x.shape[0]
        if out is None:
            out = np.empty(self.out_shape(B), dtype=np.float32)
        rc = self.lib.dit_forward_host(self.h, x.ctypes.data, t.ctypes.data, y.ctypes.data, B, float(cfg_scale),
                                       out.ctypes.data, _stream(stream))
        self._check(rc, "dit_forward_host")
        return out

    def forward_host_ptr(self, x_ptr: int, t_ptr: int, y_ptr: int, B: int, cfg_scale: float, out_ptr: int,
                         stream=None):
        rc = self.lib.dit_forward_host(self.h, x_ptr, t_ptr, y_ptr, B, float(cfg_scale), out_ptr, _stream(stream))
        self._check(rc, "dit_forward_host")

    def debug_residual(self, x, t, y, cfg_scale: float, after_block: int, stream=None):
        import torch
        B = x.shape[0]
        R = self.rows(B, cfg_scale) if not getattr(self, "_force", False) else 2 * B
        h = torch.empty((R, getattr(self.cfg, "seq_tokens", self.cfg.tokens), self.cfg.hidden), dtype=torch.float32,
                        device=x.device)
        rc = self.lib.dit_debug_residual(self.h, _ptr(x), _ptr(t), _ptr(y), B, float(cfg_scale), after_block, _ptr(h),
                                         _stream(stream))
        self._check(rc, "dit_debug_residual")
        return h

    def debug_condition(self, t, y, cfg_scale: float, stream=None):
        import torch
        B = t.shape[0]
        R = self.rows(B, cfg_scale) if not getattr(self, "_force", False) else 2 * B
        c = torch.empty((R, self.cfg.hidden), dtype=torch.float32, device=t.device)
        rc = self.lib.dit_debug_condition(self.h, _ptr(t), _ptr(y), B, float(cfg_scale), _ptr(c), _stream(stream))
        self._check(rc, "dit_debug_condition")
        return c

    def sampler_step(self, kind: int, x, model_out, a: float, b: float, x_next=None, stream=None):
        """One sampler update (DIT_SAMPLER_DDIM: a, b = abar now / next; DIT_SAMPLER_EULER:
        a, b = t now / next) of the device latent x given dit_forward's output; in place when
        x_next is x."""
        import torch
        if x_next is None:
            x_next = torch.empty_like(x)
        rc = self.lib.dit_sampler_step(self.h, int(kind), _ptr(x), _ptr(model_out), x.shape[0], float(a), float(b),
                                       _ptr(x_next), _stream(stream))
        self._check(rc, "dit_sampler_step")
        return x_next

    def sample(self, kind: int, x, y, cfg_scale: float, model_t, levels, stream=None):
        """len(model_t) steps of forward + update, in place on the device latent x."""
        mt = np.ascontiguousarray(model_t, dtype=np.float32)
        lv = np.ascontiguousarray(levels, dtype=np.float32)
        if lv.size != mt.size + 1:
            raise ValueError("levels needs one more entry than model_t")
        fp = POINTER(c_float)
        rc = self.lib.dit_sample(self.h, int(kind), _ptr(x), _ptr(y), x.shape[0], float(cfg_scale), int(mt.size),
                                 mt.ctypes.data_as(fp), lv.ctypes.data_as(fp), _stream(stream))
        self._check(rc, "dit_sample")
        return x

    def set_option(self, option: int, value: int):
        self._check(self.lib.dit_set_option(self.h, option, value), "dit_set_option")
        if option == DIT_OPT_FORCE_GUIDANCE:
            self._force = bool(value)

    def sync_status(self) -> int:
        return self.lib.dit_sync_status(self.h)

    def wait_probe(self, timeout_us: int, stream=None):
        self._check(self.lib.dit_debug_wait_probe(self.h, timeout_us, _stream(stream)), "dit_debug_wait_probe")

    def attention_rescales(self) -> int:
        """Attention reference-maximum moves (per warp of 32 query rows) since the last read."""
        n = ctypes.c_longlong(0)
        self._check(self.lib.dit_debug_attention_rescales(self.h, ctypes.byref(n)), "dit_debug_attention_rescales")
        return int(n.value)

    def launch_count(self, B: int, cfg_scale: float) -> int:
        return self.lib.dit_forward_launch_count(self.h, B, float(cfg_scale))

    def profile(self, enable: bool, kind: Optional[str] = None):
        """Per-launch event timing on (every kind, or only `kind`, one of KERNEL_KINDS) or off."""
        mode = 0 if not enable else (1 if kind is None else 2 + KERNEL_KINDS.index(kind))
        self._check(self.lib.dit_profile_enable(self.h, mode), "dit_profile_enable")

    def profile_read(self):
        """{kind: (total_ms, launches)} of the launches recorded since the last read."""
        n = len(KERNEL_KINDS)
        ms = (c_float * n)()
        cnt = (c_int * n)()
        self._check(self.lib.dit_profile_read(self.h, ms, cnt), "dit_profile_read")
        return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}

    def close(self):
        if getattr(self, "h", None):
            self.lib.dit_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def linear_bf16(x, w, b, block_n: int = 128, stream=None, pair: bool = False):
    """y = x W^T + b on the tensor-core GEMM (x, w: torch bf16 CUDA tensors);
    pair=True runs the SM-pair (cta_group::2) kernel."""
    import torch
    lib = load()
    M, K = x.shape
    N = w.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    fn = lib.dit_op_linear_bf16_pair if pair else lib.dit_op_linear_bf16
    rc = fn(_ptr(x), _ptr(w), _ptr(b), _ptr(y), M, N, K, block_n, _stream(stream))
    if rc != DIT_OK:
        raise DitError(rc, f"dit_op_linear_bf16: {status_string(rc)}")
    return y


def attention_bf16(q, k, v, o, R: int, H: int, T: int, dh: int, counters=None, stream=None):
    """The bf16 tensor-core attention kernel on the forward's workspace layouts (see
    dit_op_attention_bf16 in include/dit.h): q, k [R*H, Tpad, DP], v [R*H, DP, Tpad] and
    o [R*T, H*dh], torch bf16 CUDA tensors; counters an int32 CUDA tensor of 2 or None."""
    lib = load()
    rc = lib.dit_op_attention_bf16(_ptr(q), _ptr(k), _ptr(v), _ptr(o), R, H, T, dh, _ptr(counters), _stream(stream))
    if rc != DIT_OK:
        raise DitError(rc, f"dit_op_attention_bf16: {status_string(rc)}")
    return o


def linear_e4m3(x8, w8, sx, sw, b, block_n: int = 128, stream=None):
    """y = sx[m] sw[n] (x8 w8^T)[m, n] + b[n] on the FP8 tensor-core GEMM (x8, w8: uint8 CUDA
    tensors of E4M3 bytes; sx, sw, b: float32 CUDA tensors, b may be None)."""
    import torch
    lib = load()
    M, K = x8.shape
    N = w8.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x8.device)
    rc = lib.dit_op_linear_e4m3(_ptr(x8), _ptr(w8), _ptr(sx), _ptr(sw), _ptr(b), _ptr(y), M, N, K, block_n,
                                _stream(stream))
    if rc != DIT_OK:
        raise DitError(rc, f"dit_op_linear_e4m3: {status_string(rc)}")
    return y


# ---------------------------------------------------------------- building blocks of packed layers
# A call's own kernel may last three microseconds, so the common call goes through _fastcall (None from
# it: nothing was done, the code below decides), and the others look at each argument once and take torch's
# raw stream and device handles instead of building Stream and device objects.  A linear call of one
# token then takes the host 4.4 us instead of 9.3, one of attention over 100 keys 8.7 instead of 12.8.

_Strides8 = c_longlong * 8
_RT = None


class _Runtime:
    def __init__(self):
        import torch
        self.torch, self.lib = torch, load()
        self.linear, self.attention, self.rotary = (self.lib.dit_op_linear_fused, self.lib.dit_op_attention_packed,
                                                    self.lib.dit_op_rotary)
        self.float32, self.int32, self.int64 = torch.float32, torch.int32, torch.int64
        self.code = {torch.float32: DIT_DTYPE_F32, torch.bfloat16: DIT_DTYPE_BF16, torch.float16: DIT_DTYPE_FP16}
        self.code16 = {torch.bfloat16: DIT_DTYPE_BF16, torch.float16: DIT_DTYPE_FP16}
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent without CUDA
        self.current_device = getattr(torch._C, "_cuda_getDevice", None)
        try:
            from . import _fastcall as fast
        except ImportError:  # no headers to build it with, or another torch's
            fast = None
        else:
            fast.bind(*(ctypes.cast(f, c_void_p).value for f in (self.linear, self.attention, self.rotary)))
        self.fast = fast


def _rt() -> _Runtime:
    global _RT
    if _RT is None:
        _RT = _Runtime()
    return _RT


def _sizes(name: str, *sizes):
    """The C interface counts in int; ctypes would drop the upper bits."""
    worst = max(sizes, key=abs)
    if abs(worst) > 0x7fffffff:
        raise ValueError(f"{name}: size {worst} is beyond 32 bits")


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _no_dtype(name: str, dtype):
    raise TypeError(f"{name}: dtype {dtype} is not supported")


def _status(rt: _Runtime, name: str, status):
    """Address of the int32 that a wait which ran out writes."""
    if status.dtype != rt.int32 or status.numel() < 1:
        raise ValueError(f"{name}: status int32 [1]")
    return status.data_ptr()


def _elsewhere(rt: _Runtime, name: str, fn, dev: int, tensors, stream, args):
    """fn(*args, stream) off the common path: refuses what is not on one CUDA device, takes a given
    stream, or enters the tensors' device when another is current."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: tensors on {t.device} and {tensors[0].device}")
    if dev < 0:
        raise ValueError(f"{name}: needs CUDA tensors")
    if stream is None:
        raw = rt.raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{name}: stream on {stream.device}, tensors on {tensors[0].device}")
    else:
        raw = stream.cuda_stream
        if raw != rt.raw_stream(dev):
            for t in tensors:  # their memory is not given away before the work on this stream is done
                if t is not None:
                    t.record_stream(stream)
    with rt.torch.cuda.device(dev):
        return fn(*args, raw)


def _refused(name: str, rc: int):
    raise DitError(rc, f"{name}: {status_string(rc)}")


def _fresh(like, shape, dtype, stream):
    """An output on like's device, from the stream that will write it."""
    if stream is None:
        return like.new_empty(shape) if dtype == like.dtype else like.new_empty(shape, dtype=dtype)
    with _rt().torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _row_stride(t, name: str) -> int:
    """Stride between the rows of a matrix whose rows are contiguous; that of a single row is free."""
    rows, cols = t.shape
    if t.is_contiguous():
        return cols
    _need(cols == 1 or t.stride(1) == 1, name + ": last strides must be 1")
    return t.stride(0) if rows > 1 else cols


def linear_fused(x, w, bias=None, act: str = "none", residual=None, out=None, out_dtype=None, status=None, stream=None):
    """out = act(x w^T + bias) + residual (dit_op_linear_fused in include/dit.h).

    x [M, K] and w [N, K]: bf16 or fp16 CUDA tensors, last stride 1; bias float32 [N]; act one of
    ACTIVATIONS; residual [M, N] of out's dtype (a stride-0 row broadcasts); out [M, N] of x's
    dtype or float32, residual itself for an update in place; status int32 [1] (zeroed) receives
    a timeout.  Returns out."""
    rt, name = _RT or _rt(), "linear_fused"
    if rt.fast is not None and stream is None and status is None:
        y = rt.fast.linear(x, w, bias, ACTIVATIONS.get(act, -1), residual, out, out_dtype)
        if y is not None:
            return y if type(y) is not int else _refused(name, y)
    _need(x.dim() == 2 and w.dim() == 2, "linear_fused: x [M, K] and w [N, K]")
    (M, K), (N, kw), dtype = x.shape, w.shape, x.dtype
    code, a = rt.code16.get(dtype), ACTIVATIONS.get(act)
    if code is None:
        _no_dtype(name, dtype)
    if K != kw or w.dtype != dtype:
        raise ValueError("linear_fused: x [M, K] and w [N, K] of one dtype")
    if a is None:
        raise ValueError(f"linear_fused: act {act!r} is none of {sorted(ACTIVATIONS)}")
    _sizes(name, M, N, K)
    dev = x.get_device()
    same = w.get_device() == dev
    ldx = K if x.is_contiguous() else _row_stride(x, name)
    ldw = K if w.is_contiguous() else _row_stride(w, name)
    if out is None:
        odtype, ldy = dtype if out_dtype is None else out_dtype, N
    else:
        odtype, ldy, same = out.dtype, _row_stride(out, name), same and out.get_device() == dev
        if out.shape != (M, N) or (out_dtype is not None and odtype != out_dtype):
            raise ValueError("linear_fused: out [M, N] of out_dtype")
    ocode = code if odtype == dtype else rt.code.get(odtype)
    if ocode is None:
        _no_dtype(name, odtype)
    pb = pr = ps = None
    ldr = 0
    if bias is not None:
        if bias.shape != (N,) or bias.dtype != rt.float32 or not bias.is_contiguous():
            raise ValueError("linear_fused: bias float32 [N]")
        pb, same = bias.data_ptr(), same and bias.get_device() == dev
    if residual is not None:
        if residual.shape != (M, N) or residual.dtype != odtype or (residual.stride(1) != 1 and N > 1):
            raise ValueError("linear_fused: residual [M, N] of out's dtype")
        pr, ldr, same = residual.data_ptr(), residual.stride(0), same and residual.get_device() == dev
    if status is not None:
        ps, same = _status(rt, name, status), same and status.get_device() == dev
    if out is None:
        out = _fresh(x, (M, N), odtype, stream)
    args = (code, x.data_ptr(), ldx, w.data_ptr(), ldw, pb, a, pr, ldr, out.data_ptr(), ldy, ocode, M, N, K, ps)
    if same and stream is None and dev >= 0 and dev == rt.current_device():
        rc = rt.linear(*args, rt.raw_stream(dev))
    else:
        rc = _elsewhere(rt, name, rt.linear, dev, (x, w, out, bias, residual, status), stream, args)
    if rc != DIT_OK:
        _refused(name, rc)
    return out


def _head_strides(t, name: str):
    """Token and head stride of [tokens, heads, features]; those of a length-1 axis are free."""
    n, h, d = t.shape
    if t.is_contiguous():
        return h * d, d
    _need(d == 1 or t.stride(2) == 1, name + ": last strides must be 1")
    sh = t.stride(1) if h > 1 else -(-d // 8) * 8
    return (t.stride(0) if n > 1 else h * sh), sh


def attention_packed(q, k, v, cu_q, cu_k, max_q: int, max_k: int, causal: bool = False, scale=None, out=None,
                     return_lse: bool = False, status=None, stream=None):
    """Attention over packed sequences (dit_op_attention_packed in include/dit.h).

    q [total_q, heads, dh], k and v [total_k, kv_heads, dh]: bf16 or fp16 CUDA tensors, last
    stride 1; cu_q, cu_k int32 CUDA [n + 1]: the sequences' offsets; max_q, max_k: the longest
    lengths; causal aligns the last query with the last key; scale defaults to dh^-0.5.
    Returns out (rows outside every sequence are not written; a new out starts undefined
    there), or (out, lse float32 [heads, total_q]) with return_lse."""
    rt, name = _RT or _rt(), "attention_packed"
    if rt.fast is not None and stream is None and status is None:
        y = rt.fast.attention(q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, out, return_lse)
        if y is not None:
            return y if type(y) is not int else _refused(name, y)
    _need(q.dim() == 3 and k.dim() == 3 and k.shape == v.shape, "attention_packed: q [total_q, heads, dh], k and v "
          "[total_k, kv_heads, dh]")
    (tq, h, d), (tk, hk, dk), dtype, n = q.shape, k.shape, q.dtype, cu_q.numel() - 1
    code = rt.code16.get(dtype)
    if code is None:
        _no_dtype(name, dtype)
    if d != dk or d < 1 or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("attention_packed: q, k and v of one dtype and number of features, at least 8")
    if (cu_q.dim() != 1 or n < 0 or cu_k.shape != cu_q.shape or cu_q.dtype != rt.int32 or cu_k.dtype != rt.int32
            or not cu_q.is_contiguous() or not cu_k.is_contiguous()):
        raise ValueError("attention_packed: cu_q and cu_k contiguous int32 [n + 1]")
    _sizes(name, tq, tk, h, hk, d, n, max_q, max_k)
    dev = q.get_device()
    same = (k.get_device() == dev and v.get_device() == dev and cu_q.get_device() == dev and cu_k.get_device() == dev
            and (out is None or out.get_device() == dev) and (status is None or status.get_device() == dev))
    if out is None:
        out = _fresh(q, (tq, h, d), dtype, stream)
    elif out.shape != q.shape or out.dtype != dtype:
        raise ValueError("attention_packed: out like q")
    strides = _Strides8(*_head_strides(q, name), *_head_strides(k, name), *_head_strides(v, name), *_head_strides(out, name))
    lse = _fresh(q, (h, tq), rt.float32, stream) if return_lse else None
    args = (code, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
            cu_q.data_ptr(), cu_k.data_ptr(), n, tq, tk, max_q, max_k, h, hk, d, strides,
            d ** -0.5 if scale is None else scale, 1 if causal else 0, None if status is None else _status(rt, name, status))
    if same and stream is None and dev >= 0 and dev == rt.current_device():
        rc = rt.attention(*args, rt.raw_stream(dev))
    else:
        rc = _elsewhere(rt, name, rt.attention, dev, (q, k, v, out, lse, cu_q, cu_k, status), stream, args)
    if rc != DIT_OK:
        _refused(name, rc)
    return (out, lse) if return_lse else out


class Rotary:
    """Rotary positions for heads of head_dim features, of which the first rotary_dim turn
    (dit_op_rotary in include/dit.h).  axes coordinates per token split the turned features
    evenly; scaling is one of ROTARY_SCALINGS with its factor (and original_length for "yarn");
    freqs (radians per position, one per pair of an axis) replaces base and scaling."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, interleaved: bool = False,
                 base: float = 10000.0, axes: int = 1, scaling: str = "none", factor: float = 1.0,
                 original_length: int = 0, freqs: Optional[Sequence[float]] = None):
        lib = load()
        self.head_dim, self.axes, self.interleaved = int(head_dim), int(axes), int(bool(interleaved))
        part = self.head_dim if rotary_dim is None else int(rotary_dim)
        _need(self.axes > 0 and 0 < part <= self.head_dim and part % (2 * self.axes) == 0,
              "Rotary: rotary_dim must be a multiple of 2 * axes and at most head_dim")
        each = part // (2 * self.axes)
        if scaling not in ROTARY_SCALINGS:
            raise ValueError(f"Rotary: scaling {scaling!r} is none of {sorted(ROTARY_SCALINGS)}")
        f, amp = (c_double * each)(), c_float(1.0)
        if freqs is not None:
            _need(len(freqs) == each, f"Rotary: freqs needs {each} entries")
            f[:] = [float(v) for v in freqs]
        else:
            self._check(lib.dit_rotary_frequencies(ROTARY_SCALINGS[scaling], each, float(base), float(factor),
                                                   int(original_length), f, ctypes.byref(amp)), "dit_rotary_frequencies")
        self._plan = RotaryPlan()
        self._check(lib.dit_rotary_init(ctypes.byref(self._plan), f, each, self.axes, amp), "dit_rotary_init")
        self._ref, self._address = ctypes.byref(self._plan), ctypes.addressof(self._plan)

    @staticmethod
    def _check(rc: int, what: str):
        if rc != DIT_OK:
            raise DitError(rc, f"{what}: {status_string(rc)}")

    def apply(self, x, positions, out=None, transpose: bool = False, stream=None):
        """x [tokens, heads, head_dim] (float32, bf16 or fp16) turned by positions [tokens] or
        [tokens, axes] (int32 or int64); out=x turns in place.  transpose: the gradient of x
        from that of the result."""
        rt, name = _RT or _rt(), "Rotary.apply"
        if rt.fast is not None and stream is None:
            y = rt.fast.rotary(self._address, self.head_dim, self.axes, self.interleaved, x, positions, out, transpose)
            if y is not None:
                return y if type(y) is not int else _refused(name, y)
        _need(x.dim() == 3 and x.shape[2] == self.head_dim, "Rotary.apply: x [tokens, heads, head_dim]")
        (n, h, d), dtype, wide = x.shape, x.dtype, positions.dtype == rt.int64
        code = rt.code.get(dtype)
        if code is None:
            _no_dtype(name, dtype)
        if ((not wide and positions.dtype != rt.int32) or not positions.is_contiguous()
                or (positions.shape != (n, self.axes) and (self.axes != 1 or positions.shape != (n,)))):
            raise ValueError("Rotary.apply: positions contiguous int32 or int64 [tokens, axes]")
        _sizes(name, n, h, d)
        dev = x.get_device()
        same = positions.get_device() == dev and (out is None or out.get_device() == dev)
        xt, xh = (h * d, d) if x.is_contiguous() else _head_strides(x, name)
        if out is None:
            out, yt, yh = _fresh(x, (n, h, d), dtype, stream), h * d, d
        else:
            if out.shape != x.shape or out.dtype != dtype:
                raise ValueError("Rotary.apply: out like x")
            yt, yh = _head_strides(out, name)
        args = (self._ref, code, x.data_ptr(), xt, xh, positions.data_ptr(), 1 if wide else 0, out.data_ptr(), yt, yh, n, h, d,
                self.interleaved, 1 if transpose else 0)
        if same and stream is None and dev >= 0 and dev == rt.current_device():
            rc = rt.rotary(*args, rt.raw_stream(dev))
        else:
            rc = _elsewhere(rt, name, rt.rotary, dev, (x, positions, out), stream, args)
        if rc != DIT_OK:
            _refused(name, rc)
        return out
