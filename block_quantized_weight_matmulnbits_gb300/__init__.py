"""Python binding of libmnb (block-quantized weight-only matmul for GB300, sm_103a).

Argument marshalling only: every function forwards to the C entry point of
the same name in ``include/mnb.h`` (loaded with ctypes from the in-tree build)
and raises ``MnbError`` on a non-OK status.  Tensors are passed by device
pointer; streams default to torch's current stream.  Nothing here computes
any part of the operation, and there is no fallback: if the CUDA library
cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import threading

from . import _build

MNB_OK, MNB_ERR_INVALID_ARG, MNB_ERR_UNSUPPORTED, MNB_ERR_CUDA, MNB_ERR_NO_MEM, MNB_ERR_TIMEOUT, \
    MNB_ERR_LAYOUT_MISMATCH = range(7)
MNB_F32, MNB_F16, MNB_BF16 = 0, 1, 2
MNB_FLAG_PDL = 1
MNB_FLAG_KPERM = 2
MNB_ROTARY_INTERLEAVED, MNB_ROTARY_INVERSE = 1, 2
MNB_NORM_UNIT_OFFSET = 1
MNB_MOE_SOFTMAX, MNB_MOE_SIGMOID = 0, 1
MNB_ACT_SILU, MNB_ACT_GELU_TANH = 0, 1
MNB_ROPE_NONE, MNB_ROPE_LINEAR, MNB_ROPE_NTK, MNB_ROPE_BY_PARTS = range(4)
MNB_WF_E4M3, MNB_WF_E5M2, MNB_WF_NVFP4 = 1, 2, 3
KERNELS = {"auto": 0, "gemv": 1, "gemv_mma": 2, "gemm_tc": 3, "generic": 4, "gemv_i8": 5}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}

# Every symbol include/mnb.h declares.
EXPORTS = [
    "mnb_packed_size", "mnb_pack_weights", "mnb_unpack_codes", "mnb_dequantize", "mnb_matmul",
    "mnb_matmul_ex", "mnb_workspace_size", "mnb_quantize_activations", "mnb_select_kernel",
    "mnb_get_device_error", "mnb_status_string", "mnb_kernel_name", "mnb_abi_version", "mnb_matmul_a8_static",
    "mnb_matmul_host_io", "mnb_matmul_grouped", "mnb_fp_packed_size", "mnb_pack_fp_weights", "mnb_matmul_fp",
    "mnb_matmul_fp_ex", "mnb_packed_size_gidx", "mnb_pack_weights_gidx", "mnb_workspace_size_ex",
    "mnb_rotary_table", "mnb_rotary", "mnb_rotary_append", "mnb_paged_attention", "mnb_attention_workspace_size",
    "mnb_pages_copy", "mnb_cache_fork", "mnb_cache_resize", "mnb_cache_compact", "mnb_cache_workspace_size",
    "mnb_rms_norm", "mnb_moe_route", "mnb_moe", "mnb_moe_workspace_size", "mnb_sample",
]
MNB_A8_STATIC_SCRATCH_BYTES = 1 << 20
MNB_HOST_IO_X_BYTES = 8 << 20


class MnbError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class MatmulArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("packed_b", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("zero_points", ctypes.c_void_p), ("g_idx", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("bits", ctypes.c_int), ("block_size", ctypes.c_int), ("act_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("scale_dtype", ctypes.c_int), ("bias_dtype", ctypes.c_int),
        ("accuracy_level", ctypes.c_int), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("kernel", ctypes.c_int), ("stream", ctypes.c_void_p), ("flags", ctypes.c_int),
    ]


class KvCache(ctypes.Structure):
    """mnb_kv_cache; made by kv_cache()."""
    max_len = (1 << 30) - 1  # tokens that a row of the tables has columns for
    _fields_ = [
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("tables", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("batch", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
    ]


class RotaryArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("T", ctypes.c_int64), ("q_heads", ctypes.c_int64),
        ("rot_dim", ctypes.c_int64), ("n_pos", ctypes.c_int64), ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64), ("q_out_token_stride", ctypes.c_int64),
        ("q_out_head_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("flags", ctypes.c_int), ("stream", ctypes.c_void_p),
    ]


class AttentionArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("max_q", ctypes.c_int64), ("max_kv", ctypes.c_int64),
        ("window", ctypes.c_int64), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("o_token_stride", ctypes.c_int64), ("o_head_stride", ctypes.c_int64), ("scale", ctypes.c_float),
        ("causal", ctypes.c_int), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
    ]


class PagePlanes(ctypes.Structure):
    """mnb_page_planes; made by page_planes()."""
    _fields_ = [
        ("base", ctypes.c_void_p), ("num_planes", ctypes.c_int64), ("plane_stride", ctypes.c_int64),
        ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64), ("num_pages", ctypes.c_int64),
    ]


class CacheState(ctypes.Structure):
    """mnb_cache_state; made by cache_state()."""
    _fields_ = [
        ("refs", ctypes.c_void_p), ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64), ("num_seqs", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int),
    ]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
        ("weight", ctypes.c_void_p), ("y", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("width", ctypes.c_int64), ("block_size", ctypes.c_int64), ("x_stride", ctypes.c_int64),
        ("residual_stride", ctypes.c_int64), ("residual_out_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("eps", ctypes.c_float),
        ("flags", ctypes.c_int), ("stream", ctypes.c_void_p),
    ]


class MoeRouteArgs(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("weights", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("E", ctypes.c_int64), ("S", ctypes.c_int64), ("logits_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int), ("scoring", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float),
        ("stream", ctypes.c_void_p),
    ]


class ExpertWeights(ctypes.Structure):
    """mnb_expert_weights; made by expert_weights()."""
    _fields_ = [
        ("packed_b", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zero_points", ctypes.c_void_p),
        ("E", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("bits", ctypes.c_int),
        ("block_size", ctypes.c_int), ("scale_dtype", ctypes.c_int),
    ]


class MoeArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("gate", ctypes.POINTER(ExpertWeights)),
        ("up", ctypes.POINTER(ExpertWeights)), ("down", ctypes.POINTER(ExpertWeights)), ("x_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64), ("act_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("activation", ctypes.c_int), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
    ]


class SampleArgs(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p), ("u", ctypes.c_void_p), ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
        ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("probs", ctypes.c_void_p),
        ("B", ctypes.c_int64), ("V", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("dtype", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build: bool = True):
    """Build (if stale) and load libmnb.so; raises if that is impossible."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build() if build else _build.LIB
        lib = ctypes.CDLL(path)
        vp, i64, ci, sz, dbl = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
        sig = {
            "mnb_packed_size": (sz, [i64, i64, ci, ci]),
            "mnb_pack_weights": (ci, [vp, vp, sz, i64, i64, ci, ci, vp]),
            "mnb_packed_size_gidx": (sz, [i64, i64, ci, ci]),
            "mnb_workspace_size_ex": (sz, [i64, i64, i64, ci, ci, ci, ci]),
            "mnb_pack_weights_gidx": (ci, [vp, vp, vp, sz, i64, i64, ci, ci, vp]),
            "mnb_unpack_codes": (ci, [vp, vp, i64, i64, ci, ci, vp]),
            "mnb_dequantize": (ci, [vp, vp, vp, vp, i64, i64, ci, ci, ci, vp]),
            "mnb_matmul": (ci, [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, ci, ci, vp]),
            "mnb_matmul_ex": (ci, [ctypes.POINTER(MatmulArgs)]),
            "mnb_workspace_size": (sz, [i64, i64, i64, ci, ci, ci]),
            "mnb_quantize_activations": (ci, [vp, vp, vp, i64, i64, ci, ci, vp]),
            "mnb_select_kernel": (ci, [i64, i64, i64, ci, ci, ci, ci]),
            "mnb_get_device_error": (ci, [ctypes.POINTER(ci)]),
            "mnb_status_string": (ctypes.c_char_p, [ci]),
            "mnb_kernel_name": (ctypes.c_char_p, [ci]),
            "mnb_abi_version": (ci, []),
            "mnb_matmul_a8_static": (ci, [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, ci, ci, vp]),
            "mnb_matmul_host_io": (ci, [ctypes.POINTER(MatmulArgs)]),
            "mnb_matmul_grouped": (ci, [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, i64, i64, ci, ci, ci, ci, ci,
                                        vp]),
            "mnb_rotary_table": (ci, [vp, vp, i64, i64, dbl, ci, dbl, dbl, dbl, dbl, dbl, vp]),
            "mnb_rotary": (ci, [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, i64, ci, ci, vp]),
            "mnb_rotary_append": (ci, [ctypes.POINTER(RotaryArgs), ctypes.POINTER(KvCache)]),
            "mnb_paged_attention": (ci, [ctypes.POINTER(AttentionArgs), ctypes.POINTER(KvCache)]),
            "mnb_attention_workspace_size": (sz, [i64, i64, i64, i64, i64, i64, i64, ci]),
            "mnb_pages_copy": (ci, [ctypes.POINTER(PagePlanes), vp, vp, i64, vp]),
            "mnb_cache_workspace_size": (sz, [i64, i64, i64]),
            "mnb_cache_fork": (ci, [ctypes.POINTER(CacheState), vp, vp, i64, vp, sz, vp]),
            "mnb_cache_resize": (ci, [ctypes.POINTER(CacheState), ctypes.POINTER(PagePlanes), vp, vp, i64, vp, sz, vp]),
            "mnb_cache_compact": (ci, [ctypes.POINTER(CacheState), ctypes.POINTER(PagePlanes), vp, vp, vp, vp, sz, vp]),
            "mnb_rms_norm": (ci, [ctypes.POINTER(RmsNormArgs)]),
            "mnb_moe_route": (ci, [ctypes.POINTER(MoeRouteArgs)]),
            "mnb_moe": (ci, [ctypes.POINTER(MoeArgs), ctypes.POINTER(MoeRouteArgs)]),
            "mnb_moe_workspace_size": (sz, [i64, i64, i64, i64, i64]),
            "mnb_sample": (ci, [ctypes.POINTER(SampleArgs)]),
            "mnb_fp_packed_size": (sz, [i64, i64, ci]),
            "mnb_pack_fp_weights": (ci, [vp, vp, sz, i64, i64, ci, vp]),
            "mnb_matmul_fp": (ci, [vp, vp, vp, ctypes.c_float, vp, i64, i64, i64, ci, ci, ci, vp]),
            "mnb_matmul_fp_ex": (ci, [vp, vp, vp, ctypes.c_float, vp, i64, i64, i64, ci, ci, ci, vp, ci]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != MNB_OK:
        raise MnbError(status, what)


def status_string(status: int) -> str:
    try:
        return load().mnb_status_string(status).decode()
    except Exception:  # the library itself may be what failed to load
        return f"status {status}"


def mnb_abi_version() -> int:
    return load().mnb_abi_version()


def mnb_packed_size(N, K, bits, block_size) -> int:
    return load().mnb_packed_size(N, K, bits, block_size)


def mnb_pack_weights(b_ort, packed_b, N, K, bits, block_size, stream=None):
    _check(load().mnb_pack_weights(_ptr(b_ort), _ptr(packed_b), packed_b.numel() * packed_b.element_size(),
                                   N, K, bits, block_size, _stream(stream)), "mnb_pack_weights")


def mnb_packed_size_gidx(N, K, bits, block_size) -> int:
    return load().mnb_packed_size_gidx(N, K, bits, block_size)


def mnb_pack_weights_gidx(b_ort, g_idx, packed_b, N, K, bits, block_size, stream=None):
    """Act-order pack: depths sorted by their g_idx block, the permutation stored in the buffer
    (use it with flags=MNB_FLAG_KPERM and no g_idx)."""
    _check(load().mnb_pack_weights_gidx(_ptr(b_ort), _ptr(g_idx), _ptr(packed_b),
                                        packed_b.numel() * packed_b.element_size(), N, K, bits, block_size,
                                        _stream(stream)), "mnb_pack_weights_gidx")


def mnb_unpack_codes(packed_b, b_ort, N, K, bits, block_size, stream=None):
    _check(load().mnb_unpack_codes(_ptr(packed_b), _ptr(b_ort), N, K, bits, block_size, _stream(stream)),
           "mnb_unpack_codes")


def mnb_dequantize(packed_b, scales, zero_points, w_nk, N, K, bits, block_size, scale_dtype, stream=None):
    _check(load().mnb_dequantize(_ptr(packed_b), _ptr(scales), _ptr(zero_points), _ptr(w_nk), N, K, bits,
                                 block_size, scale_dtype, _stream(stream)), "mnb_dequantize")


def mnb_matmul(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
               scale_dtype, stream=None):
    _check(load().mnb_matmul(_ptr(x), _ptr(packed_b), _ptr(scales), _ptr(zero_points), _ptr(y), M, N, K, bits,
                             block_size, act_dtype, out_dtype, scale_dtype, _stream(stream)), "mnb_matmul")


def _matmul_args(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                 scale_dtype, g_idx, bias, bias_dtype, accuracy_level, workspace, kernel, stream, flags):
    a = MatmulArgs()
    a.x, a.packed_b, a.scales, a.zero_points = _ptr(x), _ptr(packed_b), _ptr(scales), _ptr(zero_points)
    a.g_idx, a.bias, a.y = _ptr(g_idx), _ptr(bias), _ptr(y)
    a.M, a.N, a.K, a.bits, a.block_size = M, N, K, bits, block_size
    a.act_dtype, a.out_dtype, a.scale_dtype, a.bias_dtype = act_dtype, out_dtype, scale_dtype, bias_dtype
    a.accuracy_level = accuracy_level
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.kernel = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    a.stream = _stream(stream)
    a.flags = flags
    return a


def mnb_matmul_ex(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                  scale_dtype, g_idx=None, bias=None, bias_dtype=MNB_F32, accuracy_level=0, workspace=None,
                  kernel="auto", stream=None, flags=0):
    a = _matmul_args(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                     scale_dtype, g_idx, bias, bias_dtype, accuracy_level, workspace, kernel, stream, flags)
    _check(load().mnb_matmul_ex(ctypes.byref(a)), f"mnb_matmul_ex[{kernel}]")


def mnb_matmul_host_io(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                       scale_dtype, g_idx=None, bias=None, bias_dtype=MNB_F32, accuracy_level=0, workspace=None,
                       kernel="auto", stream=None, flags=0):
    """As mnb_matmul_ex, with x and y page-locked host tensors (e.g. .pin_memory())."""
    a = _matmul_args(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                     scale_dtype, g_idx, bias, bias_dtype, accuracy_level, workspace, kernel, stream, flags)
    _check(load().mnb_matmul_host_io(ctypes.byref(a)), f"mnb_matmul_host_io[{kernel}]")


def mnb_matmul_a8_static(x, packed_b, scales, zero_points, y, M, N, K, bits, block_size, act_dtype, out_dtype,
                         scale_dtype, stream=None):
    _check(load().mnb_matmul_a8_static(_ptr(x), _ptr(packed_b), _ptr(scales), _ptr(zero_points), _ptr(y), M, N, K,
                                       bits, block_size, act_dtype, out_dtype, scale_dtype, _stream(stream)),
           "mnb_matmul_a8_static")


def mnb_matmul_grouped(x, ids, packed_b, scales, zero_points, y, T, S, E, N, K, bits, block_size, act_dtype,
                       out_dtype, scale_dtype, x_per_slot=False, stream=None):
    """Grouped (mixture-of-experts) product: y[t, s] = x_row(t, s) . dequant(B[ids[t, s]])^T."""
    _check(load().mnb_matmul_grouped(_ptr(x), _ptr(ids), _ptr(packed_b), _ptr(scales), _ptr(zero_points), _ptr(y),
                                     T, S, E, 1 if x_per_slot else 0, N, K, bits, block_size, act_dtype, out_dtype,
                                     scale_dtype, _stream(stream)), "mnb_matmul_grouped")


def mnb_fp_packed_size(N, K, fmt) -> int:
    return load().mnb_fp_packed_size(N, K, fmt)


def mnb_pack_fp_weights(w_kn, packed, N, K, fmt, stream=None):
    """Re-tile a [K, N] FP8 / NVFP4 weight (device uint8) for mnb_matmul_fp."""
    _check(load().mnb_pack_fp_weights(_ptr(w_kn), _ptr(packed), packed.numel() * packed.element_size(), N, K, fmt,
                                      _stream(stream)), "mnb_pack_fp_weights")


def mnb_matmul_fp(x, packed, scales, global_scale, y, M, N, K, fmt, act_dtype, out_dtype, stream=None, flags=0):
    """Y = X . W for an FP8 (scales f32 [N] or None) or NVFP4 (e4m3 [ceil(K/16), N] scales) weight;
    flags (MNB_FLAG_*) go through mnb_matmul_fp_ex."""
    if flags:
        _check(load().mnb_matmul_fp_ex(_ptr(x), _ptr(packed), _ptr(scales), float(global_scale), _ptr(y), M, N, K,
                                       fmt, act_dtype, out_dtype, _stream(stream), int(flags)), "mnb_matmul_fp_ex")
        return
    _check(load().mnb_matmul_fp(_ptr(x), _ptr(packed), _ptr(scales), float(global_scale), _ptr(y), M, N, K, fmt,
                                act_dtype, out_dtype, _stream(stream)), "mnb_matmul_fp")


def mnb_workspace_size_ex(M, N, K, bits, block_size, accuracy_level, flags) -> int:
    return load().mnb_workspace_size_ex(M, N, K, bits, block_size, accuracy_level, flags)


def mnb_workspace_size(M, N, K, bits, block_size, accuracy_level) -> int:
    return load().mnb_workspace_size(M, N, K, bits, block_size, accuracy_level)


def mnb_quantize_activations(x, qa, sa, M, K, block_size, act_dtype, stream=None):
    _check(load().mnb_quantize_activations(_ptr(x), _ptr(qa), _ptr(sa), M, K, block_size, act_dtype,
                                           _stream(stream)), "mnb_quantize_activations")


def mnb_select_kernel(M, N, K, bits, block_size, act_dtype, accuracy_level=0) -> str:
    return KERNEL_NAMES[load().mnb_select_kernel(M, N, K, bits, block_size, act_dtype, accuracy_level)]


# ---- between the weight products: positions, cache, attention ----------------------------------
# Sizes and strides come from the tensors: rows are [tokens, heads, dim] views with unit stride in dim.  These calls
# run between microsecond kernels, so their checks are a few attribute reads each.

_codes = {}  # torch dtype -> dtype code, filled on first use
_int8 = _int32 = _float32 = _device = _raw_stream = None


def _setup():
    global _int8, _int32, _float32, _device, _raw_stream
    import torch
    _int8, _int32, _float32 = torch.int8, torch.int32, torch.float32
    _device, _raw_stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _codes.update({torch.float32: MNB_F32, torch.float16: MNB_F16, torch.bfloat16: MNB_BF16})


def _current(stream):
    """The call's stream: torch's current one by its raw handle, without making a Stream object."""
    if stream is None and _raw_stream is not None and _device is not None:
        return _raw_stream(_device())
    return _stream(stream)


def _fail(what):
    raise ValueError(what)


def _i32(what, t):
    if t.dtype is not _int32 or not t.is_contiguous():
        _fail(f"{what}: a contiguous int32 tensor is wanted")
    return t.data_ptr()


def _table_pair(cos_table, sin_table):
    shape = cos_table.shape
    if len(shape) != 2 or sin_table.shape != shape or cos_table.dtype is not _float32 or sin_table.dtype is not _float32 or \
            not cos_table.is_contiguous() or not sin_table.is_contiguous():
        _fail("cos_table, sin_table: contiguous f32 [n_pos, rot_dim / 2] tensors of one shape are wanted")
    return shape[0], 2 * shape[1]


# Rows' strides are checked where there are rows: an empty tensor's mean nothing (one made from numpy has zeros).
def _rows_fail(what):
    _fail(f"{what}: a [tokens, heads, dim] tensor of the call's dtype with unit stride in dim is wanted")


def kv_cache(k_pages, v_pages, tables, kv_lens, order, dtype) -> KvCache:
    """The cache descriptor of one layer.  Pages are [num_pages, heads, tokens, dim] (order "hnd") or
    [num_pages, tokens, heads, dim] ("nhd") tensors of one shape and one set of strides.  The descriptor holds the
    tensors' addresses (and the tensors): make it once per layer and keep it beside them.  tables may be some columns of
    a wider array: a kv_len that needs more of them sets the status word (with positions of its own, the append takes
    the array's next column instead)."""
    if not _codes:
        _setup()
    if order not in ("hnd", "nhd"):
        _fail('order is "hnd" or "nhd"')
    if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() or k_pages.dim() != 4 or k_pages.stride(3) != 1 or \
            _codes.get(k_pages.dtype) != dtype or v_pages.dtype is not k_pages.dtype:
        _fail("k_pages, v_pages: 4-d tensors of dtype, one shape and one set of strides are wanted")
    lens_ptr = _i32("kv_lens", kv_lens)
    if tables.dtype is not _int32 or tables.dim() != 2 or (tables.shape[1] > 1 and tables.stride(1) != 1) or \
            kv_lens.numel() < tables.shape[0]:
        _fail("tables: an int32 [batch, columns] tensor with a kv_len for each row is wanted")
    c = KvCache()
    head, tok = (1, 2) if order == "hnd" else (2, 1)
    c.k_pages, c.v_pages, c.tables, c.kv_lens = k_pages.data_ptr(), v_pages.data_ptr(), tables.data_ptr(), lens_ptr
    c.batch = tables.shape[0]
    # rows are table_stride apart; a single row takes its width
    c.table_stride = tables.stride(0) if tables.shape[0] > 1 else tables.shape[1]
    if c.table_stride < tables.shape[1]:
        _fail("tables: rows overlap")
    c.num_pages, c.page_stride = k_pages.shape[0], k_pages.stride(0)
    c.token_stride, c.head_stride = k_pages.stride(tok), k_pages.stride(head)
    c.page_size, c.kv_heads, c.head_dim, c.dtype = k_pages.shape[tok], k_pages.shape[head], k_pages.shape[3], dtype
    c.max_len = min(c.max_len, tables.shape[1] * c.page_size)
    c.tensors = (k_pages, v_pages, tables, kv_lens)
    return c


def page_planes(pool) -> PagePlanes:
    """The pages of all planes (keys and values of every layer) of a [planes, pages, ...] tensor whose pages are
    contiguous, as bytes."""
    p, e = PagePlanes(), pool.element_size()
    inner = 1
    for n, st in zip(reversed(pool.shape[2:]), reversed(pool.stride()[2:])):
        if n > 1 and st != inner:
            _fail("pool: contiguous pages are wanted")
        inner *= n
    p.base, p.num_planes, p.num_pages = pool.data_ptr(), pool.shape[0], pool.shape[1]
    p.plane_stride, p.page_stride, p.page_bytes = pool.stride(0) * e, pool.stride(1) * e, inner * e
    p.tensors = (pool,)
    return p


def cache_state(refs, tables, lens, page_size) -> CacheState:
    """Reference counts [pages], page tables [sequences, columns] and lengths [sequences], contiguous int32."""
    if not _codes:
        _setup()
    s = CacheState()
    s.refs, s.tables, s.lens = _i32("refs", refs), _i32("tables", tables), _i32("lens", lens)
    if tables.dim() != 2 or lens.numel() != tables.shape[0]:
        _fail("tables: [sequences, columns] with a length for each row is wanted")
    s.num_pages, s.num_seqs, s.table_stride, s.page_size = refs.numel(), tables.shape[0], tables.shape[1], page_size
    s.tensors = (refs, tables, lens)
    return s


def mnb_rotary_table(cos_table, sin_table, base=10000.0, scaling=MNB_ROPE_NONE, factor=1.0, trained_len=0.0, low=1.0,
                     high=32.0, attn_factor=1.0, stream=None):
    """Fill the f32 [n_pos, rot_dim / 2] tables (see mnb_rope_scaling for the long-context forms)."""
    if not _codes:
        _setup()
    n_pos, rot = _table_pair(cos_table, sin_table)
    _check(load().mnb_rotary_table(_ptr(cos_table), _ptr(sin_table), n_pos, rot, base, scaling, factor, trained_len,
                                   low, high, attn_factor, _current(stream)), "mnb_rotary_table")


def mnb_rotary(x, y, positions, cos_table, sin_table, dtype, flags=0, stream=None):
    """y = x with the first rot_dim = 2 * cos_table.shape[1] depths of each head turned; x, y [T, H, D]."""
    if not _codes:
        _setup()
    n_pos, rot = _table_pair(cos_table, sin_table)
    shape, xs, ys = x.shape, x.stride(), y.stride()
    if y.shape != shape or len(shape) != 3 or xs[2] != 1 and shape[0] or ys[2] != 1 and shape[0] or _codes.get(x.dtype) != dtype or \
            y.dtype is not x.dtype:
        _rows_fail("x, y")
    pos_ptr = _i32("positions", positions)
    if positions.numel() != shape[0]:
        _fail("positions: one for each token is wanted")
    st = (_lib or load()).mnb_rotary(x.data_ptr(), y.data_ptr(), pos_ptr, cos_table.data_ptr(), sin_table.data_ptr(), shape[0], shape[1],
                                     shape[2], rot, n_pos, xs[0], xs[1], ys[0], ys[1], dtype, flags, _current(stream))
    if st:
        _check(st, "mnb_rotary")


def mnb_rotary_append(q, q_out, k, v, cos_table, sin_table, cache, q_start, positions=None, flags=0, stream=None):
    """Turn q into q_out (q None: append only) and k, and write k and v to the cache's pages."""
    if not _codes:
        _setup()
    n_pos, rot = _table_pair(cos_table, sin_table)
    dtype, ks, vs, shape = cache.dtype, k.stride(), v.stride(), k.shape
    if v.shape != shape or len(shape) != 3 or ks[2] != 1 and shape[0] or vs[2] != 1 and shape[0] or _codes.get(k.dtype) != dtype or \
            v.dtype is not k.dtype or \
            shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        _fail("k, v: [T, kv_heads, head_dim] rows of the cache's dtype are wanted")
    start_ptr, pos_ptr = _i32("q_start", q_start), None
    if q_start.numel() != cache.batch + 1:
        _fail("q_start: batch + 1 entries are wanted")
    if positions is not None:
        pos_ptr = _i32("positions", positions)
        if positions.numel() != shape[0]:
            _fail("positions: one for each token is wanted")
    elif n_pos > cache.max_len:
        n_pos = cache.max_len  # a token's position is its place, and the table's columns end there
    qp = op = None
    heads, qs, os_ = 0, (0, 0), (0, 0)
    if q is not None:
        qshape, qs, os_ = q.shape, q.stride(), q_out.stride()
        if q_out.shape != qshape or len(qshape) != 3 or qs[2] != 1 and shape[0] or os_[2] != 1 and shape[0] or \
                q.dtype is not k.dtype or q_out.dtype is not k.dtype or qshape[0] != shape[0] or qshape[2] != shape[2]:
            _fail("q, q_out: [T, q_heads, head_dim] rows of the cache's dtype are wanted")
        qp, op, heads = q.data_ptr(), q_out.data_ptr(), qshape[1]
    a = RotaryArgs(qp, op, k.data_ptr(), v.data_ptr(), cos_table.data_ptr(), sin_table.data_ptr(), start_ptr, pos_ptr, shape[0], heads, rot,
                   n_pos, qs[0], qs[1], os_[0], os_[1], ks[0], ks[1], vs[0], vs[1], flags, _current(stream))
    st = (_lib or load()).mnb_rotary_append(a, cache)
    if st:
        _check(st, "mnb_rotary_append")


def mnb_attention_workspace_size(batch, T, q_heads, kv_heads, head_dim, max_q, max_kv, dtype) -> int:
    return load().mnb_attention_workspace_size(batch, T, q_heads, kv_heads, head_dim, max_q, max_kv, dtype)


def mnb_paged_attention(q, o, cache, q_start, max_q, max_kv, scale, lse=None, causal=True, window=0, workspace=None,
                        stream=None):
    """Attention of the tokens q [T, q_heads, head_dim] over the cache; lse f32 [T, q_heads] or None."""
    if not _codes:
        _setup()
    shape, qs, os_ = q.shape, q.stride(), o.stride()
    if o.shape != shape or len(shape) != 3 or qs[2] != 1 and shape[0] or os_[2] != 1 and shape[0] or \
            _codes.get(q.dtype) != cache.dtype or o.dtype is not q.dtype or shape[2] != cache.head_dim:
        _fail("q, o: [T, q_heads, head_dim] rows of the cache's dtype are wanted")
    start_ptr, lse_ptr, ws_ptr, ws_bytes = _i32("q_start", q_start), None, None, 0
    if q_start.numel() != cache.batch + 1:
        _fail("q_start: batch + 1 entries are wanted")
    if lse is not None:
        if lse.dtype is not _float32 or lse.shape != shape[:2] or not lse.is_contiguous():
            _fail("lse: a contiguous f32 [T, q_heads] tensor is wanted")
        lse_ptr = lse.data_ptr()
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if max_kv > cache.max_len:
        max_kv = cache.max_len  # (a longer sequence has pages past its row of the tables)
    a = AttentionArgs(q.data_ptr(), o.data_ptr(), lse_ptr, start_ptr, shape[0], shape[1], max_q, max_kv, window, qs[0], qs[1], os_[0], os_[1],
                      scale, 1 if causal else 0, ws_ptr, ws_bytes, _current(stream))
    st = (_lib or load()).mnb_paged_attention(a, cache)
    if st:
        _check(st, "mnb_paged_attention")


def _pair_lists(a, b, what):
    pa, pb, n = _i32(what, a), _i32(what, b), a.numel()
    if b.numel() != n:
        _fail(f"{what}: two lists of one length are wanted")
    return pa, pb, n


def _space(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def mnb_pages_copy(planes, src, dst, stream=None):
    """Copy page src[i] to page dst[i] in every plane."""
    if not _codes:
        _setup()
    st = (_lib or load()).mnb_pages_copy(planes, *_pair_lists(src, dst, "src, dst"), _current(stream))
    if st:
        _check(st, "mnb_pages_copy")


def mnb_cache_workspace_size(num_pages, num_seqs, table_stride) -> int:
    return load().mnb_cache_workspace_size(num_pages, num_seqs, table_stride)


def mnb_cache_fork(state, src, dst, workspace=None, stream=None):
    """Sequence dst[i] becomes a fork of sequence src[i] (pages shared, nothing copied)."""
    st = (_lib or load()).mnb_cache_fork(state, *_pair_lists(src, dst, "src, dst"), *_space(workspace), _current(stream))
    if st:
        _check(st, "mnb_cache_fork")


def mnb_cache_resize(state, planes, seqs, new_lens, workspace=None, stream=None):
    """Sequence seqs[i] gets new_lens[i] tokens: pages are taken, released, or copied where a shared one grows."""
    st = (_lib or load()).mnb_cache_resize(state, planes, *_pair_lists(seqs, new_lens, "seqs, new_lens"), *_space(workspace), _current(stream))
    if st:
        _check(st, "mnb_cache_resize")


def mnb_cache_compact(state, planes, refs_out, tables_out, counts, workspace=None, stream=None):
    """Press the held pages together; counts (int32 [2]) gets the held and the moved pages."""
    ptrs = _i32("refs_out", refs_out), _i32("tables_out", tables_out), _i32("counts", counts)
    if refs_out.numel() != state.num_pages or tables_out.numel() != state.num_seqs * state.table_stride or counts.numel() != 2:
        _fail("refs_out, tables_out: arrays of the state's sizes, and counts [2], are wanted")
    st = (_lib or load()).mnb_cache_compact(state, planes, *ptrs, *_space(workspace), _current(stream))
    if st:
        _check(st, "mnb_cache_compact")


# ---- around the attention: norm, experts, the next token ----------------------------------------

# Tensors have to live on the current device, whose stream the call goes to (`dev`, asked once a call).

def _current_device():
    return -2 if _device is None else _device()


def _away(what):
    _fail(f"{what}: a tensor on the current CUDA device is wanted")


def _here(what, t, dev):
    d = t.get_device()
    if d < 0 or (d != dev and dev != -2):
        _away(what)
    return t.data_ptr()


def _row_matrix(what, t, shape, dev, dtype=None):
    """(pointer, row stride) of a [rows, columns] tensor with unit stride in a row."""
    st = t.stride()
    if len(st) != 2 or t.shape != shape or (st[1] != 1 and shape[1] > 1 and shape[0]) or (dtype is not None and t.dtype is not dtype):
        _fail(f"{what}: a [rows, columns] tensor of the call's shape and dtype with unit stride in a row is wanted")
    d = t.get_device()
    if d < 0 or (d != dev and dev != -2):
        _away(what)
    return t.data_ptr(), st[0]


def mnb_rms_norm(x, weight, eps, residual=None, residual_out=None, y=None, codes=None, scales=None, block_size=0, flags=0,
                 stream=None):
    """S = x + residual to residual_out; its norm to y and, as int8 codes with a scale for each block of block_size values,
    to codes [T, KB * block_size] and scales [T, KB].  x [T, width]; weight [width] or None."""
    if not _codes:
        _setup()
    shape, dt, dev = x.shape, x.dtype, _current_device() if x.is_cuda else -2
    code = _codes.get(dt)
    if code is None:
        _fail("x: a float32, float16 or bfloat16 tensor is wanted")
    xp, xs = _row_matrix("x", x, shape, dev)
    rp = sp = yp = wp = cp = ap = None
    rs = ss = ys = yd = wd = 0
    if residual is not None:
        rp, rs = _row_matrix("residual", residual, shape, dev, dt)
    if residual_out is not None:
        sp, ss = _row_matrix("residual_out", residual_out, shape, dev, dt)
    if y is not None:
        yp, ys = _row_matrix("y", y, shape, dev)
        yd = _codes.get(y.dtype, -1)
    if weight is not None:
        wd = _codes.get(weight.dtype, -1)
        if weight.numel() != shape[1] or not weight.is_contiguous():
            _fail("weight: a contiguous [width] tensor is wanted")
        wp = _here("weight", weight, dev)
    if codes is not None or scales is not None:
        if codes is None or scales is None or block_size < 1:
            _fail("codes, scales: both, with a block_size, are wanted")
        kb = -(-shape[1] // block_size)
        if codes.dtype is not _int8 or codes.shape != (shape[0], kb * block_size) or not codes.is_contiguous() or \
                scales.dtype is not _float32 or scales.shape != (shape[0], kb) or not scales.is_contiguous():
            _fail("codes, scales: contiguous int8 [T, KB * block_size] and f32 [T, KB] tensors are wanted")
        cp, ap = _here("codes", codes, dev), _here("scales", scales, dev)
    a = RmsNormArgs(xp, rp, sp, wp, yp, cp, ap, shape[0], shape[1], block_size, xs, rs, ss, ys, code, wd, yd, eps, flags, _current(stream))
    st = (_lib or load()).mnb_rms_norm(a)
    if st:
        _check(st, "mnb_rms_norm")


def expert_weights(packed, scales, zero_points, E, N, K, bits, block_size) -> ExpertWeights:
    """The weights [N, K] of E experts: packed back to back (mnb_packed_size(N, K, bits, block_size) bytes each), scales
    [E, N, KB], zero points [E, N, ceil(KB * bits / 8)] uint8 or None.  The descriptor holds the tensors."""
    if not _codes:
        _setup()
    kb = -(-K // block_size) if block_size > 0 else 0
    size = load().mnb_packed_size(N, K, bits, block_size)
    if E < 1 or size == 0 or packed.numel() * packed.element_size() < E * size or not packed.is_contiguous():
        _fail("packed: a contiguous buffer of E packed weights is wanted")
    if scales.dtype not in _codes or scales.numel() != E * N * kb or not scales.is_contiguous():
        _fail("scales: a contiguous [E, N, KB] tensor is wanted")
    if zero_points is not None and (zero_points.element_size() != 1 or zero_points.numel() != E * N * -(-kb * bits // 8) or
                                    not zero_points.is_contiguous()):
        _fail("zero_points: a contiguous uint8 [E, N, ceil(KB * bits / 8)] tensor is wanted")
    dev = _current_device() if packed.is_cuda else -2
    w = ExpertWeights(_here("packed", packed, dev), _here("scales", scales, dev),
                      None if zero_points is None else _here("zero_points", zero_points, dev), E, N, K, bits, block_size, _codes[scales.dtype])
    w.tensors = (packed, scales, zero_points)
    w.dev = dev
    # (ctypes.pointer(w) would hold w: a cycle that keeps the weights on the GPU until the collector runs)
    w.ref = ctypes.POINTER(ExpertWeights).from_buffer(ctypes.c_void_p(ctypes.addressof(w)))
    return w


def _route(logits, top_k, ids, weights, bias, scoring, renormalize, scale, stream, dev):
    shape, code = logits.shape, _codes.get(logits.dtype)
    if code is None:
        _fail("logits: a float32, float16 or bfloat16 tensor is wanted")
    lp, ls = _row_matrix("logits", logits, shape, dev)
    bp = ip = wp = None
    if bias is not None:
        if bias.dtype is not _float32 or bias.numel() != shape[1] or not bias.is_contiguous():
            _fail("bias: a contiguous f32 [E] tensor is wanted")
        bp = _here("bias", bias, dev)
    if ids is not None:
        ip = _i32("ids", ids)
        if ids.shape != (shape[0], top_k):
            _fail("ids: an int32 [T, top_k] tensor is wanted")
        _here("ids", ids, dev)
    if weights is not None:
        if weights.dtype is not _float32 or weights.shape != (shape[0], top_k) or not weights.is_contiguous():
            _fail("weights: a contiguous f32 [T, top_k] tensor is wanted")
        wp = _here("weights", weights, dev)
    return MoeRouteArgs(lp, bp, ip, wp, shape[0], shape[1], top_k, ls, code, scoring, 1 if renormalize else 0, scale, stream)


def mnb_moe_route(logits, ids, weights, bias=None, scoring=MNB_MOE_SOFTMAX, renormalize=True, scale=1.0, stream=None):
    """The experts (int32 [T, S]) of each token's logits [T, E] and their weights (f32 [T, S])."""
    if not _codes:
        _setup()
    dev = _current_device() if logits.is_cuda else -2
    a = _route(logits, ids.shape[-1], ids, weights, bias, scoring, renormalize, scale, _current(stream), dev)
    st = (_lib or load()).mnb_moe_route(a)
    if st:
        _check(st, "mnb_moe_route")


def mnb_moe_workspace_size(T, S, E, hidden, inner) -> int:
    return load().mnb_moe_workspace_size(T, S, E, hidden, inner)


def mnb_moe(x, logits, gate, up, down, y, top_k, ids=None, weights=None, bias=None, scoring=MNB_MOE_SOFTMAX, renormalize=True,
            scale=1.0, activation=MNB_ACT_SILU, workspace=None, stream=None):
    """y [T, hidden] = the layer's experts (expert_weights() descriptors) on x [T, hidden], selected by logits [T, E];
    ids and weights [T, top_k], where given, get the selection."""
    if not _codes:
        _setup()
    s, dev = _current(stream), _current_device() if logits.is_cuda else -2
    ws_ptr, ws_bytes = _space(workspace)
    if workspace is not None:
        if not workspace.is_contiguous():
            _fail("workspace: a contiguous buffer is wanted")
        _here("workspace", workspace, dev)
    r = _route(logits, top_k, ids, weights, bias, scoring, renormalize, scale, s, dev)
    shape = x.shape
    code, out = _codes.get(x.dtype, -1), _codes.get(y.dtype, -1)
    if len(shape) != 2 or shape[0] != r.T or shape[1] != gate.K:
        _fail("x: [T, hidden] rows, one for each row of logits, are wanted")
    if dev != -2 and not (gate.dev == up.dev == down.dev == dev):
        _away("gate, up, down")
    xp, xs = _row_matrix("x", x, shape, dev)
    yp, ys = _row_matrix("y", y, shape, dev)
    a = MoeArgs(xp, yp, gate.ref, up.ref, down.ref, xs, ys, code, out, activation, ws_ptr, ws_bytes, s)
    st = (_lib or load()).mnb_moe(a, r)
    if st:
        _check(st, "mnb_moe")


def _per_row(what, t, dtype, n, dev):
    if t is None:
        return None
    d = t.get_device()
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _fail(f"{what}: a contiguous {dtype} tensor with a value for each row is wanted")
    if d < 0 or (d != dev and dev != -2):
        _away(what)
    return t.data_ptr()


def mnb_sample(logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, stream=None):
    """A token (int32 [B]) of each row of logits [B, V] from the uniform numbers u (f32 [B]); the cuts are tensors with a
    value for each row, or None; probs (f32 [B]) gets the tokens' probabilities after the cuts."""
    if not _codes:
        _setup()
    shape, code, dev = logits.shape, _codes.get(logits.dtype), _current_device() if logits.is_cuda else -2
    if code is None:
        _fail("logits: a float32, float16 or bfloat16 tensor is wanted")
    lp, ls = _row_matrix("logits", logits, shape, dev)
    if u is None or tokens is None:
        _fail("u, tokens: a tensor with a value for each row is wanted")
    n, f = shape[0], _float32
    a = SampleArgs(lp, _per_row("u", u, f, n, dev), _per_row("temperature", temperature, f, n, dev), _per_row("top_k", top_k, _int32, n, dev),
                   _per_row("top_p", top_p, f, n, dev), _per_row("min_p", min_p, f, n, dev), _per_row("tokens", tokens, _int32, n, dev),
                   _per_row("probs", probs, f, n, dev), n, shape[1], ls, code, _current(stream))
    st = (_lib or load()).mnb_sample(a)
    if st:
        _check(st, "mnb_sample")


def mnb_get_device_error() -> int:
    code = ctypes.c_int(0)
    _check(load().mnb_get_device_error(ctypes.byref(code)), "mnb_get_device_error")
    return code.value


def mnb_status_string(status: int) -> str:
    return status_string(status)


def mnb_kernel_name(k: int) -> str:
    return load().mnb_kernel_name(k).decode()
