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
# Sizes and strides come from the tensors: rows are [tokens, heads, dim] views with unit stride in dim.

def _rows(t, what):
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError(f"{what}: a [tokens, heads, dim] tensor with unit stride in dim is wanted")
    return t.stride(0), t.stride(1)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _i32(*named):
    for what, t in named:
        if t is not None and (str(t.dtype) != "torch.int32" or not t.is_contiguous()):
            raise ValueError(f"{what}: a contiguous int32 tensor is wanted")


_DTYPE_OF = {"torch.float32": MNB_F32, "torch.float16": MNB_F16, "torch.bfloat16": MNB_BF16}


def _same_dtype(code, *named):
    for what, t in named:
        if t is not None and _DTYPE_OF.get(str(t.dtype)) != code:
            raise ValueError(f"{what}: {t.dtype} does not match the call's dtype code {code}")


def _table_pair(cos_table, sin_table):
    for t in (cos_table, sin_table):
        if t.dim() != 2 or not t.is_contiguous() or str(t.dtype) != "torch.float32" or t.shape != cos_table.shape:
            raise ValueError("cos_table, sin_table: contiguous f32 [n_pos, rot_dim / 2] tensors of one shape are wanted")
    return cos_table.shape[0], 2 * cos_table.shape[1]


def kv_cache(k_pages, v_pages, tables, kv_lens, order, dtype) -> KvCache:
    """The cache descriptor of one layer.  Pages are [num_pages, heads, tokens, dim] (order "hnd") or
    [num_pages, tokens, heads, dim] ("nhd") tensors of one shape and one set of strides.  The descriptor holds the
    tensors' addresses (and the tensors): make it once per layer and keep it beside them."""
    if order not in ("hnd", "nhd"):
        raise ValueError('order is "hnd" or "nhd"')
    if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() or k_pages.dim() != 4 or k_pages.stride(3) != 1:
        raise ValueError("k_pages, v_pages: 4-d tensors of one shape and one set of strides are wanted")
    _same_dtype(dtype, ("k_pages", k_pages), ("v_pages", v_pages))
    _i32(("kv_lens", kv_lens))
    if str(tables.dtype) != "torch.int32" or tables.dim() != 2 or (tables.shape[1] > 1 and tables.stride(1) != 1) or \
            kv_lens.numel() < tables.shape[0]:
        raise ValueError("tables: an int32 [batch, columns] tensor with a kv_len for each row is wanted")
    c = KvCache()
    head, tok = (1, 2) if order == "hnd" else (2, 1)
    c.k_pages, c.v_pages, c.tables, c.kv_lens = k_pages.data_ptr(), v_pages.data_ptr(), tables.data_ptr(), kv_lens.data_ptr()
    c.batch = tables.shape[0]
    # rows are table_stride apart; a single row, or rows apart by less than their width, take the width
    c.table_stride = tables.stride(0) if tables.shape[0] > 1 else tables.shape[1]
    if c.table_stride < tables.shape[1]:
        raise ValueError("tables: rows overlap")
    c.num_pages, c.page_stride = k_pages.shape[0], k_pages.stride(0)
    c.token_stride, c.head_stride = k_pages.stride(tok), k_pages.stride(head)
    c.page_size, c.kv_heads, c.head_dim, c.dtype = k_pages.shape[tok], k_pages.shape[head], k_pages.shape[3], dtype
    c.tensors = (k_pages, v_pages, tables, kv_lens)
    return c


def page_planes(pool) -> PagePlanes:
    """The pages of all planes (keys and values of every layer) of a [planes, pages, ...] tensor whose pages are
    contiguous, as bytes."""
    p, e = PagePlanes(), pool.element_size()
    inner = 1
    for n, st in zip(reversed(pool.shape[2:]), reversed(pool.stride()[2:])):
        if n > 1 and st != inner:
            raise ValueError("pool: contiguous pages are wanted")
        inner *= n
    p.base, p.num_planes, p.num_pages = pool.data_ptr(), pool.shape[0], pool.shape[1]
    p.plane_stride, p.page_stride, p.page_bytes = pool.stride(0) * e, pool.stride(1) * e, inner * e
    p.tensors = (pool,)
    return p


def cache_state(refs, tables, lens, page_size) -> CacheState:
    """Reference counts [pages], page tables [sequences, columns] and lengths [sequences], contiguous int32."""
    _i32(("refs", refs), ("tables", tables), ("lens", lens))
    if tables.dim() != 2 or lens.numel() != tables.shape[0]:
        raise ValueError("tables: [sequences, columns] with a length for each row is wanted")
    s = CacheState()
    s.refs, s.tables, s.lens = refs.data_ptr(), tables.data_ptr(), lens.data_ptr()
    s.num_pages, s.num_seqs, s.table_stride, s.page_size = refs.numel(), tables.shape[0], tables.shape[1], page_size
    s.tensors = (refs, tables, lens)
    return s


def mnb_rotary_table(cos_table, sin_table, base=10000.0, scaling=MNB_ROPE_NONE, factor=1.0, trained_len=0.0, low=1.0,
                     high=32.0, attn_factor=1.0, stream=None):
    """Fill the f32 [n_pos, rot_dim / 2] tables (see mnb_rope_scaling for the long-context forms)."""
    n_pos, rot = _table_pair(cos_table, sin_table)
    _check(load().mnb_rotary_table(_ptr(cos_table), _ptr(sin_table), n_pos, rot, base, scaling, factor, trained_len,
                                   low, high, attn_factor, _stream(stream)), "mnb_rotary_table")


def mnb_rotary(x, y, positions, cos_table, sin_table, dtype, flags=0, stream=None):
    """y = x with the first rot_dim = 2 * cos_table.shape[1] depths of each head turned; x, y [T, H, D]."""
    n_pos, rot = _table_pair(cos_table, sin_table)
    _same_dtype(dtype, ("x", x), ("y", y))
    _i32(("positions", positions))
    if x.shape != y.shape or positions.numel() != x.shape[0]:
        raise ValueError("x, y: one shape, with a position for each token, is wanted")
    _check(load().mnb_rotary(_ptr(x), _ptr(y), _ptr(positions), _ptr(cos_table), _ptr(sin_table), *x.shape, rot, n_pos,
                             *_rows(x, "x"), *_rows(y, "y"), dtype, flags, _stream(stream)), "mnb_rotary")


def mnb_rotary_append(q, q_out, k, v, cos_table, sin_table, cache, q_start, positions=None, flags=0, stream=None):
    """Turn q into q_out (q None: append only) and k, and write k and v to the cache's pages."""
    a = RotaryArgs()
    a.n_pos, a.rot_dim = _table_pair(cos_table, sin_table)
    _same_dtype(cache.dtype, ("q", q), ("q_out", q_out), ("k", k), ("v", v))
    _i32(("q_start", q_start), ("positions", positions))
    a.T = k.shape[0]
    if k.shape != v.shape or tuple(k.shape[1:]) != (cache.kv_heads, cache.head_dim) or q_start.numel() != cache.batch + 1 or \
            (positions is not None and positions.numel() != a.T):
        raise ValueError("k, v: [T, kv_heads, head_dim] of the cache, and q_start [batch + 1], are wanted")
    a.k_token_stride, a.k_head_stride = _rows(k, "k")
    a.v_token_stride, a.v_head_stride = _rows(v, "v")
    if q is not None:
        if q.shape != q_out.shape or q.shape[0] != a.T or q.shape[2] != cache.head_dim:
            raise ValueError("q, q_out: [T, q_heads, head_dim] is wanted")
        a.q, a.q_out, a.q_heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
        a.q_token_stride, a.q_head_stride = _rows(q, "q")
        a.q_out_token_stride, a.q_out_head_stride = _rows(q_out, "q_out")
    a.k, a.v, a.cos_table, a.sin_table = k.data_ptr(), v.data_ptr(), cos_table.data_ptr(), sin_table.data_ptr()
    a.q_start, a.positions, a.flags, a.stream = q_start.data_ptr(), _ptr(positions), flags, _stream(stream)
    _check(load().mnb_rotary_append(ctypes.byref(a), ctypes.byref(cache)), "mnb_rotary_append")


def mnb_attention_workspace_size(batch, T, q_heads, kv_heads, head_dim, max_q, max_kv, dtype) -> int:
    return load().mnb_attention_workspace_size(batch, T, q_heads, kv_heads, head_dim, max_q, max_kv, dtype)


def mnb_paged_attention(q, o, cache, q_start, max_q, max_kv, scale, lse=None, causal=True, window=0, workspace=None,
                        stream=None):
    """Attention of the tokens q [T, q_heads, head_dim] over the cache; lse f32 [T, q_heads] or None."""
    _same_dtype(cache.dtype, ("q", q), ("o", o))
    _i32(("q_start", q_start))
    if q.shape != o.shape or q.shape[2] != cache.head_dim or q_start.numel() != cache.batch + 1:
        raise ValueError("q, o: [T, q_heads, head_dim] of the cache, and q_start [batch + 1], are wanted")
    if lse is not None and (tuple(lse.shape) != tuple(q.shape[:2]) or not lse.is_contiguous() or str(lse.dtype) != "torch.float32"):
        raise ValueError("lse: a contiguous f32 [T, q_heads] tensor is wanted")
    a = AttentionArgs()
    a.q, a.o, a.lse, a.q_start = q.data_ptr(), o.data_ptr(), _ptr(lse), q_start.data_ptr()
    a.T, a.q_heads, a.max_q, a.max_kv, a.window = q.shape[0], q.shape[1], max_q, max_kv, window
    a.q_token_stride, a.q_head_stride = _rows(q, "q")
    a.o_token_stride, a.o_head_stride = _rows(o, "o")
    a.scale, a.causal = scale, 1 if causal else 0
    a.workspace, a.workspace_bytes, a.stream = _ptr(workspace), _nbytes(workspace), _stream(stream)
    _check(load().mnb_paged_attention(ctypes.byref(a), ctypes.byref(cache)), "mnb_paged_attention")


def _pair_lists(a, b, what):
    _i32((what, a), (what, b))
    if a.numel() != b.numel():
        raise ValueError(f"{what}: two lists of one length are wanted")
    return a.data_ptr(), b.data_ptr(), a.numel()


def mnb_pages_copy(planes, src, dst, stream=None):
    """Copy page src[i] to page dst[i] in every plane."""
    _check(load().mnb_pages_copy(ctypes.byref(planes), *_pair_lists(src, dst, "src, dst"), _stream(stream)), "mnb_pages_copy")


def mnb_cache_workspace_size(num_pages, num_seqs, table_stride) -> int:
    return load().mnb_cache_workspace_size(num_pages, num_seqs, table_stride)


def mnb_cache_fork(state, src, dst, workspace=None, stream=None):
    """Sequence dst[i] becomes a fork of sequence src[i] (pages shared, nothing copied)."""
    _check(load().mnb_cache_fork(ctypes.byref(state), *_pair_lists(src, dst, "src, dst"), _ptr(workspace), _nbytes(workspace),
                                 _stream(stream)), "mnb_cache_fork")


def mnb_cache_resize(state, planes, seqs, new_lens, workspace=None, stream=None):
    """Sequence seqs[i] gets new_lens[i] tokens: pages are taken, released, or copied where a shared one grows."""
    _check(load().mnb_cache_resize(ctypes.byref(state), None if planes is None else ctypes.byref(planes),
                                   *_pair_lists(seqs, new_lens, "seqs, new_lens"), _ptr(workspace), _nbytes(workspace),
                                   _stream(stream)), "mnb_cache_resize")


def mnb_cache_compact(state, planes, refs_out, tables_out, counts, workspace=None, stream=None):
    """Press the held pages together; counts (int32 [2]) gets the held and the moved pages."""
    _i32(("refs_out", refs_out), ("tables_out", tables_out), ("counts", counts))
    if refs_out.numel() != state.num_pages or tables_out.numel() != state.num_seqs * state.table_stride or counts.numel() != 2:
        raise ValueError("refs_out, tables_out: arrays of the state's sizes, and counts [2], are wanted")
    _check(load().mnb_cache_compact(ctypes.byref(state), ctypes.byref(planes), _ptr(refs_out), _ptr(tables_out),
                                    _ptr(counts), _ptr(workspace), _nbytes(workspace), _stream(stream)), "mnb_cache_compact")


def mnb_get_device_error() -> int:
    code = ctypes.c_int(0)
    _check(load().mnb_get_device_error(ctypes.byref(code)), "mnb_get_device_error")
    return code.value


def mnb_status_string(status: int) -> str:
    return status_string(status)


def mnb_kernel_name(k: int) -> str:
    return load().mnb_kernel_name(k).decode()
