"""Thin ctypes binding of liboscar (include/oscar.h). Same names as the C ABI.

Only argument marshalling happens here: tensors become device pointers and
sizes, host arrays become host pointers. Every step of the write and decode
path runs in the library's CUDA kernels. There is no fallback: if liboscar.so is
missing or fails to load, every call raises.
"""

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liboscar.so")

OSCAR_OK = 0
STATUS_NAMES = {
    0: "OSCAR_OK", -1: "OSCAR_ERR_INVALID_ARG", -2: "OSCAR_ERR_UNSUPPORTED", -3: "OSCAR_ERR_NOT_CALIBRATED",
    -4: "OSCAR_ERR_CUDA", -5: "OSCAR_ERR_BOUNDS", -6: "OSCAR_ERR_NO_MEMORY", -7: "OSCAR_ERR_WORKSPACE",
}


class OscarError(RuntimeError):
    def __init__(self, status, where, message):
        self.status = status
        super().__init__("%s: %s (%s) %s" % (where, STATUS_NAMES.get(status, status), oscar_status_string(status), message))


class oscar_config_t(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("group", ctypes.c_int), ("page_size", ctypes.c_int),
                ("sink", ctypes.c_int), ("recent", ctypes.c_int), ("sm_scale", ctypes.c_float),
                ("debug_bounds", ctypes.c_int), ("codebook", ctypes.c_int)]

OSCAR_CODEBOOK_UNIFORM, OSCAR_CODEBOOK_LLOYD_MAX = 0, 1


_lib = None
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "oscar_create": (_i, [ctypes.POINTER(oscar_config_t), ctypes.POINTER(_vp)]),
    "oscar_destroy": (None, [_vp]),
    "oscar_calibrate_upload": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp]),
    "oscar_write_tokens": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, _i64, _vp]),
    "oscar_demote_recent": (_i, [_vp, _i, _vp, _i64, _vp, _vp, _i64, _vp, _i, _vp]),
    "oscar_decode_workspace_size": (_sz, [_vp, _i, _i]),
    "oscar_decode": (_i, [_vp, _i, _vp, _vp, _i64, _vp, _i, _vp, _i, _vp, _i64, _vp, _i, _vp,
                          _vp, _vp, _sz, _i, _vp]),
    "oscar_decode_shared_prefix_workspace_size": (_sz, [_vp, _i, _i, _i]),
    "oscar_decode_shared_prefix": (_i, [_vp, _i, _vp, _vp, _i64, _vp, _i, _vp, _i, _vp, _i, _vp, _i64, _vp, _i, _vp,
                                        _vp, _vp, _sz, _i, _vp]),
    "oscar_int2_page_bytes": (_sz, [_vp]),
    "oscar_bf16_page_bytes": (_sz, [_vp]),
    "oscar_status_string": (ctypes.c_char_p, [_i]),
    "oscar_last_error": (ctypes.c_char_p, []),
    "oscar_debug_error": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_longlong)]),
    "oscar_decode_static_workspace": (_i, [_vp, _i, _vp, _vp, _i64, _vp, _i, _vp, _i, _vp, _i64, _vp, _i, _vp,
                                           _vp, _i, _vp]),
    "oscar_calibration_workspace_size": (_sz, [_i, _i, _i, _i]),
    "oscar_calibration_targets": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_double, _vp, _vp, _vp, _sz,
                                       _vp]),
    "oscar_plan_append": (_i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp]),
    "oscar_append_bf16": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _i, _vp, _i64, _vp, _vp, _vp]),
    "oscar_decode_bf16_workspace_size": (_sz, [_vp, _i, _i]),
    "oscar_decode_bf16": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _i, _vp, _i, _vp, _i, _vp, _sz, _i, _vp]),
    "oscar_sparse_capacity": (_i, [_vp, _i]),
    "oscar_decode_bf16_sparse_workspace_size": (_sz, [_vp, _i, _i, _i]),
    "oscar_decode_bf16_sparse": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i, _vp, _i, _i, _vp, _vp, _vp, _i,
                                      _vp, _sz, _i, _vp]),
    "oscar_norm_rope": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, ctypes.c_float, _vp, _i, _i,
                             ctypes.c_float, _vp, _vp, _vp, _i, _i, _vp]),
    "oscar_extend_bf16_workspace_size": (_sz, [_vp, _i, _i]),
    "oscar_extend_bf16": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp]),
    "oscar_profile_enable": (_i, [_vp, _i]),
    "oscar_profile_read": (_i, [_vp, _i, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong)]),
}

OSCAR_KERNEL_WRITE, OSCAR_KERNEL_QROT, OSCAR_KERNEL_SPLIT, OSCAR_KERNEL_MERGE = 0, 1, 2, 3
OSCAR_KERNEL_PLAN, OSCAR_KERNEL_APPEND, OSCAR_KERNEL_SELECT, OSCAR_KERNEL_ATTEND = 4, 5, 6, 7
OSCAR_KERNEL_ROPE, OSCAR_KERNEL_EXTEND = 8, 9
OSCAR_OUT_FP32, OSCAR_OUT_BF16 = 0, 1
OSCAR_ROPE_HALF, OSCAR_ROPE_INTERLEAVED = 0, 1


def lib():
    """Load liboscar.so once. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("liboscar.so not found at %s: build it with "
                               "`python -m bit_kv_cache_write_gb300.build`" % LIB_PATH)
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(handle, name)
            f.restype = res
            f.argtypes = args
        _lib = handle
    return _lib


def oscar_status_string(status):
    return lib().oscar_status_string(int(status)).decode()


def oscar_last_error():
    return lib().oscar_last_error().decode()


def _check(status, where):
    if status != OSCAR_OK:
        raise OscarError(status, where, oscar_last_error())


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dptr(t, dtype, name):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def oscar_create(n_layers, n_q_heads, n_kv_heads, head_dim, group, page_size=16, sink=64, recent=256,
                 sm_scale=0.0, debug_bounds=0, codebook=OSCAR_CODEBOOK_UNIFORM):
    """Create a context on the current CUDA device; returns an opaque handle (int)."""
    cfg = oscar_config_t(n_layers, n_q_heads, n_kv_heads, head_dim, group, page_size, sink, recent,
                         float(sm_scale), int(debug_bounds), int(codebook))
    ctx = _vp()
    _check(lib().oscar_create(ctypes.byref(cfg), ctypes.byref(ctx)), "oscar_create")
    device = _torch_device()
    if device is not None:
        _configs[ctx.value] = (n_q_heads, n_kv_heads, head_dim, device, lib().oscar_sparse_capacity(ctx, 0))
    return ctx.value


def _torch_device():
    """The current device as torch counts it, or None: the calls that check their tensors' device need it, no other."""
    try:
        import torch
        return torch.cuda.current_device()
    except (ImportError, AssertionError, RuntimeError):
        return None


def oscar_destroy(ctx):
    _configs.pop(ctx, None)
    lib().oscar_destroy(ctx)


def oscar_calibrate_upload(ctx, layer, R_k, R_v, T_k, T_v, stream=None):
    """R_k, R_v: host fp32 [H_kv][d][d]; T_k, T_v: host fp32 [H_kv][d]."""
    arrs = [np.ascontiguousarray(a, dtype=np.float32) for a in (R_k, R_v, T_k, T_v)]
    ptrs = [a.ctypes.data_as(_vp) for a in arrs]
    _check(lib().oscar_calibrate_upload(ctx, layer, *ptrs, _stream(stream)), "oscar_calibrate_upload")


def oscar_int2_page_bytes(ctx):
    return lib().oscar_int2_page_bytes(ctx)


def oscar_bf16_page_bytes(ctx):
    return lib().oscar_bf16_page_bytes(ctx)


def oscar_write_tokens(ctx, layer, k, v, slots, int2_pool, stream=None):
    """k, v: bf16 [n][H_kv][d]; slots: int64 [n]; int2_pool: uint8 tensor of whole pages."""
    import torch
    n = slots.numel()
    pages = int2_pool.numel() // oscar_int2_page_bytes(ctx)
    _check(lib().oscar_write_tokens(ctx, layer, _dptr(k, torch.bfloat16, "k"), _dptr(v, torch.bfloat16, "v"),
                                    _dptr(slots, torch.int64, "slots"), n, _dptr(int2_pool, torch.uint8, "int2_pool"),
                                    pages, _stream(stream)), "oscar_write_tokens")


def oscar_demote_recent(ctx, layer, bf16_pool, src_slots, int2_pool, dst_slots, stream=None):
    import torch
    if src_slots.numel() != dst_slots.numel():
        raise ValueError("src_slots and dst_slots differ in length")
    bf_pages = bf16_pool.numel() * 2 // oscar_bf16_page_bytes(ctx)
    i2_pages = int2_pool.numel() // oscar_int2_page_bytes(ctx)
    _check(lib().oscar_demote_recent(ctx, layer, _dptr(bf16_pool, torch.bfloat16, "bf16_pool"), bf_pages,
                                     _dptr(src_slots, torch.int64, "src_slots"),
                                     _dptr(int2_pool, torch.uint8, "int2_pool"), i2_pages,
                                     _dptr(dst_slots, torch.int64, "dst_slots"), src_slots.numel(),
                                     _stream(stream)), "oscar_demote_recent")


def oscar_decode_workspace_size(ctx, batch, max_hist):
    return lib().oscar_decode_workspace_size(ctx, batch, max_hist)


def oscar_decode(ctx, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool, bf16_tables, bf16_len,
                 out, workspace, stream=None):
    """q: bf16 [B][H_q][d]; tables int32 [B][stride]; lengths int32 [B]; out fp32 [B][H_q][d]; workspace uint8."""
    import torch
    batch = q.shape[0]
    i2_pages = int2_pool.numel() // oscar_int2_page_bytes(ctx) if int2_pool is not None else 0
    bf_pages = bf16_pool.numel() * 2 // oscar_bf16_page_bytes(ctx)
    _check(lib().oscar_decode(
        ctx, layer, _dptr(q, torch.bfloat16, "q"),
        _dptr(int2_pool, torch.uint8, "int2_pool"), i2_pages,
        _dptr(int2_tables, torch.int32, "int2_tables"), int2_tables.shape[1] if int2_tables is not None else 0,
        _dptr(hist_len, torch.int32, "hist_len"), int(max_hist),
        _dptr(bf16_pool, torch.bfloat16, "bf16_pool"), bf_pages,
        _dptr(bf16_tables, torch.int32, "bf16_tables"), bf16_tables.shape[1],
        _dptr(bf16_len, torch.int32, "bf16_len"),
        _dptr(out, torch.float32, "out"), _dptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), batch, _stream(stream)), "oscar_decode")


def oscar_decode_shared_prefix_workspace_size(ctx, batch, prefix_pages, max_hist):
    return lib().oscar_decode_shared_prefix_workspace_size(ctx, batch, prefix_pages, max_hist)


def oscar_decode_shared_prefix(ctx, layer, q, int2_pool, prefix_table, int2_tables, hist_len, max_hist, bf16_pool,
                               bf16_tables, bf16_len, out, workspace, stream=None):
    """oscar_decode with a prefix shared by the whole batch: prefix_table int32 [P] (full pages), then each
    sequence's own pages in int2_tables [B][stride] with hist_len counting the tokens after the prefix."""
    import torch
    batch = q.shape[0]
    i2_pages = int2_pool.numel() // oscar_int2_page_bytes(ctx)
    bf_pages = bf16_pool.numel() * 2 // oscar_bf16_page_bytes(ctx)
    _check(lib().oscar_decode_shared_prefix(
        ctx, layer, _dptr(q, torch.bfloat16, "q"),
        _dptr(int2_pool, torch.uint8, "int2_pool"), i2_pages,
        _dptr(prefix_table, torch.int32, "prefix_table"), prefix_table.numel() if prefix_table is not None else 0,
        _dptr(int2_tables, torch.int32, "int2_tables"), int2_tables.shape[1] if int2_tables is not None else 0,
        _dptr(hist_len, torch.int32, "hist_len"), int(max_hist),
        _dptr(bf16_pool, torch.bfloat16, "bf16_pool"), bf_pages,
        _dptr(bf16_tables, torch.int32, "bf16_tables"), bf16_tables.shape[1],
        _dptr(bf16_len, torch.int32, "bf16_len"),
        _dptr(out, torch.float32, "out"), _dptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), batch, _stream(stream)), "oscar_decode_shared_prefix")


def oscar_calibration_workspace_size(n, n_q_heads, n_kv_heads, head_dim):
    return lib().oscar_calibration_workspace_size(n, n_q_heads, n_kv_heads, head_dim)


def oscar_calibration_targets(q_cal, k_cal, v_cal, sm_scale, target_k, target_v, workspace, stream=None):
    """q_cal fp32 [n][H_q][d], k_cal/v_cal fp32 [m][H_kv][d] -> target_k/target_v fp64 [H_kv][d][d] (device)."""
    import torch
    n, h_q, d = q_cal.shape
    m, h_kv = k_cal.shape[0], k_cal.shape[1]
    _check(lib().oscar_calibration_targets(
        _dptr(q_cal, torch.float32, "q_cal"), _dptr(k_cal, torch.float32, "k_cal"),
        _dptr(v_cal, torch.float32, "v_cal"), n, m, h_q, h_kv, d, float(sm_scale),
        _dptr(target_k, torch.float64, "target_k"), _dptr(target_v, torch.float64, "target_v"),
        _dptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream)),
        "oscar_calibration_targets")


def oscar_decode_static_workspace(ctx, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool,
                                  bf16_tables, bf16_len, out, stream=None):
    """oscar_decode for callers that cannot allocate: the scratch is the library's static device array.

    Same arguments as oscar_decode without the workspace. The library rejects
    sizes whose workspace exceeds its fixed maximum. Calls that overlap on the
    GPU share that array and race.
    """
    import torch
    batch = q.shape[0]
    i2_pages = int2_pool.numel() // oscar_int2_page_bytes(ctx) if int2_pool is not None else 0
    bf_pages = bf16_pool.numel() * 2 // oscar_bf16_page_bytes(ctx)
    _check(lib().oscar_decode_static_workspace(
        ctx, layer, _dptr(q, torch.bfloat16, "q"),
        _dptr(int2_pool, torch.uint8, "int2_pool"), i2_pages,
        _dptr(int2_tables, torch.int32, "int2_tables"), int2_tables.shape[1] if int2_tables is not None else 0,
        _dptr(hist_len, torch.int32, "hist_len"), int(max_hist),
        _dptr(bf16_pool, torch.bfloat16, "bf16_pool"), bf_pages,
        _dptr(bf16_tables, torch.int32, "bf16_tables"), bf16_tables.shape[1],
        _dptr(bf16_len, torch.int32, "bf16_len"),
        _dptr(out, torch.float32, "out"), batch, _stream(stream)), "oscar_decode_static_workspace")


# context handle -> (H_q, H_kv, d, device, pages that a sparse decode always keeps at most) of the contexts created
# here, for the checks below
_configs = {}


def _config_of(ctx):
    try:
        return _configs[ctx]
    except KeyError:
        raise ValueError("the context was not created by oscar_create, or torch saw no device then") from None


def _stream_on(stream, device):
    """Raw handle of the stream, by default of the device's current one."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # a 30th of current_stream()'s cost
        return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(t, dtype, n, device, name):
    """Says why _ptr does not take a tensor."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.get_device() != device:
        raise ValueError("%s is on device %d, the context on %d" % (name, t.get_device(), device))
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must hold %d elements, holds %d" % (name, n, t.numel()))


def _ptr(t, dtype, n, device, name):
    """Pointer of a contiguous tensor of n elements on the context's device."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, n, device, name)


def _rows(t, bf16, heads, d, device, name):
    """(pointer, row stride in elements) of bf16 rows [n][heads][d] whose heads lie together."""
    try:
        n, h, c = t.shape
        row, head, one = t.stride()
        if h == heads and c == d and t.dtype is bf16 and t.get_device() == device and (
                n == 0 or (one == 1 and (head == d or heads == 1))):
            return t.data_ptr(), row if n > 1 else heads * d
    except (AttributeError, ValueError):
        pass
    if getattr(t, "dim", lambda: 0)() == 3 and tuple(t.shape[1:]) == (heads, d) and t.dtype is bf16 and \
            t.get_device() == device:
        raise ValueError("%s: a row's heads must be contiguous (strides %s)" % (name, t.stride()))
    if getattr(t, "is_cuda", False) and t.dtype is bf16 and t.get_device() == device:
        raise ValueError("%s must be [n][%d][%d], got %s" % (name, heads, d, tuple(t.shape)))
    _refuse(t, bf16, 0, device, name)


def _bound(value, name):
    """An int that the C ABI takes whole (ctypes would cut it to 32 bits)."""
    if not -0x80000000 <= value <= 0x7fffffff:
        raise ValueError("%s %s does not fit in 32 bits" % (name, value))
    return value


def _table(t, batch, dtype, device):
    """(pointer, row length) of contiguous block tables [batch][stride]."""
    try:
        rows, stride = t.shape
    except ValueError:
        rows = -1
    if rows != batch:
        raise ValueError("tables must be [%d][stride], got %s" % (batch, tuple(t.shape)))
    _bound(batch, "batch")
    _bound(stride, "table stride")
    return _ptr(t, dtype, rows * stride, device, "tables"), stride


def _output(out, n, device, torch):
    """(pointer, oscar_out_type) of an output of n elements."""
    dtype = out.dtype
    if dtype is torch.float32:
        return _ptr(out, dtype, n, device, "out"), OSCAR_OUT_FP32
    if dtype is torch.bfloat16:
        return _ptr(out, dtype, n, device, "out"), OSCAR_OUT_BF16
    raise ValueError("out must be torch.float32 or torch.bfloat16, got %s" % dtype)


def _scratch(workspace, device):
    """(pointer, bytes) of a workspace tensor or None."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != device or not workspace.is_contiguous():
        _refuse(workspace, workspace.dtype, 0, device, "workspace")
    return workspace.data_ptr(), workspace.nbytes


def oscar_plan_append(ctx, seq_len, new_len, free_pages, free_head, tables, slots, row_start, total_len, state,
                      stream=None):
    """seq_len, new_len int32 [B]; free_pages int32; free_head int32 [1]; tables int32 [B][stride] (in and out);
    out: slots int64, row_start int32 [B + 1], total_len int32 [B], state int32 [4]."""
    import torch
    dev = _config_of(ctx)[3]
    i32, batch, n_free, n_slots = torch.int32, seq_len.numel(), free_pages.numel(), slots.numel()
    tp, ts = _table(tables, batch, i32, dev)
    st = lib().oscar_plan_append(
        ctx, _ptr(seq_len, i32, batch, dev, "seq_len"), _ptr(new_len, i32, batch, dev, "new_len"), batch,
        _ptr(free_pages, i32, n_free, dev, "free_pages"), _bound(n_free, "free_pages"),
        _ptr(free_head, i32, 1, dev, "free_head"), tp, ts, _ptr(slots, torch.int64, n_slots, dev, "slots"),
        _bound(n_slots, "slots"), _ptr(row_start, i32, batch + 1, dev, "row_start"),
        _ptr(total_len, i32, batch, dev, "total_len"), _ptr(state, i32, 4, dev, "state"), _stream_on(stream, dev))
    if st:
        _check(st, "oscar_plan_append")


def oscar_append_bf16(ctx, k, v, slots, bf16_pool, key_steps=None, key_bounds=None, stream=None):
    """k, v: bf16 [n][H_kv][d], rows at any stride; slots int64 [n]; bf16_pool: whole pages; key_steps int8
    [H_kv][d] and key_bounds int8 [pages][H_kv][2][d], or neither."""
    import torch
    _, h_kv, d, dev, _ = _config_of(ctx)
    bf16 = torch.bfloat16
    kp, ks = _rows(k, bf16, h_kv, d, dev, "k")
    vp, vs = _rows(v, bf16, h_kv, d, dev, "v")
    n, size = k.shape[0], bf16_pool.numel()
    if v.shape[0] != n:
        raise ValueError("k and v differ in length")
    pages = size // (h_kv * 32 * d)
    steps = bounds = None
    if key_steps is not None or key_bounds is not None:
        steps = _ptr(key_steps, torch.int8, h_kv * d, dev, "key_steps")
        bounds = _ptr(key_bounds, torch.int8, pages * h_kv * 2 * d, dev, "key_bounds")
    st = lib().oscar_append_bf16(ctx, kp, ks, vp, vs, _ptr(slots, torch.int64, n, dev, "slots"), _bound(n, "tokens"),
                                 _ptr(bf16_pool, bf16, size, dev, "bf16_pool"), pages, steps, bounds,
                                 _stream_on(stream, dev))
    if st:
        _check(st, "oscar_append_bf16")


def oscar_decode_bf16_workspace_size(ctx, batch, max_len):
    return lib().oscar_decode_bf16_workspace_size(ctx, _bound(batch, "batch"), _bound(max_len, "max_len"))


def oscar_decode_bf16(ctx, q, bf16_pool, tables, seq_len, max_len, out, workspace, stream=None):
    """q: bf16 [B][H_q][d], rows at any stride; tables int32 [B][stride]; seq_len int32 [B], at most max_len;
    out fp32 or bf16 [B][H_q][d]; workspace uint8."""
    import torch
    h_q, h_kv, d, dev, _ = _config_of(ctx)
    qp, qs = _rows(q, torch.bfloat16, h_q, d, dev, "q")
    batch, size = q.shape[0], bf16_pool.numel()
    tp, ts = _table(tables, batch, torch.int32, dev)
    op, ot = _output(out, batch * h_q * d, dev, torch)
    wp, ws = _scratch(workspace, dev)
    st = lib().oscar_decode_bf16(
        ctx, qp, qs, _ptr(bf16_pool, torch.bfloat16, size, dev, "bf16_pool"), size // (h_kv * 32 * d), tp, ts,
        _ptr(seq_len, torch.int32, batch, dev, "seq_len"), _bound(max_len, "max_len"), op, ot, wp, ws, batch,
        _stream_on(stream, dev))
    if st:
        _check(st, "oscar_decode_bf16")


def oscar_sparse_capacity(ctx, top_pages):
    return lib().oscar_sparse_capacity(ctx, _bound(top_pages, "top_pages"))


def oscar_decode_bf16_sparse_workspace_size(ctx, batch, max_len, top_pages):
    return lib().oscar_decode_bf16_sparse_workspace_size(ctx, _bound(batch, "batch"), _bound(max_len, "max_len"),
                                                         _bound(top_pages, "top_pages"))


def oscar_decode_bf16_sparse(ctx, q, bf16_pool, key_steps, key_bounds, tables, seq_len, max_len, top_pages, chosen,
                             n_chosen, out, workspace, stream=None):
    """oscar_decode_bf16 over the sink, the recent window and the top_pages best pages by their key bounds; chosen
    int32 [B][H_kv][oscar_sparse_capacity(ctx, top_pages)] and n_chosen int32 [B][H_kv] say which."""
    import torch
    h_q, h_kv, d, dev, kept = _config_of(ctx)
    i8, i32 = torch.int8, torch.int32
    qp, qs = _rows(q, torch.bfloat16, h_q, d, dev, "q")
    batch, size = q.shape[0], bf16_pool.numel()
    pages = size // (h_kv * 32 * d)
    tp, ts = _table(tables, batch, i32, dev)
    op, ot = _output(out, batch * h_q * d, dev, torch)
    wp, ws = _scratch(workspace, dev)
    listed = 0 <= _bound(top_pages, "top_pages") <= 65536        # else the library refuses it
    st = lib().oscar_decode_bf16_sparse(
        ctx, qp, qs, _ptr(bf16_pool, torch.bfloat16, size, dev, "bf16_pool"), pages,
        _ptr(key_steps, i8, h_kv * d, dev, "key_steps"), _ptr(key_bounds, i8, pages * h_kv * 2 * d, dev, "key_bounds"),
        tp, ts, _ptr(seq_len, i32, batch, dev, "seq_len"), _bound(max_len, "max_len"), top_pages,
        _ptr(chosen, i32, batch * h_kv * (kept + top_pages), dev, "chosen") if listed else None,
        _ptr(n_chosen, i32, batch * h_kv, dev, "n_chosen"), op, ot, wp, ws, batch, _stream_on(stream, dev))
    if st:
        _check(st, "oscar_decode_bf16_sparse")


def _pair(x, out, weight, fp32, bf16, heads, d, n, device, name):
    """Pointers and strides of rows, their output's rows and their weights; nothing of either for None."""
    if x is None and out is None:
        return None, 0, None, 0, None
    xp, xs = _rows(x, bf16, heads, d, device, name)
    if x.shape[0] != n:
        raise ValueError("%s must have %d rows, has %d" % (name, n, x.shape[0]))
    if out is not None and out.is_contiguous():
        op, os_ = _ptr(out, bf16, n * heads * d, device, name + "_out"), heads * d
    else:
        op, os_ = _rows(out, bf16, heads, d, device, name + "_out")
        if out.shape[0] != n:
            raise ValueError("%s_out must have %d rows, has %d" % (name, n, out.shape[0]))
    return xp, xs, op, os_, None if weight is None else _ptr(weight, fp32, d, device, name + "_weight")


def oscar_norm_rope(ctx, q, k, q_out, k_out, turns, positions=None, row_start=None, total_len=None, q_weight=None,
                    k_weight=None, eps=1e-6, layout=OSCAR_ROPE_HALF, scale=1.0, stream=None):
    """q bf16 [n][H_q][d] -> q_out, k bf16 [n][H_kv][d] -> k_out, rows at any stride, either pair None; turns int64
    [rot_dim / 2] (rope.rope_turns) or None; positions int32 [n], or row_start int32 [B + 1] and total_len int32 [B]
    of the plan; weights fp32 [d] or None."""
    import torch
    h_q, h_kv, d, dev, _ = _config_of(ctx)
    bf16, fp32, i32 = torch.bfloat16, torch.float32, torch.int32
    n = q.shape[0] if q is not None else k.shape[0] if k is not None else 0
    qp, qs, qop, qos, qw = _pair(q, q_out, q_weight, fp32, bf16, h_q, d, n, dev, "q")
    kp, ks, kop, kos, kw = _pair(k, k_out, k_weight, fp32, bf16, h_kv, d, n, dev, "k")
    half = turns.numel() if turns is not None else 0
    pp = _ptr(positions, i32, n, dev, "positions") if positions is not None else None
    batch, rp, tp = 0, None, None
    if pp is None:
        if row_start is None or total_len is None:
            raise ValueError("positions, or row_start and total_len, must be given")
        batch = total_len.numel()
        rp, tp = _ptr(row_start, i32, batch + 1, dev, "row_start"), _ptr(total_len, i32, batch, dev, "total_len")
    st = lib().oscar_norm_rope(
        ctx, qp, qs, qop, qos, kp, ks, kop, kos, qw, kw, eps,
        _ptr(turns, torch.int64, half, dev, "turns") if half else None, _bound(2 * half, "rot_dim"),
        _bound(layout, "layout"), scale, pp, rp, tp, _bound(batch, "batch"), _bound(n, "tokens"),
        _stream_on(stream, dev))
    if st:
        _check(st, "oscar_norm_rope")


def oscar_extend_bf16_workspace_size(ctx, batch, n):
    return lib().oscar_extend_bf16_workspace_size(ctx, _bound(batch, "batch"), _bound(n, "tokens"))


def oscar_extend_bf16(ctx, q, bf16_pool, tables, row_start, total_len, out, workspace, stream=None):
    """q: bf16 [n][H_q][d], rows at any stride; tables int32 [B][stride]; row_start int32 [B + 1] and total_len int32
    [B] of the plan; out bf16 [n][H_q][d]; workspace uint8."""
    import torch
    h_q, h_kv, d, dev, _ = _config_of(ctx)
    bf16, i32 = torch.bfloat16, torch.int32
    qp, qs = _rows(q, bf16, h_q, d, dev, "q")
    n, batch, size = q.shape[0], total_len.numel(), bf16_pool.numel()
    tp, ts = _table(tables, batch, i32, dev)
    wp, ws = _scratch(workspace, dev)
    st = lib().oscar_extend_bf16(
        ctx, qp, qs, _ptr(bf16_pool, bf16, size, dev, "bf16_pool"), size // (h_kv * 32 * d), tp, ts,
        _ptr(row_start, i32, batch + 1, dev, "row_start"), _ptr(total_len, i32, batch, dev, "total_len"), batch,
        _bound(n, "tokens"), _ptr(out, bf16, n * h_q * d, dev, "out"), wp, ws, _stream_on(stream, dev))
    if st:
        _check(st, "oscar_extend_bf16")


def oscar_debug_error(ctx):
    """Returns (status, kind, index) and clears the device error word."""
    kind = _i(0)
    index = ctypes.c_longlong(0)
    st = lib().oscar_debug_error(ctx, ctypes.byref(kind), ctypes.byref(index))
    return st, kind.value, index.value


def oscar_profile_enable(ctx, enable):
    _check(lib().oscar_profile_enable(ctx, int(bool(enable))), "oscar_profile_enable")


def oscar_profile_read(ctx, kernel):
    """(total_ms, launches) of one kernel class since the last read; synchronizes."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_longlong(0)
    _check(lib().oscar_profile_read(ctx, int(kernel), ctypes.byref(ms), ctypes.byref(n)), "oscar_profile_read")
    return ms.value, n.value


class Oscar:
    """Owning wrapper around one context: the same calls as methods, with ctx bound."""

    def __init__(self, **cfg):
        self.cfg = dict(cfg)
        self.ctx = oscar_create(**cfg)

    def close(self):
        if self.ctx:
            oscar_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def calibrate_upload(self, layer, R_k, R_v, T_k, T_v, stream=None):
        oscar_calibrate_upload(self.ctx, layer, R_k, R_v, T_k, T_v, stream)

    def write_tokens(self, layer, k, v, slots, int2_pool, stream=None):
        oscar_write_tokens(self.ctx, layer, k, v, slots, int2_pool, stream)

    def demote_recent(self, layer, bf16_pool, src_slots, int2_pool, dst_slots, stream=None):
        oscar_demote_recent(self.ctx, layer, bf16_pool, src_slots, int2_pool, dst_slots, stream)

    def decode_workspace_size(self, batch, max_hist):
        return oscar_decode_workspace_size(self.ctx, batch, max_hist)

    def decode(self, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool, bf16_tables, bf16_len,
               out, workspace, stream=None):
        oscar_decode(self.ctx, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool, bf16_tables,
                     bf16_len, out, workspace, stream)

    def decode_static_workspace(self, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool, bf16_tables,
                                bf16_len, out, stream=None):
        oscar_decode_static_workspace(self.ctx, layer, q, int2_pool, int2_tables, hist_len, max_hist, bf16_pool,
                                      bf16_tables, bf16_len, out, stream)

    def decode_shared_prefix_workspace_size(self, batch, prefix_pages, max_hist):
        return oscar_decode_shared_prefix_workspace_size(self.ctx, batch, prefix_pages, max_hist)

    def decode_shared_prefix(self, layer, q, int2_pool, prefix_table, int2_tables, hist_len, max_hist, bf16_pool,
                             bf16_tables, bf16_len, out, workspace, stream=None):
        oscar_decode_shared_prefix(self.ctx, layer, q, int2_pool, prefix_table, int2_tables, hist_len, max_hist,
                                   bf16_pool, bf16_tables, bf16_len, out, workspace, stream)

    def plan_append(self, seq_len, new_len, free_pages, free_head, tables, slots, row_start, total_len, state,
                    stream=None):
        oscar_plan_append(self.ctx, seq_len, new_len, free_pages, free_head, tables, slots, row_start, total_len,
                          state, stream)

    def append_bf16(self, k, v, slots, bf16_pool, key_steps=None, key_bounds=None, stream=None):
        oscar_append_bf16(self.ctx, k, v, slots, bf16_pool, key_steps, key_bounds, stream)

    def decode_bf16_workspace_size(self, batch, max_len):
        return oscar_decode_bf16_workspace_size(self.ctx, batch, max_len)

    def decode_bf16(self, q, bf16_pool, tables, seq_len, max_len, out, workspace, stream=None):
        oscar_decode_bf16(self.ctx, q, bf16_pool, tables, seq_len, max_len, out, workspace, stream)

    def sparse_capacity(self, top_pages):
        return oscar_sparse_capacity(self.ctx, top_pages)

    def decode_bf16_sparse_workspace_size(self, batch, max_len, top_pages):
        return oscar_decode_bf16_sparse_workspace_size(self.ctx, batch, max_len, top_pages)

    def decode_bf16_sparse(self, q, bf16_pool, key_steps, key_bounds, tables, seq_len, max_len, top_pages, chosen,
                           n_chosen, out, workspace, stream=None):
        oscar_decode_bf16_sparse(self.ctx, q, bf16_pool, key_steps, key_bounds, tables, seq_len, max_len, top_pages,
                                 chosen, n_chosen, out, workspace, stream)

    def norm_rope(self, q, k, q_out, k_out, turns, positions=None, row_start=None, total_len=None, q_weight=None,
                  k_weight=None, eps=1e-6, layout=OSCAR_ROPE_HALF, scale=1.0, stream=None):
        oscar_norm_rope(self.ctx, q, k, q_out, k_out, turns, positions, row_start, total_len, q_weight, k_weight, eps,
                        layout, scale, stream)

    def extend_bf16_workspace_size(self, batch, n):
        return oscar_extend_bf16_workspace_size(self.ctx, batch, n)

    def extend_bf16(self, q, bf16_pool, tables, row_start, total_len, out, workspace, stream=None):
        oscar_extend_bf16(self.ctx, q, bf16_pool, tables, row_start, total_len, out, workspace, stream)

    def int2_page_bytes(self):
        return oscar_int2_page_bytes(self.ctx)

    def bf16_page_bytes(self):
        return oscar_bf16_page_bytes(self.ctx)

    def debug_error(self):
        return oscar_debug_error(self.ctx)

    def profile_enable(self, enable):
        oscar_profile_enable(self.ctx, enable)

    def profile_read(self, kernel):
        return oscar_profile_read(self.ctx, kernel)
