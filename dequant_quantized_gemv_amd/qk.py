"""Thin Python binding of libqk (include/qk.h).

Argument marshalling only: tensors are passed as device pointers with the
current HIP stream; every step of the computation runs in the library's gfx950
kernels.  The library must be built (``python -m dequant_quantized_gemv_amd.build``
or ``__graft_entry__.build()``); loading fails loudly otherwise, and there is no
CPU fallback.
"""
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqk.so")

# enum qk_format / qk_dtype / qk_status (include/qk.h)
QK_Q4_0, QK_Q4_1, QK_Q8_0, QK_Q5_0, QK_Q5_1 = 1, 2, 3, 4, 5
QK_F32, QK_F16, QK_X8 = 0, 1, 2
QK_KV_F16, QK_KV_I8 = 0, 1
QK_SOFTMAX, QK_SIGMOID = 0, 1
QK_OK, QK_ERR_INVALID_ARG, QK_ERR_UNSUPPORTED, QK_ERR_ALIGNMENT, QK_ERR_LAUNCH = 0, 1, 2, 3, 4

FORMATS = {"q4_0": QK_Q4_0, "q4_1": QK_Q4_1, "q8_0": QK_Q8_0, "q5_0": QK_Q5_0, "q5_1": QK_Q5_1}
SYMBOLS = ("qk_block_bytes", "qk_row_bytes", "qk_status_string", "qk_version",
           "qk_dequantize", "qk_mul_mat_vec", "qk_mul_mat_vec_x8", "qk_mul_mat_vec_batched",
           "qk_mul_mat_vec_id", "qk_mul_mat", "qk_mul_mat_vec_x8q", "qk_rms_norm", "qk_kv_store",
           "qk_attn_decode", "qk_attn_decode_workspace", "qk_moe_route")
QK_MAX_BATCH = 16
X8_BLOCK_BYTES = 36  # an 8-bit activation block: fp32 scale, 32 int8 codes


class MatVecItem(ctypes.Structure):
    """struct qk_mat_vec_item (include/qk.h)."""
    _fields_ = [("w", ctypes.c_void_p), ("m", ctypes.c_int64), ("k", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class KVCacheDesc(ctypes.Structure):
    """struct qk_kv_cache (include/qk.h)."""
    _fields_ = [("type", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("n_heads", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_slot_stride", ctypes.c_int64)]


class QKError(RuntimeError):
    def __init__(self, status, call):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} (status {status})")


_lib = None


def load():
    """Load libqk.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "or python -m dequant_quantized_gemv_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.qk_block_bytes.argtypes = [ci]
    lib.qk_block_bytes.restype = ctypes.c_size_t
    lib.qk_row_bytes.argtypes = [ci, i64]
    lib.qk_row_bytes.restype = ctypes.c_size_t
    lib.qk_status_string.argtypes = [ci]
    lib.qk_status_string.restype = ctypes.c_char_p
    lib.qk_version.argtypes = []
    lib.qk_version.restype = ci
    lib.qk_dequantize.argtypes = [ci, vp, i64, i64, ci, vp, vp]
    lib.qk_dequantize.restype = ci
    lib.qk_mul_mat_vec.argtypes = [ci, vp, i64, i64, vp, i64, i64, vp, i64, vp]
    lib.qk_mul_mat_vec.restype = ci
    lib.qk_mul_mat_vec_x8.argtypes = [ci, vp, i64, i64, vp, i64, i64, vp, i64, vp]
    lib.qk_mul_mat_vec_x8.restype = ci
    lib.qk_mul_mat_vec_batched.argtypes = [ci, ctypes.POINTER(MatVecItem), ci, i64, vp]
    lib.qk_mul_mat_vec_batched.restype = ci
    lib.qk_mul_mat_vec_id.argtypes = [ci, vp, i64, i64, i64, i64, vp, i64, i64, i64,
                                      vp, i64, i64, vp, i64, i64, vp]
    lib.qk_mul_mat_vec_id.restype = ci
    lib.qk_mul_mat.argtypes = [ci, vp, i64, i64, vp, i64, i64, vp, i64, vp]
    lib.qk_mul_mat.restype = ci
    lib.qk_mul_mat_vec_x8q.argtypes = [ci, vp, i64, i64, vp, i64, i64, vp, i64, vp]
    lib.qk_mul_mat_vec_x8q.restype = ci
    lib.qk_rms_norm.argtypes = [ci, vp, i64, vp, i64, vp, ctypes.c_double, i64, i64, vp, i64, ci, vp, i64, vp]
    lib.qk_rms_norm.restype = ci
    cache = ctypes.POINTER(KVCacheDesc)
    lib.qk_kv_store.argtypes = [cache, vp, i64, i64, vp, i64, i64, i64, vp, i64, i64, i64, vp, vp, vp]
    lib.qk_kv_store.restype = ci
    lib.qk_attn_decode.argtypes = [cache, vp, i64, i64, i64, i64, vp, i64, vp, i64, ctypes.c_float, i64, i64,
                                   ci, vp, i64, i64, vp, ctypes.c_size_t, vp]
    lib.qk_attn_decode.restype = ci
    lib.qk_attn_decode_workspace.argtypes = [cache, i64, i64, i64, i64, i64]
    lib.qk_attn_decode_workspace.restype = ctypes.c_size_t
    lib.qk_moe_route.argtypes = [vp, i64, i64, i64, i64, ci, vp, i64, i64, i64, ci, ctypes.c_float,
                                 vp, i64, vp, i64, vp]
    lib.qk_moe_route.restype = ci
    _lib = lib
    return lib


def status_string(status):
    return load().qk_status_string(int(status)).decode()


def block_bytes(fmt):
    return load().qk_block_bytes(_fmt(fmt))


def row_bytes(fmt, k):
    return load().qk_row_bytes(_fmt(fmt), int(k))


def _fmt(fmt):
    if isinstance(fmt, str):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}")
        return FORMATS[fmt]
    return int(fmt)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(stream) if not hasattr(stream, "cuda_stream") else stream.cuda_stream


def _check(status, call):
    if status != QK_OK:
        raise QKError(status, call)


# ---------------------------------------------------------------------------
# Raw entry points (pointers and sizes, same names and argument order as C)
# ---------------------------------------------------------------------------

def qk_dequantize(fmt, w_ptr, rows, k, out_dtype, out_ptr, stream=0):
    return load().qk_dequantize(_fmt(fmt), w_ptr, rows, k, out_dtype, out_ptr, stream)


def qk_mul_mat_vec(fmt, w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream=0):
    return load().qk_mul_mat_vec(_fmt(fmt), w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream)


def qk_mul_mat_vec_x8(fmt, w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream=0):
    return load().qk_mul_mat_vec_x8(_fmt(fmt), w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream)


def make_items(items):
    """ctypes array of MatVecItem from (w_ptr, m, k, x_ptr, ldx, y_ptr, ldy) tuples."""
    arr = (MatVecItem * max(len(items), 1))()
    for i, it in enumerate(items):
        arr[i] = MatVecItem(*it)
    return arr


def qk_mul_mat_vec_batched(fmt, items, count, n, stream=0):
    """items: a ctypes MatVecItem array (see make_items) or None."""
    return load().qk_mul_mat_vec_batched(_fmt(fmt), items, count, n, stream)


def qk_mul_mat_vec_id(fmt, w_ptr, n_experts, expert_stride, m, k, ids_ptr, ld_ids, n_used,
                      n_tokens, x_ptr, x_slot, x_tok, y_ptr, y_slot, y_tok, stream=0):
    return load().qk_mul_mat_vec_id(_fmt(fmt), w_ptr, n_experts, expert_stride, m, k, ids_ptr,
                                    ld_ids, n_used, n_tokens, x_ptr, x_slot, x_tok, y_ptr,
                                    y_slot, y_tok, stream)


def qk_mul_mat(fmt, w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream=0):
    return load().qk_mul_mat(_fmt(fmt), w_ptr, m, k, x_ptr, n, ldx, y_ptr, ldy, stream)


def qk_mul_mat_vec_x8q(fmt, w_ptr, m, k, xq_ptr, n, ldx, y_ptr, ldy, stream=0):
    return load().qk_mul_mat_vec_x8q(_fmt(fmt), w_ptr, m, k, xq_ptr, n, ldx, y_ptr, ldy, stream)


def qk_rms_norm(x_dtype, x_ptr, ldx, residual_ptr, ldr, weight_ptr, eps, n, k, sum_ptr, lds, y_dtype, y_ptr,
                ldy, stream=0):
    return load().qk_rms_norm(x_dtype, x_ptr, ldx, residual_ptr, ldr, weight_ptr, eps, n, k, sum_ptr, lds,
                              y_dtype, y_ptr, ldy, stream)


def qk_kv_store(cache, k_ptr, k_tok, k_head, v_ptr, v_tok, v_head, n_tokens, table_ptr, ld_table, n_seqs,
                max_pages, seq_ptr, pos_ptr, stream=0):
    """cache: a KVCacheDesc or None."""
    return load().qk_kv_store(cache, k_ptr, k_tok, k_head, v_ptr, v_tok, v_head, n_tokens, table_ptr, ld_table,
                              n_seqs, max_pages, seq_ptr, pos_ptr, stream)


def qk_attn_decode(cache, q_ptr, q_seq, q_head, n_seqs, n_q_heads, table_ptr, ld_table, lens_ptr, max_len, scale,
                   window, sinks, y_dtype, y_ptr, y_seq, y_head, workspace_ptr, workspace_bytes, stream=0):
    """cache: a KVCacheDesc or None."""
    return load().qk_attn_decode(cache, q_ptr, q_seq, q_head, n_seqs, n_q_heads, table_ptr, ld_table, lens_ptr,
                                 max_len, scale, window, sinks, y_dtype, y_ptr, y_seq, y_head, workspace_ptr,
                                 workspace_bytes, stream)


def qk_attn_decode_workspace(cache, n_seqs, n_q_heads, max_len, window=0, sinks=0):
    return load().qk_attn_decode_workspace(cache, n_seqs, n_q_heads, max_len, window, sinks)


def qk_moe_route(logits_ptr, ldx, n_tokens, n_experts, n_used, score, bias_ptr, n_groups, topk_groups, group_top,
                 renorm, scale, ids_ptr, ld_ids, weights_ptr, ldw, stream=0):
    return load().qk_moe_route(logits_ptr, ldx, n_tokens, n_experts, n_used, score, bias_ptr, n_groups,
                               topk_groups, group_top, renorm, scale, ids_ptr, ld_ids, weights_ptr, ldw, stream)


# ---------------------------------------------------------------------------
# torch-tensor conveniences (allocation by torch, compute by libqk)
#
# The C ABI sees only pointers, so these wrappers check every tensor on the
# host before anything is launched: dtype, shape, a contiguous innermost
# dimension, enough weight bytes, one CUDA device for all operands.  A
# mismatch raises TypeError or ValueError and enqueues nothing.
# ---------------------------------------------------------------------------

_BLOCK_BYTES = {QK_Q4_0: 18, QK_Q4_1: 20, QK_Q8_0: 34, QK_Q5_0: 22, QK_Q5_1: 24}


def _weight_check(fmt, w, rows, k):
    import torch
    code = _fmt(fmt)
    if code not in _BLOCK_BYTES:
        raise ValueError(f"unknown format {fmt!r}")
    if rows < 0 or k < 0 or k % 32 != 0:
        raise ValueError(f"bad shape rows={rows}, k={k} (k must be a non-negative multiple of 32)")
    if not isinstance(w, torch.Tensor) or w.dtype != torch.uint8:
        raise TypeError("w must be a uint8 tensor of block bytes")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    need = rows * (k // 32) * _BLOCK_BYTES[code]
    if w.numel() < need:
        raise ValueError(f"w holds {w.numel()} bytes, a {rows} x {k} matrix needs {need}")


def _cols_check(t, name, dtype, n, length):
    """t is (n, >= length) of dtype with contiguous rows (ggml columns)."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.dim() != 2 or t.shape[0] != n or t.shape[1] < length:
        raise ValueError(f"{name} must have shape ({n}, >= {length}), got {tuple(t.shape)}")
    if n > 0 and length > 0 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous columns (stride(1) == 1)")


def _same_device(*ts):
    dev = ts[0].device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")


def _on_stream(stream, t, call, *args):
    """call(*args) with the caller's stream as the current one of t's device.
    What a call allocates then comes from the pool of the stream that it runs
    on; a block of another stream's pool may be in use there still."""
    import torch
    device = t.get_device() if isinstance(t, torch.Tensor) else -1
    handle = _stream(stream)
    if device < 0 or handle == torch._C._cuda_getCurrentRawStream(device):
        return call(*args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    elif stream.device_index != device:
        raise ValueError(f"stream of device {stream.device_index}, tensors on device {device}")
    with torch.cuda.stream(stream):
        return call(*args)


def dequantize(fmt, w, rows, k, out_dtype="f32", out=None, stream=None):
    """Dequantize a rows x k matrix held as block bytes in a uint8 CUDA tensor."""
    import torch
    if stream is not None:
        return _on_stream(stream, w, dequantize, fmt, w, rows, k, out_dtype, out)
    if out_dtype not in ("f32", "f16"):
        raise ValueError(f"out_dtype must be 'f32' or 'f16', got {out_dtype!r}")
    dt = {"f32": (QK_F32, torch.float32), "f16": (QK_F16, torch.float16)}[out_dtype]
    _weight_check(fmt, w, rows, k)
    if out is None:
        out = torch.empty((rows, k), dtype=dt[1], device=w.device)
    if not isinstance(out, torch.Tensor) or out.dtype != dt[1]:
        raise TypeError(f"out must be a {dt[1]} tensor for out_dtype {out_dtype!r}")
    if tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous ({rows}, {k}) tensor")
    _same_device(w, out)
    st = qk_dequantize(fmt, w.data_ptr(), rows, k, dt[0], out.data_ptr(), _stream(None))
    _check(st, "qk_dequantize")
    return out


def _gemv_args(fmt, w, m, k, x, y):
    import torch
    if x.dim() == 1:
        x = x.view(1, -1)
    n = x.shape[0]
    if not 1 <= n <= 8:
        raise ValueError(f"1..8 activation columns, got {n}")
    _weight_check(fmt, w, m, k)
    _cols_check(x, "x", torch.float32, n, k)
    if y is None:
        y = torch.empty((n, m), dtype=torch.float32, device=x.device)
    _cols_check(y, "y", torch.float32, n, m)
    _same_device(w, x, y)
    return x, y, n


def mul_mat_vec(fmt, w, m, k, x, y=None, stream=None):
    """y (n, m) = x (n, k) @ W^T for 1..8 fp32 columns; rows of x and y are the
    ggml columns (contiguous, ldx = x.stride(0), ldy = y.stride(0))."""
    if stream is not None:
        return _on_stream(stream, x, mul_mat_vec, fmt, w, m, k, x, y)
    x, y, n = _gemv_args(fmt, w, m, k, x, y)
    st = qk_mul_mat_vec(fmt, w.data_ptr(), m, k, x.data_ptr(), n, x.stride(0),
                        y.data_ptr(), y.stride(0), _stream(None))
    _check(st, "qk_mul_mat_vec")
    return y


def mul_mat_vec_x8(fmt, w, m, k, x, y=None, stream=None):
    """As mul_mat_vec, with the activations quantized to 8 bits per 32-element
    block inside the kernel and integer dot products (qk_mul_mat_vec_x8)."""
    if stream is not None:
        return _on_stream(stream, x, mul_mat_vec_x8, fmt, w, m, k, x, y)
    x, y, n = _gemv_args(fmt, w, m, k, x, y)
    st = qk_mul_mat_vec_x8(fmt, w.data_ptr(), m, k, x.data_ptr(), n, x.stride(0),
                           y.data_ptr(), y.stride(0), _stream(None))
    _check(st, "qk_mul_mat_vec_x8")
    return y


def mul_mat_vec_batched(fmt, problems, ys=None, stream=None):
    """One launch for several GEMVs of one format and column count.
    problems: list of (w, m, k, x) with x shaped (n, k) fp32; returns the ys."""
    import torch
    if not problems:
        return []
    if stream is not None:
        return _on_stream(stream, problems[0][0], mul_mat_vec_batched, fmt, problems, ys)
    if len(problems) > QK_MAX_BATCH:
        raise ValueError(f"at most {QK_MAX_BATCH} problems per launch")
    n = problems[0][3].shape[0] if problems[0][3].dim() == 2 else 1
    if ys is None:
        ys = [torch.empty((n, m), dtype=torch.float32, device=x.device) for (_, m, _, x) in problems]
    if len(ys) != len(problems):
        raise ValueError("one output per problem")
    tup = []
    for (w, m, k, x), y in zip(problems, ys):
        x2 = x.view(1, -1) if x.dim() == 1 else x
        if x2.shape[0] != n:
            raise ValueError("every x must have the same number of columns")
        x2, y, _ = _gemv_args(fmt, w, m, k, x2, y)
        _same_device(problems[0][0], w)
        tup.append((w.data_ptr(), m, k, x2.data_ptr(), x2.stride(0), y.data_ptr(), y.stride(0)))
    arr = make_items(tup)
    st = qk_mul_mat_vec_batched(fmt, arr, len(tup), n, _stream(None))
    _check(st, "qk_mul_mat_vec_batched")
    return ys


def mul_mat_vec_id(fmt, w, n_experts, m, k, ids, x, y=None, expert_stride=None, stream=None):
    """Expert-indexed GEMV: y[t, s] = W[ids[t, s]] @ x[t] (x shaped (n_tokens, k),
    shared by a token's slots) or x[t, s] (x shaped (n_tokens, n_used, k)).
    w: uint8 CUDA tensor holding n_experts matrices, expert_stride bytes apart
    (default: packed); ids: int32 CUDA tensor (n_tokens, n_used).  Returns y
    shaped (n_tokens, n_used, m) fp32."""
    import torch
    if stream is not None:
        return _on_stream(stream, x, mul_mat_vec_id, fmt, w, n_experts, m, k, ids, x, y, expert_stride)
    if not isinstance(ids, torch.Tensor) or ids.dtype != torch.int32 or ids.dim() != 2 or ids.stride(1) != 1:
        raise TypeError("ids must be int32 (n_tokens, n_used) with contiguous rows")
    n_tokens, n_used = ids.shape
    if not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or x.stride(-1) != 1:
        raise TypeError("x must be float32 with contiguous vectors")
    if x.dim() == 2 and x.shape[0] == n_tokens and x.shape[1] >= k:
        x_slot, x_tok = 0, x.stride(0)
    elif x.dim() == 3 and tuple(x.shape[:2]) == (n_tokens, n_used) and x.shape[2] >= k:
        x_slot, x_tok = x.stride(1), x.stride(0)
    else:
        raise ValueError(f"x must be ({n_tokens}, >= {k}) or ({n_tokens}, {n_used}, >= {k}), "
                         f"got {tuple(x.shape)}")
    one = m * (k // 32) * _BLOCK_BYTES.get(_fmt(fmt), 0)
    if expert_stride is None:
        expert_stride = one
    if n_experts < 1 or expert_stride < one:
        raise ValueError("n_experts >= 1 and expert_stride >= one expert matrix")
    _weight_check(fmt, w, m, k)
    if w.numel() < (n_experts - 1) * expert_stride + one:
        raise ValueError(f"w holds {w.numel()} bytes, the stack needs {(n_experts - 1) * expert_stride + one}")
    if y is None:
        y = torch.empty((n_tokens, n_used, m), dtype=torch.float32, device=x.device)
    if not isinstance(y, torch.Tensor) or y.dtype != torch.float32:
        raise TypeError("y must be a float32 tensor")
    if tuple(y.shape) != (n_tokens, n_used, m) or (m > 0 and y.stride(2) != 1):
        raise ValueError(f"y must have shape ({n_tokens}, {n_used}, {m}) with contiguous rows")
    _same_device(w, ids, x, y)
    st = qk_mul_mat_vec_id(fmt, w.data_ptr(), n_experts, expert_stride, m, k, ids.data_ptr(),
                           ids.stride(0), n_used, n_tokens, x.data_ptr(), x_slot, x_tok,
                           y.data_ptr(), y.stride(1), y.stride(0), _stream(None))
    _check(st, "qk_mul_mat_vec_id")
    return y


def mul_mat(fmt, w, m, k, x, y=None, stream=None):
    """y (n, m) = x (n, k, fp16) @ f16(W)^T on the matrix cores."""
    import torch
    if stream is not None:
        return _on_stream(stream, x, mul_mat, fmt, w, m, k, x, y)
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a 2-D float16 tensor (n, k)")
    n = x.shape[0]
    _weight_check(fmt, w, m, k)
    _cols_check(x, "x", torch.float16, n, k)
    if y is None:
        y = torch.empty((n, m), dtype=torch.float32, device=x.device)
    _cols_check(y, "y", torch.float32, n, m)
    _same_device(w, x, y)
    st = qk_mul_mat(fmt, w.data_ptr(), m, k, x.data_ptr(), n, x.stride(0),
                    y.data_ptr(), y.stride(0), _stream(None))
    _check(st, "qk_mul_mat")
    return y


# The calls below run between the products of a decode step, where the time to
# make them counts: the checks that a well-formed call passes are a few
# attribute reads, and what refuses is left to the slower helpers above.

def _stream_of(t, stream=None):
    """Handle of the caller's stream, or of the current one on t's device."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return _stream(stream)


def _on_device(*ts):
    """_same_device, over tensors of which some may be None."""
    d = ts[0].get_device()
    for t in ts:
        if t is not None and (d < 0 or t.get_device() != d):
            _same_device(*[u for u in ts if u is not None])


def _rows_check(t, name, dtype, n, length):
    """_cols_check, quick where t is as it should be; the stride of its rows."""
    import torch
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == (n, length) and t.is_contiguous():
        return length
    _cols_check(t, name, dtype, n, length)
    return t.stride(0)


def _vec_check(t, name, n):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous ({n},) tensor, got {tuple(t.shape)}")


def mul_mat_vec_x8q(fmt, w, m, k, xq, y=None, stream=None):
    """As mul_mat_vec_x8, over activations in 8 bits already: xq (n, >= k/32*36)
    uint8, rows of 36-byte blocks as rms_norm(..., out_dtype="x8") gives them."""
    import torch
    if stream is not None:
        return _on_stream(stream, xq, mul_mat_vec_x8q, fmt, w, m, k, xq, y)
    _weight_check(fmt, w, m, k)
    if not isinstance(xq, torch.Tensor) or xq.dtype is not torch.uint8:
        raise TypeError("xq must be a uint8 tensor of 8-bit activation blocks")
    if xq.dim() == 1:
        xq = xq.view(1, -1)
    n = xq.shape[0]
    if not 1 <= n <= 8:
        raise ValueError(f"1..8 activation columns, got {n}")
    ldx = _rows_check(xq, "xq", torch.uint8, n, k // 32 * X8_BLOCK_BYTES)
    if y is None:
        y, ldy = xq.new_empty((n, m), dtype=torch.float32), m
    else:
        ldy = _rows_check(y, "y", torch.float32, n, m)
    _on_device(w, xq, y)
    st = load().qk_mul_mat_vec_x8q(_fmt(fmt), w.data_ptr(), m, k, xq.data_ptr(), n, ldx, y.data_ptr(), ldy,
                                   _stream_of(xq))
    _check(st, "qk_mul_mat_vec_x8q")
    return y


def _row_stride(t):
    """Stride of a tensor's first dimension, 0 where it has no second row."""
    return t.stride(0) if t.shape[0] > 1 else 0


_NORM_OUT = {"f32": QK_F32, "f16": QK_F16, "x8": QK_X8}


def rms_norm(x, weight=None, eps=1e-5, residual=None, out_dtype="f32", y=None, residual_out=None, stream=None):
    """Root-mean-square norm of the rows of x (n, k), fp32 or fp16, after
    adding `residual` (as x): returns y, or (y, x + residual) with a residual.
    out_dtype "f32", "f16", or "x8" (y uint8 (n, k/32*36), 8-bit activation
    blocks for mul_mat_vec_x8q).  residual_out may be x or residual itself."""
    import torch
    if stream is not None:
        return _on_stream(stream, x, rms_norm, x, weight, eps, residual, out_dtype, y, residual_out)
    dtype = x.dtype if isinstance(x, torch.Tensor) else None
    if dtype is torch.float32:
        code = QK_F32
    elif dtype is torch.float16:
        code = QK_F16
    else:
        raise TypeError("x must be a float32 or float16 tensor")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"x must have shape (n, k) with k >= 1, got {tuple(x.shape)}")
    ycode = _NORM_OUT.get(out_dtype)
    if ycode is None:
        raise ValueError(f"out_dtype must be 'f32', 'f16' or 'x8', got {out_dtype!r}")
    n, k = x.shape
    if ycode == QK_X8:
        if k % 32 != 0:
            raise ValueError(f"k must be a multiple of 32 for out_dtype 'x8', got {k}")
        ydtype, row = torch.uint8, k // 32 * X8_BLOCK_BYTES
    else:
        ydtype, row = torch.float32 if ycode == QK_F32 else torch.float16, k
    ldx = _rows_check(x, "x", dtype, n, k)
    r, ldr, s, lds = None, 0, None, 0
    if residual is not None:
        ldr = _rows_check(residual, "residual", dtype, n, k)
        if residual_out is None:
            # (empty_like is the quicker call; of whole rows it gives whole rows)
            residual_out, lds = torch.empty_like(residual) if ldr == k else x.new_empty((n, k)), k
        else:
            lds = _rows_check(residual_out, "residual_out", dtype, n, k)
        r, s = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    if weight is not None:
        _vec_check(weight, "weight", k)
    if y is None:
        y = torch.empty_like(x) if ydtype is dtype and ldx == k else x.new_empty((n, row), dtype=ydtype)
        ldy = row
    else:
        ldy = _rows_check(y, "y", ydtype, n, row)
    _on_device(x, y, residual, residual_out, weight)
    st = load().qk_rms_norm(code, x.data_ptr(), ldx, r, ldr, weight.data_ptr() if weight is not None else None,
                            eps, n, k, s, lds, ycode, y.data_ptr(), ldy, _stream_of(x))
    _check(st, "qk_rms_norm")
    return y if residual is None else (y, residual_out)


class KVCache:
    """A paged key-value cache over tensors that the caller keeps.

    k, v: (n_pages, n_kv_heads, page_size, head_dim), float16, or int8 with
    k_scale, v_scale float32 (n_pages, n_kv_heads, page_size): an element is
    code * scale.  Any strides with contiguous rows, the same for k and v
    (tokens outside heads: pass a view transposed to this order)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor) or k.dtype != v.dtype \
                or k.dtype not in (torch.float16, torch.int8):
            raise TypeError("k and v must be float16 or int8 tensors")
        if k.dim() != 4 or k.shape != v.shape or min(k.shape) < 1:
            raise ValueError("k and v must both be (n_pages, n_kv_heads, page_size, head_dim), "
                             f"got {tuple(k.shape)} and {tuple(v.shape)}")
        i8 = k.dtype == torch.int8
        pages, heads, page, dim = k.shape
        if dim % 32 != 0 or dim > 256:
            raise ValueError(f"head_dim must be a multiple of 32 up to 256, got {dim}")

        def strides(t, n):
            return [t.stride(i) if t.shape[i] > 1 else 0 for i in range(n)]

        if k.stride(3) != 1 or v.stride(3) != 1 or strides(k, 3) != strides(v, 3):
            raise ValueError("k and v must have contiguous rows and the same strides")
        if any(s * k.element_size() % 16 for s in strides(k, 3)) or k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("rows of k and v must begin at multiples of 16 bytes")
        if i8 != (k_scale is not None) or i8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to int8 caches, and only to them")
        sc = [0, 0, 0]
        if i8:
            for t in (k_scale, v_scale):
                if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
                    raise TypeError("k_scale and v_scale must be float32 tensors")
                if tuple(t.shape) != (pages, heads, page):
                    raise ValueError(f"k_scale and v_scale must be ({pages}, {heads}, {page}), got {tuple(t.shape)}")
            sc = strides(k_scale, 3)
            if strides(v_scale, 3) != sc:
                raise ValueError("k_scale and v_scale must have the same strides")
        _same_device(k, v, *([k_scale, v_scale] if i8 else []))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.device = k.device
        self.desc = KVCacheDesc(QK_KV_I8 if i8 else QK_KV_F16, k.data_ptr(), v.data_ptr(),
                                k_scale.data_ptr() if i8 else None, v_scale.data_ptr() if i8 else None,
                                pages, heads, page, dim, *strides(k, 3), *sc)

    @classmethod
    def empty(cls, n_pages, n_heads, page_size, head_dim, dtype="f16", device="cuda"):
        """A cache of its own tensors; dtype "f16" or "i8"."""
        import torch
        if dtype not in ("f16", "i8"):
            raise ValueError(f"dtype must be 'f16' or 'i8', got {dtype!r}")
        shape = (n_pages, n_heads, page_size, head_dim)
        kv = [torch.zeros(shape, dtype=torch.float16 if dtype == "f16" else torch.int8, device=device)
              for _ in range(2)]
        if dtype == "i8":
            kv += [torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*kv)


def _int32_check(t, name, dim):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if t.dim() != dim or (not t.is_contiguous() and t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be {dim}-dimensional with contiguous rows, got {tuple(t.shape)}")


def _heads_check(t, name, dtype, n, heads, dim):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != (n, heads, dim) or (not t.is_contiguous() and t.stride(2) != 1):
        raise ValueError(f"{name} must have shape ({n}, {heads}, {dim}) with contiguous rows, got {tuple(t.shape)}")


def kv_store(cache, k, v, table, pos, seq=None, stream=None):
    """Write new keys and values into a paged cache: token i of k and v
    (n_tokens, n_kv_heads, head_dim) fp32 goes to position pos[i] of sequence
    seq[i] (i itself without seq), whose pages are table[seq[i]].  table int32
    (n_seqs, max_pages); pos, seq int32 (n_tokens,).  A token with no place in
    the table or the pool is left out."""
    import torch
    _int32_check(table, "table", 2)
    _int32_check(pos, "pos", 1)
    n = pos.shape[0]
    if seq is not None:
        _int32_check(seq, "seq", 1)
        if seq.shape[0] != n:
            raise ValueError(f"seq has {seq.shape[0]} tokens, pos {n}")
    elif table.shape[0] < n:
        raise ValueError(f"table has {table.shape[0]} sequences for {n} tokens")
    for t, name in ((k, "k"), (v, "v")):
        _heads_check(t, name, torch.float32, n, cache.n_heads, cache.head_dim)
    _on_device(cache.k, k, v, table, pos, seq)
    st = load().qk_kv_store(cache.desc, k.data_ptr(), _row_stride(k), k.stride(1) if cache.n_heads > 1 else 0,
                            v.data_ptr(), _row_stride(v), v.stride(1) if cache.n_heads > 1 else 0,
                            n, table.data_ptr(), table.stride(0), table.shape[0], table.shape[1],
                            seq.data_ptr() if seq is not None else None, pos.data_ptr(), _stream_of(pos, stream))
    _check(st, "qk_kv_store")


def attn_decode_workspace(cache, n_seqs, n_q_heads, max_len, window=0, sinks=0):
    """Scratch for attn_decode calls of up to these sizes (n_seqs, max_len, and a
    window and sinks where they are given): a uint8 tensor, or None where none
    is needed.  One tensor serves one stream at a time."""
    import torch
    need = qk_attn_decode_workspace(cache.desc, n_seqs, n_q_heads, max_len, window, sinks)
    return torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None


def attn_decode(cache, q, table, lens, scale=None, window=0, sinks=0, max_len=None, out_dtype="f32", y=None,
                workspace=None, stream=None):
    """Attention of one new token per sequence over a paged cache.  q (n_seqs,
    n_q_heads, head_dim) fp32; table int32 (n_seqs, max_pages); lens int32
    (n_seqs,), the new token counted.  scale: 1/sqrt(head_dim) unless given.
    window > 0: the last `window` tokens and the first `sinks` are seen.
    max_len bounds the lengths (default: all of the table's pages) and sizes
    the split over the cache; a length above it gives NaN.  Returns y (n_seqs,
    n_q_heads, head_dim), fp32 or (out_dtype "f16") fp16."""
    import torch
    if stream is not None:
        return _on_stream(stream, q, attn_decode, cache, q, table, lens, scale, window, sinks, max_len, out_dtype, y,
                          workspace)
    if out_dtype == "f32":
        code, dt = QK_F32, torch.float32
    elif out_dtype == "f16":
        code, dt = QK_F16, torch.float16
    else:
        raise ValueError(f"out_dtype must be 'f32' or 'f16', got {out_dtype!r}")
    _int32_check(table, "table", 2)
    _int32_check(lens, "lens", 1)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a float32 tensor (n_seqs, n_q_heads, head_dim)")
    n, heads, dim = q.shape[0], q.shape[1], cache.head_dim
    _heads_check(q, "q", torch.float32, n, heads, dim)
    if heads < 1 or heads % cache.n_heads != 0:
        raise ValueError(f"{heads} query heads over {cache.n_heads} key-value heads")
    if table.shape[0] != n or lens.shape[0] != n:
        raise ValueError(f"q has {n} sequences, table {table.shape[0]}, lens {lens.shape[0]}")
    room = table.shape[1] * cache.page_size
    max_len = room if max_len is None else int(max_len)
    if not 1 <= max_len <= room:
        raise ValueError(f"max_len {max_len}: the table has room for {room} tokens")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    if y is None:
        y = q.new_empty((n, heads, dim), dtype=dt)
    else:
        _heads_check(y, "y", dt, n, heads, dim)
    _on_device(cache.k, q, table, lens, y, workspace)
    if workspace is None:
        need = qk_attn_decode_workspace(cache.desc, n, heads, max_len, window, sinks)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    q_head, y_head = (q.stride(1), y.stride(1)) if heads > 1 else (0, 0)
    st = load().qk_attn_decode(cache.desc, q.data_ptr(), _row_stride(q), q_head, n, heads, table.data_ptr(),
                               table.stride(0), lens.data_ptr(), max_len, dim ** -0.5 if scale is None else scale,
                               window, sinks, code, y.data_ptr(), _row_stride(y), y_head,
                               workspace.data_ptr() if workspace is not None else None,
                               workspace.numel() if workspace is not None else 0, _stream_of(q))
    _check(st, "qk_attn_decode")
    return y


_SCORES = {"softmax": QK_SOFTMAX, "sigmoid": QK_SIGMOID}


def moe_route(logits, n_used, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=True,
              scale=1.0, ids=None, weights=None, stream=None):
    """Choose n_used experts for each token from logits (n_tokens, n_experts)
    fp32: (ids int32, weights fp32), both (n_tokens, n_used), the ids as
    mul_mat_vec_id takes them.  score "softmax" or "sigmoid"; bias
    (n_experts,) fp32 is added for the choice only; with n_groups > 1 only the
    topk_groups best groups of neighbouring experts take part, by the sum of
    their group_top (1 or 2) largest values."""
    import torch
    if stream is not None:
        return _on_stream(stream, logits, moe_route, logits, n_used, score, bias, n_groups, topk_groups, group_top,
                          renorm, scale, ids, weights)
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    if not isinstance(logits, torch.Tensor) or logits.dtype is not torch.float32:
        raise TypeError("logits must be a float32 tensor")
    if logits.dim() != 2 or (not logits.is_contiguous() and logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be (n_tokens, n_experts) with contiguous rows, got {tuple(logits.shape)}")
    n, experts = logits.shape
    if bias is not None:
        _vec_check(bias, "bias", experts)
    if not 1 <= n_used <= 64:
        raise ValueError(f"n_used must be 1..64, got {n_used}")
    if ids is None:
        ids, ld_ids = logits.new_empty((n, n_used), dtype=torch.int32), n_used
    else:
        ld_ids = _rows_check(ids, "ids", torch.int32, n, n_used)
    if weights is None:
        weights, ldw = logits.new_empty((n, n_used)), n_used
    else:
        ldw = _rows_check(weights, "weights", torch.float32, n, n_used)
    _on_device(logits, ids, weights, bias)
    st = load().qk_moe_route(logits.data_ptr(), logits.stride(0), n, experts, n_used, code,
                             bias.data_ptr() if bias is not None else None, n_groups, topk_groups, group_top,
                             1 if renorm else 0, scale, ids.data_ptr(), ld_ids, weights.data_ptr(), ldw,
                             _stream_of(logits))
    _check(st, "qk_moe_route")
    return ids, weights
