"""Thin Python binding of libhdq (C ABI in include/hdq.h).

Argument marshalling only: torch provides device memory and the current
stream; every step of the path runs in libhdq's HIP kernels.  The names
follow the C entry points: select_precision, quantize, linear.  Importing
this module loads libhdq.so and raises if it is missing (build it with
__graft_entry__.build() or `python bit_quantized_video_amd/build.py`); there
is no CPU fallback.
"""
import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhdq.so")

# status codes
OK, ERR_INVALID, ERR_SHAPE, ERR_UNSUPPORTED, ERR_HIP, ERR_WORKSPACE, ERR_TOO_LARGE = 0, -1, -2, -3, -4, -5, -6
NOALLOC_SCRATCH_BYTES = 2 << 20      # HDQ_NOALLOC_SCRATCH_BYTES
# formats
FMT_INT8_ROW, FMT_INT4_ROW, FMT_NVFP4, FMT_NVFP4_MX, FMT_NVFP4_P2 = 0, 1, 2, 3, 4
# precisions
PREC_NVFP4, PREC_INT8, PREC_BF16 = 0, 1, 2
# output dtypes
DTYPE_F32, DTYPE_BF16, DTYPE_I32 = 0, 1, 2
# workspace ops
OP_SELECT, OP_QUANTIZE, OP_LINEAR, OP_SELECT_Q8, OP_DQ_QUANTIZE, OP_DQ_LINEAR = 0, 1, 2, 3, 4, 5
# FP8 scale layouts: per 128 elements of a row, per 128 x 128 block
FP8_ROWS, FP8_BLOCKS = 0, 1
FP8_BLOCK = 128
FP8_MAX_COLS, FP8_MAX_ROWS = 1 << 22, 0x7ffffc00   # HDQ_FP8_MAX_*
# activations of the group norms
ACT_NONE, ACT_SILU = 0, 1
GROUP_NORM_MAX_CHANNELS = 8192   # HDQ_GROUP_NORM_MAX_CHANNELS
# buffers of 4-bit weights
W4_CODES, W4_SCALE, W4_ZERO = 0, 1, 2
W4_MAX_ROWS, W4_MAX_TOKENS = 1 << 27, 1 << 20   # HDQ_W4_MAX_*
# head norms, rotary layouts and frequency scalings, cache formats
HEAD_MAX_DIM, HEAD_MAX_HEADS = 512, 1 << 20   # HDQ_HEAD_MAX_*
HEAD_NORM_NONE, HEAD_NORM_LAYER, HEAD_NORM_RMS = 0, 1, 2
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_MAX_AXES = 3
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_RAMP = 0, 1, 2, 3
CACHE_INT8, CACHE_FP8, CACHE_INT4 = 0, 1, 2

EXPORTS = ("hdq_select_precision", "hdq_delta_sums", "hdq_select_precision_sums",
           "hdq_select_quantize_int8", "hdq_select_quantize_int8_noalloc", "hdq_linear_dispatch", "hdq_linear_dispatch_delta",
           "hdq_tdc_decide", "hdq_quantize", "hdq_dq_cubes", "hdq_dq_quantize", "hdq_dq_decode_weights",
           "hdq_dq_linear", "hdq_dq_linear_workspace_bytes",
           "hdq_fp8_quantize", "hdq_fp8_linear_workspace_bytes", "hdq_fp8_linear",
           "hdq_group_norm_workspace_bytes", "hdq_group_norm", "hdq_group_norm_fp8",
           "hdq_w4_bytes", "hdq_w4_pack", "hdq_w4_quantize", "hdq_w4_linear",
           "hdq_w4_linear_workspace_bytes",
           "hdq_rope_turns", "hdq_qk_norm_rope", "hdq_qkv_to_cache", "hdq_cache_read",
           "hdq_linear", "hdq_workspace_bytes",
           "hdq_status_string", "hdq_version")

_c = ctypes
_p = _c.c_void_p


class QTensorDesc(_c.Structure):
    """hdq_qtensor."""
    _fields_ = [("fmt", _c.c_int32), ("had_block", _c.c_int32), ("rows", _c.c_int64),
                ("cols", _c.c_int64), ("codes", _p), ("row_scale", _p), ("blk_scale", _p),
                ("tensor_scale", _p), ("dec", _p)]


class DeltaSlice(_c.Structure):
    """hdq_delta_slice."""
    _fields_ = [("prev_in", _p), ("prev_out", _p), ("numel", _c.c_int64), ("chunk_begin", _c.c_int64),
                ("chunk_end", _c.c_int64), ("partials", _p)]


DELTA_CHUNK = 65536       # HDQ_DELTA_CHUNK
DELTA_MAX_SLICES = 4      # HDQ_DELTA_MAX_SLICES


def delta_chunks(numel):
    """Chunks (and partial pairs) of a module's difference statistic."""
    return (numel + DELTA_CHUNK - 1) // DELTA_CHUNK


class DqGridDesc(_c.Structure):
    """hdq_dq_grid."""
    _fields_ = [("frames", _c.c_int64), ("height", _c.c_int64), ("width", _c.c_int64),
                ("cube_f", _c.c_int32), ("cube_h", _c.c_int32), ("cube_w", _c.c_int32)]


class Fp8TensorDesc(_c.Structure):
    """hdq_fp8_tensor."""
    _fields_ = [("layout", _c.c_int32), ("had_block", _c.c_int32), ("rows", _c.c_int64), ("cols", _c.c_int64),
                ("codes", _p), ("scale", _p)]


class W4TensorDesc(_c.Structure):
    """hdq_w4_tensor."""
    _fields_ = [("N", _c.c_int64), ("K", _c.c_int64), ("group", _c.c_int32), ("codes", _p), ("scale", _p), ("zero", _p)]


class HeadsDesc(_c.Structure):
    """hdq_heads."""
    _fields_ = [("data", _p), ("dtype", _c.c_int32), ("heads", _c.c_int32), ("batch_stride", _c.c_int64),
                ("token_stride", _c.c_int64), ("head_stride", _c.c_int64)]


class HeadNormDesc(_c.Structure):
    """hdq_head_norm."""
    _fields_ = [("kind", _c.c_int32), ("eps", _c.c_float), ("q_weight", _p), ("q_bias", _p), ("k_weight", _p),
                ("k_bias", _p)]


class RopeDesc(_c.Structure):
    """hdq_rope."""
    _fields_ = [("layout", _c.c_int32), ("dim", _c.c_int32), ("axes", _c.c_int32), ("axis_dim", _c.c_int32 * 3),
                ("scale", _c.c_float), ("turns", _p), ("positions", _p), ("pos_axis_stride", _c.c_int64),
                ("pos_batch_stride", _c.c_int64), ("pos_token_stride", _c.c_int64)]


class KvCacheDesc(_c.Structure):
    """hdq_kv_cache."""
    _fields_ = [("fmt", _c.c_int32), ("group", _c.c_int32), ("had_block", _c.c_int32), ("heads", _c.c_int32),
                ("dim", _c.c_int32), ("slots", _c.c_int64), ("k_codes", _p), ("k_scale", _p), ("v_codes", _p),
                ("v_scale", _p)]


class WeightsDesc(_c.Structure):
    """hdq_weights."""
    _fields_ = [("N", _c.c_int64), ("K", _c.c_int64), ("w_bf16", _p), ("w_int4", QTensorDesc),
                ("w_fp4", QTensorDesc)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libhdq.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = _c.CDLL(LIB_PATH)
    L.hdq_select_precision.restype = _c.c_int
    L.hdq_select_precision.argtypes = [_p, _p, _c.c_int64, _p, _c.c_int64, _c.c_int64, _c.c_int32,
                                       _c.c_float, _c.c_float, _p, _p, _p, _c.c_size_t, _p]
    L.hdq_delta_sums.restype = _c.c_int
    L.hdq_delta_sums.argtypes = [_p, _p, _c.c_int64, _p, _p, _c.c_size_t, _p]
    L.hdq_select_precision_sums.restype = _c.c_int
    L.hdq_select_precision_sums.argtypes = [_p, _c.c_int64, _p, _c.c_int64, _c.c_int64, _c.c_int32,
                                            _c.c_float, _c.c_float, _p, _p, _p, _c.c_size_t, _p]
    L.hdq_select_quantize_int8.restype = _c.c_int
    L.hdq_select_quantize_int8.argtypes = [_p, _c.c_int64, _p, _c.c_int64, _c.c_int64, _c.c_int32,
                                           _c.c_float, _c.c_float, _p, _p, _c.POINTER(QTensorDesc), _p,
                                           _c.c_size_t, _p]
    L.hdq_select_quantize_int8_noalloc.restype = _c.c_int
    L.hdq_select_quantize_int8_noalloc.argtypes = [_p, _c.c_int64, _p, _c.c_int64, _c.c_int64, _c.c_int32,
                                                   _c.c_float, _c.c_float, _p, _p, _c.POINTER(QTensorDesc), _p]
    L.hdq_linear_dispatch.restype = _c.c_int
    L.hdq_linear_dispatch.argtypes = [_p, _p, _c.POINTER(QTensorDesc), _c.POINTER(QTensorDesc),
                                      _c.c_int64, _c.c_int64, _c.POINTER(WeightsDesc), _p, _c.c_int32, _p]
    L.hdq_linear_dispatch_delta.restype = _c.c_int
    L.hdq_linear_dispatch_delta.argtypes = [_p, _p, _c.POINTER(QTensorDesc), _c.POINTER(QTensorDesc),
                                            _c.c_int64, _c.c_int64, _c.POINTER(WeightsDesc), _p,
                                            _c.c_int32, _c.POINTER(DeltaSlice), _c.c_int32, _p, _p]
    L.hdq_tdc_decide.restype = _c.c_int
    L.hdq_tdc_decide.argtypes = [_p, _p, _p, _p, _p, _p, _c.c_int64, _c.c_float, _c.c_float, _p]
    L.hdq_quantize.restype = _c.c_int
    L.hdq_quantize.argtypes = [_p, _c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32, _p, _p,
                               _c.POINTER(QTensorDesc), _p, _c.c_size_t, _p]
    L.hdq_linear.restype = _c.c_int
    L.hdq_linear.argtypes = [_c.c_int32, _p, _p, _c.POINTER(QTensorDesc), _p, _c.c_int64,
                             _c.c_int64, _c.POINTER(WeightsDesc), _p, _c.c_int32, _p,
                             _c.c_size_t, _p]
    L.hdq_dq_cubes.restype = _c.c_int64
    L.hdq_dq_cubes.argtypes = [_c.POINTER(DqGridDesc)]
    L.hdq_dq_quantize.restype = _c.c_int
    L.hdq_dq_quantize.argtypes = [_p, _c.c_int64, _c.POINTER(DqGridDesc), _c.c_int32, _p, _p, _p,
                                  _c.POINTER(QTensorDesc), _p, _c.c_size_t, _p]
    L.hdq_dq_decode_weights.restype = _c.c_int
    L.hdq_dq_decode_weights.argtypes = [_c.POINTER(QTensorDesc), _p, _p]
    L.hdq_dq_linear.restype = _c.c_int
    L.hdq_dq_linear.argtypes = [_c.POINTER(DqGridDesc), _p, _p, _p, _c.POINTER(QTensorDesc),
                                _c.POINTER(QTensorDesc), _p, _p, _c.c_int32, _p, _c.c_size_t, _p]
    L.hdq_dq_linear_workspace_bytes.restype = _c.c_size_t
    L.hdq_dq_linear_workspace_bytes.argtypes = [_c.POINTER(DqGridDesc), _c.c_int64, _c.c_int64, _c.c_int32]
    L.hdq_fp8_quantize.restype = _c.c_int
    L.hdq_fp8_quantize.argtypes = [_p, _c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32, _c.POINTER(Fp8TensorDesc), _p]
    L.hdq_fp8_linear_workspace_bytes.restype = _c.c_size_t
    L.hdq_fp8_linear_workspace_bytes.argtypes = [_c.c_int64, _c.c_int64, _c.c_int64, _c.c_int32]
    L.hdq_fp8_linear.restype = _c.c_int
    L.hdq_fp8_linear.argtypes = [_p, _c.POINTER(Fp8TensorDesc), _c.c_int64, _c.c_int64, _c.POINTER(Fp8TensorDesc), _p,
                                 _c.c_int32, _p, _c.c_size_t, _p]
    L.hdq_group_norm_workspace_bytes.restype = _c.c_size_t
    L.hdq_group_norm_workspace_bytes.argtypes = [_c.c_int64, _c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32]
    norm = [_p, _c.c_int32, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int32, _p, _p, _c.c_float, _c.c_int32]
    L.hdq_group_norm.restype = _c.c_int
    L.hdq_group_norm.argtypes = norm + [_p, _c.c_int32, _p, _c.c_size_t, _p]
    L.hdq_group_norm_fp8.restype = _c.c_int
    L.hdq_group_norm_fp8.argtypes = norm + [_c.c_int32, _c.POINTER(Fp8TensorDesc), _p, _c.c_size_t, _p]
    L.hdq_w4_bytes.restype = _c.c_size_t
    L.hdq_w4_bytes.argtypes = [_c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32]
    w4 = _c.POINTER(W4TensorDesc)
    L.hdq_w4_pack.restype = _c.c_int
    L.hdq_w4_pack.argtypes = [_p, _p, _p, w4, _p]
    L.hdq_w4_quantize.restype = _c.c_int
    L.hdq_w4_quantize.argtypes = [_p, w4, _p]
    L.hdq_w4_linear.restype = _c.c_int
    L.hdq_w4_linear.argtypes = [_p, _c.c_int64, w4, _p, _c.c_int32, _p, _c.c_size_t, _p]
    L.hdq_w4_linear_workspace_bytes.restype = _c.c_size_t
    L.hdq_w4_linear_workspace_bytes.argtypes = [_c.c_int64, _c.c_int64, _c.c_int64]
    L.hdq_rope_turns.restype = _c.c_int
    L.hdq_rope_turns.argtypes = [_c.c_int32, _c.c_double, _c.c_int32, _c.c_double, _c.c_double, _c.c_double,
                                 _c.c_double, _c.POINTER(_c.c_double)]
    heads, norm, rope, cache = (_c.POINTER(t) for t in (HeadsDesc, HeadNormDesc, RopeDesc, KvCacheDesc))
    L.hdq_qk_norm_rope.restype = _c.c_int
    L.hdq_qk_norm_rope.argtypes = [heads, heads, _c.c_int64, _c.c_int64, _c.c_int32, norm, rope, heads, heads, _p]
    L.hdq_qkv_to_cache.restype = _c.c_int
    L.hdq_qkv_to_cache.argtypes = [heads, heads, heads, _c.c_int64, _c.c_int64, norm, rope, heads, _p, cache, _p]
    L.hdq_cache_read.restype = _c.c_int
    L.hdq_cache_read.argtypes = [cache, _p, _c.c_int64, _p, _p, _c.c_int32, _p]
    L.hdq_workspace_bytes.restype = _c.c_size_t
    L.hdq_workspace_bytes.argtypes = [_c.c_int32, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int32]
    L.hdq_status_string.restype = _c.c_char_p
    L.hdq_status_string.argtypes = [_c.c_int]
    L.hdq_version.restype = _c.c_int
    L.hdq_version.argtypes = []
    return L


lib = _load()


class HdqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {lib.hdq_status_string(status).decode()} ({status})")


def _check(fn, status):
    if status != OK:
        raise HdqError(fn, status)


def _ptr(t):
    return None if t is None else _p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return _p(s.cuda_stream)


def _bf16(t, name):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    return t


def linear_dispatch(decision, x, xq8, xq4, w, y=None, y_dtype=DTYPE_BF16, stream=None):
    """hdq_linear_dispatch: the GEMM of the device decision's precision in
    one launch (INT8 from xq8, NVFP4 from xq4, bf16 from x)."""
    x = _bf16(x, "x")
    M, K = x.shape
    if y is None:
        dt = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16}[y_dtype]
        y = torch.empty(M, w.N, dtype=dt, device=x.device)
    wd, d8, d4 = w.desc(), xq8.desc(), xq4.desc()
    st = lib.hdq_linear_dispatch(_ptr(decision), _ptr(x), _c.byref(d8), _c.byref(d4), M, K,
                                 _c.byref(wd), _ptr(y), y_dtype, _stream(stream))
    _check("hdq_linear_dispatch", st)
    return y


def linear_dispatch_delta(decision, x, xq8, xq4, w, slices, queue, y=None, y_dtype=DTYPE_BF16,
                          stream=None):
    """hdq_linear_dispatch_delta: linear_dispatch's GEMM, plus the chunk
    partials of difference statistics on extra workgroups of the launch.
    slices: up to DELTA_MAX_SLICES tuples (prev_in, prev_out, chunk_begin,
    chunk_end, partials), partials float64 [delta_chunks(numel), 2];
    queue: int32 [2] on the device, zero before the first call (each call
    leaves it zero)."""
    x = _bf16(x, "x")
    M, K = x.shape
    if y is None:
        dt = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16}[y_dtype]
        y = torch.empty(M, w.N, dtype=dt, device=x.device)
    arr = (DeltaSlice * max(1, len(slices)))()
    for i, (pi, po, c0, c1, parts) in enumerate(slices):
        _bf16(pi, "prev_in")
        _bf16(po, "prev_out")
        if pi.numel() != po.numel():
            raise ValueError("prev_in and prev_out differ in size")
        if parts.dtype != torch.float64 or parts.numel() < 2 * delta_chunks(pi.numel()):
            raise ValueError("partials: float64 [delta_chunks(numel), 2] expected")
        arr[i] = DeltaSlice(_ptr(pi), _ptr(po), pi.numel(), c0, c1, _ptr(parts))
    if queue.dtype != torch.int32 or queue.numel() < 2:
        raise ValueError("queue: int32 [2] expected")
    wd, d8, d4 = w.desc(), xq8.desc(), xq4.desc()
    st = lib.hdq_linear_dispatch_delta(_ptr(decision), _ptr(x), _c.byref(d8), _c.byref(d4), M, K,
                                       _c.byref(wd), _ptr(y), y_dtype, arr, len(slices), _ptr(queue),
                                       _stream(stream))
    _check("hdq_linear_dispatch_delta", st)
    return y


def workspace_bytes(op, M, K, N=0, fmt=-1):
    return int(lib.hdq_workspace_bytes(op, M, K, N, fmt))


def _workspace(ws, nbytes, device):
    if nbytes == 0:
        return ws
    if ws is None or ws.numel() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


class QuantizedTensor:
    """A quantized tensor: torch buffers plus the hdq_qtensor descriptor.
    decoded (NVFP4 formats): also a bf16 [rows, cols] buffer for the codes'
    exact values, which hdq_quantize fills and the plain-NVFP4 GEMM reads."""

    def __init__(self, fmt, rows, cols, had_block, device, decoded=False):
        self.fmt, self.rows, self.cols, self.had_block = fmt, rows, cols, had_block
        self.row_scale = self.blk_scale = self.tensor_scale = self.dec = None
        if fmt == FMT_INT8_ROW:
            self.codes = torch.empty(rows, cols, dtype=torch.int8, device=device)
        else:
            self.codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=device)
        if fmt in (FMT_INT8_ROW, FMT_INT4_ROW):
            self.row_scale = torch.empty(rows, dtype=torch.float32, device=device)
        else:
            self.blk_scale = torch.empty(rows, cols // 16, dtype=torch.uint8, device=device)
            self.tensor_scale = torch.empty(1, dtype=torch.float32, device=device)
            if decoded:
                self.dec = torch.empty(rows, cols, dtype=torch.bfloat16, device=device)

    def desc(self):
        return QTensorDesc(self.fmt, self.had_block, self.rows, self.cols, _ptr(self.codes),
                           _ptr(self.row_scale), _ptr(self.blk_scale), _ptr(self.tensor_scale),
                           _ptr(self.dec))


def select_precision(prev_in, prev_out, cur_in, had_block=0, delta_thresh=0.1, ratio_thresh=50.0,
                     decision=None, stats=None, ws=None, stream=None):
    """hdq_select_precision.  prev_in/prev_out None = no history.  Returns the
    device tensors (decision int32[1], stats float32[5])."""
    cur_in = _bf16(cur_in, "cur_in")
    rows, cols = cur_in.shape
    dev = cur_in.device
    if (prev_in is None) != (prev_out is None):
        raise ValueError("prev_in and prev_out must both be given or both be None")
    n_prev = 0
    if prev_in is not None:
        _bf16(prev_in, "prev_in")
        _bf16(prev_out, "prev_out")
        if prev_in.numel() != prev_out.numel():
            raise ValueError("prev_in and prev_out differ in size")
        n_prev = prev_in.numel()
    decision = torch.empty(1, dtype=torch.int32, device=dev) if decision is None else decision
    stats = torch.empty(5, dtype=torch.float32, device=dev) if stats is None else stats
    ws = _workspace(ws, workspace_bytes(OP_SELECT, rows, cols, n_prev), dev)
    st = lib.hdq_select_precision(_ptr(prev_in), _ptr(prev_out), n_prev, _ptr(cur_in), rows, cols,
                                  had_block, delta_thresh, ratio_thresh, _ptr(decision),
                                  _ptr(stats), _ptr(ws), ws.numel(), _stream(stream))
    _check("hdq_select_precision", st)
    return decision, stats


def delta_sums(prev_in, prev_out, sums=None, ws=None, stream=None):
    """hdq_delta_sums: device double[2] {sum|prev_out - prev_in|, sum|prev_in|}."""
    _bf16(prev_in, "prev_in")
    _bf16(prev_out, "prev_out")
    if prev_in.numel() != prev_out.numel():
        raise ValueError("prev_in and prev_out differ in size")
    n = prev_in.numel()
    dev = prev_in.device
    sums = torch.empty(2, dtype=torch.float64, device=dev) if sums is None else sums
    ws = _workspace(ws, workspace_bytes(OP_SELECT, 1, n, n), dev)
    st = lib.hdq_delta_sums(_ptr(prev_in), _ptr(prev_out), n, _ptr(sums), _ptr(ws), ws.numel(),
                            _stream(stream))
    _check("hdq_delta_sums", st)
    return sums


def tdc_decide(sums, state, c, acc, skip=None, tau_skip=0.05, tau_acc=0.15, stream=None, offsets=None):
    """hdq_tdc_decide over n modules: sums float64 [n, 2] (or, with offsets
    int64 [n + 1], pairs [P, 2] of which module i's are rows offsets[i] ..
    offsets[i + 1] - 1), state int32 [n], c and acc float32 [n] (updated in
    place); returns skip int32 [n]."""
    n = state.numel()
    pairs = (n, 2) if offsets is None else (sums.shape[0], 2)
    checks = [(sums, torch.float64, pairs), (state, torch.int32, (n,)),
              (c, torch.float32, (n,)), (acc, torch.float32, (n,))]
    if offsets is not None:
        checks.append((offsets, torch.int64, (n + 1,)))
    for t, dt, shape in checks:
        if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"tdc_decide: expected {dt} {shape} contiguous, got {t.dtype} {tuple(t.shape)}")
    skip = torch.empty(n, dtype=torch.int32, device=state.device) if skip is None else skip
    st = lib.hdq_tdc_decide(_ptr(sums), _ptr(offsets), _ptr(state), _ptr(c), _ptr(acc), _ptr(skip), n,
                            float(tau_skip), float(tau_acc), _stream(stream))
    _check("hdq_tdc_decide", st)
    return skip


def _delta_parts(delta_sums):
    """(pointer, pairs) of a difference-sums argument: None, or float64 with
    an even number of elements -- one pair from delta_sums(), or the chunk
    partials of linear_dispatch_delta()."""
    if delta_sums is None:
        return None, 0
    if delta_sums.dtype != torch.float64 or not delta_sums.is_contiguous() or delta_sums.numel() % 2 or \
            delta_sums.numel() == 0:
        raise ValueError("delta sums: expected contiguous float64 pairs")
    return _ptr(delta_sums), delta_sums.numel() // 2


def select_precision_sums(delta_sums, cur_in, had_block=0, delta_thresh=0.1, ratio_thresh=50.0,
                          decision=None, stats=None, ws=None, stream=None):
    """hdq_select_precision_sums: the selection with the difference sums of
    delta_sums() (None = no history).  Returns (decision, stats)."""
    cur_in = _bf16(cur_in, "cur_in")
    rows, cols = cur_in.shape
    dev = cur_in.device
    decision = torch.empty(1, dtype=torch.int32, device=dev) if decision is None else decision
    stats = torch.empty(5, dtype=torch.float32, device=dev) if stats is None else stats
    ws = _workspace(ws, workspace_bytes(OP_SELECT, rows, cols, 0), dev)
    dp, parts = _delta_parts(delta_sums)
    st = lib.hdq_select_precision_sums(dp, parts, _ptr(cur_in), rows, cols, had_block,
                                       delta_thresh, ratio_thresh, _ptr(decision), _ptr(stats),
                                       _ptr(ws), ws.numel(), _stream(stream))
    _check("hdq_select_precision_sums", st)
    return decision, stats


def select_quantize_int8(delta_sums, cur_in, had_block, delta_thresh=0.1, ratio_thresh=50.0,
                         decision=None, stats=None, out=None, ws=None, stream=None):
    """hdq_select_quantize_int8: the selection (difference sums from
    delta_sums(), None = no history) fused with the INT8 per-token
    quantization of cur_in.  Returns (decision, stats, QuantizedTensor)."""
    cur_in = _bf16(cur_in, "cur_in")
    rows, cols = cur_in.shape
    dev = cur_in.device
    decision = torch.empty(1, dtype=torch.int32, device=dev) if decision is None else decision
    stats = torch.empty(5, dtype=torch.float32, device=dev) if stats is None else stats
    out = QuantizedTensor(FMT_INT8_ROW, rows, cols, had_block, dev) if out is None else out
    ws = _workspace(ws, workspace_bytes(OP_SELECT_Q8, rows, cols, 0), dev)
    d = out.desc()
    dp, parts = _delta_parts(delta_sums)
    st = lib.hdq_select_quantize_int8(dp, parts, _ptr(cur_in), rows, cols, had_block,
                                      delta_thresh, ratio_thresh, _ptr(decision), _ptr(stats),
                                      _c.byref(d), _ptr(ws), ws.numel(), _stream(stream))
    _check("hdq_select_quantize_int8", st)
    out.fmt, out.had_block, out.rows, out.cols = d.fmt, d.had_block, d.rows, d.cols
    return decision, stats, out


def select_quantize_int8_noalloc(delta_sums, cur_in, had_block, decision, stats, out, delta_thresh=0.1,
                                 ratio_thresh=50.0, stream=None):
    """hdq_select_quantize_int8_noalloc: select_quantize_int8 with the
    library's fixed per-GPU scratch instead of a workspace; the caller passes
    every output (decision int32[1], stats float32[5], an INT8 QuantizedTensor),
    so the call allocates nothing."""
    cur_in = _bf16(cur_in, "cur_in")
    rows, cols = cur_in.shape
    d = out.desc()
    dp, parts = _delta_parts(delta_sums)
    st = lib.hdq_select_quantize_int8_noalloc(dp, parts, _ptr(cur_in), rows, cols, had_block,
                                              delta_thresh, ratio_thresh, _ptr(decision), _ptr(stats),
                                              _c.byref(d), _stream(stream))
    _check("hdq_select_quantize_int8_noalloc", st)
    out.fmt, out.had_block, out.rows, out.cols = d.fmt, d.had_block, d.rows, d.cols
    return decision, stats, out


def quantize(x, had_block, fmt, tensor_amax=None, out=None, ws=None, stream=None, decision=None,
             decoded=False):
    """hdq_quantize: rotate + quantize a bf16 [rows, cols] tensor (only when
    the device decision matches the format's precision, if one is given).
    decoded: a new output also gets the NVFP4 codes' exact bf16 values."""
    x = _bf16(x, "x")
    rows, cols = x.shape
    out = QuantizedTensor(fmt, rows, cols, had_block, x.device, decoded) if out is None else out
    d = out.desc()
    nbytes = workspace_bytes(OP_QUANTIZE, rows, cols, 0, fmt) if tensor_amax is None else 0
    ws = _workspace(ws, nbytes, x.device)
    st = lib.hdq_quantize(_ptr(x), rows, cols, had_block, fmt, _ptr(tensor_amax), _ptr(decision),
                          _c.byref(d),
                          _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check("hdq_quantize", st)
    return out


# ---- DeltaQuant cube-delta quantization --------------------------------------

def dq_cubes(grid):
    """Cubes of grid = (frames, height, width, (cube_f, cube_h, cube_w))."""
    n = lib.hdq_dq_cubes(_c.byref(_dq_grid(grid)))
    if n < 0:
        raise ValueError(f"bad DeltaQuant grid {grid}")
    return n


def _dq_grid(grid):
    F, H, W, (cf, ch, cw) = grid
    return DqGridDesc(F, H, W, cf, ch, cw)


def dq_core_needs_bf16(fmt, cubes, K, N=None):
    """Whether hdq_dq_linear's core GEMM runs on the bf16 core values and
    decoded weights: unless the weights' block scales are powers of two (MX
    or per-16 format), K % 128 == 0, and the core codes and (N given) the
    FP4 weight codes fit 32-bit offsets -- the library's own rule."""
    fits = cubes * K < 2 ** 31 and (N is None or N * K // 2 < 2 ** 31)
    return not (fmt in (FMT_NVFP4_MX, FMT_NVFP4_P2) and K % 128 == 0 and fits)


class DqActivations:
    """hdq_dq_quantize's outputs: core codes [cubes, K], core scales [cubes],
    the differences' NVFP4 tensor and, when asked for (by default when the
    core GEMM needs them, see dq_core_needs_bf16), the core code values as
    bf16 [cubes, K]."""

    def __init__(self, grid, K, fmt, device, core_bf16=None):
        self.grid, self.K = grid, K
        n, M = dq_cubes(grid), grid[0] * grid[1] * grid[2]
        self.core = torch.empty(n, K, dtype=torch.uint8, device=device)
        self.core_scale = torch.empty(n, dtype=torch.float32, device=device)
        want = dq_core_needs_bf16(fmt, n, K) if core_bf16 is None else core_bf16
        self.core_bf16 = torch.empty(n, K, dtype=torch.bfloat16, device=device) if want else None
        self.delta = QuantizedTensor(fmt, M, K, 1, device)


def dq_quantize(x, grid, fmt, out=None, ws=None, stream=None, core_bf16=None):
    """hdq_dq_quantize: cube cores in FP8 and the differences in NVFP4."""
    x = _bf16(x, "x")
    M, K = x.shape
    out = DqActivations(grid, K, fmt, x.device, core_bf16) if out is None else out
    ws = _workspace(ws, workspace_bytes(OP_DQ_QUANTIZE, M, K), x.device)
    d = out.delta.desc()
    st = lib.hdq_dq_quantize(_ptr(x), K, _c.byref(_dq_grid(grid)), fmt, _ptr(out.core), _ptr(out.core_scale),
                             _ptr(out.core_bf16), _c.byref(d), _ptr(ws), ws.numel(), _stream(stream))
    _check("hdq_dq_quantize", st)
    return out


def dq_decode_weights(w_fp4, stream=None):
    """hdq_dq_decode_weights: bf16 [N, K] of E2M1 x block scale."""
    out = torch.empty(w_fp4.rows, w_fp4.cols, dtype=torch.bfloat16, device=w_fp4.codes.device)
    d = w_fp4.desc()
    _check("hdq_dq_decode_weights", lib.hdq_dq_decode_weights(_c.byref(d), _ptr(out), _stream(stream)))
    return out


def dq_linear_workspace_bytes(grid, K, N, fmt):
    """hdq_dq_linear_workspace_bytes: the scratch hdq_dq_linear needs on its route."""
    return lib.hdq_dq_linear_workspace_bytes(_c.byref(_dq_grid(grid)), K, N, fmt)


def dq_linear(a, w_fp4, w_dec=None, y=None, y_dtype=DTYPE_BF16, ws=None, stream=None):
    """hdq_dq_linear: y = differences x W^T + cube cores x W^T.  w_dec and
    the activations' bf16 core values are needed only when the core GEMM runs
    in bf16 (dq_core_needs_bf16 with N: plain NVFP4, K % 128 != 0, or codes
    past 32-bit offsets); the library returns HDQ_ERR_INVALID without them."""
    M, N = a.delta.rows, w_fp4.rows
    if y is None:
        dt = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16}[y_dtype]
        y = torch.empty(M, N, dtype=dt, device=a.core.device)
    ws = _workspace(ws, dq_linear_workspace_bytes(a.grid, a.delta.cols, N, a.delta.fmt), a.core.device)
    dd, wd = a.delta.desc(), w_fp4.desc()
    st = lib.hdq_dq_linear(_c.byref(_dq_grid(a.grid)), _ptr(a.core), _ptr(a.core_bf16), _ptr(a.core_scale), _c.byref(dd),
                           _c.byref(wd), _ptr(w_dec), _ptr(y), y_dtype, _ptr(ws), ws.numel(), _stream(stream))
    _check("hdq_dq_linear", st)
    return y


class LinearWeights:
    """A linear layer's weights in every form a precision may need:
    bf16 (unrotated, for the full-precision fallback), INT4 per output
    channel, and NVFP4 (or its MX-compatible variant).  fp4_decoded: the
    NVFP4 weights also as their exact bf16 values (N x K x 2 bytes), which
    the plain-NVFP4 GEMM reads when the activations carry theirs too."""

    def __init__(self, w_bf16, had_block, fp4_fmt=FMT_NVFP4, keep_bf16=True, stream=None, fp4_decoded=False):
        w_bf16 = _bf16(w_bf16, "w")
        self.N, self.K = w_bf16.shape
        self.had_block = had_block
        self.w_bf16 = w_bf16 if keep_bf16 else None
        self.w_int4 = quantize(w_bf16, had_block, FMT_INT4_ROW, stream=stream)
        self.w_fp4 = (quantize(w_bf16, had_block, fp4_fmt, stream=stream, decoded=fp4_decoded)
                      if fp4_fmt is not None else None)

    def desc(self):
        empty = QTensorDesc(-1, 0, 0, 0, None, None, None, None, None)
        return WeightsDesc(self.N, self.K, _ptr(self.w_bf16), self.w_int4.desc(),
                           self.w_fp4.desc() if self.w_fp4 is not None else empty)


def linear(precision, x, w, decision=None, xq=None, x_amax=None, y=None, y_dtype=DTYPE_BF16,
           ws=None, stream=None):
    """hdq_linear: Y[M, N] = quantized X[M, K] @ W^T.  precision -1 reads the
    decision tensor on the device; a fixed precision with a decision tensor
    runs only when the device decision equals it."""
    if x is not None:
        x = _bf16(x, "x")
        M, K = x.shape
        dev = x.device
    else:
        M, K = xq.rows, xq.cols
        dev = xq.codes.device
    if y is None:
        dt = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16, DTYPE_I32: torch.int32}[y_dtype]
        y = torch.empty(M, w.N, dtype=dt, device=dev)
    wd = w.desc()
    fp4_fmt = w.w_fp4.fmt if w.w_fp4 is not None else -1
    nbytes = 0 if xq is not None else workspace_bytes(OP_LINEAR, M, K, w.N, fp4_fmt)
    ws = _workspace(ws, nbytes, dev)
    xqd = xq.desc() if xq is not None else None
    st = lib.hdq_linear(precision, _ptr(decision), _ptr(x), _c.byref(xqd) if xqd is not None else None,
                        _ptr(x_amax), M, K, _c.byref(wd), _ptr(y), y_dtype, _ptr(ws),
                        0 if ws is None else ws.numel(), _stream(stream))
    _check("hdq_linear", st)
    return y


# ---- FP8 block-128 linear layers ----------------------------------------------

def _torch_call(name, public):
    """torch's own binding `name`, which builds no Python object on the way, or
    `public` in a torch that lacks it."""
    return getattr(torch._C, name, public)


_current_device = _torch_call("_cuda_getDevice", torch.cuda.current_device)
_current_stream = _torch_call("_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, stream, call):
    """call(raw stream) with `dev` the current device and `stream` (None: the
    device's current stream) the current stream, so that what the call
    allocates belongs to the stream its kernels run on."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors are on {dev}, not on a GPU")
    if stream is None:
        if dev.index == _current_device():
            return call(_current_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_current_stream(dev.index))
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _operand(t, name, dtype, shape, dev):
    """Checks a tensor the library reads or writes in place."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name}: expected a contiguous {dtype} {shape} tensor on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t


def _scratch(ws, nbytes, dev):
    """The caller's workspace if it is large enough, else a new one, or None
    where none is needed: (tensor, pointer, bytes)."""
    if nbytes == 0:
        return None, None, 0
    if ws is not None:
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws: expected a contiguous tensor on {dev}")
        size = ws.numel() * ws.element_size()
        if size >= nbytes:
            return ws, ws.data_ptr(), size
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws, ws.data_ptr(), nbytes


class Fp8Tensor:
    """An FP8 (E4M3) tensor with one float32 scale per block of 128: torch
    buffers plus the hdq_fp8_tensor fields.  codes uint8 (or float8_e4m3fn)
    [rows, 128 * kb] with zeros past cols, kb = ceil(cols / 128); scale float32
    [kb, rows] (FP8_ROWS) or [ceil(rows / 128), kb] (FP8_BLOCKS).  Buffers that
    are not given are allocated on `device`; given ones (an FP8 checkpoint's
    weights and block scales) are used as they are."""

    def __init__(self, rows, cols, had_block=1, layout=FP8_ROWS, device=None, codes=None, scale=None):
        if layout not in (FP8_ROWS, FP8_BLOCKS):
            raise ValueError(f"unknown FP8 layout {layout}")
        self.rows, self.cols, self.had_block, self.layout = rows, cols, had_block, layout
        kb = -(-cols // FP8_BLOCK)
        cshape = (rows, kb * FP8_BLOCK)
        sshape = (kb, rows) if layout == FP8_ROWS else (-(-rows // FP8_BLOCK), kb)
        dev = codes.device if codes is not None else scale.device if scale is not None else device
        if codes is None:
            codes = torch.empty(*cshape, dtype=torch.uint8, device=dev)
        else:
            codes = codes.view(torch.uint8) if codes.dtype == torch.float8_e4m3fn else codes
            _operand(codes, "codes", torch.uint8, cshape, dev)
        if scale is None:
            scale = torch.empty(*sshape, dtype=torch.float32, device=dev)
        else:
            _operand(scale, "scale", torch.float32, sshape, dev)
        self.codes, self.scale = codes, scale

    def desc(self):
        return Fp8TensorDesc(self.layout, self.had_block, self.rows, self.cols, self.codes.data_ptr(),
                             self.scale.data_ptr())


def fp8_quantize(x, had_block=1, layout=FP8_ROWS, out=None, stream=None):
    """hdq_fp8_quantize: rotate a bf16 [rows, cols] tensor and quantize it to
    FP8 with one scale per 128 elements of a row (activations) or per
    128 x 128 block (FP8_BLOCKS, weights)."""
    x = _bf16(x, "x")
    rows, cols = x.shape
    dev = x.device
    if out is not None and ((out.rows, out.cols, out.layout) != (rows, cols, layout) or out.codes.device != dev):
        raise ValueError("out does not fit x")

    def call(s):
        q = Fp8Tensor(rows, cols, had_block, layout, dev) if out is None else out
        d = q.desc()
        _check("hdq_fp8_quantize", lib.hdq_fp8_quantize(x.data_ptr(), rows, cols, had_block, layout, _c.byref(d), s))
        q.had_block = had_block
        return q
    return _launch(dev, stream, call)


def fp8_linear_workspace_bytes(M, K, N, y_dtype=DTYPE_BF16):
    """hdq_fp8_linear_workspace_bytes: the scratch fp8_linear needs without xq."""
    return lib.hdq_fp8_linear_workspace_bytes(M, K, N, y_dtype)


def fp8_linear(x, w, xq=None, y=None, y_dtype=DTYPE_BF16, ws=None, stream=None):
    """hdq_fp8_linear: Y[M, N] = X[M, K] @ W[N, K]^T for FP8_BLOCKS weights;
    x bf16 is quantized within the call (with the weights' had_block), or
    xq holds the activations already quantized (FP8_ROWS; x is then unused)."""
    if xq is None:
        x = _bf16(x, "x")
        (M, K), dev = x.shape, x.device
    else:
        M, K, dev = xq.rows, xq.cols, xq.codes.device
    if w.codes.device != dev:
        raise ValueError(f"the weights are on {w.codes.device}, the activations on {dev}")
    N = w.rows
    dt = torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16
    if y is not None:
        _operand(y, "y", dt, (M, N), dev)

    def call(s):
        out = torch.empty(M, N, dtype=dt, device=dev) if y is None else y
        wd = w.desc()
        if xq is None:
            _keep, wp, wn = _scratch(ws, lib.hdq_fp8_linear_workspace_bytes(M, K, N, y_dtype), dev)
            st = lib.hdq_fp8_linear(x.data_ptr(), None, M, K, _c.byref(wd), out.data_ptr(), y_dtype, wp, wn, s)
        else:
            xd = xq.desc()
            st = lib.hdq_fp8_linear(None, _c.byref(xd), M, K, _c.byref(wd), out.data_ptr(), y_dtype, None, 0, s)
        _check("hdq_fp8_linear", st)
        return out
    return _launch(dev, stream, call)


# ---- group norm, channels last --------------------------------------------------

def group_norm_workspace_bytes(n, length, channels, groups, fp8=False):
    """hdq_group_norm_workspace_bytes: the scratch group_norm or (fp8) group_norm_fp8 needs."""
    return lib.hdq_group_norm_workspace_bytes(n, length, channels, groups, int(fp8))


_NORM_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _norm_input(x, weight, bias):
    """(x's dtype code, n, length, channels, weight and bias pointers)."""
    xt, shape, dev = _NORM_DTYPES.get(x.dtype), x.shape, x.device
    if xt is None or not x.is_cuda or not x.is_contiguous() or len(shape) < 2:
        raise ValueError("x must be a contiguous bfloat16 or float32 CUDA tensor [n, ..., channels]")
    n, C, numel = shape[0], shape[-1], x.numel()
    if numel == 0:
        raise ValueError("x is empty")
    wp = _operand(weight, "weight", torch.float32, (C,), dev).data_ptr() if weight is not None else None
    bp = _operand(bias, "bias", torch.float32, (C,), dev).data_ptr() if bias is not None else None
    return xt, n, numel // (n * C), C, wp, bp


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, act=ACT_NONE, y=None, y_dtype=None, ws=None, stream=None):
    """hdq_group_norm of x [n, ..., channels] (bf16 or float32, channels last)
    with float32 weight and bias [channels] (None: 1 and 0), and a SiLU for
    ACT_SILU.  y (may be x) or a new tensor of y_dtype (DTYPE_*; None: x's)."""
    xt, n, length, C, wp, bp = _norm_input(x, weight, bias)
    yt = (xt if y is None else _NORM_DTYPES.get(y.dtype)) if y_dtype is None else y_dtype
    dt = torch.float32 if yt == DTYPE_F32 else torch.bfloat16
    dev = x.device
    if y is not None:
        _operand(y, "y", dt, x.shape, dev)

    def call(s):
        out = torch.empty_like(x, dtype=dt) if y is None else y
        _keep, sp, sn = _scratch(ws, lib.hdq_group_norm_workspace_bytes(n, length, C, groups, 0), dev)
        st = lib.hdq_group_norm(x.data_ptr(), xt, n, length, C, groups, wp, bp, eps, act, out.data_ptr(), yt, sp, sn, s)
        _check("hdq_group_norm", st)
        return out
    return _launch(dev, stream, call)


def group_norm_fp8(x, groups, weight=None, bias=None, eps=1e-5, act=ACT_NONE, had_block=1, out=None, ws=None,
                   stream=None):
    """hdq_group_norm_fp8: group_norm's float32 result rotated and quantized
    to an FP8_ROWS tensor [n * length, channels], an fp8_linear's xq."""
    xt, n, length, C, wp, bp = _norm_input(x, weight, bias)
    dev = x.device
    if out is not None and ((out.rows, out.cols, out.layout) != (n * length, C, FP8_ROWS) or out.codes.device != dev):
        raise ValueError("out does not fit x")

    def call(s):
        q = Fp8Tensor(n * length, C, had_block, FP8_ROWS, dev) if out is None else out
        _keep, sp, sn = _scratch(ws, lib.hdq_group_norm_workspace_bytes(n, length, C, groups, 1), dev)
        d = q.desc()
        st = lib.hdq_group_norm_fp8(x.data_ptr(), xt, n, length, C, groups, wp, bp, eps, act, had_block, _c.byref(d),
                                    sp, sn, s)
        _check("hdq_group_norm_fp8", st)
        q.had_block = had_block
        return q
    return _launch(dev, stream, call)


# ---- linear layers of few tokens, 4-bit weights in groups ---------------------------

class W4Weights:
    """4-bit weights [N, K] with one bf16 scale (and, with zero_points, a zero
    point) per group of 32, 64 or 128 columns of a row, packed in tiles as
    hdq_w4_tensor describes.  w4_pack and w4_quantize make them."""

    def __init__(self, N, K, group=128, zero_points=False, device=None):
        sizes = [lib.hdq_w4_bytes(N, K, group, b) for b in (W4_CODES, W4_SCALE, W4_ZERO)]
        if sizes[0] == 0:
            raise ValueError(f"no 4-bit weights of {N} x {K} in groups of {group}")
        self.N, self.K, self.group = N, K, group
        self.codes = torch.empty(sizes[0], dtype=torch.uint8, device=device)
        self.scale = torch.empty(sizes[1] // 2, dtype=torch.bfloat16, device=device)
        self.zero = torch.empty(sizes[2], dtype=torch.uint8, device=device) if zero_points else None
        self._desc = W4TensorDesc(N, K, group, self.codes.data_ptr(), self.scale.data_ptr(),
                                  self.zero.data_ptr() if zero_points else None)
        self._ref = _c.byref(self._desc)

    def desc(self):
        return self._ref


def w4_pack(codes, scale, zero=None, stream=None):
    """hdq_w4_pack: codes uint8 [N, K / 2] (even columns in the low nibbles),
    scale bf16 [N, K / group] and zero points uint8 [N, K / group] or None, to
    W4Weights."""
    if codes.dtype != torch.uint8 or codes.dim() != 2 or scale.dim() != 2 or scale.shape[1] == 0:
        raise ValueError("expected uint8 codes [N, K / 2] and scales [N, K / group]")
    (N, half), dev = codes.shape, codes.device
    K, group = 2 * half, 2 * half // scale.shape[1]
    _operand(codes, "codes", torch.uint8, (N, half), dev)
    if group == 0 or K % group:
        raise ValueError(f"{scale.shape[1]} scales a row do not divide {K} columns")
    _operand(scale, "scale", torch.bfloat16, (N, K // group), dev)
    if zero is not None:
        _operand(zero, "zero", torch.uint8, (N, K // group), dev)

    def call(s):
        w = W4Weights(N, K, group, zero is not None, dev)
        _check("hdq_w4_pack", lib.hdq_w4_pack(codes.data_ptr(), scale.data_ptr(), zero.data_ptr() if zero is not None else None,
                                              w.desc(), s))
        return w
    return _launch(dev, stream, call)


def w4_quantize(w, group=128, zero_points=False, stream=None):
    """hdq_w4_quantize: bf16 weights [N, K], rounded to nearest, to W4Weights."""
    w = _bf16(w, "w")
    N, K = w.shape

    def call(s):
        q = W4Weights(N, K, group, zero_points, w.device)
        _check("hdq_w4_quantize", lib.hdq_w4_quantize(w.data_ptr(), q.desc(), s))
        return q
    return _launch(w.device, stream, call)


def w4_linear_workspace_bytes(M, N, K):
    """hdq_w4_linear_workspace_bytes: the scratch w4_linear needs."""
    return lib.hdq_w4_linear_workspace_bytes(M, N, K)


def w4_linear(x, w, y=None, y_dtype=DTYPE_BF16, ws=None, stream=None):
    """hdq_w4_linear: Y[M, N] = X[M, K] @ W[N, K]^T, x bf16, w W4Weights."""
    x = _bf16(x, "x")
    (M, K), dev = x.shape, x.device
    if K != w.K or w.codes.device != dev:
        raise ValueError(f"the weights are {w.N} x {w.K} on {w.codes.device}, x {M} x {K} on {dev}")
    dt = torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16
    if y is not None:
        _operand(y, "y", dt, (M, w.N), dev)

    def call(s):
        out = x.new_empty((M, w.N), dtype=dt) if y is None else y
        # few tokens in short rows need none
        need = 0 if M <= 16 and M * K <= 24576 else lib.hdq_w4_linear_workspace_bytes(M, w.N, K)
        _keep, wp, wn = _scratch(ws, need, dev)
        _check("hdq_w4_linear", lib.hdq_w4_linear(x.data_ptr(), M, w.desc(), out.data_ptr(), y_dtype, wp, wn, s))
        return out
    return _launch(dev, stream, call)


# ---- heads: norms, rotary positions, a quantized key-value cache ----------------------

def rope_turns(dim, base=10000.0, scaling=ROPE_SCALE_NONE, factor=1.0, length=0.0, ramp=(1.0, 32.0)):
    """hdq_rope_turns: float64 [dim / 2] (on the host) of one axis' turns per
    position; ramp is (slow, fast) of ROPE_SCALE_RAMP."""
    out = torch.empty(max(dim, 0) // 2, dtype=torch.float64)
    ptr = _c.cast(out.data_ptr(), _c.POINTER(_c.c_double)) if out.numel() else (_c.c_double * 1)()
    _check("hdq_rope_turns", lib.hdq_rope_turns(dim, base, scaling, factor, length, *ramp, ptr))
    return out


class Rope:
    """Rotary positions (hdq_rope without the positions): dims are the rotated
    elements of each position axis (one to three, even), layout ROPE_HALF or
    ROPE_INTERLEAVED; scale multiplies the rotated elements.  turns: float64
    [sum(dims) / 2] on the device, or None for rope_turns of each axis with the
    remaining arguments."""

    def __init__(self, dims, layout=ROPE_INTERLEAVED, base=10000.0, scaling=ROPE_SCALE_NONE, factor=1.0, length=0.0,
                 ramp=(1.0, 32.0), scale=1.0, turns=None, device=None):
        dims = (dims,) if isinstance(dims, int) else tuple(dims)
        if not 1 <= len(dims) <= ROPE_MAX_AXES or any(d <= 0 or d % 2 for d in dims):
            raise ValueError(f"rotary dims {dims}: one to {ROPE_MAX_AXES} even numbers")
        if layout not in (ROPE_INTERLEAVED, ROPE_HALF):
            raise ValueError(f"unknown rotary layout {layout}")
        if turns is None:
            turns = torch.cat([rope_turns(d, base, scaling, factor, length, ramp) for d in dims]).to(device or "cuda")
        _operand(turns, "turns", torch.float64, (sum(dims) // 2,), turns.device)
        self.dims, self.dim, self.axes, self.layout, self.scale, self.turns = dims, sum(dims), len(dims), layout, scale, turns
        self._device = turns.device
        self._fixed = (layout, self.dim, self.axes, *dims, *(0,) * (3 - len(dims)), scale, turns.data_ptr())

    def desc(self, positions, batch, length, dev):
        """hdq_rope with positions int64 [axes, batch, length]; [batch, length] or
        [length] for one axis and [axes, length], the same in every sequence."""
        if positions.dtype is not _I64 or positions.device != dev or self._device != dev:
            raise ValueError(f"positions: expected int64 on {dev}, got {positions.dtype} on {positions.device}; "
                             f"turns on {self._device}")
        shape, st, axes = positions.shape, positions.stride(), self.axes
        if shape == (axes, batch, length):
            a, b, t = st
        elif axes == 1 and shape == (batch, length):
            a, (b, t) = 0, st
        elif axes == 1 and shape == (length,):
            a, b, t = 0, 0, st[0]
        elif shape == (axes, length):
            a, b, t = st[0], 0, st[1]
        else:
            raise ValueError(f"positions {tuple(shape)} for {axes} axes, {batch} sequences of {length}")
        return _ROPE.pack(*self._fixed, positions.data_ptr(), a, b, t)


_F32, _BF16, _I64 = torch.float32, torch.bfloat16, torch.int64
# hdq_heads, hdq_head_norm and hdq_rope as bytes, in C's layout (see HeadsDesc, HeadNormDesc, RopeDesc): several
# of them are made for every call, and packing takes a fraction of a ctypes structure's time
_HEADS, _NORM, _ROPE = struct.Struct("Piiqqq"), struct.Struct("ifPPPP"), struct.Struct("iii3ifPPqqq")


def _entry(name, pointers):
    """lib's function `name` with these arguments taken as addresses or bytes."""
    f = lib[name]
    f.restype, types = _c.c_int, list(getattr(lib, name).argtypes)
    for i in pointers:
        types[i] = _c.c_char_p
    f.argtypes = types
    return f


_qk_norm_rope = _entry("hdq_qk_norm_rope", (0, 1, 5, 6, 7, 8))
_qkv_to_cache = _entry("hdq_qkv_to_cache", (0, 1, 2, 5, 6, 7))


def _head_shape(x, name):
    """(batch, length, heads, dim) of a view [batch, length, heads, dim] or [length, heads, dim]."""
    shape = x.shape
    if len(shape) == 4:
        return shape
    if len(shape) != 3:
        raise ValueError(f"{name}: expected [batch, length, heads, dim] or [length, heads, dim], got {tuple(shape)}")
    return (1, *shape)


def _row_dtype(dtype):
    return DTYPE_BF16 if dtype is _BF16 else DTYPE_F32 if dtype is _F32 else -1


def _heads(x, name, heads, dim, dev):
    """hdq_heads of a view of `heads` heads whose last dimension is contiguous."""
    st, dt = x.stride(), _row_dtype(x.dtype)
    if dt < 0 or x.device != dev or (st[-1] != 1 and dim != 1):
        raise ValueError(f"{name}: expected bfloat16 or float32 on {dev} with contiguous heads, got {x.dtype} on "
                         f"{x.device}, strides {st}")
    if len(st) == 4:
        b, t, h, _ = st
    else:
        b, (t, h, _) = 0, st
    return _HEADS.pack(x.data_ptr(), dt, heads, b, t, h)


def _head_norm(kind, eps, dim, dev, qw, qb, kw, kb):
    if kind == HEAD_NORM_NONE:
        return None
    shape = (dim,)
    return _NORM.pack(kind, eps, 0 if qw is None else _operand(qw, "q_weight", _F32, shape, dev).data_ptr(),
                      0 if qb is None else _operand(qb, "q_bias", _F32, shape, dev).data_ptr(),
                      0 if kw is None else _operand(kw, "k_weight", _F32, shape, dev).data_ptr(),
                      0 if kb is None else _operand(kb, "k_bias", _F32, shape, dev).data_ptr())


def _out_heads(out, x, shape, y_dtype, name, dev):
    """(out or a new contiguous tensor of y_dtype (None: x's), its hdq_heads)."""
    B, T, H, D = shape
    dtype = x.dtype if y_dtype is None else _F32 if y_dtype == DTYPE_F32 else _BF16 if y_dtype == DTYPE_BF16 else None
    if dtype is None or (out is not None and y_dtype is not None and out.dtype is not dtype):
        raise ValueError(f"{name}: y_dtype {y_dtype}" + ("" if out is None else f" for a tensor of {out.dtype}"))
    if out is not None:
        if out.shape != x.shape:
            raise ValueError(f"{name} {tuple(out.shape)} for an input {tuple(x.shape)}")
        return out, _heads(out, name, H, D, dev)
    if dtype is not x.dtype:
        out = x.new_empty((B, T, H, D) if x.dim() == 4 else (T, H, D), dtype=dtype)
    else:                       # the quicker forms
        out = x.new_empty(B, T, H, D) if x.dim() == 4 else x.new_empty(T, H, D)
    return out, _HEADS.pack(out.data_ptr(), _row_dtype(out.dtype), H, T * H * D, H * D, D)


def _rope_desc(rope, positions, batch, length, dev):
    if rope is None:
        return None
    if positions is None:
        raise ValueError("rotary positions are missing")
    return rope.desc(positions, batch, length, dev)


def qk_norm_rope(q, k=None, norm=HEAD_NORM_NONE, q_weight=None, k_weight=None, q_bias=None, k_bias=None, eps=1e-6,
                 positions=None, rope=None, q_out=None, k_out=None, y_dtype=None, stream=None):
    """hdq_qk_norm_rope: queries [batch, length, heads, dim] (or [length, heads,
    dim]) and, with their own number of heads, keys, normed over each head and
    rotated.  Any strides but the last; outputs are new contiguous tensors (of
    y_dtype, DTYPE_F32 or DTYPE_BF16; None: the input's) or q_out and k_out (which
    may be q and k).
    Returns (q_out, k_out), or q_out alone without k."""
    shape, dev = _head_shape(q, "q"), q.device
    B, T, H, D = shape
    if k is not None:
        kshape = _head_shape(k, "k")
        if (kshape[0], kshape[1], kshape[3]) != (B, T, D):
            raise ValueError(f"queries {tuple(q.shape)}, keys {tuple(k.shape)}")

    def call(s):
        qd = _heads(q, "q", H, D, dev)
        qo, qod = _out_heads(q_out, q, shape, y_dtype, "q_out", dev)
        ko = kd = kod = None
        if k is not None:
            kd = _heads(k, "k", kshape[2], D, dev)
            ko, kod = _out_heads(k_out, k, kshape, y_dtype, "k_out", dev)
        nd = _head_norm(norm, eps, D, dev, q_weight, q_bias, k_weight, k_bias)
        rd = _rope_desc(rope, positions, B, T, dev)
        if B * T:
            _check("hdq_qk_norm_rope", _qk_norm_rope(qd, kd, B, T, D, nd, rd, qod, kod, s))
        return qo if k is None else (qo, ko)
    return _launch(dev, stream, call)


def rope(x, positions, rope, out=None, y_dtype=None, stream=None):
    """Rotary positions of one tensor [batch, length, heads, dim] (hdq_qk_norm_rope
    without a norm); out may be x."""
    return qk_norm_rope(x, positions=positions, rope=rope, q_out=out, y_dtype=y_dtype, stream=stream)


class KvCache:
    """A cache of `slots` tokens' keys and values (hdq_kv_cache): CACHE_INT8,
    CACHE_FP8 or CACHE_INT4 codes with a float32 scale per group of elements
    (None: the head), rotated in Hadamard blocks of had_block.  Buffers
    (k_codes and v_codes uint8 [slots, heads, dim], or dim / 2 for INT4;
    k_scale and v_scale float32 [slots, heads, dim / group]) are the given
    ones or new ones on `device`, zeroed.  Calls with a cache of 0 slots, whose
    buffers have no address, are refused."""

    def __init__(self, slots, heads, dim, fmt=CACHE_FP8, group=None, had_block=1, device=None, k_codes=None, k_scale=None,
                 v_codes=None, v_scale=None):
        group = dim if group is None else group
        if fmt not in (CACHE_INT8, CACHE_FP8, CACHE_INT4) or group < 1 or dim % group or dim % 8:
            raise ValueError(f"no cache of format {fmt}, dim {dim}, groups of {group}")
        cshape, sshape = (slots, heads, dim // 2 if fmt == CACHE_INT4 else dim), (slots, heads, dim // group)
        given = next((t for t in (k_codes, k_scale, v_codes, v_scale) if t is not None), None)
        dev = given.device if given is not None else torch.device(device or "cuda")
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())

        def buffer(t, name, dtype, shape):
            return torch.zeros(shape, dtype=dtype, device=dev) if t is None else _operand(t, name, dtype, shape, dev)
        self.slots, self.heads, self.dim, self.fmt, self.group, self.had_block = slots, heads, dim, fmt, group, had_block
        self.device = dev
        self.k_codes = buffer(k_codes, "k_codes", torch.uint8, cshape)
        self.k_scale = buffer(k_scale, "k_scale", torch.float32, sshape)
        self.v_codes = buffer(v_codes, "v_codes", torch.uint8, cshape)
        self.v_scale = buffer(v_scale, "v_scale", torch.float32, sshape)
        self._desc = KvCacheDesc(fmt, group, had_block, heads, dim, slots, self.k_codes.data_ptr(), self.k_scale.data_ptr(),
                                 self.v_codes.data_ptr(), self.v_scale.data_ptr())
        self._ref = _c.byref(self._desc)

    def desc(self):
        return self._ref


def _slots(slots, n, dev):
    if slots.dtype is not _I64 or slots.numel() != n or not slots.is_contiguous() or slots.device != dev:
        raise ValueError(f"slots: expected {n} contiguous int64 on {dev}, got {slots.dtype} {tuple(slots.shape)} on {slots.device}")
    return slots.data_ptr()


def qkv_to_cache(cache, q, k, v, slots, norm=HEAD_NORM_NONE, q_weight=None, k_weight=None, q_bias=None, k_bias=None, eps=1e-6,
                 positions=None, rope=None, q_out=None, y_dtype=None, stream=None):
    """hdq_qkv_to_cache: queries normed and rotated, keys normed, rotated and
    quantized into the cache's slots (int64 [batch * length]), values quantized
    as they are.  Views as qk_norm_rope's.  Returns q_out (None without q)."""
    B, T, Hk, D = _head_shape(k, "k")
    dev = k.device
    if v is None:
        raise ValueError("v is missing")
    if v.shape != k.shape:
        raise ValueError(f"values {tuple(v.shape)}, keys {tuple(k.shape)}")
    if q is not None:
        shape = _head_shape(q, "q")
        if (shape[0], shape[1], shape[3]) != (B, T, D):
            raise ValueError(f"queries {tuple(q.shape)}, keys {tuple(k.shape)}")
    if Hk != cache.heads or D != cache.dim or cache.device != dev:
        raise ValueError(f"keys {tuple(k.shape)} on {dev}, a cache of {cache.heads} heads of {cache.dim} on {cache.device}")

    def call(s):
        qo = qd = qod = None
        if q is not None:
            qd = _heads(q, "q", shape[2], D, dev)
            qo, qod = _out_heads(q_out, q, shape, y_dtype, "q_out", dev)
        kd, vd = _heads(k, "k", Hk, D, dev), _heads(v, "v", Hk, D, dev)
        nd = _head_norm(norm, eps, D, dev, q_weight, q_bias, k_weight, k_bias)
        rd = _rope_desc(rope, positions, B, T, dev)
        sp = _slots(slots, B * T, dev)
        if B * T:
            _check("hdq_qkv_to_cache", _qkv_to_cache(qd, kd, vd, B, T, nd, rd, qod, sp, cache.desc(), s))
        return qo
    return _launch(dev, stream, call)


def cache_write(cache, k, v, slots, stream=None):
    """Keys and values as they are, quantized into the cache's slots
    (hdq_qkv_to_cache without queries, norm and rotation)."""
    qkv_to_cache(cache, None, k, v, slots, stream=stream)


def cache_read(cache, slots, k_out=None, v_out=None, y_dtype=DTYPE_BF16, stream=None):
    """hdq_cache_read: (keys, values) [tokens, heads, dim] of slots (int64
    [tokens]), new or k_out and v_out; slots that are not there read zeros."""
    n, dev = slots.numel(), cache.device
    shape, dt = (n, cache.heads, cache.dim), torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16
    sp = _slots(slots, n, dev)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            _operand(t, name, dt, shape, dev)

    def call(s):
        ko = slots.new_empty(shape, dtype=dt) if k_out is None else k_out
        vo = slots.new_empty(shape, dtype=dt) if v_out is None else v_out
        if n:
            _check("hdq_cache_read", lib.hdq_cache_read(cache.desc(), sp, n, ko.data_ptr(), vo.data_ptr(), y_dtype, s))
        return ko, vo
    return _launch(dev, stream, call)
