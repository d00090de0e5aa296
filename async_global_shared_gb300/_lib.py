"""ctypes binding of libasyncpipe: argument marshalling only.

Every function has the C entry point's name and arguments. Buffers may be
given as torch tensors (float32, on the current CUDA device, contiguous) or as
raw integer device addresses; ``stream`` may be a ``torch.cuda.Stream``, a raw
``cudaStream_t`` integer, or None for torch's current stream. The 8-bit
block-scaled operators (``ap_rms_norm`` and those after it) take torch tensors
only: their shapes, types and row strides fill in the C call's sizes, element
types and leading dimensions. A status other than AP_OK raises :class:`APError`. Nothing here computes: every step runs in
the library's CUDA kernels, and a missing library raises instead of falling
back to anything else.
"""

from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libasyncpipe.so")

AP_OK = 0
STATUS_NAMES = {
    0: "AP_OK",
    1: "AP_ERR_NULL",
    2: "AP_ERR_SHAPE",
    3: "AP_ERR_ALIGN",
    4: "AP_ERR_ALIAS",
    5: "AP_ERR_STAGES",
    6: "AP_ERR_CLUSTER",
    7: "AP_ERR_SMEM",
    8: "AP_ERR_CUDA",
    9: "AP_ERR_DEVICE_TIMEOUT",
    10: "AP_ERR_UNSUPPORTED_DEVICE",
    11: "AP_ERR_ARG",
}
globals().update({name: code for code, name in STATUS_NAMES.items()})

AP_MIN_STAGES = 2
AP_MAX_STAGES = 6
AP_POLY_MAX_DEGREE = 1023

# ap_debug_key
AP_DBG_FORCE_PATH = 1
AP_DBG_EXPECT_TX_EXTRA = 2
AP_DBG_TIMEOUT_NS = 3
AP_DBG_STAGE_BYTES = 4
AP_DBG_GRID = 5
AP_DBG_CTAS_PER_SM = 6
AP_DBG_ROLL_STAGES = 7
AP_DBG_CONSUMER_WARPS = 8
AP_DBG_EXCHANGE_STORE = 9
AP_DBG_DEVICE_CHECKS = 11
AP_DBG_EXCHANGE_GROUP = 13
AP_DBG_STRICT_ALIGN = 14
AP_DBG_EXCHANGE_LANES = 15
AP_DBG_EXCHANGE_BATCH = 16
AP_DBG_EXCHANGE_SEND_SLOTS = 17
AP_DBG_RING_RUN = 18
AP_DBG_CONSUMER_GROUPS = 19
AP_DBG_GIVE_UP = 20
AP_DBG_LAST_PATH = 100
AP_DBG_LAST_GRID = 101
AP_DBG_LAST_STAGE_ELEMS = 102
AP_DBG_LAST_SMEM = 103
AP_DBG_LAST_STAGES = 104
AP_DBG_LAST_FLAGS = 105
AP_DBG_LAST_SITE = 106
AP_DBG_LAST_RUN = 107
AP_DBG_LAST_WARPS = 108
AP_DBG_LAST_GROUPS = 109
AP_DBG_LAST_CHAINS = 110

# Every symbol the headers under include/ declare.
EXPORTED = (
    "ap_scale",
    "ap_scale_sync",
    "ap_row_roll",
    "ap_poly",
    "ap_cluster_exchange",
    "ap_cluster_exchange_ex",
    "ap_cluster_all_to_all",
    "ap_masked_copy",
    "ap_autotune",
    "ap_autotune_reset",
    "ap_check",
    "ap_status_string",
    "ap_debug_set",
    "ap_debug_get",
    "ap_debug_emulate_ring",
    "ap_debug_emulate_ring_tensor",
    "ap_debug_fma_probe",
    "ap_debug_fma_probe_horner",
    "ap_debug_scale_pages_async",
    "ap_debug_norm_grad_ctas",
    "ap_debug_block_scale",
    "ap_rms_norm",
    "ap_rms_norm_backward",
    "ap_rms_norm_backward_workspace",
    "ap_quantize",
    "ap_matmul_fp8",
)


AP_TUNE_SCALE = 1
AP_TUNE_ROW_ROLL = 2
AP_TUNE_POLY = 3

# ap_dtype
AP_F32 = 0
AP_BF16 = 1
AP_F16 = 2


class RingShape(ctypes.Structure):
    _fields_ = [("stage_bytes", ctypes.c_int64), ("ctas_per_sm", ctypes.c_int), ("consumer_warps", ctypes.c_int),
                ("stages_per_cta", ctypes.c_int), ("consumer_groups", ctypes.c_int), ("gbs", ctypes.c_double)]


class APError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} failed: {STATUS_NAMES.get(status, status)}")


_lib = None
_f32p = ctypes.c_void_p
_i64 = ctypes.c_int64


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libasyncpipe.so (built by ``async_global_shared_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"libasyncpipe is not built ({p} missing); run `python -c \"import __graft_entry__ as g; g.build()\"`"
        )
    lib = ctypes.CDLL(p)
    vp = ctypes.c_void_p
    lib.ap_scale.argtypes = [vp, vp, _i64, _i64, ctypes.c_float, ctypes.c_int, vp]
    lib.ap_scale_sync.argtypes = [vp, vp, _i64, _i64, ctypes.c_float, vp]
    lib.ap_row_roll.argtypes = [vp, vp, _i64, _i64, _i64, vp]
    lib.ap_poly.argtypes = [vp, vp, _i64, vp, ctypes.c_int, ctypes.c_int, vp]
    lib.ap_cluster_exchange.argtypes = [vp, vp, _i64, ctypes.c_int, _i64, vp]
    lib.ap_cluster_exchange_ex.argtypes = [vp, vp, _i64, ctypes.c_int, _i64, _i64, vp]
    lib.ap_cluster_all_to_all.argtypes = [vp, vp, _i64, ctypes.c_int, _i64, vp]
    lib.ap_masked_copy.argtypes = [vp, vp, _i64, vp, ctypes.c_int, vp]
    lib.ap_autotune.argtypes = [ctypes.c_int, vp, vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(RingShape), vp]
    lib.ap_autotune_reset.argtypes = []
    lib.ap_check.argtypes = [vp]
    lib.ap_status_string.argtypes = [ctypes.c_int]
    lib.ap_status_string.restype = ctypes.c_char_p
    lib.ap_debug_set.argtypes = [ctypes.c_int, _i64]
    lib.ap_debug_get.argtypes = [ctypes.c_int]
    lib.ap_debug_get.restype = _i64
    lib.ap_debug_emulate_ring.argtypes = [vp, vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _i64]
    lib.ap_debug_fma_probe.argtypes = [vp, _i64, _i64, vp]
    lib.ap_debug_fma_probe_horner.argtypes = [vp, _i64, _i64, vp]
    lib.ap_debug_scale_pages_async.argtypes = [vp, vp, _i64, _i64, ctypes.c_float, vp]
    lib.ap_debug_emulate_ring_tensor.argtypes = [vp, vp, _i64, _i64, _i64, _i64, _i64]
    f32, i32 = ctypes.c_float, ctypes.c_int
    lib.ap_rms_norm.argtypes = [vp, _i64, i32, vp, vp, _i64, i32, vp, i32, f32, _i64, _i64, vp, _i64, vp, _i64, vp, vp, vp]
    lib.ap_rms_norm_backward.argtypes = [vp, _i64, i32, vp, _i64, i32, vp, i32, vp, vp, _i64, _i64, _i64, vp, _i64, vp,
                                         vp, vp]
    lib.ap_rms_norm_backward_workspace.argtypes = [_i64, _i64]
    lib.ap_rms_norm_backward_workspace.restype = _i64
    lib.ap_quantize.argtypes = [vp, _i64, i32, _i64, _i64, i32, vp, _i64, vp, vp, _i64, vp, vp]
    lib.ap_matmul_fp8.argtypes = [vp, _i64, vp, vp, _i64, vp, i32, vp, _i64, i32, _i64, _i64, _i64, vp]
    lib.ap_debug_norm_grad_ctas.argtypes = [_i64, _i64, i32, i32, i32, i32]
    lib.ap_debug_norm_grad_ctas.restype = _i64
    lib.ap_debug_block_scale.argtypes = [vp, vp, vp, _i64, vp]
    for name in ("ap_rms_norm", "ap_rms_norm_backward", "ap_quantize", "ap_matmul_fp8", "ap_scale", "ap_scale_sync", "ap_row_roll", "ap_poly", "ap_cluster_exchange",
                 "ap_cluster_exchange_ex", "ap_cluster_all_to_all", "ap_masked_copy", "ap_autotune", "ap_autotune_reset", "ap_check",
                 "ap_debug_set", "ap_debug_emulate_ring", "ap_debug_emulate_ring_tensor", "ap_debug_fma_probe",
                 "ap_debug_fma_probe_horner", "ap_debug_scale_pages_async", "ap_debug_block_scale"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _addr(buf) -> int | None:
    """Device-accessible address of a tensor (checked: float32, contiguous, on
    the GPU or in pinned host memory, which the GPU reads and writes over the
    host link) or an int."""
    if buf is None:
        return None
    if isinstance(buf, int):
        return buf
    if hasattr(buf, "data_ptr"):
        import torch

        if buf.dtype != torch.float32:
            raise TypeError("libasyncpipe works on float32 tensors")
        if not buf.is_cuda and not buf.is_pinned():
            raise TypeError("libasyncpipe needs CUDA tensors or pinned host tensors")
        if not buf.is_contiguous():
            raise TypeError("libasyncpipe needs contiguous tensors")
        return buf.data_ptr()
    raise TypeError(f"cannot take a device address of {type(buf).__name__}")


_cuda_available = None  # torch.cuda.is_available(), asked once


def _current_stream() -> int | None:
    """torch's current CUDA stream on the current device, as a raw handle."""
    global _cuda_available
    try:
        import torch
    except ImportError:
        return None
    if _cuda_available is None:
        _cuda_available = bool(torch.cuda.is_available())
    if not _cuda_available:
        return None
    # The raw handle without building a Stream object (about 0.3 us against
    # 3 us for current_stream() per call); the public call where a torch
    # build lacks it.
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, call: str):
    if status != AP_OK:
        raise APError(status, call)


def ap_scale(inp, out, n_tiles: int, tile_elems: int, alpha: float, stages: int, stream=None):
    _check(load().ap_scale(_addr(inp), _addr(out), n_tiles, tile_elems, alpha, stages, _stream(stream)), "ap_scale")


def ap_scale_sync(inp, out, n_tiles: int, tile_elems: int, alpha: float, stream=None):
    _check(load().ap_scale_sync(_addr(inp), _addr(out), n_tiles, tile_elems, alpha, _stream(stream)),
           "ap_scale_sync")


def ap_row_roll(A, B, rows: int, cols: int, shift: int, stream=None):
    _check(load().ap_row_roll(_addr(A), _addr(B), rows, cols, shift, _stream(stream)), "ap_row_roll")


def ap_poly(inp, out, n: int, coeffs, degree: int, stages: int, stream=None):
    """``coeffs`` is a HOST sequence of degree + 1 floats (copied by the call)."""
    c = (ctypes.c_float * max(1, len(coeffs)))(*[float(v) for v in coeffs])
    if len(coeffs) < degree + 1:
        raise ValueError("ap_poly needs degree + 1 coefficients")
    _check(load().ap_poly(_addr(inp), _addr(out), n, ctypes.cast(c, ctypes.c_void_p), degree, stages,
                          _stream(stream)), "ap_poly")


def ap_cluster_exchange(inp, out, n: int, cluster_size: int, chunk_bytes: int, stream=None):
    _check(load().ap_cluster_exchange(_addr(inp), _addr(out), n, cluster_size, chunk_bytes, _stream(stream)),
           "ap_cluster_exchange")


def ap_cluster_exchange_ex(inp, out, n: int, cluster_size: int, chunk_bytes: int, shift: int, stream=None):
    _check(load().ap_cluster_exchange_ex(_addr(inp), _addr(out), n, cluster_size, chunk_bytes, shift,
                                         _stream(stream)), "ap_cluster_exchange_ex")


def ap_cluster_all_to_all(inp, out, n: int, cluster_size: int, chunk_bytes: int, stream=None):
    _check(load().ap_cluster_all_to_all(_addr(inp), _addr(out), n, cluster_size, chunk_bytes, _stream(stream)),
           "ap_cluster_all_to_all")


def ap_masked_copy(inp, out, n_chunks: int, codes, stages: int, stream=None):
    """``codes``: a CUDA int8 tensor (or device address) of n_chunks codes."""
    if hasattr(codes, "data_ptr"):
        import torch

        if codes.dtype != torch.int8 or not codes.is_cuda or not codes.is_contiguous():
            raise TypeError("codes must be a contiguous CUDA int8 tensor")
        codes = codes.data_ptr()
    _check(load().ap_masked_copy(_addr(inp), _addr(out), n_chunks, codes, stages, _stream(stream)),
           "ap_masked_copy")


def ap_autotune(op: int, inp, out, n: int, stages: int, degree: int = 0, stream=None) -> dict:
    """Time the ring's shapes over inp/out, install the fastest; returns it."""
    shape = RingShape()
    _check(load().ap_autotune(op, _addr(inp), _addr(out), n, stages, degree, ctypes.byref(shape), _stream(stream)),
           "ap_autotune")
    return {"stage_bytes": shape.stage_bytes, "ctas_per_sm": shape.ctas_per_sm,
            "consumer_warps": shape.consumer_warps, "stages_per_cta": shape.stages_per_cta,
            "consumer_groups": shape.consumer_groups, "gbs": shape.gbs}


def ap_autotune_reset():
    _check(load().ap_autotune_reset(), "ap_autotune_reset")


def ap_check(stream=None) -> int:
    """Wait for the stream and return (not raise) the device status, then clear it."""
    return load().ap_check(_stream(stream))


def ap_status_string(status: int) -> str:
    return load().ap_status_string(status).decode()


def ap_debug_set(key: int, value: int):
    _check(load().ap_debug_set(key, value), "ap_debug_set")


def ap_debug_get(key: int) -> int:
    return load().ap_debug_get(key)


def ap_debug_emulate_ring(in_host, out_host, n: int, off: int, in_mis: int, out_mis: int, stage_elems: int) -> int:
    """Host emulation (numpy float32 arrays); returns the status code."""
    import numpy as np

    assert in_host.dtype == np.float32 and out_host.dtype == np.float32
    return load().ap_debug_emulate_ring(in_host.ctypes.data, out_host.ctypes.data, n, off, in_mis, out_mis,
                                        stage_elems)


def ap_debug_emulate_ring_tensor(in_host, out_host, rows: int, cols: int, shift: int, line_boxes: int,
                                 stage_elems: int) -> int:
    """Host emulation of the tensor-map producer's row shift (numpy float32 arrays); returns the status code."""
    import numpy as np

    assert in_host.dtype == np.float32 and out_host.dtype == np.float32
    return load().ap_debug_emulate_ring_tensor(in_host.ctypes.data, out_host.ctypes.data, rows, cols, shift,
                                               line_boxes, stage_elems)


def ap_debug_fma_probe(out, out_elems: int, iters: int, stream=None):
    _check(load().ap_debug_fma_probe(_addr(out), out_elems, iters, _stream(stream)), "ap_debug_fma_probe")


def ap_debug_fma_probe_horner(out, out_elems: int, iters: int, stream=None):
    _check(load().ap_debug_fma_probe_horner(_addr(out), out_elems, iters, _stream(stream)),
           "ap_debug_fma_probe_horner")


def ap_debug_scale_pages_async(inp, out, n_tiles: int, tile_elems: int, alpha: float, stream=None):
    _check(load().ap_debug_scale_pages_async(_addr(inp), _addr(out), n_tiles, tile_elems, alpha, _stream(stream)),
           "ap_debug_scale_pages_async")


def ap_debug_norm_grad_ctas(rows: int, cols: int, type: int, residual_type: int, dresidual: bool, sms: int) -> int:
    return load().ap_debug_norm_grad_ctas(rows, cols, type, residual_type, int(dresidual), sms)


def ap_debug_block_scale(amax, scale, inv, n: int, stream=None):
    _check(load().ap_debug_block_scale(_addr(amax), _addr(scale), _addr(inv), n, _stream(stream)), "ap_debug_block_scale")


# ------------------------------------------------------------------ 8-bit block-scaled operators
#
# These calls are made once a layer and token, so their checks are written for
# few attribute look-ups: one look at a tensor's device, shape, strides, type
# and address each.

SCALE_BLOCK = 128  # values of a row that share a scale

_DTYPES = None  # torch dtype -> ap_dtype; the dtypes that hold e4m3 codes; the current device's number; float32


def _dtypes():
    global _DTYPES
    if _DTYPES is None:
        import torch

        _DTYPES = ({torch.float32: AP_F32, torch.bfloat16: AP_BF16, torch.float16: AP_F16},
                   (torch.float8_e4m3fn, torch.uint8), torch._C._cuda_getDevice, torch.float32)
    return _DTYPES


def _device(t, name: str) -> int:
    """The device of a call's first tensor, which must be the current one."""
    dev = t.get_device()  # -1 for a host tensor
    if dev < 0 or dev != _dtypes()[2]():
        raise TypeError(f"{name} must be a tensor on the current CUDA device")
    return dev


def _where(t, name: str, dev: int):
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on the current CUDA device")


def _kind(t, name: str) -> int:
    kind = _DTYPES[0].get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return kind


def _matrix(t, name: str, shape, dev: int) -> int:
    """Leading dimension of a matrix of this shape with unit column stride, on this device."""
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on the current CUDA device")
    if t.shape != shape:
        raise ValueError(f"{name} must be a matrix of shape {tuple(shape)}, got {tuple(t.shape)}")
    rows, cols = shape
    ld, col_stride = t.stride()
    if rows <= 1:
        # a single row's stride is never used: give one its columns fit in and
        # that the 16-byte rule of the products accepts
        ld = -(-cols // 16) * 16
    elif ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    if col_stride != 1 and cols > 1:
        raise ValueError(f"{name} must have a column stride of 1")
    return ld


def _codes(t, name: str, shape, dev: int) -> int:
    if t.dtype not in _DTYPES[1]:
        raise TypeError(f"{name} must be float8_e4m3fn (or uint8 codes), got {t.dtype}")
    return _matrix(t, name, shape, dev)


def _floats(t, name: str, shape, dev: int) -> int:
    """Address of a contiguous float32 tensor of this shape."""
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on the current CUDA device")
    if t.dtype != _DTYPES[3] or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _weight(t, cols: int, dev: int) -> int:
    _where(t, "weight", dev)
    if t.shape != (cols,) or not t.is_contiguous():
        raise ValueError(f"weight must be a contiguous vector of {cols}, got {tuple(t.shape)}")
    return _kind(t, "weight")


def _shape2(t, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(shape)}")
    return shape


def ap_rms_norm(x, weight, eps: float, y=None, q=None, q_scales=None, residual=None, residual_out=None, rstd=None,
                stream=None):
    """h = x + residual; r = 1 / sqrt(mean(h^2) + eps); y = h * r * weight over each row of x (rows x cols).

    ``y``: the output in x's type; ``q`` (float8_e4m3fn or uint8) and ``q_scales`` (float32, rows x ceil(cols / 128)):
    the output in 8 bits. ``residual`` and ``residual_out`` (the same tensor for in place) are of x's type or float32
    and share a row stride; ``rstd`` receives r, which the gradient needs."""
    dev = _device(x, "x")
    shape = _shape2(x, "x")
    rows, cols = shape
    ldx = _matrix(x, "x", shape, dev)
    rtype = kind = _kind(x, "x")
    res = out = yp = qp = sp = rp = None
    ldr = ldy = ldq = cols
    if residual is not None:
        if residual_out is None:
            raise ValueError("residual needs residual_out (the same tensor for in place)")
        ldr = _matrix(residual, "residual", shape, dev)
        rtype = _kind(residual, "residual")
        res = out = residual.data_ptr()
        if residual_out is not residual:
            if residual_out.dtype != residual.dtype or _matrix(residual_out, "residual_out", shape, dev) != ldr:
                raise ValueError("residual_out must match residual in type and row stride")
            out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    if y is not None:
        ldy = _matrix(y, "y", shape, dev)
        if y.dtype != x.dtype:
            raise TypeError("y must have x's type")
        yp = y.data_ptr()
    if q is not None:
        if q_scales is None:
            raise ValueError("q needs q_scales")
        ldq = _codes(q, "q", shape, dev)
        qp = q.data_ptr()
    if q_scales is not None:
        sp = _floats(q_scales, "q_scales", (rows, (cols + 127) // 128), dev)
    if rstd is not None:
        rp = _floats(rstd, "rstd", (rows,), dev)
    wtype = _weight(weight, cols, dev)
    status = (_lib or load()).ap_rms_norm(x.data_ptr(), ldx, kind, res, out, ldr, rtype, weight.data_ptr(), wtype, eps, rows,
                                          cols, yp, ldy, qp, ldq, sp, rp, _stream(stream))
    if status:
        raise APError(status, "ap_rms_norm")


def ap_rms_norm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace ap_rms_norm_backward needs for these sizes."""
    size = (_lib or load()).ap_rms_norm_backward_workspace(rows, cols)
    if size < 0:
        raise APError(2, "ap_rms_norm_backward_workspace")
    return size


def ap_rms_norm_backward(dy, h, weight, rstd, dx, dweight=None, workspace=None, dresidual=None, stream=None):
    """Gradient of ap_rms_norm: ``dx`` (of h's type, the gradient of x and of residual) and ``dweight`` (float32).

    ``h``: the forward call's residual_out, or its x where there was no residual; ``dresidual``: a gradient of h from
    elsewhere, added to dx; ``workspace``: a contiguous uint8 tensor of at least ap_rms_norm_backward_workspace(rows,
    cols) bytes, needed with dweight."""
    dev = _device(dy, "dy")
    shape = _shape2(dy, "dy")
    rows, cols = shape
    lddy, ldh, lddx = _matrix(dy, "dy", shape, dev), _matrix(h, "h", shape, dev), _matrix(dx, "dx", shape, dev)
    kind, rtype = _kind(dy, "dy"), _kind(h, "h")
    if dx.dtype != h.dtype:
        raise TypeError("dx must have h's type")
    dp = wp = sp = None
    lddr = cols
    if dresidual is not None:
        lddr = _matrix(dresidual, "dresidual", shape, dev)
        if dresidual.dtype != h.dtype:
            raise TypeError("dresidual must have h's type")
        dp = dresidual.data_ptr()
    if dweight is not None:
        wp = _floats(dweight, "dweight", (cols,), dev)
    if workspace is not None:
        _where(workspace, "workspace", dev)
        if not workspace.is_contiguous() or (
                wp is not None and workspace.nbytes < ap_rms_norm_backward_workspace(rows, cols)):
            raise ValueError(f"workspace must be contiguous, of at least {ap_rms_norm_backward_workspace(rows, cols)} bytes")
        sp = workspace.data_ptr()
    wtype = _weight(weight, cols, dev)
    status = (_lib or load()).ap_rms_norm_backward(
        dy.data_ptr(), lddy, kind, h.data_ptr(), ldh, rtype, weight.data_ptr(), wtype, _floats(rstd, "rstd", (rows,), dev), dp,
        lddr, rows, cols, dx.data_ptr(), lddx, wp, sp, _stream(stream))
    if status:
        raise APError(status, "ap_rms_norm_backward")


def ap_quantize(x, block_rows: int, q=None, scales=None, qt=None, scales_t=None, stream=None):
    """e4m3 codes and scales of x (rows x cols): ``q`` and ``scales`` as it stands, ``qt`` and ``scales_t`` transposed.

    ``block_rows`` 1: a scale for 128 consecutive values of a row of the output (scales rows x ceil(cols / 128),
    scales_t cols x ceil(rows / 128)); 128: a scale for each 128 x 128 tile."""
    dev = _device(x, "x")
    shape = _shape2(x, "x")
    rows, cols = shape
    ldx = _matrix(x, "x", shape, dev)
    kind = _kind(x, "x")
    tile = block_rows if block_rows == 1 or block_rows == 128 else 1  # other values are the library's to refuse
    ldq, ldqt = cols, rows
    qp = sp = qtp = stp = None
    if q is not None:
        if scales is None:
            raise ValueError("q needs scales")
        ldq = _codes(q, "q", shape, dev)
        qp = q.data_ptr()
    if scales is not None:
        sp = _floats(scales, "scales", ((rows + tile - 1) // tile, (cols + 127) // 128), dev)
    if qt is not None:
        if scales_t is None:
            raise ValueError("qt needs scales_t")
        ldqt = _codes(qt, "qt", (cols, rows), dev)
        qtp = qt.data_ptr()
    if scales_t is not None:
        stp = _floats(scales_t, "scales_t", ((cols + tile - 1) // tile, (rows + 127) // 128), dev)
    status = (_lib or load()).ap_quantize(x.data_ptr(), ldx, kind, rows, cols, block_rows, qp, ldq, sp, qtp, ldqt, stp,
                                          _stream(stream))
    if status:
        raise APError(status, "ap_quantize")


def ap_matmul_fp8(a, a_scales, b, b_scales, c, b_block_rows: int = SCALE_BLOCK, stream=None):
    """c = a * b^T of e4m3 matrices: a (m x k) scaled by row blocks, b (n x k) by 128 x 128 tiles (``b_block_rows`` 128)
    or by row blocks (1), c (m x n) float32, bfloat16 or float16. Rows of a and b start on 16-byte boundaries."""
    dev = _device(a, "a")
    m, k = _shape2(a, "a")
    n, kb = _shape2(b, "b")
    if k != kb:
        raise ValueError(f"shapes do not match: a {tuple(a.shape)}, b {tuple(b.shape)}")
    lda, ldb, ldc = _codes(a, "a", a.shape, dev), _codes(b, "b", b.shape, dev), _matrix(c, "c", (m, n), dev)
    kind = _kind(c, "c")
    tile = b_block_rows if b_block_rows == 1 or b_block_rows == 128 else 1
    blocks = (k + 127) // 128
    status = (_lib or load()).ap_matmul_fp8(
        a.data_ptr(), lda, _floats(a_scales, "a_scales", (m, blocks), dev), b.data_ptr(), ldb,
        _floats(b_scales, "b_scales", ((n + tile - 1) // tile, blocks), dev), b_block_rows, c.data_ptr(), ldc, kind, m, n, k,
        _stream(stream))
    if status:
        raise APError(status, "ap_matmul_fp8")
