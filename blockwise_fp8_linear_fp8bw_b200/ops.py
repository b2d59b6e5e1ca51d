"""Python binding of the C ABI: the same entry points, taking torch tensors.

Argument marshalling only (tensor -> device pointer, shape -> int64, the
current CUDA stream -> cudaStream_t); every step of the computation runs in
the CUDA library. The `fp8bw_*` functions take pre-allocated outputs; the
short-named helpers allocate the outputs with torch and call them.
"""
import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _native

FP8BW_OK = 0
FP8BW_ERR_NULL = -1
FP8BW_ERR_SHAPE = -2
FP8BW_ERR_ALIGN = -3
FP8BW_ERR_DEVICE = -4
FP8BW_ERR_LAUNCH = -5
FP8BW_ERR_DEVICE_TIMEOUT = -6
FP8BW_ERR_CUDA = -7
FP8BW_ERR_ALIAS = -8
FP8BW_ERR_SCALE = -9

_lib = _native.load()

from . import _layer_binding as _fast  # noqa: E402  (built by load() if missing)


def _bind(lib):
    _fast.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
        "fp8bw_rmsnorm_quantize", "fp8bw_rmsnorm_quantize_pow2",
        "fp8bw_rmsnorm_backward_workspace", "fp8bw_rmsnorm_backward",
        "fp8bw_swiglu_quantize", "fp8bw_swiglu_quantize_pow2",
        "fp8bw_swiglu_backward_quantize", "fp8bw_swiglu_backward_quantize_pow2",
        "fp8bw_newton_schulz_workspace", "fp8bw_newton_schulz")))


_bind(_lib)


class Fp8bwError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        msg = _lib.fp8bw_status_string(status).decode()
        super().__init__("%s failed: %s (%d)" % (call, msg, status))


def _check(status: int, call: str) -> None:
    if status != FP8BW_OK:
        raise Fp8bwError(status, call)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream, dev=None):
    """The raw handle of `stream`; None means the current stream of `dev`
    (of the current device when `dev` is None). A torch stream must belong
    to `dev`."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if hasattr(stream, "cuda_stream"):
        if dev is not None and stream.device != dev:
            raise ValueError("stream is on %s, the tensors on %s"
                             % (stream.device, dev))
        return stream.cuda_stream
    return int(stream)


def _device_of(tensors):
    """The one CUDA device that holds every (non-None) tensor."""
    devs = set()
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        devs.add(t.device)
    if len(devs) != 1:
        raise ValueError("expected tensors on one CUDA device, got %s"
                         % sorted(str(d) for d in devs))
    return devs.pop()


def _call(name, tensors, stream, *args):
    """Call entry point `name` with `args` and the stream handle, on the
    device that holds `tensors`: the library launches on the current device,
    so a call for another device runs under a device guard."""
    dev = _device_of(tensors)
    handle = _stream(stream, dev)
    fn = getattr(_lib, name)
    if dev.index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    _check(status, name)


def _expect(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected %s %s, got %s %s" %
                         (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


def _cdiv(a, b):
    return (a + b - 1) // b


def _fn(name, pow2):
    """The entry point, or its power-of-two-scale variant."""
    return name + "_pow2" if pow2 else name


# ----------------------------------------------------------- raw entry points

def fp8bw_quantize_rowwise(x, q, s, stream=None, pow2=False):
    rows, cols = x.shape
    _expect(x, torch.bfloat16, (rows, cols), "x")
    _expect(q, torch.uint8, (rows, cols), "q")
    _expect(s, torch.float32, (_cdiv(cols, 128), rows), "s")
    _call(_fn('fp8bw_quantize_rowwise', pow2), (x, q, s), stream,
          _ptr(x), rows, cols, _ptr(q), _ptr(s))


def fp8bw_quantize_colwise(x, q_t, s_t, q_row=None, s_row=None, stream=None,
                           pow2=False):
    rows, cols = x.shape
    _expect(x, torch.bfloat16, (rows, cols), "x")
    _expect(q_t, torch.uint8, (cols, rows), "q_t")
    _expect(s_t, torch.float32, (_cdiv(rows, 128), cols), "s_t")
    if q_row is not None:
        _expect(q_row, torch.uint8, (rows, cols), "q_row")
        _expect(s_row, torch.float32, (_cdiv(cols, 128), rows), "s_row")
    _call(_fn('fp8bw_quantize_colwise', pow2), (x, q_t, s_t, q_row, s_row),
          stream, _ptr(x), rows, cols, _ptr(q_t), _ptr(s_t), _ptr(q_row),
          _ptr(s_row))


def fp8bw_quantize_weight_block(w, q, s, q_t=None, stream=None,
                                pow2=False):
    n, k = w.shape
    _expect(w, torch.bfloat16, (n, k), "w")
    _expect(q, torch.uint8, (n, k), "q")
    _expect(s, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "s")
    if q_t is not None:
        _expect(q_t, torch.uint8, (k, n), "q_t")
    _call(_fn('fp8bw_quantize_weight_block', pow2), (w, q, s, q_t), stream,
          _ptr(w), n, k, _ptr(q), _ptr(s), _ptr(q_t))


def fp8bw_quantize_weight_block_batch(ws, qs, ss, q_ts=None, stream=None,
                                      pow2=False):
    """Block quantisation of up to 8 weights in one launch: job i is
    fp8bw_quantize_weight_block(ws[i], qs[i], ss[i], q_ts[i])."""
    count = len(ws)
    if q_ts is None:
        q_ts = [None] * count
    if not (len(qs) == len(ss) == len(q_ts) == count):
        raise ValueError("ws, qs, ss and q_ts must have one entry per weight")
    if count == 0:
        return
    jobs = (_native.WeightBlockJob * count)()
    tensors = []
    for i, (w, q, s, q_t) in enumerate(zip(ws, qs, ss, q_ts)):
        n, k = w.shape
        _expect(w, torch.bfloat16, (n, k), "ws[%d]" % i)
        _expect(q, torch.uint8, (n, k), "qs[%d]" % i)
        _expect(s, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "ss[%d]" % i)
        if q_t is not None:
            _expect(q_t, torch.uint8, (k, n), "q_ts[%d]" % i)
        jobs[i] = _native.WeightBlockJob(_ptr(w), n, k, _ptr(q), _ptr(s), _ptr(q_t))
        tensors += [w, q, s, q_t]
    _call(_fn("fp8bw_quantize_weight_block_batch", pow2), tensors, stream,
          ctypes.cast(jobs, ctypes.c_void_p), count)


def fp8bw_gemm_fprop(qx, sx, qw, sw, y, stream=None, pow2=False):
    m, k = qx.shape
    n = qw.shape[0]
    _expect(qx, torch.uint8, (m, k), "qx")
    _expect(qw, torch.uint8, (n, k), "qw")
    _expect(sx, torch.float32, (_cdiv(k, 128), m), "sx")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(y, torch.bfloat16, (m, n), "y")
    _call(_fn('fp8bw_gemm_fprop', pow2), (qx, sx, qw, sw, y), stream,
          _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), m, n, k, _ptr(y))


def fp8bw_gemm_dgrad(qdy, sdy, qw, qw_is_transposed, sw, dx, stream=None,
                     pow2=False):
    m, n = qdy.shape
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    _expect(qdy, torch.uint8, (m, n), "qdy")
    _expect(qw, torch.uint8, (k, n) if qw_is_transposed else (n, k), "qw")
    _expect(sdy, torch.float32, (_cdiv(n, 128), m), "sdy")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(dx, torch.bfloat16, (m, k), "dx")
    _call(_fn('fp8bw_gemm_dgrad', pow2), (qdy, sdy, qw, sw, dx), stream,
          _ptr(qdy), _ptr(sdy), _ptr(qw), 1 if qw_is_transposed else 0,
          _ptr(sw), m, n, k, _ptr(dx))


def fp8bw_gemm_wgrad(qdy_t, sdy_t, qx_t, sx_t, dw, stream=None, pow2=False):
    n, m = qdy_t.shape
    k = qx_t.shape[0]
    _expect(qdy_t, torch.uint8, (n, m), "qdy_t")
    _expect(qx_t, torch.uint8, (k, m), "qx_t")
    _expect(sdy_t, torch.float32, (_cdiv(m, 128), n), "sdy_t")
    _expect(sx_t, torch.float32, (_cdiv(m, 128), k), "sx_t")
    _expect(dw, torch.bfloat16, (n, k), "dw")
    _call(_fn('fp8bw_gemm_wgrad', pow2), (qdy_t, sdy_t, qx_t, sx_t, dw),
          stream, _ptr(qdy_t), _ptr(sdy_t), _ptr(qx_t), _ptr(sx_t), m, n, k,
          _ptr(dw))


def fp8bw_gemm_wgrad_f32(qdy_t, sdy_t, qx_t, sx_t, dw, accumulate=False,
                         stream=None, pow2=False):
    n, m = qdy_t.shape
    k = qx_t.shape[0]
    _expect(qdy_t, torch.uint8, (n, m), "qdy_t")
    _expect(qx_t, torch.uint8, (k, m), "qx_t")
    _expect(sdy_t, torch.float32, (_cdiv(m, 128), n), "sdy_t")
    _expect(sx_t, torch.float32, (_cdiv(m, 128), k), "sx_t")
    _expect(dw, torch.float32, (n, k), "dw")
    _call(_fn("fp8bw_gemm_wgrad_f32", pow2), (qdy_t, sdy_t, qx_t, sx_t, dw),
          stream, _ptr(qdy_t), _ptr(sdy_t), _ptr(qx_t), _ptr(sx_t), m, n, k,
          _ptr(dw), 1 if accumulate else 0)


def _wgrad_jobs(jobs, dtype):
    """ctypes array of fp8bw_wgrad_job from (qdy_t, sdy_t, qx_t, sx_t, dw)
    tuples, and the tensors it points into."""
    arr = (_native.WgradJob * len(jobs))()
    tensors = []
    for i, (qdy_t, sdy_t, qx_t, sx_t, dw) in enumerate(jobs):
        n, m = qdy_t.shape
        k = qx_t.shape[0]
        _expect(qdy_t, torch.uint8, (n, m), "jobs[%d].qdy_t" % i)
        _expect(qx_t, torch.uint8, (k, m), "jobs[%d].qx_t" % i)
        _expect(sdy_t, torch.float32, (_cdiv(m, 128), n), "jobs[%d].sdy_t" % i)
        _expect(sx_t, torch.float32, (_cdiv(m, 128), k), "jobs[%d].sx_t" % i)
        _expect(dw, dtype, (n, k), "jobs[%d].dw" % i)
        arr[i] = _native.WgradJob(_ptr(qdy_t), _ptr(sdy_t), _ptr(qx_t),
                                  _ptr(sx_t), m, n, k, _ptr(dw))
        tensors += [qdy_t, sdy_t, qx_t, sx_t, dw]
    return arr, tensors


def fp8bw_gemm_wgrad_batch(jobs, stream=None, pow2=False):
    """Up to 4 weight gradients over the same tokens in one launch: each job
    (qdy_t, sdy_t, qx_t, sx_t, dw) is fp8bw_gemm_wgrad of its arguments (bf16
    dw)."""
    if not jobs:
        return
    arr, tensors = _wgrad_jobs(jobs, torch.bfloat16)
    _call(_fn("fp8bw_gemm_wgrad_batch", pow2), tensors, stream,
          ctypes.cast(arr, ctypes.c_void_p), len(jobs))


def fp8bw_gemm_wgrad_f32_batch(jobs, accumulate=False, stream=None,
                               pow2=False):
    """The fp32-dW form of fp8bw_gemm_wgrad_batch (each job as
    fp8bw_gemm_wgrad_f32, the same `accumulate` for all)."""
    if not jobs:
        return
    arr, tensors = _wgrad_jobs(jobs, torch.float32)
    _call(_fn("fp8bw_gemm_wgrad_f32_batch", pow2), tensors, stream,
          ctypes.cast(arr, ctypes.c_void_p), len(jobs), 1 if accumulate else 0)


def fp8bw_gemm_fprop_quant(qx, sx, qw, sw, y, qy, sy, stream=None):
    m, k = qx.shape
    n = qw.shape[0]
    _expect(qx, torch.uint8, (m, k), "qx")
    _expect(qw, torch.uint8, (n, k), "qw")
    _expect(sx, torch.float32, (_cdiv(k, 128), m), "sx")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(y, torch.bfloat16, (m, n), "y")
    _expect(qy, torch.uint8, (m, n), "qy")
    _expect(sy, torch.float32, (_cdiv(n, 128), m), "sy")
    _call("fp8bw_gemm_fprop_quant", (qx, sx, qw, sw, y, qy, sy), stream,
          _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), m, n, k, _ptr(y), _ptr(qy),
          _ptr(sy))


def fp8bw_gemm_dgrad_quant(qdy, sdy, qw, qw_is_transposed, sw, dx, qdx, sdx,
                           stream=None):
    m, n = qdy.shape
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    _expect(qdy, torch.uint8, (m, n), "qdy")
    _expect(qw, torch.uint8, (k, n) if qw_is_transposed else (n, k), "qw")
    _expect(sdy, torch.float32, (_cdiv(n, 128), m), "sdy")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(dx, torch.bfloat16, (m, k), "dx")
    _expect(qdx, torch.uint8, (m, k), "qdx")
    _expect(sdx, torch.float32, (_cdiv(k, 128), m), "sdx")
    _call("fp8bw_gemm_dgrad_quant", (qdy, sdy, qw, sw, dx, qdx, sdx), stream,
          _ptr(qdy), _ptr(sdy), _ptr(qw), 1 if qw_is_transposed else 0,
          _ptr(sw), m, n, k, _ptr(dx), _ptr(qdx), _ptr(sdx))


def fp8bw_gemm_fprop_quant_rowcol(qx, sx, qw, sw, y, qy, sy, qy_t, sy_t,
                                  stream=None):
    m, k = qx.shape
    n = qw.shape[0]
    _expect(qx, torch.uint8, (m, k), "qx")
    _expect(qw, torch.uint8, (n, k), "qw")
    _expect(sx, torch.float32, (_cdiv(k, 128), m), "sx")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(y, torch.bfloat16, (m, n), "y")
    _expect(qy, torch.uint8, (m, n), "qy")
    _expect(sy, torch.float32, (_cdiv(n, 128), m), "sy")
    _expect(qy_t, torch.uint8, (n, m), "qy_t")
    _expect(sy_t, torch.float32, (_cdiv(m, 128), n), "sy_t")
    _call("fp8bw_gemm_fprop_quant_rowcol", (qx, sx, qw, sw, y, qy, sy, qy_t, sy_t),
          stream, _ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), m, n, k, _ptr(y),
          _ptr(qy), _ptr(sy), _ptr(qy_t), _ptr(sy_t))


def fp8bw_gemm_dgrad_quant_rowcol(qdy, sdy, qw, qw_is_transposed, sw, dx, qdx,
                                  sdx, qdx_t, sdx_t, stream=None):
    m, n = qdy.shape
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    _expect(qdy, torch.uint8, (m, n), "qdy")
    _expect(qw, torch.uint8, (k, n) if qw_is_transposed else (n, k), "qw")
    _expect(sdy, torch.float32, (_cdiv(n, 128), m), "sdy")
    _expect(sw, torch.float32, (_cdiv(n, 128), _cdiv(k, 128)), "sw")
    _expect(dx, torch.bfloat16, (m, k), "dx")
    _expect(qdx, torch.uint8, (m, k), "qdx")
    _expect(sdx, torch.float32, (_cdiv(k, 128), m), "sdx")
    _expect(qdx_t, torch.uint8, (k, m), "qdx_t")
    _expect(sdx_t, torch.float32, (_cdiv(m, 128), k), "sdx_t")
    _call("fp8bw_gemm_dgrad_quant_rowcol",
          (qdy, sdy, qw, sw, dx, qdx, sdx, qdx_t, sdx_t), stream,
          _ptr(qdy), _ptr(sdy), _ptr(qw), 1 if qw_is_transposed else 0,
          _ptr(sw), m, n, k, _ptr(dx), _ptr(qdx), _ptr(sdx), _ptr(qdx_t),
          _ptr(sdx_t))


def _device_call(name, stream, device, *args):
    """Call a device-wide entry point (no tensor arguments) for one device:
    `device` if given, else the device of a torch `stream`, else the current
    device. The library works on the current device, so another device's
    call runs under a device guard."""
    if device is None and hasattr(stream, "device"):
        device = stream.device
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    if dev.type != "cuda" or dev.index is None:
        raise ValueError("expected a CUDA device with an index, got %s" % dev)
    handle = _stream(stream, dev)
    fn = getattr(_lib, name)
    if dev.index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    _check(status, name)


def fp8bw_selftest_wait_timeout(limit_ns, stream=None, device=None):
    _device_call("fp8bw_selftest_wait_timeout", stream, device, int(limit_ns))


def fp8bw_check_device_error(stream=None, device=None):
    """Synchronise `stream` and raise Fp8bwError if a kernel of the library on
    that device (`device`, else the stream's, else the current one) recorded
    an expired wait or a bad power-of-two scale since the last check."""
    # the layer operators keep a record of their own: both are read and cleared
    try:
        _device_call("fp8bw_layer_check_device_error", stream, device)
    finally:
        _device_call("fp8bw_check_device_error", stream, device)


# ----------------------------------------------------------- layer operators
# (include/fp8bw_layer.h)

_NS_COEFFS = (3.4445, -4.7750, 2.0315)


def _pad16(rows):
    return (rows + 15) // 16 * 16


def _gamma_is_f32(gamma, cols):
    if gamma.dtype not in (torch.bfloat16, torch.float32) or \
            tuple(gamma.shape) != (cols,):
        raise ValueError("gamma: expected bf16 or fp32 (%d,), got %s %s"
                         % (cols, gamma.dtype, tuple(gamma.shape)))
    return 1 if gamma.dtype == torch.float32 else 0


def _expect_2d(t, dtype, name):
    if t.dtype != dtype or len(t.shape) != 2:
        raise ValueError("%s: expected a 2-D %s tensor, got %s %s"
                         % (name, dtype, t.dtype, tuple(t.shape)))


def _expect_codes(q, s, q_t, s_t, rows, cols):
    """Codes of a [rows, cols] tensor: rows padded to a multiple of 16."""
    rp = _pad16(rows)
    for name, t, dtype, shape in (
            ("q", q, torch.uint8, (rp, cols)),
            ("s", s, torch.float32, (_cdiv(cols, 128), rp)),
            ("q_t", q_t, torch.uint8, (cols, rp)),
            ("s_t", s_t, torch.float32, (_cdiv(rp, 128), cols))):
        if t is not None:
            _expect(t, dtype, shape, name)


def fp8bw_rmsnorm_quantize(x, gamma, residual=None, eps=1e-6, h=None,
                           rstd=None, y=None, q=None, s=None, q_t=None,
                           s_t=None, stream=None, pow2=False):
    """h = bf16(x + residual) (x itself without a residual), its root-mean-
    square norm times gamma: as bf16 (y), as row-wise (q, s) and as column-wise
    codes (q_t, s_t), each if given."""
    _expect_2d(x, torch.bfloat16, "x")
    rows, cols = x.shape
    is_f32 = _gamma_is_f32(gamma, cols)
    for name, t in (("residual", residual), ("h", h), ("y", y)):
        if t is not None:
            _expect(t, torch.bfloat16, (rows, cols), name)
    if rstd is not None:
        _expect(rstd, torch.float32, (rows,), "rstd")
    _expect_codes(q, s, q_t, s_t, rows, cols)
    _call(_fn("fp8bw_rmsnorm_quantize", pow2),
          (x, gamma, residual, h, rstd, y, q, s, q_t, s_t), stream, _ptr(x),
          _ptr(residual), _ptr(gamma), is_f32, rows, cols, eps, _ptr(h),
          _ptr(rstd), _ptr(y), _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t))


def fp8bw_rmsnorm_backward(dy, h, rstd, gamma, dres, dh, dgamma, workspace,
                           stream=None):
    """dh (bf16) and dgamma (fp32) of the norm; `workspace` is a uint8 tensor
    of at least rmsnorm_backward_workspace(rows, cols) bytes."""
    _expect_2d(h, torch.bfloat16, "h")
    rows, cols = h.shape
    is_f32 = _gamma_is_f32(gamma, cols)
    for name, t in (("dy", dy), ("dres", dres), ("dh", dh)):
        if t is not None:
            _expect(t, torch.bfloat16, (rows, cols), name)
    _expect(rstd, torch.float32, (rows,), "rstd")
    _expect(dgamma, torch.float32, (cols,), "dgamma")
    _expect(workspace, torch.uint8, (workspace.numel(),), "workspace")
    _call("fp8bw_rmsnorm_backward",
          (dy, h, rstd, gamma, dres, dh, dgamma, workspace), stream, _ptr(dy),
          _ptr(h), _ptr(rstd), _ptr(gamma), is_f32, _ptr(dres), rows, cols,
          _ptr(dh), _ptr(dgamma), _ptr(workspace), workspace.numel())


def _glu_shape(gu):
    _expect_2d(gu, torch.bfloat16, "gu")
    rows, f2 = gu.shape
    if f2 % 2:
        raise ValueError("gu: expected an even number of columns, got %d" % f2)
    return rows, f2 // 2


def fp8bw_swiglu_quantize(gu, q, s, q_t=None, s_t=None, stream=None,
                          pow2=False):
    """Codes of silu(gate) * up, gu = [gate | up]."""
    rows, f = _glu_shape(gu)
    _expect_codes(q, s, q_t, s_t, rows, f)
    _call(_fn("fp8bw_swiglu_quantize", pow2), (gu, q, s, q_t, s_t), stream,
          _ptr(gu), rows, f, _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t))


def fp8bw_swiglu_backward_quantize(da, gu, q, s, q_t, s_t, stream=None,
                                   pow2=False):
    """Codes of [dgate | dup], da being the gradient of silu(gate) * up."""
    rows, f = _glu_shape(gu)
    _expect(da, torch.bfloat16, (rows, f), "da")
    _expect_codes(q, s, q_t, s_t, rows, 2 * f)
    _call(_fn("fp8bw_swiglu_backward_quantize", pow2),
          (da, gu, q, s, q_t, s_t), stream, _ptr(da), _ptr(gu), rows, f,
          _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t))


def accumulates_on_default_stream(leaf):
    """Whether a graph that is still alive has the gradient of `leaf` (a CUDA tensor)
    accumulated on its device's default stream."""
    return _fast.accumulates_on_default_stream(leaf)


def _workspace_size(name, *args):
    size = getattr(_lib, name)(*args)
    if size < 0:
        raise Fp8bwError(size, name)
    return size


def rmsnorm_backward_workspace(rows, cols):
    """Bytes of workspace that fp8bw_rmsnorm_backward needs."""
    return _workspace_size("fp8bw_rmsnorm_backward_workspace", rows, cols)


def _ns_jobs(gs, outs):
    dtype = gs[0].dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("gs: expected bf16 or fp32 tensors, got %s" % dtype)
    arr = (_native.NsJob * len(gs))()
    for i, (g, out) in enumerate(zip(gs, outs)):
        _expect_2d(g, dtype, "gs[%d]" % i)
        if out is not None:
            _expect(out, torch.bfloat16, tuple(g.shape), "outs[%d]" % i)
        arr[i] = _native.NsJob(_ptr(g), g.shape[0], g.shape[1], _ptr(out))
    return arr, 1 if dtype == torch.float32 else 0


def newton_schulz_workspace(gs):
    """Bytes of workspace that fp8bw_newton_schulz needs for `gs`."""
    if not gs:
        return 0
    arr, _ = _ns_jobs(gs, [None] * len(gs))
    return _workspace_size("fp8bw_newton_schulz_workspace",
                           ctypes.cast(arr, ctypes.c_void_p), len(gs))


def fp8bw_newton_schulz(gs, outs, workspace, steps=5, coeffs=_NS_COEFFS,
                        eps=1e-7, stream=None):
    """Orthogonalise up to 8 matrices of one dtype (bf16 or fp32) into the
    bf16 `outs`; `workspace` is a uint8 tensor of at least
    newton_schulz_workspace(gs) bytes."""
    if len(gs) != len(outs):
        raise ValueError("gs and outs must have one entry per matrix")
    if not gs:
        return
    arr, is_f32 = _ns_jobs(gs, outs)
    _expect(workspace, torch.uint8, (workspace.numel(),), "workspace")
    a, b, c = coeffs
    _call("fp8bw_newton_schulz", (*gs, *outs, workspace), stream,
          ctypes.cast(arr, ctypes.c_void_p), len(gs), is_f32, steps, a, b, c,
          eps, _ptr(workspace), workspace.numel())


# ----------------------------------------------------------- allocating helpers

_HERE = contextlib.nullcontext()


def _allocating(stream, dev):
    """Context whose allocations on `dev` belong to the stream a call runs on,
    so that memory freed on another stream is not reused under it."""
    if stream is None:
        return _HERE
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle \
            else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


class Codes(NamedTuple):
    """E4M3 codes and scales of a [rows, cols] tensor whose rows are padded to
    rp = 16 * ceil(rows / 16): row-wise q [rp, cols], s [ceil(cols/128)][rp];
    column-wise q_t [cols, rp], s_t [ceil(rp/128)][cols] (None if not asked
    for)."""
    q: torch.Tensor
    s: torch.Tensor
    q_t: Optional[torch.Tensor]
    s_t: Optional[torch.Tensor]


class NormCodes(NamedTuple):
    """Codes of a norm's output (see Codes), with what its backward pass
    needs: h (the sum that was normalised) and rstd."""
    q: torch.Tensor
    s: torch.Tensor
    q_t: Optional[torch.Tensor]
    s_t: Optional[torch.Tensor]
    h: torch.Tensor
    rstd: torch.Tensor


def _fast_call(fn, name, like, stream, *args):
    """Call `fn` of the native binding (checks, allocation and launch on the
    current stream of the tensors' device) with `stream` current."""
    if stream is None:
        r = fn(*args)
    else:
        dev = like.device
        if not like.is_cuda:
            raise ValueError("expected a CUDA tensor")
        _stream(stream, dev)            # refuses another device's stream
        with _allocating(stream, dev):
            r = fn(*args)
    if r[0] != FP8BW_OK:
        _check(r[0], name)
    return r[1:]


def rmsnorm_quantize(x, gamma, residual=None, eps=1e-6, colwise=False,
                     stream=None, pow2=False):
    """-> NormCodes of the root-mean-square norm of x (+ residual) times
    gamma; h is the bf16 sum (x itself without a residual)."""
    return NormCodes._make(_fast_call(
        _fast.rmsnorm, "fp8bw_rmsnorm_quantize", x, stream, x, gamma, residual,
        eps, True, colwise, pow2))


def rmsnorm(x, gamma, residual=None, eps=1e-6, stream=None):
    """-> (y, h, rstd): the norm's bf16 output without quantisation (for what
    is not an FP8 linear: a final norm, a router)."""
    return _fast_call(_fast.rmsnorm, "fp8bw_rmsnorm_quantize", x, stream, x,
                      gamma, residual, eps, False, False, False)


def rmsnorm_backward(dy, h, rstd, gamma, dres=None, stream=None):
    """-> (dh, dgamma): the gradient of x (and of the residual), bf16, and the
    fp32 gradient of gamma. `dres` is the gradient that reaches h directly."""
    return _fast_call(_fast.rmsnorm_backward, "fp8bw_rmsnorm_backward", h,
                      stream, dy, h, rstd, gamma, dres)


def swiglu_quantize(gu, colwise=False, stream=None, pow2=False):
    """-> Codes of silu(gate) * up, gu = [gate | up] ([rows, 2f])."""
    return Codes._make(_fast_call(_fast.swiglu, "fp8bw_swiglu_quantize", gu,
                                  stream, gu, colwise, pow2))


def swiglu_backward_quantize(da, gu, stream=None, pow2=False):
    """-> Codes (both ways) of [dgate | dup] ([rows, 2f])."""
    return Codes._make(_fast_call(
        _fast.swiglu_backward, "fp8bw_swiglu_backward_quantize", gu, stream,
        da, gu, pow2))


def newton_schulz_batch(gs, steps=5, coeffs=_NS_COEFFS, eps=1e-7, stream=None):
    """-> [bf16 orthogonalised update] for each matrix of `gs` (all bf16 or
    all fp32), up to 8 per launch; the workspace is shared by the launches."""
    gs = list(gs)
    if not gs:
        return []
    a, b, c = coeffs
    return list(_fast_call(_fast.newton_schulz, "fp8bw_newton_schulz", gs[0],
                           stream, gs, steps, a, b, c, eps))


def newton_schulz(g, steps=5, coeffs=_NS_COEFFS, eps=1e-7, stream=None):
    """-> the bf16 orthogonalised update of one matrix."""
    return newton_schulz_batch([g], steps, coeffs, eps, stream)[0]


def quantize_rowwise(x, stream=None, pow2=False):
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    s = torch.empty((_cdiv(cols, 128), rows), dtype=torch.float32,
                    device=x.device)
    fp8bw_quantize_rowwise(x, q, s, stream, pow2=pow2)
    return q, s


def quantize_colwise(x, with_rowwise=False, stream=None, pow2=False):
    """-> (q_t, s_t) or (q_t, s_t, q_row, s_row) when with_rowwise."""
    rows, cols = x.shape
    dev = x.device
    q_t = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
    s_t = torch.empty((_cdiv(rows, 128), cols), dtype=torch.float32,
                      device=dev)
    q_row = s_row = None
    if with_rowwise:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        s_row = torch.empty((_cdiv(cols, 128), rows), dtype=torch.float32,
                            device=dev)
    fp8bw_quantize_colwise(x, q_t, s_t, q_row, s_row, stream, pow2=pow2)
    return (q_t, s_t, q_row, s_row) if with_rowwise else (q_t, s_t)


def quantize_weight_block(w, transposed=True, stream=None, pow2=False):
    n, k = w.shape
    dev = w.device
    q = torch.empty((n, k), dtype=torch.uint8, device=dev)
    s = torch.empty((_cdiv(n, 128), _cdiv(k, 128)), dtype=torch.float32,
                    device=dev)
    q_t = torch.empty((k, n), dtype=torch.uint8, device=dev) if transposed \
        else None
    fp8bw_quantize_weight_block(w, q, s, q_t, stream, pow2=pow2)
    return q, s, q_t


def gemm_fprop(qx, sx, qw, sw, stream=None, pow2=False):
    y = torch.empty((qx.shape[0], qw.shape[0]), dtype=torch.bfloat16,
                    device=qx.device)
    fp8bw_gemm_fprop(qx, sx, qw, sw, y, stream, pow2=pow2)
    return y


def gemm_dgrad(qdy, sdy, qw, sw, qw_is_transposed=True, stream=None,
               pow2=False):
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    dx = torch.empty((qdy.shape[0], k), dtype=torch.bfloat16,
                     device=qdy.device)
    fp8bw_gemm_dgrad(qdy, sdy, qw, qw_is_transposed, sw, dx, stream,
                     pow2=pow2)
    return dx


def gemm_wgrad(qdy_t, sdy_t, qx_t, sx_t, stream=None, pow2=False):
    dw = torch.empty((qdy_t.shape[0], qx_t.shape[0]), dtype=torch.bfloat16,
                     device=qdy_t.device)
    fp8bw_gemm_wgrad(qdy_t, sdy_t, qx_t, sx_t, dw, stream, pow2=pow2)
    return dw


def gemm_wgrad_f32(qdy_t, sdy_t, qx_t, sx_t, main_grad=None, stream=None,
                   pow2=False):
    """fp32 dW; with `main_grad` given, dW is added into it in place and it is
    returned."""
    if main_grad is not None:
        fp8bw_gemm_wgrad_f32(qdy_t, sdy_t, qx_t, sx_t, main_grad, True, stream,
                             pow2=pow2)
        return main_grad
    dw = torch.empty((qdy_t.shape[0], qx_t.shape[0]), dtype=torch.float32,
                     device=qdy_t.device)
    fp8bw_gemm_wgrad_f32(qdy_t, sdy_t, qx_t, sx_t, dw, False, stream, pow2=pow2)
    return dw


def gemm_wgrad_batch(operands, stream=None, pow2=False):
    """-> [bf16 dW] for each (qdy_t, sdy_t, qx_t, sx_t) in `operands` (same
    token count), computed in one launch."""
    dws = [torch.empty((o[0].shape[0], o[2].shape[0]), dtype=torch.bfloat16,
                       device=o[0].device) for o in operands]
    fp8bw_gemm_wgrad_batch([tuple(o) + (dw,) for o, dw in zip(operands, dws)],
                           stream, pow2=pow2)
    return dws


def gemm_wgrad_f32_batch(operands, main_grads=None, stream=None, pow2=False):
    """fp32 dWs of fp8bw_gemm_wgrad_f32_batch; with `main_grads` given (one
    fp32 tensor per job), each dW is added into its main-grad in place and the
    main-grads are returned."""
    if main_grads is not None:
        fp8bw_gemm_wgrad_f32_batch([tuple(o) + (g,) for o, g in zip(operands, main_grads)],
                                   True, stream, pow2=pow2)
        return list(main_grads)
    dws = [torch.empty((o[0].shape[0], o[2].shape[0]), dtype=torch.float32,
                       device=o[0].device) for o in operands]
    fp8bw_gemm_wgrad_f32_batch([tuple(o) + (dw,) for o, dw in zip(operands, dws)],
                               False, stream, pow2=pow2)
    return dws


def gemm_fprop_quant(qx, sx, qw, sw, stream=None):
    """-> (y, qy, sy): the bf16 product and its row-wise quantisation."""
    m, n = qx.shape[0], qw.shape[0]
    dev = qx.device
    y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    qy = torch.empty((m, n), dtype=torch.uint8, device=dev)
    sy = torch.empty((_cdiv(n, 128), m), dtype=torch.float32, device=dev)
    fp8bw_gemm_fprop_quant(qx, sx, qw, sw, y, qy, sy, stream)
    return y, qy, sy


def gemm_dgrad_quant(qdy, sdy, qw, sw, qw_is_transposed=True, stream=None):
    """-> (dx, qdx, sdx): the bf16 product and its row-wise quantisation."""
    m = qdy.shape[0]
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    dev = qdy.device
    dx = torch.empty((m, k), dtype=torch.bfloat16, device=dev)
    qdx = torch.empty((m, k), dtype=torch.uint8, device=dev)
    sdx = torch.empty((_cdiv(k, 128), m), dtype=torch.float32, device=dev)
    fp8bw_gemm_dgrad_quant(qdy, sdy, qw, qw_is_transposed, sw, dx, qdx, sdx,
                           stream)
    return dx, qdx, sdx


def gemm_fprop_quant_rowcol(qx, sx, qw, sw, stream=None):
    """-> (y, qy, sy, qy_t, sy_t): the bf16 product with its row-wise and its
    transposed column-wise quantisation."""
    m, n = qx.shape[0], qw.shape[0]
    dev = qx.device
    y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    qy = torch.empty((m, n), dtype=torch.uint8, device=dev)
    sy = torch.empty((_cdiv(n, 128), m), dtype=torch.float32, device=dev)
    qy_t = torch.empty((n, m), dtype=torch.uint8, device=dev)
    sy_t = torch.empty((_cdiv(m, 128), n), dtype=torch.float32, device=dev)
    fp8bw_gemm_fprop_quant_rowcol(qx, sx, qw, sw, y, qy, sy, qy_t, sy_t, stream)
    return y, qy, sy, qy_t, sy_t


def gemm_dgrad_quant_rowcol(qdy, sdy, qw, sw, qw_is_transposed=True,
                            stream=None):
    """-> (dx, qdx, sdx, qdx_t, sdx_t): the bf16 product with its row-wise
    and its transposed column-wise quantisation."""
    m = qdy.shape[0]
    k = qw.shape[0] if qw_is_transposed else qw.shape[1]
    dev = qdy.device
    dx = torch.empty((m, k), dtype=torch.bfloat16, device=dev)
    qdx = torch.empty((m, k), dtype=torch.uint8, device=dev)
    sdx = torch.empty((_cdiv(k, 128), m), dtype=torch.float32, device=dev)
    qdx_t = torch.empty((k, m), dtype=torch.uint8, device=dev)
    sdx_t = torch.empty((_cdiv(m, 128), k), dtype=torch.float32, device=dev)
    fp8bw_gemm_dgrad_quant_rowcol(qdy, sdy, qw, qw_is_transposed, sw, dx, qdx,
                                  sdx, qdx_t, sdx_t, stream)
    return dx, qdx, sdx, qdx_t, sdx_t


def quantize_weight_block_batch(ws, transposed=True, stream=None, pow2=False):
    """-> [(q, s, q_t)] for each weight, all quantised in one launch."""
    out = []
    for w in ws:
        n, k = w.shape
        dev = w.device
        out.append((torch.empty((n, k), dtype=torch.uint8, device=dev),
                    torch.empty((_cdiv(n, 128), _cdiv(k, 128)), dtype=torch.float32,
                                device=dev),
                    torch.empty((k, n), dtype=torch.uint8, device=dev)
                    if transposed else None))
    fp8bw_quantize_weight_block_batch(ws, [o[0] for o in out], [o[1] for o in out],
                                      [o[2] for o in out], stream, pow2=pow2)
    return out
