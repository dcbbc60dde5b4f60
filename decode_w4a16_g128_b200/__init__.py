"""Python binding of libw4a16.so, the B200 W4A16 group-128 linear layer.

Marshalling only: every function below checks tensor metadata, passes raw
device pointers and the current CUDA stream to the C ABI declared in
``include/w4a16.h`` and turns a non-zero status into ``W4A16Error``.  All
arithmetic runs in the library's CUDA kernels; there is no fallback, and
importing this package fails loudly when the shared library has not been
built (``python decode_w4a16_g128_b200/build.py``).

Tensors: ``x`` bf16 [M, K]; ``wq`` int32/uint32 [N, K/8] (eight 4-bit codes
per word, low nibble first); ``scales``/``biases`` bf16 [N, K/128]; the result
``y`` is bf16 [M, N].  All on the same CUDA device, contiguous.

With ``stream``, the work runs on that stream, behind what is on it alone: the
caller orders it behind the work that makes the inputs, and uses of the outputs
behind it.  New outputs are then that stream's memory, and every tensor of the
call may be dropped before its work is done.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libw4a16.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_CUDA = 4
ERR_NO_MEMORY = 5
ERR_DEVICE = 6
ERR_TIMEOUT = 7

PATH_AUTO = 0
PATH_MATVEC = 1
PATH_GEMM = 2
PATH_MATVEC_ROWS = 3

DTYPE_F32 = 0
DTYPE_BF16 = 1

FLAG_NO_PDL = 1
FLAG_STATIC_WEIGHTS = 2
FLAG_TEST_DROP_COPY = 4


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("splits", ctypes.c_int32), ("workers", ctypes.c_int32),
                ("sm_count", ctypes.c_int32), ("flags", ctypes.c_int32), ("row_blocks", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 2)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("splits", ctypes.c_int32), ("grid_x", ctypes.c_int32),
                ("grid_y", ctypes.c_int32), ("grid_z", ctypes.c_int32), ("block", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("cluster", ctypes.c_int32), ("tiles", ctypes.c_int64),
                ("units", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64), ("row_blocks", ctypes.c_int32),
                ("slices", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError(f"{LIBRARY_PATH} is missing: build it with "
                          "`python decode_w4a16_g128_b200/build.py` (needs nvcc)")
    lib = ctypes.CDLL(LIBRARY_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.w4a16_matmul.argtypes = [p, p, p, p, p, i64, i64, i64, p]
    lib.w4a16_matmul_ex.argtypes = [p, p, p, p, p, i64, i64, i64, p, ctypes.POINTER(Options)]
    lib.w4a16_matmul_last_rows.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p]
    lib.w4a16_plan.argtypes = [i64, i64, i64, ctypes.POINTER(Options), ctypes.POINTER(PlanInfo)]
    lib.w4a16_device_status.argtypes = [p]
    lib.w4a16_release.argtypes = []
    lib.w4a16_release.restype = None
    lib.w4a16_status_string.argtypes = [i32]
    lib.w4a16_status_string.restype = ctypes.c_char_p
    lib.w4a16_last_cuda_error.argtypes = []
    lib.w4a16_version.argtypes = []
    lib.w4a16_streamk_owner.argtypes = [i64, i64, i64]
    lib.w4a16_streamk_owner.restype = i64
    lib.w4a16_matvec_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, p]
    lib.w4a16_quantize.argtypes = [p, ctypes.c_int32, p, p, p, i64, i64, p]
    lib.w4a16_gate_up.argtypes = [p, p, p, p, p, i64, i64, i64, p]
    lib.w4a16_matmul_bits.argtypes = [p, p, p, p, p, i64, i64, i64, ctypes.c_int32, p]
    lib.w4a16_mx_quantize.argtypes = [p, ctypes.c_int32, p, p, i64, i64, p]
    lib.w4a16_mx_dequantize.argtypes = [p, p, p, ctypes.c_int32, i64, i64, p]
    lib.w4a16_mx_matmul.argtypes = [p, p, p, p, i64, i64, i64, p]
    lib.w4a16_mx_matmul_a4.argtypes = [p, p, p, p, p, i64, i64, i64, p]
    lib.w4a16_mx_gate_up.argtypes = [p, p, p, p, i64, i64, i64, p]
    lib.w4a16_mx_matmul_backward.argtypes = [p, p, p, p, i64, i64, i64, p]
    lib.w4a16_mx_gate_up_backward.argtypes = [p, p, p, p, p, p, i64, i64, i64, p]
    for name in ("w4a16_matmul", "w4a16_matmul_ex", "w4a16_matmul_last_rows", "w4a16_plan",
                 "w4a16_device_status", "w4a16_last_cuda_error", "w4a16_version", "w4a16_matvec_noalloc",
                 "w4a16_quantize", "w4a16_gate_up", "w4a16_matmul_bits", "w4a16_mx_quantize", "w4a16_mx_dequantize",
                 "w4a16_mx_matmul", "w4a16_mx_matmul_a4", "w4a16_mx_gate_up", "w4a16_mx_matmul_backward",
                 "w4a16_mx_gate_up_backward"):
        getattr(lib, name).restype = i32
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.w4a16_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise W4A16Error(status, where)


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _side_stream(stream, device):
    """A stream that was given as torch's, or None where it is the device's current one."""
    import torch
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == 1:                    # the other name of the default stream, which torch calls 0
        handle = 0
    if handle == torch._C._cuda_getCurrentRawStream(device):
        return None
    if handle == 0:                    # for torch a stream without a handle is a new one
        return torch.cuda.default_stream(device)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device)


def _empty_on(stream, device, like, shape, dtype):
    """A new output for work on a stream that was given, on the device of `like`.  Memory of the current
    stream would not do: what it hands out may be memory that was freed there with work in front of it
    still pending, which the given stream does not wait for.  So the block comes from the given stream's
    memory, and is not reused there before the current stream, on which the caller may use it, has come
    past its end."""
    import torch
    side = _side_stream(stream, device)
    if side is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(side):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _keep_for(stream, device, *tensors):
    """The tensors' memory is not reused before work on a stream that was given is done with it."""
    side = _side_stream(stream, device)
    if side is not None:
        for t in tensors:
            t.record_stream(side)


def _new(like, shape, dtype, stream):
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    return _empty_on(stream, like.get_device(), like, shape, dtype)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check_tensors(x, wq, scales, biases, y):
    import torch
    if x.dtype != torch.bfloat16 or scales.dtype != torch.bfloat16 or biases.dtype != torch.bfloat16:
        raise TypeError("x, scales and biases must be bfloat16")
    if wq.dtype not in (torch.int32, torch.uint32):
        raise TypeError("wq must be int32 or uint32 (packed codes)")
    for name, t in (("x", x), ("wq", wq), ("scales", scales), ("biases", biases)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    M, K = x.shape
    N = wq.shape[0]
    if tuple(wq.shape) != (N, K // 8) or tuple(scales.shape) != (N, K // 128) or \
            tuple(biases.shape) != (N, K // 128):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, wq {tuple(wq.shape)}, "
                         f"scales {tuple(scales.shape)}, biases {tuple(biases.shape)}")
    if y is not None and (y.dtype != torch.bfloat16 or not y.is_cuda or not y.is_contiguous()):
        raise ValueError("y must be a contiguous bfloat16 CUDA tensor")
    return M, N, K


def w4a16_matmul(x, wq, scales, biases, y=None, stream=None):
    """y = x . dequant(wq)^T on the current (or given) CUDA stream; returns y."""
    import torch
    M, N, K = _check_tensors(x, wq, scales, biases, y)
    if y is None:
        y = _new(x, (M, N), torch.bfloat16, stream)
    elif tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    _check(lib.w4a16_matmul(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(y), M, N, K,
                            _stream_handle(stream)), "w4a16_matmul")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, y)
    return y


def make_options(path=PATH_AUTO, splits=0, workers=0, sm_count=0, flags=0, row_blocks=0) -> Options:
    return Options(int(path), int(splits), int(workers), int(sm_count), int(flags), int(row_blocks))


def w4a16_matmul_ex(x, wq, scales, biases, y=None, stream=None, path=PATH_AUTO, splits=0, workers=0,
                    flags=0, row_blocks=0):
    """w4a16_matmul with a forced path / split count / worker count / row blocks per CTA."""
    import torch
    M, N, K = _check_tensors(x, wq, scales, biases, y)
    if y is None:
        y = _new(x, (M, N), torch.bfloat16, stream)
    elif tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    opt = make_options(path, splits, workers, 0, flags, row_blocks)
    _check(lib.w4a16_matmul_ex(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(y), M, N, K,
                               _stream_handle(stream), ctypes.byref(opt)), "w4a16_matmul_ex")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, y)
    return y


def w4a16_matmul_last_rows(x, wq, scales, biases, keep: int, y=None, stream=None):
    """Project only the last ``keep`` rows of x (0 = every row); returns y [keep, N]."""
    import torch
    M, N, K = _check_tensors(x, wq, scales, biases, None)
    rows = M if keep == 0 else keep
    if y is None:
        y = _new(x, (rows, N), torch.bfloat16, stream)
    elif tuple(y.shape) != (rows, N):
        raise ValueError("y must be [keep, N]")
    _check(lib.w4a16_matmul_last_rows(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(y), M,
                                      int(keep), N, K, _stream_handle(stream)),
           "w4a16_matmul_last_rows")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, y)
    return y


NOALLOC_MAX_N = 1048576


def w4a16_matvec_noalloc(x, wq, scales, biases, y, stream=None):
    """The matvec (M <= 8) without any allocation, for callers that cannot allocate
    device memory: its split-row scratch is a fixed array inside the library, so
    calls that can overlap on the GPU must be serialised.  y must be given."""
    M, N, K = _check_tensors(x, wq, scales, biases, y)
    if tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    _check(lib.w4a16_matvec_noalloc(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(y), M, N, K,
                                    _stream_handle(stream)), "w4a16_matvec_noalloc")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, y)
    return y


def interleave_gate_up(gate, up):
    """Row-interleave a gate and an up tensor [N2, ...] (codes, scales or biases of the two
    layers) in blocks of 8, the weight layout w4a16_gate_up reads (layout only)."""
    import torch
    if gate.shape != up.shape or gate.shape[0] % 8:
        raise ValueError("gate and up need the same shape and a row count divisible by 8")
    n2 = gate.shape[0]
    return torch.stack([gate.reshape(n2 // 8, 8, -1), up.reshape(n2 // 8, 8, -1)], dim=1).reshape(2 * n2, -1)


def w4a16_gate_up(x, wq, scales, biases, h=None, stream=None):
    """Fused gate/up projection, M <= 8: h [M, N2] = bf16(silu(x . gate^T) * (x . up^T)) with the
    two layers' rows interleaved in blocks of 8 in wq, scales and biases (2 N2 rows)."""
    import torch
    M, N, K = _check_tensors(x, wq, scales, biases, h)
    if N % 16:
        raise ValueError("the interleaved gate/up rows come in blocks of 16")
    N2 = N // 2
    if h is None:
        h = _new(x, (M, N2), torch.bfloat16, stream)
    elif tuple(h.shape) != (M, N2):
        raise ValueError("h must be [M, N2]")
    _check(lib.w4a16_gate_up(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(h), M, N2, K,
                             _stream_handle(stream)), "w4a16_gate_up")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, h)
    return h


def w4a16_matmul_bits(x, wq, scales, biases, bits: int, y=None, stream=None):
    """y = x . dequant(wq)^T with b-bit codes (b = 2, 4 or 8): wq int32/uint32 [N, K b / 32], 32 / b
    codes per word, the lowest code in the lowest bits.  2 and 8 bits: M <= 32."""
    import torch
    if bits not in (2, 4, 8):
        raise W4A16Error(ERR_UNSUPPORTED, "w4a16_matmul_bits")
    if x.dtype != torch.bfloat16 or scales.dtype != torch.bfloat16 or biases.dtype != torch.bfloat16:
        raise TypeError("x, scales and biases must be bfloat16")
    if wq.dtype not in (torch.int32, torch.uint32):
        raise TypeError("wq must be int32 or uint32 (packed codes)")
    for name, t in (("x", x), ("wq", wq), ("scales", scales), ("biases", biases)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    M, K = x.shape
    N = wq.shape[0]
    if tuple(wq.shape) != (N, K * bits // 32) or tuple(scales.shape) != (N, K // 128) or \
            tuple(biases.shape) != (N, K // 128):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, wq {tuple(wq.shape)}, "
                         f"scales {tuple(scales.shape)}, biases {tuple(biases.shape)} for {bits}-bit codes")
    if y is None:
        y = _new(x, (M, N), torch.bfloat16, stream)
    elif tuple(y.shape) != (M, N) or y.dtype != torch.bfloat16 or not y.is_cuda or not y.is_contiguous():
        raise ValueError("y must be a contiguous bfloat16 CUDA tensor [M, N]")
    _check(lib.w4a16_matmul_bits(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(y), M, N, K, int(bits),
                                 _stream_handle(stream)), "w4a16_matmul_bits")
    if stream is not None:
        _keep_for(stream, x.get_device(), x, wq, scales, biases, y)
    return y


def w4a16_quantize(w, wq=None, scales=None, biases=None, stream=None):
    """Quantise weights W [N, K] (float32 or bfloat16, CUDA, contiguous) on the GPU into the
    packed format: returns (wq int32 [N, K/8], scales bf16 [N, K/128], biases bf16 [N, K/128])."""
    import torch
    if w.dim() != 2 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous 2-D CUDA tensor")
    if w.dtype == torch.float32:
        dt = DTYPE_F32
    elif w.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    else:
        raise TypeError("w must be float32 or bfloat16")
    N, K = w.shape
    if K % 128:
        raise W4A16Error(ERR_UNSUPPORTED, "w4a16_quantize")
    if wq is None:
        wq = _new(w, (N, K // 8), torch.int32, stream)
    if scales is None:
        scales = _new(w, (N, K // 128), torch.bfloat16, stream)
    if biases is None:
        biases = _new(w, (N, K // 128), torch.bfloat16, stream)
    if tuple(wq.shape) != (N, K // 8) or tuple(scales.shape) != (N, K // 128) or tuple(biases.shape) != (N, K // 128):
        raise ValueError("output shapes must be [N, K/8], [N, K/128], [N, K/128]")
    _check(lib.w4a16_quantize(_ptr(w), dt, _ptr(wq), _ptr(scales), _ptr(biases), N, K, _stream_handle(stream)),
           "w4a16_quantize")
    if stream is not None:
        _keep_for(stream, w.get_device(), w, wq, scales, biases)
    return wq, scales, biases


# ---------------------------------------------------------------- MXFP4 (microscaled 4-bit float)
#
# wq int32/uint32 [N, K/8] codes and scales uint8 [N, K/32], as in include/w4a16.h.  Tensors are
# contiguous and on one CUDA device, which need not be the current one; outputs that are not given
# are allocated there.  A decode loop runs these functions for every token, so each looks at what it
# was given in one expression, and only a call that fails it goes on to find out why.
#
# The C functions take scales that start on 16 bytes, which rows cut out of a larger array (a shard, the
# last token of a quantised prompt) seldom do, as a row has K/32 of them.  Such scales are copied first, by
# every call: a program that uses them often clones them once.  Scales to be written have to be aligned.

MX_BLOCK = 32

_torch = None            # torch and what the checks compare with, bound by the first call
_Tensor = _bf16 = _f32 = _i32 = _u32 = _u8 = None


def _mx_setup():
    global _torch, _Tensor, _bf16, _f32, _i32, _u32, _u8
    import torch
    _Tensor = torch.Tensor
    _bf16, _f32, _i32, _u32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint32, torch.uint8
    _torch = torch


def _mx_ok(t, dtype, rows, cols, device):
    """A contiguous CUDA matrix of this type and shape on this device (by index)."""
    return t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == device and t.is_contiguous()


def _mx_refuse(name, t, dtypes, shape, device=None):
    """Raises if a tensor is not what its function needs, and says why."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device} like the first argument")


def _mx_rows(name, t):
    """Rows, columns and device of the first argument, bfloat16."""
    if _torch is None:
        _mx_setup()
    if isinstance(t, _Tensor) and t.dtype is _bf16 and t.is_contiguous():
        shape, device = t.shape, t.get_device()
        if len(shape) == 2 and device >= 0:
            return shape[0], shape[1], device
    _mx_refuse(name, t, (_bf16,), None)


def _mx_stored(codes, scales, K, device, names=("wq", "scales")):
    """Rows N and device of stored codes [N, K/8] with their scales [N, K/32]; K and the device
    (by index) are those of the first argument, or None where that is `codes`."""
    if _torch is None:
        _mx_setup()
    if isinstance(codes, _Tensor) and (codes.dtype is _i32 or codes.dtype is _u32) and codes.is_contiguous():
        shape, on = codes.shape, codes.get_device()
        if len(shape) == 2 and on >= 0:
            N, words = shape
            if (K is None or words * 8 == K and on == device) and words % 4 == 0 and isinstance(scales, _Tensor) and (
                    _mx_ok(scales, _u8, N, words // 4, on)):
                return N, words * 8, on
    if K is None:
        _mx_refuse(names[0], codes, (_i32, _u32), None)
        K, device = codes.shape[1] * 8, codes.get_device()
    if K % MX_BLOCK:
        raise W4A16Error(ERR_UNSUPPORTED, f"rows of {K} values: K must be a multiple of {MX_BLOCK}")
    N = codes.shape[0] if isinstance(codes, _Tensor) and codes.dim() == 2 else 0
    _mx_refuse(names[0], codes, (_i32, _u32), (N, K // 8), device)
    _mx_refuse(names[1], scales, (_u8,), (N, K // MX_BLOCK), device)


def _mx_out(name, t, like, dtype, rows, cols, device, stream):
    """A given output, checked, or a new one."""
    if t is None:
        if stream is None:
            t = like.new_empty((rows, cols)) if dtype is like.dtype else like.new_empty((rows, cols), dtype=dtype)
        else:
            t = _empty_on(stream, device, like, (rows, cols), dtype)
    elif not (isinstance(t, _Tensor) and (_mx_ok(t, dtype, rows, cols, device) or (
            dtype is _i32 and _mx_ok(t, _u32, rows, cols, device)))):
        _mx_refuse(name, t, (_i32, _u32) if dtype is _i32 else (dtype,), (rows, cols), device)
    return t


def _mx_aligned(scales, device, stream):
    """A copy, on the call's stream, of scales that do not start on 16 bytes."""
    side = None if stream is None else _side_stream(stream, device)
    if side is None:
        return scales.clone()
    with _torch.cuda.stream(side):
        return scales.clone()


def _mx_run(fn, device, stream, *args):
    """Calls a C entry point on `device`, made current for the call, and its stream."""
    if stream is None:
        handle = _torch._C._cuda_getCurrentRawStream(device)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if device == _torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with _torch.cuda.device(device):
            status = fn(*args, handle)
    if status != OK:
        raise W4A16Error(status, fn.__name__)


def w4a16_mx_quantize(w, wq=None, scales=None, stream=None):
    """Quantise w [N, K] (float32 or bfloat16: weights, or activations for w4a16_mx_matmul_a4) to
    MXFP4: returns (wq int32 [N, K/8], scales uint8 [N, K/32])."""
    if _torch is None:
        _mx_setup()
    if not (isinstance(w, _Tensor) and (w.dtype is _bf16 or w.dtype is _f32) and w.is_contiguous() and w.dim() == 2
            and w.is_cuda):
        _mx_refuse("w", w, (_f32, _bf16), None)
    (N, K), device = w.shape, w.get_device()
    if K % MX_BLOCK:
        raise W4A16Error(ERR_UNSUPPORTED, "w4a16_mx_quantize")
    wq = _mx_out("wq", wq, w, _i32, N, K // 8, device, stream)
    scales = _mx_out("scales", scales, w, _u8, N, K // MX_BLOCK, device, stream)
    _mx_run(lib.w4a16_mx_quantize, device, stream, w.data_ptr(), DTYPE_F32 if w.dtype is _f32 else DTYPE_BF16,
            wq.data_ptr(), scales.data_ptr(), N, K)
    if stream is not None:
        _keep_for(stream, device, w, wq, scales)
    return wq, scales


def w4a16_mx_dequantize(wq, scales, w=None, dtype=None, stream=None):
    """The values of stored codes [N, K], bfloat16 (default) or float32; both hold them exactly."""
    N, K, device = _mx_stored(wq, scales, None, None)
    if dtype is None:
        dtype = _bf16 if w is None else w.dtype
    if dtype is not _f32 and dtype is not _bf16:
        raise TypeError("values come in float32 or bfloat16")
    w = _mx_out("w", w, wq, dtype, N, K, device, stream)
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_dequantize, device, stream, wq.data_ptr(), ws, w.data_ptr(),
            DTYPE_F32 if dtype is _f32 else DTYPE_BF16, N, K)
    if stream is not None:
        _keep_for(stream, device, wq, scales, w)
    return w


def w4a16_mx_matmul(x, wq, scales, y=None, stream=None):
    """y [M, N] = x . W^T for W in MXFP4; x and y bfloat16, any M."""
    M, K, device = _mx_rows("x", x)
    N = _mx_stored(wq, scales, K, device)[0]
    y = _mx_out("y", y, x, _bf16, M, N, device, stream)
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_matmul, device, stream, x.data_ptr(), wq.data_ptr(), ws, y.data_ptr(), M, N, K)
    if stream is not None:
        _keep_for(stream, device, x, wq, scales, y)
    return y


def w4a16_mx_matmul_a4(xq, xscales, wq, scales, y=None, stream=None):
    """y [M, N] = X . W^T with both operands in MXFP4 (X from w4a16_mx_quantize of the activations)."""
    M, K, device = _mx_stored(xq, xscales, None, None, ("xq", "xscales"))
    N = _mx_stored(wq, scales, K, device)[0]
    y = _mx_out("y", y, xq, _bf16, M, N, device, stream)
    xs = xscales.data_ptr()
    if xs & 15:
        xcopy = _mx_aligned(xscales, device, stream)
        xs = xcopy.data_ptr()
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_matmul_a4, device, stream, xq.data_ptr(), xs, wq.data_ptr(), ws,
            y.data_ptr(), M, N, K)
    if stream is not None:
        _keep_for(stream, device, xq, xscales, wq, scales, y)
    return y


def w4a16_mx_gate_up(x, wq, scales, h=None, stream=None):
    """Gated block, any M: h [M, N2] = bf16(silu(x . gate^T) * (x . up^T)), the two layers' rows
    interleaved in blocks of 8 (interleave_gate_up) in wq and scales (2 N2 rows)."""
    M, K, device = _mx_rows("x", x)
    N = _mx_stored(wq, scales, K, device)[0]
    if N % 16:
        raise ValueError("the interleaved gate/up rows come in blocks of 16")
    h = _mx_out("h", h, x, _bf16, M, N // 2, device, stream)
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_gate_up, device, stream, x.data_ptr(), wq.data_ptr(), ws, h.data_ptr(), M, N // 2, K)
    if stream is not None:
        _keep_for(stream, device, x, wq, scales, h)
    return h


def w4a16_mx_matmul_backward(dy, wq, scales, dx=None, stream=None):
    """The input's gradient of w4a16_mx_matmul: dx [M, K] = dy [M, N] . W; N a multiple of 8."""
    M, N, device = _mx_rows("dy", dy)
    rows, K, on = _mx_stored(wq, scales, None, None)
    if on != device:
        _mx_refuse("wq", wq, (_i32, _u32), None, device)
    if rows != N:
        raise ValueError(f"dy has {N} columns, W {rows} rows")
    dx = _mx_out("dx", dx, dy, _bf16, M, K, device, stream)
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_matmul_backward, device, stream, dy.data_ptr(), wq.data_ptr(), ws, dx.data_ptr(),
            M, N, K)
    if stream is not None:
        _keep_for(stream, device, dy, wq, scales, dx)
    return dx


def w4a16_mx_gate_up_backward(x, wq, scales, dh, dx=None, dgu=None, stream=None):
    """Backward pass of w4a16_mx_gate_up from x and dh [M, N2]: returns (dx [M, K], dgu [M, 2 N2]),
    dgu the gradients of both projections' outputs with columns interleaved like the rows of W."""
    M, K, device = _mx_rows("x", x)
    N = _mx_stored(wq, scales, K, device)[0]
    if N % 16:
        raise ValueError("the interleaved gate/up rows come in blocks of 16")
    if not (isinstance(dh, _Tensor) and _mx_ok(dh, _bf16, M, N // 2, device)):
        _mx_refuse("dh", dh, (_bf16,), (M, N // 2), device)
    dx = _mx_out("dx", dx, x, _bf16, M, K, device, stream)
    dgu = _mx_out("dgu", dgu, x, _bf16, M, N, device, stream)
    ws = scales.data_ptr()
    if ws & 15:
        copy = _mx_aligned(scales, device, stream)
        ws = copy.data_ptr()
    _mx_run(lib.w4a16_mx_gate_up_backward, device, stream, x.data_ptr(), wq.data_ptr(), ws, dh.data_ptr(),
            dgu.data_ptr(), dx.data_ptr(), M, N // 2, K)
    if stream is not None:
        _keep_for(stream, device, x, wq, scales, dh, dx, dgu)
    return dx, dgu


def w4a16_plan(M: int, N: int, K: int, path=PATH_AUTO, splits=0, workers=0, sm_count=0, row_blocks=0) -> dict:
    opt = make_options(path, splits, workers, sm_count, 0, row_blocks)
    info = PlanInfo()
    _check(lib.w4a16_plan(M, N, K, ctypes.byref(opt), ctypes.byref(info)), "w4a16_plan")
    return {name: getattr(info, name) for name, _ in PlanInfo._fields_ if name != "reserved"}


def w4a16_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return lib.w4a16_device_status(_stream_handle(stream))


def w4a16_release() -> None:
    lib.w4a16_release()


def w4a16_version() -> int:
    return lib.w4a16_version()


def w4a16_streamk_owner(units: int, workers: int, u: int) -> int:
    return lib.w4a16_streamk_owner(units, workers, u)


__all__ = [
    "w4a16_matmul", "w4a16_matmul_ex", "w4a16_matmul_last_rows", "w4a16_plan", "w4a16_device_status",
    "w4a16_release", "w4a16_version", "w4a16_streamk_owner", "w4a16_matvec_noalloc", "w4a16_quantize",
    "w4a16_gate_up", "interleave_gate_up", "w4a16_matmul_bits",
    "w4a16_mx_quantize", "w4a16_mx_dequantize", "w4a16_mx_matmul", "w4a16_mx_matmul_a4", "w4a16_mx_gate_up",
    "w4a16_mx_matmul_backward", "w4a16_mx_gate_up_backward",
    "status_string", "W4A16Error", "Options",
    "PlanInfo", "make_options", "lib", "LIBRARY_PATH",
]
