"""Python binding of libhalo.so, the MI355X Hadamard-rotated low-precision linear layer.

Argument marshalling only: torch tensors supply device pointers and the current HIP stream;
every step of the computation runs in the library's gfx950 kernels.  The library must be
built (``python -m hadamard_rotated_precision_halo_amd.build``); importing the functions below
without it raises immediately -- there is no fallback path.

Method: "HALO: Hadamard-Assisted Lower-Precision Optimization for LLMs" (abstract: rotations
in the forward and backward pass, all large products in 8 bits; key design 2: INT8 or FP8),
with the orthonormal Walsh-Hadamard transform and absmax quantiser of
"QWHA方法：基于Walsh-Hadamard变换的高效大模型微调技术" s2.1-s2.2, applied blockwise (s3.1), with
the zero padding and stochastic rounding of its s5, and the seeded randomised transform H D of
"企业官网建设流程全解析" s4.2.
"""
import ctypes
import os
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhalo.so")

# halo_dtype / halo_axis / halo_status values of include/halo.h
F32, BF16, I8, E4M3, E5M2, I32 = range(6)
ROWS, COLS = 0, 1
NEAREST, STOCHASTIC = 0, 1  # halo_rounding
NOALLOC_SCRATCH_BYTES = 1 << 20  # HALO_NOALLOC_SCRATCH_BYTES
STATUS = {0: "HALO_OK", 1: "HALO_ERR_NULL", 2: "HALO_ERR_SHAPE", 3: "HALO_ERR_BLOCK",
          4: "HALO_ERR_DTYPE", 5: "HALO_ERR_ALIGN", 6: "HALO_ERR_WORKSPACE", 7: "HALO_ERR_HIP",
          8: "HALO_ERR_OPTION"}

EXPORTS = ("halo_fwht_quant", "halo_fwht_quant_ex", "halo_fwht_quant_noalloc",
           "halo_fwht_quant_workspace_bytes",
           "halo_gemm_i8", "halo_gemm_fp8", "halo_linear_workspace_bytes",
           "halo_linear_workspace_bytes_ex", "halo_linear_fwd", "halo_linear_fwd_ex",
           "halo_linear_bwd", "halo_linear_bwd_ex", "halo_fwht_quant_dual",
           "halo_fwht_quant_dual_workspace_bytes", "halo_mfma_rate_probe", "halo_status_str",
           "halo_block_norm_fwd", "halo_block_norm_bwd", "halo_block_norm_bwd_workspace_bytes",
           "halo_distill_fwd", "halo_distill_bwd", "halo_distill_fwd_bwd",
           "halo_linear_act_fwd", "halo_linear_act_q", "halo_linear_act_q_workspace_bytes",
           "halo_linear_act_bwd", "halo_linear_act_bwd_workspace_bytes",
           "halo_linear_act_bwd_workspace_bytes_ex",
           "halo_checkpoint_pack", "halo_checkpoint_unpack", "halo_linear_act_fwd_kept",
           "halo_linear_act_bwd_kept", "halo_linear_act_bwd_kept_workspace_bytes",
           "halo_linear_glu_fwd", "halo_linear_glu_q", "halo_linear_glu_bwd",
           "halo_linear_glu_bwd_workspace_bytes")
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3, "gelu_erf": 4}  # halo_activation


class QuantOpts(ctypes.Structure):
    """halo_quant_opts of include/halo.h."""
    _fields_ = [("signs", ctypes.c_void_p), ("rounding", ctypes.c_int32),
                ("seed", ctypes.c_uint32 * 2), ("counter", ctypes.c_uint32 * 2),
                ("exchange_polls", ctypes.c_uint32)]


class LinearOpts(ctypes.Structure):
    """halo_linear_opts of include/halo.h."""
    _fields_ = [("signs_k", ctypes.c_void_p), ("signs_n", ctypes.c_void_p),
                ("signs_m", ctypes.c_void_p), ("grad_rounding", ctypes.c_int32),
                ("seed", ctypes.c_uint32 * 2), ("counter", ctypes.c_uint32 * 2),
                ("exchange_polls", ctypes.c_uint32)]


class Epilogue(ctypes.Structure):
    """halo_epilogue of include/halo.h."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("activation", ctypes.c_int32)]


class Kept(ctypes.Structure):
    """halo_kept of include/halo.h."""
    _fields_ = [("data", ctypes.c_void_p), ("powers", ctypes.c_void_p), ("type", ctypes.c_int)]


class Checkpoint(NamedTuple):
    """Activations kept in 8 bits (checkpoint_pack): codes [rows, cols] (int8 or float8_e4m3fn) and
    powers [rows, ceil(cols / 32)] (uint8): codes[r, c] * 2 ** (powers[r, c // 32] - 127)."""
    codes: torch.Tensor
    powers: torch.Tensor


_TORCH_CODE = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8,
               torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2, torch.int32: I32}


class HaloError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_status_str(status)})")


_lib = None


def lib():
    """The loaded libhalo.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run "
                              "`python -m hadamard_rotated_precision_halo_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        e = ctypes.c_int  # enums
        L.halo_fwht_quant.argtypes = [vp, e, i64, i64, i64, e, i32, e, vp, i64, vp, vp, sz, vp]
        L.halo_fwht_quant_workspace_bytes.argtypes = [i64, i64, e, i32, e]
        L.halo_fwht_quant_workspace_bytes.restype = sz
        L.halo_gemm_i8.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, e, i64, vp]
        L.halo_gemm_fp8.argtypes = [vp, e, i64, vp, vp, e, i64, vp, i64, i64, i64, vp, e, i64, vp]
        L.halo_linear_workspace_bytes.argtypes = [i64, i64, i64, e, ctypes.c_int]
        L.halo_linear_workspace_bytes.restype = sz
        L.halo_linear_fwd.argtypes = [vp, vp, e, i64, i64, i64, i32, e, vp, e, vp, sz, vp]
        L.halo_linear_bwd.argtypes = [vp, vp, vp, e, i64, i64, i64, i32, e, e, vp, vp, vp, sz, vp]
        qo, lo = ctypes.POINTER(QuantOpts), ctypes.POINTER(LinearOpts)
        L.halo_fwht_quant_ex.argtypes = [vp, e, i64, i64, i64, e, i32, e, vp, i64, vp, qo, vp, sz,
                                         vp]
        L.halo_fwht_quant_noalloc.argtypes = [vp, e, i64, i64, i64, e, i32, e, vp, i64, vp, qo,
                                              vp]
        L.halo_linear_workspace_bytes_ex.argtypes = [i64, i64, i64, i32, e, ctypes.c_int]
        L.halo_linear_workspace_bytes_ex.restype = sz
        L.halo_linear_fwd_ex.argtypes = [vp, vp, e, i64, i64, i64, i32, e, vp, e, lo, vp, sz, vp]
        L.halo_linear_bwd_ex.argtypes = [vp, vp, vp, e, i64, i64, i64, i32, e, e, vp, vp, lo, vp,
                                         sz, vp]
        L.halo_mfma_rate_probe.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_int64), vp]
        L.halo_fwht_quant_dual_workspace_bytes.argtypes = [i64, i64, i32, e]
        L.halo_fwht_quant_dual_workspace_bytes.restype = sz
        L.halo_fwht_quant_dual.argtypes = [vp, e, i64, i64, i64, i32, e, vp, i64, vp, vp, i64, vp,
                                           qo, qo, vp, sz, vp]
        f32 = ctypes.c_float
        L.halo_block_norm_fwd.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, vp, e, i64, i64, f32,
                                          f32, vp, i64, vp, i64, vp, vp, vp]
        L.halo_block_norm_bwd_workspace_bytes.argtypes = [i64, i64, i64, e]
        L.halo_block_norm_bwd_workspace_bytes.restype = sz
        L.halo_block_norm_bwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, vp,
                                          vp, vp, e, i64, i64, f32, vp, i64, vp, i64, vp, vp, vp,
                                          vp, sz, vp]
        L.halo_distill_fwd.argtypes = [vp, e, i64, vp, i64, vp, e, i64, i64, i64, i64, f32, vp, vp,
                                       vp]
        L.halo_distill_bwd.argtypes = [vp, vp, e, i64, vp, vp, i64, vp, e, i64, i64, i64, i64, f32,
                                       vp, i64, vp]
        L.halo_distill_fwd_bwd.argtypes = [vp, e, i64, vp, i64, vp, e, i64, vp, i64, i64, i64, f32,
                                           vp, vp, vp, i64, vp]
        ep = ctypes.POINTER(Epilogue)
        L.halo_linear_act_fwd.argtypes = [vp, vp, e, i64, i64, i64, i32, e, vp, e, ep, lo, vp, sz,
                                          vp]
        L.halo_linear_act_q_workspace_bytes.argtypes = [i64, i64, i32]
        L.halo_linear_act_q_workspace_bytes.restype = sz
        L.halo_linear_act_q.argtypes = [vp, e, vp, e, vp, i64, i64, i64, i32, vp, e, ep, vp, vp, sz,
                                        vp]
        L.halo_linear_act_bwd_workspace_bytes.argtypes = [i64, i64, i64, i32, e]
        L.halo_linear_act_bwd_workspace_bytes.restype = sz
        L.halo_linear_act_bwd_workspace_bytes_ex.argtypes = [i64, i64, i64, i32, e, e, e, i32, e]
        L.halo_linear_act_bwd_workspace_bytes_ex.restype = sz
        L.halo_linear_act_bwd.argtypes = [vp, vp, e, vp, vp, e, i64, i64, i64, i32, e, e, vp, vp,
                                          vp, lo, vp, sz, vp]
        kp = ctypes.POINTER(Kept)
        L.halo_checkpoint_pack.argtypes = [vp, e, i64, i64, i64, e, vp, i64, vp, i64, vp]
        L.halo_checkpoint_unpack.argtypes = [vp, e, i64, vp, i64, i64, i64, vp, e, i64, vp]
        L.halo_linear_act_fwd_kept.argtypes = [vp, vp, e, i64, i64, i64, i32, e, vp, e, ep, kp, lo,
                                               vp, sz, vp]
        L.halo_linear_glu_fwd.argtypes = [vp, vp, e, i64, i64, i64, i32, e, vp, e, vp, e, kp, lo, vp,
                                          sz, vp]
        L.halo_linear_glu_q.argtypes = [vp, e, vp, e, vp, i64, i64, i64, i32, vp, e, vp, e, vp, vp,
                                        sz, vp]
        for f in (L.halo_linear_act_bwd_kept, L.halo_linear_glu_bwd):
            f.argtypes = [vp, kp, e, kp, vp, e, i64, i64, i64, i32, e, e, vp, vp, vp, lo, vp, sz, vp]
        for f in (L.halo_linear_act_bwd_kept_workspace_bytes, L.halo_linear_glu_bwd_workspace_bytes):
            f.argtypes = [i64, i64, i64, i32, e, e, e, e, e, i32, e]
            f.restype = sz
        L.halo_status_str.argtypes = [e]
        L.halo_status_str.restype = ctypes.c_char_p
        for f in ("halo_fwht_quant", "halo_fwht_quant_ex", "halo_fwht_quant_noalloc",
                  "halo_gemm_i8", "halo_gemm_fp8",
                  "halo_linear_fwd", "halo_linear_fwd_ex", "halo_linear_bwd",
                  "halo_linear_bwd_ex", "halo_fwht_quant_dual", "halo_mfma_rate_probe",
                  "halo_block_norm_fwd", "halo_block_norm_bwd", "halo_distill_fwd",
                  "halo_distill_bwd", "halo_distill_fwd_bwd", "halo_linear_act_fwd",
                  "halo_linear_act_q", "halo_linear_act_bwd", "halo_checkpoint_pack",
                  "halo_checkpoint_unpack", "halo_linear_act_fwd_kept",
                  "halo_linear_act_bwd_kept", "halo_linear_glu_fwd", "halo_linear_glu_q",
                  "halo_linear_glu_bwd"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _status_str(s):
    try:
        return lib().halo_status_str(int(s)).decode()
    except Exception:  # pragma: no cover
        return "?"


def _code(dtype):
    try:
        return _TORCH_CODE[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# The current device's index; torch's own handle, where this torch has it, at a fraction of
# torch.cuda.current_device's time.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _off_device(t):
    """Whether a tensor is on a GPU that is not the current device: the library launches on the
    current one."""
    return t.is_cuda and t.device.index != _current_device()


def _on(stream, device, call, *args, **kw):
    """call(..) with `device` the current device and `stream` (None: the device's current one) its
    current stream, so that the kernels run on the tensors' device and the outputs and workspaces
    they need belong to the stream they run on: the allocator hands out memory in the order of one
    stream's work."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif not (isinstance(stream, torch.cuda.Stream) and stream.device == device):
        raise ValueError(f"stream must be a torch.cuda.Stream of {device}")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _check(status, what):
    if status != 0:
        raise HaloError(status, what)


def _ld(t):
    assert t.dim() == 2, "matrices are 2-D"
    if t.numel() == 0:  # an empty matrix has no meaningful stride; any aligned value works
        return max(t.shape[1], 16)
    assert t.stride(1) == 1, "matrices must be row-major with unit column stride"
    return t.stride(0)


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _matrix(t, name, shape, dtype=None, contiguous=False):
    """A 2-D matrix argument of exactly `shape` (and `dtype`): row-major with unit column stride
    and a row stride of at least its width, or contiguous for the layer calls, which take no
    leading dimension.  The kernels trust the shapes the call passes: a tensor smaller than
    that would be read or written past its end."""
    _require(isinstance(t, torch.Tensor) and t.dim() == 2, f"{name} must be a 2-D tensor")
    _require(tuple(t.shape) == tuple(shape),
             f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if dtype is not None:
        _require(t.dtype == dtype, f"{name} has dtype {t.dtype}, the call needs {dtype}")
    if contiguous:
        _require(t.is_contiguous(), f"{name} must be contiguous (row-major, no row padding)")
    elif t.numel() > 0:
        _require(t.stride(1) == 1 and t.stride(0) >= t.shape[1],
                 f"{name} must be row-major with unit column stride")


def _vector(t, name, n, dtype):
    """A contiguous 1-D argument of at least n entries of dtype."""
    _require(isinstance(t, torch.Tensor) and t.dim() == 1 and t.dtype == dtype
             and t.is_contiguous() and t.numel() >= n,
             f"{name} must be a contiguous 1-D {dtype} tensor of at least {n} entries")


def _bytes(t, name):
    """A workspace: a contiguous 1-D uint8 tensor (its size is checked by the library)."""
    _require(isinstance(t, torch.Tensor) and t.dim() == 1 and t.dtype == torch.uint8
             and t.is_contiguous(), f"{name} must be a contiguous 1-D uint8 tensor")


def _same_gpu(ref, **tensors):
    """The reference input on a GPU and every other tensor argument on the same device."""
    _require(isinstance(ref, torch.Tensor) and ref.is_cuda, "the inputs must be GPU tensors")
    for name, t in tensors.items():
        if t is not None:
            _require(t.device == ref.device, f"{name} is on {t.device}, the inputs on {ref.device}")


def _sign_words(length):
    return -(-int(length) // 32)


def contraction_len(dim, block):
    """Contraction length of a layer product: the dimension padded with zeros to a multiple of
    the block and of 32; a layer call's sign array covers this length."""
    step = max(int(block), 32)
    return -(-int(dim) // step) * step


def padded_len(length, block):
    """Rotated length of a vector of `length` elements: rounded up to a multiple of block
    (the zero padding)."""
    return -(-int(length) // int(block)) * int(block)


def hadamard_signs(length, seed, device=None):
    """Packed random signs of the randomised transform H D for vectors of `length` elements:
    ceil(length / 32) 32-bit words (bit i set = element i negated), drawn on the host from
    `seed`, so every process that uses the same seed gets the same transform.  Returned as an
    int32 tensor (the words' bit patterns) on `device`."""
    g = torch.Generator(device="cpu")
    g.manual_seed(int(seed))
    words = torch.randint(-(2 ** 31), 2 ** 31, (-(-int(length) // 32),), dtype=torch.int32,
                          generator=g)
    return words.to(device) if device is not None else words


def _u32x2(v):
    v = int(v)
    return (ctypes.c_uint32 * 2)(v & 0xFFFFFFFF, (v >> 32) & 0xFFFFFFFF)


_ROUNDING = {"nearest": NEAREST, "stochastic": STOCHASTIC, NEAREST: NEAREST,
             STOCHASTIC: STOCHASTIC}


def _rounding(r):
    try:
        return _ROUNDING[r]
    except KeyError:
        raise ValueError(f"rounding must be 'nearest' or 'stochastic', not {r!r}") from None


def fwht_quant_workspace_bytes(rows, cols, axis, block, x_dtype=torch.bfloat16):
    return int(lib().halo_fwht_quant_workspace_bytes(rows, cols, axis, int(block),
                                                     _code(x_dtype)))


def fwht_quant(x, axis=ROWS, block=256, q_dtype=torch.int8, q=None, scale=None, workspace=None,
               stream=None, signs=None, rounding="nearest", seed=0, counter=0,
               exchange_polls=0):
    """Rotate + quantise the rows (axis ROWS) or columns (axis COLS) of x.

    Returns (q, scale): q is [rows x Lp] (ROWS) or [cols x Lp] (COLS) of q_dtype
    (torch.int8 / float8_e4m3fn / float8_e5m2, or torch.float32 for the rotated values
    themselves), Lp the vector length padded with zeros to a multiple of block; scale is
    float32 with one entry per vector.  `workspace` is the optional scratch of the single-read
    columns pass: a uint8 device tensor, allocated here when None and the shape can use one;
    pass False to run without it.  `signs`: the randomised transform's packed sign words (an
    int32 device tensor, see hadamard_signs) or None.  `rounding`: "nearest" or "stochastic"
    (Philox key `seed`, counter words 2-3 `counter`, each a 64-bit integer).
    `exchange_polls`: for columns longer than 4096 rows, the polls a waiting workgroup makes
    before it stops waiting (the strip is then stored by a follow-up launch, with the same
    codes); 0 = the library's default.
    """
    _require(isinstance(x, torch.Tensor) and x.dim() == 2, "x must be a 2-D tensor")
    if stream is not None or _off_device(x):
        return _on(stream, x.device, fwht_quant, x, axis, block, q_dtype, q, scale, workspace,
                   signs=signs, rounding=rounding, seed=seed, counter=counter,
                   exchange_polls=exchange_polls)
    rows, cols = x.shape
    nvec, L = (rows, cols) if axis == ROWS else (cols, rows)
    Lp = padded_len(L, block)
    if q is None:
        q = torch.empty((nvec, Lp), dtype=q_dtype, device=x.device)
    _matrix(q, "q", (nvec, Lp))
    if scale is None:
        scale = torch.empty(nvec, dtype=torch.float32, device=x.device)
    _vector(scale, "scale", nvec, torch.float32)
    if signs is not None:
        _vector(signs, "signs", _sign_words(Lp), torch.int32)
    if workspace is not None and workspace is not False:
        _bytes(workspace, "workspace")
    _same_gpu(x, q=q, scale=scale, signs=signs,
              workspace=workspace if workspace is not False else None)
    if workspace is False:
        ws_ptr, ws_bytes = None, 0
    else:
        need = fwht_quant_workspace_bytes(rows, cols, axis, block, x.dtype)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        if workspace is None:
            ws_ptr, ws_bytes = None, 0
        else:
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()
    opts = None
    rnd = _rounding(rounding)
    if signs is not None or rnd != NEAREST or exchange_polls:
        opts = QuantOpts(_ptr(signs), rnd, _u32x2(seed), _u32x2(counter), int(exchange_polls))
    st = lib().halo_fwht_quant_ex(_ptr(x), _code(x.dtype), rows, cols, _ld(x), axis, int(block),
                                  _code(q.dtype), _ptr(q), _ld(q), _ptr(scale),
                                  ctypes.byref(opts) if opts is not None else None, ws_ptr,
                                  ws_bytes, _stream(stream))
    _check(st, "halo_fwht_quant_ex")
    return q, scale


def fwht_quant_dual_workspace_bytes(rows, cols, block, x_dtype=torch.bfloat16):
    return int(lib().halo_fwht_quant_dual_workspace_bytes(int(rows), int(cols), int(block),
                                                          _code(x_dtype)))


def _quant_opts(signs, rounding, seed, counter, exchange_polls):
    rnd = _rounding(rounding)
    if signs is None and rnd == NEAREST and not exchange_polls:
        return None
    return QuantOpts(_ptr(signs), rnd, _u32x2(seed), _u32x2(counter), int(exchange_polls))


def fwht_quant_dual(x, block=256, q_dtype=torch.int8, qr=None, scale_r=None, qc=None,
                    scale_c=None, workspace=None, stream=None, row_signs=None, col_signs=None,
                    rounding="nearest", seed=0, row_counter=0, col_counter=0, exchange_polls=0):
    """Both passes of x from one read where the shape allows (halo_fwht_quant_dual): returns
    (qr, scale_r, qc, scale_c), the codes and scales of fwht_quant along the rows and along
    the columns.  `row_signs` / `col_signs`: each pass's sign words (along the columns of a row
    / the rows of a column); `rounding`, `seed`, the counters and `exchange_polls` as in
    fwht_quant (the counter of each pass its own).  `workspace`: the scratch, allocated here
    when None; False runs without it."""
    _require(isinstance(x, torch.Tensor) and x.dim() == 2, "x must be a 2-D tensor")
    if stream is not None or _off_device(x):
        return _on(stream, x.device, fwht_quant_dual, x, block, q_dtype, qr, scale_r, qc, scale_c,
                   workspace, row_signs=row_signs, col_signs=col_signs, rounding=rounding,
                   seed=seed, row_counter=row_counter, col_counter=col_counter,
                   exchange_polls=exchange_polls)
    rows, cols = x.shape
    if qr is None:
        qr = torch.empty((rows, padded_len(cols, block)), dtype=q_dtype, device=x.device)
    if scale_r is None:
        scale_r = torch.empty(rows, dtype=torch.float32, device=x.device)
    if qc is None:
        qc = torch.empty((cols, padded_len(rows, block)), dtype=q_dtype, device=x.device)
    if scale_c is None:
        scale_c = torch.empty(cols, dtype=torch.float32, device=x.device)
    _matrix(qr, "qr", (rows, padded_len(cols, block)), dtype=q_dtype)
    _matrix(qc, "qc", (cols, padded_len(rows, block)), dtype=q_dtype)
    _vector(scale_r, "scale_r", rows, torch.float32)
    _vector(scale_c, "scale_c", cols, torch.float32)
    if row_signs is not None:
        _vector(row_signs, "row_signs", _sign_words(padded_len(cols, block)), torch.int32)
    if col_signs is not None:
        _vector(col_signs, "col_signs", _sign_words(padded_len(rows, block)), torch.int32)
    if workspace is not None and workspace is not False:
        _bytes(workspace, "workspace")
    _same_gpu(x, qr=qr, qc=qc, scale_r=scale_r, scale_c=scale_c, row_signs=row_signs,
              col_signs=col_signs, workspace=workspace if workspace is not False else None)
    if workspace is False:
        ws_ptr, ws_bytes = None, 0
    else:
        need = fwht_quant_dual_workspace_bytes(rows, cols, block, x.dtype)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace),
                                                                workspace.numel())
    ro = _quant_opts(row_signs, rounding, seed, row_counter, exchange_polls)
    co = _quant_opts(col_signs, rounding, seed, col_counter, exchange_polls)
    st = lib().halo_fwht_quant_dual(_ptr(x), _code(x.dtype), rows, cols, _ld(x), int(block),
                                    _code(q_dtype), _ptr(qr), _ld(qr), _ptr(scale_r), _ptr(qc),
                                    _ld(qc), _ptr(scale_c),
                                    ctypes.byref(ro) if ro is not None else None,
                                    ctypes.byref(co) if co is not None else None, ws_ptr,
                                    ws_bytes, _stream(stream))
    _check(st, "halo_fwht_quant_dual")
    return qr, scale_r, qc, scale_c


MFMA_PROBE_KINDS = {0: "v_mfma_i32_32x32x32_i8", 1: "v_mfma_scale_f32_32x32x64_f8f6f4 (E4M3)",
                    2: "v_mfma_scale_f32_16x16x128_f8f6f4 (E4M3)"}


def mfma_rate_probe(kind, iters, stream=None):
    """One launch of the matrix-core rate probe (halo_mfma_rate_probe) on `stream`; returns the
    operations it performs.  A measurement aid: time it with events on the same stream."""
    if stream is not None and stream.device.index != _current_device():
        return _on(stream, stream.device, mfma_rate_probe, kind, iters)
    ops = ctypes.c_int64(0)
    _check(lib().halo_mfma_rate_probe(int(kind), int(iters), ctypes.byref(ops), _stream(stream)),
           "halo_mfma_rate_probe")
    return ops.value


def fwht_quant_noalloc(x, q, scale, axis=ROWS, block=256, stream=None, signs=None,
                       rounding="nearest", seed=0, counter=0, exchange_polls=0):
    """fwht_quant into caller-provided q and scale with the library's fixed scratch in place of
    a workspace (halo_fwht_quant_noalloc): nothing is allocated.  Calls that may overlap on one
    device share that scratch and must be ordered by the caller."""
    _require(isinstance(x, torch.Tensor) and x.dim() == 2, "x must be a 2-D tensor")
    if stream is not None or _off_device(x):
        return _on(stream, x.device, fwht_quant_noalloc, x, q, scale, axis, block, signs=signs,
                   rounding=rounding, seed=seed, counter=counter, exchange_polls=exchange_polls)
    rows, cols = x.shape
    nvec, L = (rows, cols) if axis == ROWS else (cols, rows)
    Lp = padded_len(L, block)
    _matrix(q, "q", (nvec, Lp))
    _vector(scale, "scale", nvec, torch.float32)
    if signs is not None:
        _vector(signs, "signs", _sign_words(Lp), torch.int32)
    _same_gpu(x, q=q, scale=scale, signs=signs)
    opts = None
    rnd = _rounding(rounding)
    if signs is not None or rnd != NEAREST or exchange_polls:
        opts = QuantOpts(_ptr(signs), rnd, _u32x2(seed), _u32x2(counter), int(exchange_polls))
    st = lib().halo_fwht_quant_noalloc(_ptr(x), _code(x.dtype), rows, cols, _ld(x), axis,
                                       int(block), _code(q.dtype), _ptr(q), _ld(q), _ptr(scale),
                                       ctypes.byref(opts) if opts is not None else None,
                                       _stream(stream))
    _check(st, "halo_fwht_quant_noalloc")
    return q, scale


def gemm_i8(a, sa, b, sb, out_dtype=torch.bfloat16, c=None, stream=None):
    """c = (a . b^T) * sa[:, None] * sb[None, :] with int8 codes (int32 raw if out is int32)."""
    _require(isinstance(a, torch.Tensor) and a.dim() == 2 and isinstance(b, torch.Tensor)
             and b.dim() == 2, "a and b must be 2-D tensors")
    if stream is not None or _off_device(a):
        return _on(stream, a.device, gemm_i8, a, sa, b, sb, out_dtype, c)
    m, k = a.shape
    n = b.shape[0]
    _matrix(b, "b", (n, k))
    if c is None:
        c = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _matrix(c, "c", (m, n))
    if c.dtype != torch.int32:  # the raw int32 output takes no scales
        _vector(sa, "sa", m, torch.float32)
        _vector(sb, "sb", n, torch.float32)
    _same_gpu(a, b=b, c=c, sa=sa, sb=sb)
    st = lib().halo_gemm_i8(_ptr(a), _ld(a), _ptr(sa), _ptr(b), _ld(b), _ptr(sb), m, n, k,
                            _ptr(c), _code(c.dtype), _ld(c), _stream(stream))
    _check(st, "halo_gemm_i8")
    return c


def gemm_fp8(a, sa, b, sb, out_dtype=torch.bfloat16, c=None, stream=None):
    """c = (dec(a) . dec(b)^T) * sa[:, None] * sb[None, :] with fp8 codes (E4M3 / E5M2)."""
    _require(isinstance(a, torch.Tensor) and a.dim() == 2 and isinstance(b, torch.Tensor)
             and b.dim() == 2, "a and b must be 2-D tensors")
    if stream is not None or _off_device(a):
        return _on(stream, a.device, gemm_fp8, a, sa, b, sb, out_dtype, c)
    m, k = a.shape
    n = b.shape[0]
    _matrix(b, "b", (n, k))
    if c is None:
        c = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _matrix(c, "c", (m, n))
    if c.dtype != torch.int32:  # the raw int32 output takes no scales
        _vector(sa, "sa", m, torch.float32)
        _vector(sb, "sb", n, torch.float32)
    _same_gpu(a, b=b, c=c, sa=sa, sb=sb)
    st = lib().halo_gemm_fp8(_ptr(a), _code(a.dtype), _ld(a), _ptr(sa), _ptr(b), _code(b.dtype),
                             _ld(b), _ptr(sb), m, n, k, _ptr(c), _code(c.dtype), _ld(c),
                             _stream(stream))
    _check(st, "halo_gemm_fp8")
    return c


def linear_workspace_bytes(m, n, k, q_dtype=torch.int8, backward=False, block=None):
    """Workspace bytes of the layer calls: for one block size, or for every block (None)."""
    if block is None:
        return int(lib().halo_linear_workspace_bytes(m, n, k, _code(q_dtype),
                                                     1 if backward else 0))
    return int(lib().halo_linear_workspace_bytes_ex(m, n, k, int(block), _code(q_dtype),
                                                    1 if backward else 0))


def _workspace(nbytes, device, ws):
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    return ws


def linear_fwd(x, w, block, q_dtype=torch.int8, y=None, y_dtype=None, workspace=None,
               stream=None, signs_k=None):
    """Y = X W^T with both operands rotated and quantised along K (the layer's forward);
    signs_k: the randomised transform's sign words along K (see hadamard_signs) or None."""
    _require(isinstance(x, torch.Tensor) and x.dim() == 2 and isinstance(w, torch.Tensor)
             and w.dim() == 2, "x and w must be 2-D tensors")
    if stream is not None or _off_device(x):
        return _on(stream, x.device, linear_fwd, x, w, block, q_dtype, y, y_dtype, workspace,
                   signs_k=signs_k)
    m, k = x.shape
    n = w.shape[0]
    _matrix(x, "x", (m, k), contiguous=True)
    _matrix(w, "w", (n, k), dtype=x.dtype, contiguous=True)
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype or x.dtype, device=x.device)
    _matrix(y, "y", (m, n), contiguous=True)
    if signs_k is not None:
        _vector(signs_k, "signs_k", _sign_words(contraction_len(k, block)), torch.int32)
    if workspace is not None:
        _bytes(workspace, "workspace")
    _same_gpu(x, w=w, y=y, signs_k=signs_k, workspace=workspace)
    need = linear_workspace_bytes(m, n, k, q_dtype, False, block)
    ws = _workspace(need, x.device, workspace)
    opts = LinearOpts(_ptr(signs_k), None, None, NEAREST) if signs_k is not None else None
    st = lib().halo_linear_fwd_ex(_ptr(x), _ptr(w), _code(x.dtype), m, n, k, int(block),
                                  _code(q_dtype), _ptr(y), _code(y.dtype),
                                  ctypes.byref(opts) if opts is not None else None, _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "halo_linear_fwd_ex")
    return y


def linear_bwd(dy, x, w, block, q_dtype=torch.int8, grad_q_dtype=None, want_dx=True,
               want_dw=True, dx=None, dw=None, workspace=None, stream=None, signs_n=None,
               signs_m=None, grad_rounding="nearest", seed=0, counter=0, exchange_polls=0):
    """dX = dY W (rotated along N) and dW = dY^T X (rotated along M), 8-bit products.

    signs_n / signs_m: the randomised transform's sign words along N / M (or None).
    grad_rounding: "nearest" or "stochastic" rounding of the dY codes (Philox key `seed`,
    counter words 2-3 `counter`; the columns of dY draw with counter word 3 ^ 2^31).
    exchange_polls: as in fwht_quant, for the columns along m."""
    _require(all(isinstance(t, torch.Tensor) and t.dim() == 2 for t in (dy, x, w)),
             "dy, x and w must be 2-D tensors")
    if stream is not None or _off_device(x):
        return _on(stream, x.device, linear_bwd, dy, x, w, block, q_dtype, grad_q_dtype, want_dx,
                   want_dw, dx, dw, workspace, signs_n=signs_n, signs_m=signs_m,
                   grad_rounding=grad_rounding, seed=seed, counter=counter,
                   exchange_polls=exchange_polls)
    m, k = x.shape
    n = w.shape[0]
    _matrix(x, "x", (m, k), contiguous=True)
    _matrix(w, "w", (n, k), dtype=x.dtype, contiguous=True)
    _matrix(dy, "dy", (m, n), dtype=x.dtype, contiguous=True)
    grad_q_dtype = grad_q_dtype or q_dtype
    if want_dx and dx is None:
        dx = torch.empty((m, k), dtype=x.dtype, device=x.device)
    if want_dw and dw is None:
        dw = torch.empty((n, k), dtype=x.dtype, device=x.device)
    if want_dx:
        _matrix(dx, "dx", (m, k), contiguous=True)
    if want_dw:
        _matrix(dw, "dw", (n, k), contiguous=True)
    if signs_n is not None:
        _vector(signs_n, "signs_n", _sign_words(contraction_len(n, block)), torch.int32)
    if signs_m is not None:
        _vector(signs_m, "signs_m", _sign_words(contraction_len(m, block)), torch.int32)
    if workspace is not None:
        _bytes(workspace, "workspace")
    _same_gpu(x, dy=dy, w=w, dx=dx if want_dx else None, dw=dw if want_dw else None,
              signs_n=signs_n, signs_m=signs_m, workspace=workspace)
    need = linear_workspace_bytes(m, n, k, q_dtype, True, block)
    ws = _workspace(need, x.device, workspace)
    rnd = _rounding(grad_rounding)
    opts = None
    if signs_n is not None or signs_m is not None or rnd != NEAREST or exchange_polls:
        opts = LinearOpts(None, _ptr(signs_n), _ptr(signs_m), rnd, _u32x2(seed),
                          _u32x2(counter), int(exchange_polls))
    st = lib().halo_linear_bwd_ex(_ptr(dy), _ptr(x), _ptr(w), _code(x.dtype), m, n, k,
                                  int(block), _code(q_dtype), _code(grad_q_dtype),
                                  _ptr(dx) if want_dx else None, _ptr(dw) if want_dw else None,
                                  ctypes.byref(opts) if opts is not None else None, _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "halo_linear_bwd_ex")
    return (dx if want_dx else None), (dw if want_dw else None)


# ---------------------------------------------------------------------------
# the join between two blocks, and the distillation loss
# ---------------------------------------------------------------------------

def _rows(t, name, shape, dtype, device):
    """A 2-D argument of exactly shape and dtype with unit column stride and any row stride of
    at least its width; returns the row stride."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.device == device):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    rows, cols = shape
    if t.is_contiguous():
        return cols
    ld = t.stride(0) if rows > 1 else cols  # one row: its stride says nothing
    if t.numel() and ((cols > 1 and t.stride(1) != 1) or ld < cols):
        raise ValueError(f"{name} must be row-major with unit column stride")
    return max(ld, cols)


def _vec(t, name, n, dtype, device):
    """A contiguous 1-D argument of exactly n entries."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 1 and t.shape[0] == n and t.dtype is dtype
            and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} entries on {device}")


def _io_2d(t, name):
    if not (isinstance(t, torch.Tensor) and t.dim() == 2):
        raise ValueError(f"{name} must be a 2-D tensor")
    dt = t.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"unsupported dtype {dt}")
    if not t.is_cuda:
        raise ValueError("the inputs must be GPU tensors")
    return dt, t.device


# The handle of the current stream of the device of that index: torch's raw one, a twentieth of the
# time of building the torch.cuda.Stream object for it, where this torch has it.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dense_like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _p(t):
    return None if t is None else t.data_ptr()


def block_norm_fwd(r, y=None, gate=None, post_weight=None, pre_weight=None, scale=1.0, eps=1e-6,
                   r_out=None, h=None, stream=None):
    """The join between two blocks (halo_block_norm_fwd): the block output y enters the residual
    stream r under a norm, a gate and a residual scale, and the next block's input is normalised,

        a = 1 / sqrt(mean(y^2) + eps),      r_out = r + scale * gate * (y * a * post_weight),
        b = 1 / sqrt(mean(r_out^2) + eps),  h = r_out * b * pre_weight,

    each mean over the features of a token (a row of r and y, bf16 or fp32).  y None: only
    h = norm(r).  gate: [groups, dim] (or [dim]), row g for the g-th run of tokens / groups
    consecutive tokens, or None.  post_weight None: y joins without a norm; pre_weight None: no
    norm after the join.  Returns (r_out, h, rstd_post, rstd_pre): r itself without y, None for h
    and for the fp32 factors of norms that were not asked for.
    """
    dt, dev = _io_2d(r, "r")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, block_norm_fwd, r, y, gate, post_weight, pre_weight, scale, eps,
                   r_out, h)
    t, d = shape = r.shape
    ldr = _rows(r, "r", shape, dt, dev)
    ldy = ldro = ldh = ldg = 0
    groups = 1
    rstd_post = rstd_pre = None
    if y is not None:
        ldy = _rows(y, "y", shape, dt, dev)
        if gate is not None:
            if gate.dim() == 1:
                gate = gate.unsqueeze(0)
            groups = gate.shape[0]
            ldg = _rows(gate, "gate", (groups, d), dt, dev)
        if post_weight is not None:
            _vec(post_weight, "post_weight", d, dt, dev)
            rstd_post = torch.empty(t, dtype=torch.float32, device=dev)
        if r_out is None:
            r_out, ldro = _dense_like(r), d
        else:
            ldro = _rows(r_out, "r_out", shape, dt, dev)
    elif gate is not None or post_weight is not None or r_out is not None:
        raise ValueError("gate, post_weight and r_out need y")
    if pre_weight is not None:
        _vec(pre_weight, "pre_weight", d, dt, dev)
        rstd_pre = torch.empty(t, dtype=torch.float32, device=dev)
        if h is None:
            h, ldh = _dense_like(r), d
        else:
            ldh = _rows(h, "h", shape, dt, dev)
    elif h is not None:
        raise ValueError("h needs pre_weight")
    st = lib().halo_block_norm_fwd(_p(r), ldr, _p(y), ldy, _p(gate), ldg, groups, _p(post_weight),
                                   _p(pre_weight), _TORCH_CODE[dt], t, d, scale, eps, _p(r_out),
                                   ldro, _p(h), ldh, _p(rstd_post), _p(rstd_pre),
                                   _current_stream(dev.index))
    _check(st, "halo_block_norm_fwd")
    return (r if y is None else r_out), h, rstd_post, rstd_pre


def block_norm_bwd_workspace_bytes(tokens, dim, groups=1, dtype=torch.bfloat16):
    return int(lib().halo_block_norm_bwd_workspace_bytes(tokens, dim, groups, _code(dtype)))


def block_norm_bwd(dr_out, dh, r_out, y=None, gate=None, post_weight=None, pre_weight=None,
                   rstd_post=None, rstd_pre=None, scale=1.0, dr=None, dy=None, want_dgate=True,
                   want_dpost=True, want_dpre=True, workspace=None, stream=None):
    """Gradient of block_norm_fwd: from dr_out (the gradient arriving at the residual stream, or
    None) and dh, with the forward's r_out, y, weights and factors, returns (dr, dy, dgate,
    dpost_weight, dpre_weight); None for what does not exist or is not wanted.  dgate is
    [groups, dim].  The parameter gradients are fp32 sums in a fixed order, rounded once."""
    ref = dr_out if dr_out is not None else dh
    dt, dev = _io_2d(ref, "dr_out" if dr_out is not None else "dh")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, block_norm_bwd, dr_out, dh, r_out, y, gate, post_weight,
                   pre_weight, rstd_post, rstd_pre, scale, dr, dy, want_dgate, want_dpost,
                   want_dpre, workspace)
    t, d = shape = ref.shape
    if t == 0:
        raise ValueError("the gradient needs at least one token")
    lddro = lddh = ldro = ldy = ldg = lddy = 0
    groups = 1
    dgate = dpost = dpre = None
    if dr_out is not None:
        lddro = _rows(dr_out, "dr_out", shape, dt, dev)
    if pre_weight is not None:
        _vec(pre_weight, "pre_weight", d, dt, dev)
        _vec(rstd_pre, "rstd_pre", t, torch.float32, dev)
        lddh = _rows(dh, "dh", shape, dt, dev)
        ldro = _rows(r_out, "r_out", shape, dt, dev)
        if want_dpre:
            dpre = torch.empty(d, dtype=dt, device=dev)
    elif dh is not None:
        raise ValueError("dh needs pre_weight")
    if y is not None:
        ldy = _rows(y, "y", shape, dt, dev)
        if gate is not None:
            if gate.dim() == 1:
                gate = gate.unsqueeze(0)
            groups = gate.shape[0]
            ldg = _rows(gate, "gate", (groups, d), dt, dev)
            if want_dgate:
                dgate = torch.empty((groups, d), dtype=dt, device=dev)
        if post_weight is not None:
            _vec(post_weight, "post_weight", d, dt, dev)
            _vec(rstd_post, "rstd_post", t, torch.float32, dev)
            if want_dpost:
                dpost = torch.empty(d, dtype=dt, device=dev)
        if dy is None:
            dy, lddy = _dense_like(y), d
        else:
            lddy = _rows(dy, "dy", shape, dt, dev)
    elif gate is not None or post_weight is not None or dy is not None:
        raise ValueError("gate, post_weight and dy need y")
    if dr is None:
        dr, lddr = _dense_like(ref), d
    else:
        lddr = _rows(dr, "dr", shape, dt, dev)
    L = lib()
    code = _TORCH_CODE[dt]
    if workspace is None:
        need = L.halo_block_norm_bwd_workspace_bytes(t, d, groups, code)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _bytes(workspace, "workspace")
        _same_gpu(ref, workspace=workspace)
    st = L.halo_block_norm_bwd(_p(dr_out), lddro, _p(dh), lddh,
                               _p(r_out) if pre_weight is not None else None, ldro, _p(y), ldy,
                               _p(gate), ldg, groups, _p(post_weight), _p(pre_weight),
                               _p(rstd_post) if post_weight is not None else None, _p(rstd_pre),
                               code, t, d, scale, _p(dr), lddr, _p(dy), lddy, _p(dgate),
                               _p(dpost), _p(dpre), _p(workspace), workspace.numel(),
                               _current_stream(dev.index))
    _check(st, "halo_block_norm_bwd")
    return dr, dy, dgate, dpost, dpre


def _distill_args(logits, idx, tlogits):
    dt, dev = _io_2d(logits, "logits")
    t, v = shape = logits.shape
    ldl = _rows(logits, "logits", shape, dt, dev)
    if not (isinstance(tlogits, torch.Tensor) and tlogits.dim() == 2):
        raise ValueError("tlogits must be a 2-D tensor")
    tt = tlogits.dtype
    if tt is not torch.float32 and tt is not torch.bfloat16:
        raise TypeError(f"unsupported dtype {tt}")
    top = tlogits.shape[1]
    shape = (t, top)
    ldt = _rows(tlogits, "tlogits", shape, tt, dev)
    ldi = _rows(idx, "idx", shape, torch.int32, dev)
    return dt, dev, t, v, top, ldl, ldi, ldt, _TORCH_CODE[tt]


def distill_fwd(logits, idx, tlogits, temperature=1.0, loss=None, lse=None, stream=None):
    """Distillation loss of every token from a teacher's top logits (halo_distill_fwd):
    temperature^2 * sum_k p_k (log p_k - log q[idx_k]) with p the softmax of the kept teacher
    logits (tlogits [tokens, top], at vocabulary indices idx, int32; an index outside the
    vocabulary, such as -1, is no entry) and q the softmax of the student's logits, both at the
    temperature.  Returns (loss, lse), fp32 per token; lse = log sum exp(logits / temperature)."""
    dt, dev, t, v, top, ldl, ldi, ldt, tc = _distill_args(logits, idx, tlogits)
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, distill_fwd, logits, idx, tlogits, temperature, loss, lse)
    loss = _out_vec(loss, "loss", t, dev)
    lse = _out_vec(lse, "lse", t, dev)
    st = lib().halo_distill_fwd(_p(logits), _TORCH_CODE[dt], ldl, _p(idx), ldi, _p(tlogits), tc,
                                ldt, t, v, top, temperature, _p(loss), _p(lse),
                                _current_stream(dev.index))
    _check(st, "halo_distill_fwd")
    return loss, lse


def _out_vec(t, name, n, dev):
    if t is None:
        return torch.empty(n, dtype=torch.float32, device=dev)
    _vec(t, name, n, torch.float32, dev)
    return t


def distill_bwd(dloss, logits, lse, idx, tlogits, temperature=1.0, dlogits=None, stream=None):
    """Gradient of distill_fwd for the logits: dloss[t] * temperature * (q - p) per token, from
    the forward's lse.  dlogits may be logits itself."""
    dt, dev, t, v, top, ldl, ldi, ldt, tc = _distill_args(logits, idx, tlogits)
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, distill_bwd, dloss, logits, lse, idx, tlogits, temperature,
                   dlogits)
    _vec(dloss, "dloss", t, torch.float32, dev)
    _vec(lse, "lse", t, torch.float32, dev)
    if dlogits is None:
        dlogits, ldd = _dense_like(logits), v
    else:
        ldd = _rows(dlogits, "dlogits", logits.shape, dt, dev)
    st = lib().halo_distill_bwd(_p(dloss), _p(logits), _TORCH_CODE[dt], ldl, _p(lse), _p(idx), ldi,
                                _p(tlogits), tc, ldt, t, v, top, temperature, _p(dlogits), ldd,
                                _current_stream(dev.index))
    _check(st, "halo_distill_bwd")
    return dlogits


def distill_fwd_bwd(logits, idx, tlogits, dloss, temperature=1.0, loss=None, lse=None,
                    dlogits=None, stream=None):
    """distill_fwd and distill_bwd from one read of the logits, for training steps that know each
    token's weight in the loss beforehand (dloss; 0 leaves a token out).  Returns (loss, lse,
    dlogits); dlogits may be logits itself."""
    dt, dev, t, v, top, ldl, ldi, ldt, tc = _distill_args(logits, idx, tlogits)
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, distill_fwd_bwd, logits, idx, tlogits, dloss, temperature, loss,
                   lse, dlogits)
    _vec(dloss, "dloss", t, torch.float32, dev)
    loss = _out_vec(loss, "loss", t, dev)
    lse = _out_vec(lse, "lse", t, dev)
    if dlogits is None:
        dlogits, ldd = _dense_like(logits), v
    else:
        ldd = _rows(dlogits, "dlogits", logits.shape, dt, dev)
    st = lib().halo_distill_fwd_bwd(_p(logits), _TORCH_CODE[dt], ldl, _p(idx), ldi, _p(tlogits),
                                    tc, ldt, _p(dloss), t, v, top, temperature, _p(loss), _p(lse),
                                    _p(dlogits), ldd, _current_stream(dev.index))
    _check(st, "halo_distill_fwd_bwd")
    return loss, lse, dlogits


# ---------------------------------------------------------------------------
# the layer with its epilogue
# ---------------------------------------------------------------------------

def _dense(t, name, shape, dtype, device):
    """A contiguous 2-D argument of exactly shape and dtype."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, not {name!r}") from None


def _epilogue(bias, activation, residual, z, shape, dtype, device):
    if bias is not None:
        _vec(bias, "bias", shape[1], dtype, device)
    if residual is not None:
        _dense(residual, "residual", shape, dtype, device)
    if z is not None:
        _dense(z, "z", shape, dtype, device)
    return Epilogue(_p(bias), _p(residual), _p(z), _activation(activation))


def _scratch(workspace, need, ref):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=ref.device)
    _bytes(workspace, "workspace")
    _same_gpu(ref, workspace=workspace)
    return workspace


def linear_act_fwd(x, w, block, q_dtype=torch.int8, bias=None, activation="none", residual=None,
                   y=None, y_dtype=None, want_z=False, z=None, workspace=None, stream=None,
                   signs_k=None):
    """The layer with its epilogue (halo_linear_act_fwd): z = X W^T + bias (rotated 8-bit product,
    as linear_fwd), y = act(z) + residual, rounded once.  activation: "none", "relu", "silu",
    "gelu_tanh" or "gelu_erf"; bias [n], residual, y and z [m, n] share y's type.  Returns y, or
    (y, z) when the pre-activation is wanted (want_z or a z to write it to): linear_act_bwd takes
    it.  want_z=torch.int8 or torch.float8_e4m3fn keeps it in 8 bits: z is then a Checkpoint.
    residual may be y itself."""
    dt, dev = _io_2d(x, "x")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, linear_act_fwd, x, w, block, q_dtype, bias, activation, residual,
                   y, y_dtype, want_z, z, workspace, signs_k=signs_k)
    if not (isinstance(w, torch.Tensor) and w.dim() == 2):
        raise ValueError("w must be a 2-D tensor")
    m, k = x.shape
    n = w.shape[0]
    _dense(x, "x", (m, k), dt, dev)
    _dense(w, "w", (n, k), dt, dev)
    yt = y.dtype if y is not None else (y_dtype or dt)
    if y is None:
        y = torch.empty((m, n), dtype=yt, device=dev)
    else:
        _dense(y, "y", (m, n), yt, dev)
    z = _new_kept(want_z, z, m, n, yt, dev)
    kept = _kept(z, "z", m, n, yt, dev) if isinstance(z, tuple) else None
    ep = _epilogue(bias, activation, residual, None if kept else z, (m, n), yt, dev)
    opts = None
    if signs_k is not None:
        _vector(signs_k, "signs_k", _sign_words(contraction_len(k, block)), torch.int32)
        _same_gpu(x, signs_k=signs_k)
        opts = ctypes.byref(LinearOpts(_p(signs_k), None, None, NEAREST))
    L, qc = lib(), _code(q_dtype)
    ws = _scratch(workspace, L.halo_linear_workspace_bytes_ex(m, n, k, int(block), qc, 0)
                  if workspace is None else 0, x)
    if kept is not None:
        st = L.halo_linear_act_fwd_kept(_p(x), _p(w), _TORCH_CODE[dt], m, n, k, int(block), qc, _p(y),
                                        _code(yt), ctypes.byref(ep), ctypes.byref(kept), opts, _p(ws),
                                        ws.numel(), _current_stream(dev.index))
        _check(st, "halo_linear_act_fwd_kept")
        return y, z
    st = L.halo_linear_act_fwd(_p(x), _p(w), _TORCH_CODE[dt], m, n, k, int(block), qc, _p(y),
                               _code(yt), ctypes.byref(ep), opts, _p(ws), ws.numel(),
                               _current_stream(dev.index))
    _check(st, "halo_linear_act_fwd")
    return y if z is None else (y, z)


def linear_act_q_workspace_bytes(m, k, block):
    return int(lib().halo_linear_act_q_workspace_bytes(m, k, int(block)))


def linear_act_q(x, qw, sw, block, bias=None, activation="none", residual=None, y=None,
                 y_dtype=None, z=None, workspace=None, stream=None, signs_k=None):
    """linear_act_fwd on weights quantised once, for serving: (qw, sw) = fwht_quant(w, ROWS, block,
    q_dtype[, signs=signs_k]) of the weights [n, k] (k padded to a multiple of block, of 32 at
    least).  Only x is rotated and quantised here; up to 16 rows of x take a kernel bound by
    reading qw once.  Returns y (and z when a z to write it to is given)."""
    dt, dev = _io_2d(x, "x")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, linear_act_q, x, qw, sw, block, bias, activation, residual, y,
                   y_dtype, z, workspace, signs_k=signs_k)
    m, k = x.shape
    if not (isinstance(qw, torch.Tensor) and qw.dim() == 2):
        raise ValueError("qw must be a 2-D tensor")
    n, block = qw.shape[0], int(block)
    _dense(x, "x", x.shape, dt, dev)
    if qw.dtype is not torch.int8 and qw.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"unsupported dtype {qw.dtype}")
    kq = contraction_len(k, block) if block > 0 else k  # the library refuses a bad block
    _dense(qw, "qw", (n, kq), qw.dtype, dev)
    _vec(sw, "sw", n, torch.float32, dev)
    yt = y.dtype if y is not None else (y_dtype or dt)
    if y is None:
        y = torch.empty((m, n), dtype=yt, device=dev)
    else:
        _dense(y, "y", (m, n), yt, dev)
    ep = _epilogue(bias, activation, residual, z, (m, n), yt, dev)
    if signs_k is not None:
        _vector(signs_k, "signs_k", _sign_words(kq), torch.int32)
        _same_gpu(x, signs_k=signs_k)
    L = lib()
    if workspace is None:
        need = L.halo_linear_act_q_workspace_bytes(m, k, block)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _scratch(workspace, 0, x)
    st = L.halo_linear_act_q(x.data_ptr(), _TORCH_CODE[dt], qw.data_ptr(), _TORCH_CODE[qw.dtype],
                             sw.data_ptr(), m, n, k, block, y.data_ptr(), _code(yt),
                             ctypes.byref(ep), _p(signs_k), _p(workspace),
                             0 if workspace is None else workspace.numel(),
                             _current_stream(dev.index))
    _check(st, "halo_linear_act_q")
    return y if z is None else (y, z)


def linear_act_bwd_workspace_bytes(m, n, k, block, q_dtype=torch.int8, dtype=None,
                                   activation="none", want_dx=True, want_dw=True, want_db=True,
                                   grad_rounding="nearest"):
    """Workspace bytes of linear_act_bwd: for a call on tensors of dtype with these arguments, or,
    with dtype None, for every form."""
    if dtype is None:
        return int(lib().halo_linear_act_bwd_workspace_bytes(m, n, k, int(block), _code(q_dtype)))
    return int(lib().halo_linear_act_bwd_workspace_bytes_ex(
        m, n, k, int(block), _code(dtype), _code(q_dtype), _activation(activation),
        1 * bool(want_dx) + 2 * bool(want_dw) + 4 * bool(want_db), _rounding(grad_rounding)))


def linear_act_bwd(dy, z, x, w, block, q_dtype=torch.int8, grad_q_dtype=None, activation="none",
                   want_dx=True, want_dw=True, want_db=True, dx=None, dw=None, db=None,
                   workspace=None, stream=None, signs_n=None, signs_m=None,
                   grad_rounding="nearest", seed=0, counter=0, exchange_polls=0):
    """Gradient of linear_act_fwd: dz = dy act'(z) (fp32 until its codes), then linear_bwd's
    products dX = dz W and dW = dz^T X, and db = dz summed over the rows.  z may be None with
    activation "none".  x and z may each be a Checkpoint (activations kept in 8 bits).  The
    residual's gradient is dy.  Returns (dx, dw, db), None where not wanted; options as
    linear_bwd."""
    if isinstance(x, tuple) or isinstance(z, tuple):
        return _bwd_kept(False, dy, z, x, w, block, q_dtype, grad_q_dtype, activation, want_dx,
                         want_dw, want_db, dx, dw, db, workspace, stream, signs_n, signs_m,
                         grad_rounding, seed, counter, exchange_polls)
    dt, dev = _io_2d(dy, "dy")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, linear_act_bwd, dy, z, x, w, block, q_dtype, grad_q_dtype,
                   activation, want_dx, want_dw, want_db, dx, dw, db, workspace, signs_n=signs_n,
                   signs_m=signs_m, grad_rounding=grad_rounding, seed=seed, counter=counter,
                   exchange_polls=exchange_polls)
    if not all(isinstance(t, torch.Tensor) and t.dim() == 2 for t in (x, w)):
        raise ValueError("x and w must be 2-D tensors")
    m, k = x.shape
    n = w.shape[0]
    _dense(dy, "dy", (m, n), dt, dev)
    _dense(x, "x", (m, k), dt, dev)
    _dense(w, "w", (n, k), dt, dev)
    act = _activation(activation)
    if act != 0 or z is not None:
        _dense(z, "z", (m, n), dt, dev)
    if want_dx:
        dx = torch.empty((m, k), dtype=dt, device=dev) if dx is None else dx
        _dense(dx, "dx", (m, k), dt, dev)
    if want_dw:
        dw = torch.empty((n, k), dtype=dt, device=dev) if dw is None else dw
        _dense(dw, "dw", (n, k), dt, dev)
    if want_db:
        db = torch.empty(n, dtype=dt, device=dev) if db is None else db
        _vec(db, "db", n, dt, dev)
    if signs_n is not None:
        _vector(signs_n, "signs_n", _sign_words(contraction_len(n, block)), torch.int32)
    if signs_m is not None:
        _vector(signs_m, "signs_m", _sign_words(contraction_len(m, block)), torch.int32)
    _same_gpu(dy, signs_n=signs_n, signs_m=signs_m)
    rnd = _rounding(grad_rounding)
    opts = None
    if signs_n is not None or signs_m is not None or rnd != NEAREST or exchange_polls:
        opts = ctypes.byref(LinearOpts(None, _p(signs_n), _p(signs_m), rnd, _u32x2(seed),
                                       _u32x2(counter), int(exchange_polls)))
    L, qc = lib(), _code(q_dtype)
    ws = _scratch(workspace, L.halo_linear_act_bwd_workspace_bytes_ex(
        m, n, k, int(block), _TORCH_CODE[dt], qc, act, 1 * bool(want_dx) + 2 * bool(want_dw)
        + 4 * bool(want_db), rnd) if workspace is None else 0, dy)
    st = L.halo_linear_act_bwd(_p(dy), _p(z), act, _p(x), _p(w), _TORCH_CODE[dt], m, n, k,
                               int(block), qc, _code(grad_q_dtype or q_dtype),
                               _p(dx) if want_dx else None, _p(dw) if want_dw else None,
                               _p(db) if want_db else None, opts, _p(ws), ws.numel(),
                               _current_stream(dev.index))
    _check(st, "halo_linear_act_bwd")
    return (dx if want_dx else None), (dw if want_dw else None), (db if want_db else None)


# ---------------------------------------------------------------------------
# activations kept in 8 bits, and the gated layer
# ---------------------------------------------------------------------------

_KEPT_DTYPES = (torch.int8, torch.float8_e4m3fn)


def _groups(cols):
    return -(-cols // 32)


def _parts(a, name):
    if not (isinstance(a, tuple) and len(a) == 2 and isinstance(a[0], torch.Tensor)
            and isinstance(a[1], torch.Tensor)):
        raise ValueError(f"{name} must be a tensor or a Checkpoint")
    if a[0].dtype not in _KEPT_DTYPES:
        raise TypeError(f"unsupported dtype {a[0].dtype}")
    return a


def _kept(a, name, rows, cols, dtype, device, shape=None):
    """A kept activation, [rows, cols] as a Checkpoint or `shape` (the same by default) as a plain
    tensor of dtype."""
    if isinstance(a, torch.Tensor):
        _dense(a, name, shape or (rows, cols), dtype, device)
        return Kept(a.data_ptr(), None, _TORCH_CODE[dtype])
    codes, powers = _parts(a, name)
    _dense(codes, f"{name}'s codes", (rows, cols), codes.dtype, device)
    _dense(powers, f"{name}'s powers", (rows, _groups(cols)), torch.uint8, device)
    return Kept(codes.data_ptr(), powers.data_ptr(), _TORCH_CODE[codes.dtype])


def _new_checkpoint(rows, cols, q_dtype, device):
    if q_dtype not in _KEPT_DTYPES:
        raise TypeError(f"unsupported dtype {q_dtype}")
    return Checkpoint(torch.empty((rows, cols), dtype=q_dtype, device=device),
                      torch.empty((rows, -(-cols // 32)), dtype=torch.uint8, device=device))


def _new_kept(want, a, rows, cols, dtype, device, shape=None):
    """The place a forward writes z to: the caller's, or a new one in the form wanted."""
    if a is not None or want is False or want is None:
        return a
    if isinstance(want, torch.dtype) and want is not dtype:
        return _new_checkpoint(rows, cols, want, device)
    return torch.empty(shape or (rows, cols), dtype=dtype, device=device) if want else None


def checkpoint_pack(x, q_dtype=torch.int8, out=None, stream=None):
    """Activations in 8 bits for the backward pass (halo_checkpoint_pack): every 32 values of a row
    of x (bf16 or fp32, any row stride) share the least power of two that brings the largest of them
    to at most 127 (torch.int8) or 448 (torch.float8_e4m3fn), and are rounded once, ties to even.
    Returns a Checkpoint (`out` to write into, dense or with longer rows).  Its values are bf16 numbers
    exactly; a group with an infinity or a NaN becomes NaN throughout."""
    dt, dev = _io_2d(x, "x")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, checkpoint_pack, x, q_dtype, out)
    rows, cols = shape = x.shape
    ldx = _rows(x, "x", shape, dt, dev)
    ldc, ldp = cols, _groups(cols)
    if out is None:
        out = codes, powers = _new_checkpoint(rows, cols, q_dtype, dev)
    else:
        codes, powers = _parts(out, "out")
        ldc = _rows(codes, "out's codes", shape, q_dtype, dev)
        ldp = _rows(powers, "out's powers", (rows, ldp), torch.uint8, dev)
    st = lib().halo_checkpoint_pack(x.data_ptr(), _TORCH_CODE[dt], rows, cols, ldx, _code(q_dtype),
                                    codes.data_ptr(), ldc, powers.data_ptr(), ldp,
                                    _current_stream(dev.index))
    _check(st, "halo_checkpoint_pack")
    return out


def checkpoint_unpack(kept, dtype=torch.bfloat16, x=None, stream=None):
    """The values a Checkpoint stands for, as bf16 or fp32 rows (halo_checkpoint_unpack; `x` to write
    into)."""
    codes, powers = _parts(kept, "kept")
    if codes.dim() != 2 or not codes.is_cuda:
        raise ValueError("a checkpoint's codes must be a 2-D GPU tensor")
    dev = codes.device
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, checkpoint_unpack, kept, dtype, x)
    rows, cols = shape = codes.shape
    ldc = _rows(codes, "codes", shape, codes.dtype, dev)
    ldp = _rows(powers, "powers", (rows, _groups(cols)), torch.uint8, dev)
    if x is None:
        x, ldx = torch.empty(shape, dtype=dtype, device=dev), cols
    else:
        ldx = _rows(x, "x", shape, dtype, dev)
    st = lib().halo_checkpoint_unpack(codes.data_ptr(), _TORCH_CODE[codes.dtype], ldc,
                                      powers.data_ptr(), ldp, rows, cols, x.data_ptr(), _code(dtype),
                                      ldx, _current_stream(dev.index))
    _check(st, "halo_checkpoint_unpack")
    return x


def linear_glu_fwd(x, w, block, q_dtype=torch.int8, bias=None, activation="silu", y=None,
                   y_dtype=None, want_z=False, z=None, workspace=None, stream=None, signs_k=None):
    """The gated feed-forward layer (halo_linear_glu_fwd): w [2 n, k] holds the gate's n rows, then
    the up projection's; z = X W^T + bias (one rotated 8-bit product), y = act(z[:, :n]) z[:, n:],
    rounded once.  Returns y [m, n], or (y, z) when the pre-activations are wanted for
    linear_glu_bwd: want_z True for z [m, 2 n] of y's type, torch.int8 or torch.float8_e4m3fn for a
    Checkpoint of 2 m rows of n (a token's gate half, then its up half), or z to write them to.
    Workspace as linear_fwd's of 2 n output features."""
    dt, dev = _io_2d(x, "x")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, linear_glu_fwd, x, w, block, q_dtype, bias, activation, y, y_dtype,
                   want_z, z, workspace, signs_k=signs_k)
    if not (isinstance(w, torch.Tensor) and w.dim() == 2 and w.shape[0] % 2 == 0):
        raise ValueError("w must be a 2-D tensor of 2 n rows")
    m, k = x.shape
    n = w.shape[0] // 2
    _dense(x, "x", (m, k), dt, dev)
    _dense(w, "w", (2 * n, k), dt, dev)
    yt = y.dtype if y is not None else (y_dtype or dt)
    if y is None:
        y = torch.empty((m, n), dtype=yt, device=dev)
    else:
        _dense(y, "y", (m, n), yt, dev)
    if bias is not None:
        _vec(bias, "bias", 2 * n, yt, dev)
    z = _new_kept(want_z, z, 2 * m, n, yt, dev, (m, 2 * n))
    kept = None if z is None else _kept(z, "z", 2 * m, n, yt, dev, (m, 2 * n))
    opts = None
    if signs_k is not None:
        _vector(signs_k, "signs_k", _sign_words(contraction_len(k, block)), torch.int32)
        _same_gpu(x, signs_k=signs_k)
        opts = ctypes.byref(LinearOpts(_p(signs_k), None, None, NEAREST))
    L, qc = lib(), _code(q_dtype)
    ws = _scratch(workspace, L.halo_linear_workspace_bytes_ex(m, 2 * n, k, int(block), qc, 0)
                  if workspace is None else 0, x)
    st = L.halo_linear_glu_fwd(_p(x), _p(w), _TORCH_CODE[dt], m, n, k, int(block), qc, _p(y),
                               _code(yt), _p(bias), _activation(activation),
                               None if kept is None else ctypes.byref(kept), opts, _p(ws),
                               ws.numel(), _current_stream(dev.index))
    _check(st, "halo_linear_glu_fwd")
    return y if z is None else (y, z)


def linear_glu_q(x, qw, sw, block, bias=None, activation="silu", y=None, y_dtype=None,
                 workspace=None, stream=None, signs_k=None):
    """linear_glu_fwd on weights quantised once, for serving: (qw, sw) = fwht_quant(w, ROWS, block,
    q_dtype[, signs=signs_k]) of the stacked weights [2 n, k], as for linear_act_q.  Returns y."""
    dt, dev = _io_2d(x, "x")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, linear_glu_q, x, qw, sw, block, bias, activation, y, y_dtype,
                   workspace, signs_k=signs_k)
    m, k = x.shape
    if not (isinstance(qw, torch.Tensor) and qw.dim() == 2 and qw.shape[0] % 2 == 0):
        raise ValueError("qw must be a 2-D tensor of 2 n rows")
    n, block = qw.shape[0] // 2, int(block)
    _dense(x, "x", x.shape, dt, dev)
    if qw.dtype not in _KEPT_DTYPES:
        raise TypeError(f"unsupported dtype {qw.dtype}")
    kq = contraction_len(k, block) if block > 0 else k  # the library refuses a bad block
    _dense(qw, "qw", (2 * n, kq), qw.dtype, dev)
    _vec(sw, "sw", 2 * n, torch.float32, dev)
    yt = y.dtype if y is not None else (y_dtype or dt)
    if y is None:
        y = torch.empty((m, n), dtype=yt, device=dev)
    else:
        _dense(y, "y", (m, n), yt, dev)
    if bias is not None:
        _vec(bias, "bias", 2 * n, yt, dev)
    if signs_k is not None:
        _vector(signs_k, "signs_k", _sign_words(kq), torch.int32)
        _same_gpu(x, signs_k=signs_k)
    L = lib()
    if workspace is None:
        need = L.halo_linear_act_q_workspace_bytes(m, k, block)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _scratch(workspace, 0, x)
    st = L.halo_linear_glu_q(x.data_ptr(), _TORCH_CODE[dt], qw.data_ptr(), _TORCH_CODE[qw.dtype],
                             sw.data_ptr(), m, n, k, block, y.data_ptr(), _code(yt), _p(bias),
                             _activation(activation), _p(signs_k), _p(workspace),
                             0 if workspace is None else workspace.numel(),
                             _current_stream(dev.index))
    _check(st, "halo_linear_glu_q")
    return y


def linear_glu_bwd(dy, z, x, w, block, q_dtype=torch.int8, grad_q_dtype=None, activation="silu",
                   want_dx=True, want_dw=True, want_db=True, dx=None, dw=None, db=None,
                   workspace=None, stream=None, signs_n=None, signs_m=None,
                   grad_rounding="nearest", seed=0, counter=0, exchange_polls=0):
    """Gradient of linear_glu_fwd for dy [m, n]: with g, u the halves of z,
    dz = [dy u act'(g), dy act(g)] [m, 2 n] (fp32 until its codes), dX = dz W and dW = dz^T X as
    linear_bwd's products over 2 n output features, db [2 n] = dz summed over the rows.  x and z are
    the forward's, each a tensor or a Checkpoint.  Returns (dx, dw, db), None where not wanted;
    options as linear_bwd (signs_n covers 2 n)."""
    return _bwd_kept(True, dy, z, x, w, block, q_dtype, grad_q_dtype, activation, want_dx, want_dw,
                     want_db, dx, dw, db, workspace, stream, signs_n, signs_m, grad_rounding, seed,
                     counter, exchange_polls)


def _type_of(a, dt):
    """halo_dtype of a kept activation (None: plain)."""
    return _TORCH_CODE[a[0].dtype if isinstance(a, tuple) else dt]


def linear_kept_bwd_workspace_bytes(glu, m, n, k, block, q_dtype=torch.int8, dtype=torch.bfloat16,
                                    activation="none", z_dtype=None, x_dtype=None, want_dx=True,
                                    want_dw=True, want_db=True, grad_rounding="nearest"):
    """Workspace bytes of linear_glu_bwd (glu True; n output features, w [2 n, k]), or of linear_act_bwd
    with a Checkpoint among x and z, for a call of these types (z_dtype, x_dtype: torch.int8 or
    torch.float8_e4m3fn for a Checkpoint, None for a tensor of dtype)."""
    L = lib()
    f = L.halo_linear_glu_bwd_workspace_bytes if glu else L.halo_linear_act_bwd_kept_workspace_bytes
    return int(f(m, n, k, int(block), _code(dtype), _code(q_dtype), _activation(activation),
                 _code(z_dtype or dtype), _code(x_dtype or dtype),
                 1 * bool(want_dx) + 2 * bool(want_dw) + 4 * bool(want_db), _rounding(grad_rounding)))


def _bwd_kept(glu, dy, z, x, w, block, q_dtype, grad_q_dtype, activation, want_dx, want_dw, want_db,
              dx, dw, db, workspace, stream, signs_n, signs_m, grad_rounding, seed, counter,
              exchange_polls):
    dt, dev = _io_2d(dy, "dy")
    if stream is not None or dev.index != _current_device():
        return _on(stream, dev, _bwd_kept, glu, dy, z, x, w, block, q_dtype, grad_q_dtype, activation,
                   want_dx, want_dw, want_db, dx, dw, db, workspace, None, signs_n, signs_m,
                   grad_rounding, seed, counter, exchange_polls)
    m, n = dy.shape
    nz = 2 * n if glu else n
    if not (isinstance(w, torch.Tensor) and w.dim() == 2):
        raise ValueError("w must be a 2-D tensor")
    k = w.shape[1]
    _dense(dy, "dy", (m, n), dt, dev)
    _dense(w, "w", (nz, k), dt, dev)
    kx = _kept(x, "x", m, k, dt, dev)
    act = _activation(activation)
    kz = None
    if glu or act != 0 or z is not None:
        kz = _kept(z, "z", 2 * m if glu else m, n, dt, dev, (m, nz))
    if want_dx:
        dx = torch.empty((m, k), dtype=dt, device=dev) if dx is None else dx
        _dense(dx, "dx", (m, k), dt, dev)
    if want_dw:
        dw = torch.empty((nz, k), dtype=dt, device=dev) if dw is None else dw
        _dense(dw, "dw", (nz, k), dt, dev)
    if want_db:
        db = torch.empty(nz, dtype=dt, device=dev) if db is None else db
        _vec(db, "db", nz, dt, dev)
    if signs_n is not None:
        _vector(signs_n, "signs_n", _sign_words(contraction_len(nz, block)), torch.int32)
    if signs_m is not None:
        _vector(signs_m, "signs_m", _sign_words(contraction_len(m, block)), torch.int32)
    _same_gpu(dy, signs_n=signs_n, signs_m=signs_m)
    rnd = _rounding(grad_rounding)
    opts = None
    if signs_n is not None or signs_m is not None or rnd != NEAREST or exchange_polls:
        opts = ctypes.byref(LinearOpts(None, _p(signs_n), _p(signs_m), rnd, _u32x2(seed),
                                       _u32x2(counter), int(exchange_polls)))
    L, qc, code = lib(), _code(q_dtype), _TORCH_CODE[dt]
    query, call, name = (
        (L.halo_linear_glu_bwd_workspace_bytes, L.halo_linear_glu_bwd, "halo_linear_glu_bwd") if glu
        else (L.halo_linear_act_bwd_kept_workspace_bytes, L.halo_linear_act_bwd_kept,
              "halo_linear_act_bwd_kept"))
    ws = _scratch(workspace, query(m, n, k, int(block), code, qc, act, _type_of(z, dt),
                                   _type_of(x, dt), 1 * bool(want_dx) + 2 * bool(want_dw)
                                   + 4 * bool(want_db), rnd) if workspace is None else 0, dy)
    st = call(_p(dy), None if kz is None else ctypes.byref(kz), act, ctypes.byref(kx), _p(w), code, m,
              n, k, int(block), qc, _code(grad_q_dtype or q_dtype), _p(dx) if want_dx else None,
              _p(dw) if want_dw else None, _p(db) if want_db else None, opts, _p(ws), ws.numel(),
              _current_stream(dev.index))
    _check(st, name)
    return (dx if want_dx else None), (dw if want_dw else None), (db if want_db else None)
