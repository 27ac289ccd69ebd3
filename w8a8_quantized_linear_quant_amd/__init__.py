"""MI355X (gfx950) W8A8 quantized linear: Python binding of libw8a8.so.

Argument marshalling only.  Every step of the path runs in the HIP kernels of
the shared library (C ABI in include/w8a8.h); torch provides device memory and
the current stream.  The functions carry the C names:

  w8a8_quant_weight_tensorwise  tensor-wise int8 / e4m3 weight quantization
  w8a8_quant_act_rowwise        row-wise (token-wise) activation quantization
  w8a8_quant_act_rowwise_hadamard   the same on Hadamard-rotated rows
  w8a8_hadamard_rotate          rows rotated by the block Walsh-Hadamard matrix -> bf16
  w8a8_linear                   8-bit product + fused dequant epilogue -> bf16
  w8a8_linear_backward_dx       dX = dY . W from quantized dY and W^T codes
  w8a8_gemm_i32                 raw int32 accumulators (test export)
  svdq_linear                   residual 8-bit product + bf16 low-rank branch
  svdq_linear_noalloc           the same with its workspace in a fixed per-GPU scratch (allocates nothing)
  svdq_prepare                  W -> bf16 low-rank pair (truncated SVD) + bf16 residual
  q8_0_quantize / q8_0_dequantize / q8_0_nbytes   GGUF Q8_0 blocks
  gguf_a8_requant_q8_0          Q8_0 weight -> int8 / e4m3 codes, one scale per output channel
  gguf_a8_linear                8-bit product with per-channel weight scales -> bf16
  lora_plan                     which rows of a batch use which low-rank adapter (host -> device, once per batch)
  lora_forward / lora_backward  adapters of many requests added to a shared projection, and their gradients
  layer_norm_forward / layer_norm_backward   layer norm over rows, and its gradients
  w8a8_quant_act_rowwise_layer_norm   row-wise activation quantization of the layer norm, in one pass
  probe_mfma_i8                 diagnostic: sustained int8 MFMA loop (include/w8a8_probe.h)
  probe_cvt_e4m3                diagnostic: the hardware e4m3 conversion on consecutive f32 bit patterns
  probe_gemm_tile_n             diagnostic: the tile width along N w8a8_linear picks for an M x N output

Codes are torch.int8 (int8) or torch.float8_e4m3fn (e4m3); bf16 tensors are
torch.bfloat16; scales are float32.  Output tensors may be passed in (`out=`)
or are allocated on the input's device.  Nothing falls back to the CPU: if the
library is missing, importing this package raises.
"""
import ctypes
import os
import re

import torch

from .build import LIB as _LIB_PATH

INT8 = 0
FP8_E4M3 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(os.path.dirname(_HERE), "include", "w8a8.h")
BLOCK_HEADER = os.path.join(os.path.dirname(_HERE), "include", "w8a8_block.h")
PROBE_HEADER = os.path.join(os.path.dirname(_HERE), "include", "w8a8_probe.h")


class W8A8Error(RuntimeError):
    """A non-OK status returned by the library."""


def _load_library():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is not built; run `python -m w8a8_quantized_linear_quant_amd.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sigs = {
        "w8a8_status_str": (ctypes.c_char_p, [I]),
        "w8a8_weight_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
        "w8a8_quant_weight_tensorwise": (I, [I, P, I64, I64, P, P, P, P, P]),
        "w8a8_quant_act_rowwise": (I, [I, P, I64, I64, I64, P, I64, P, P]),
        "w8a8_linear": (I, [I, P, P, P, P, P, I64, I64, I64, P, P]),
        "w8a8_linear_backward_dx": (I, [I, P, P, P, P, I64, I64, I64, P, P]),
        "w8a8_gemm_i32": (I, [P, P, I64, I64, I64, P, P]),
        "svdq_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
        "svdq_linear": (I, [I, P, I64, I64, P, P, P, P, I64, P, I64, P, P, P, P, P]),
        "svdq_linear_noalloc": (I, [I, P, I64, I64, P, P, P, P, I64, P, I64, P, P, P, P]),
        "q8_0_nbytes": (ctypes.c_size_t, [I64]),
        "q8_0_quantize": (I, [P, I64, P, P]),
        "q8_0_dequantize": (I, [P, I64, P, P]),
        "gguf_a8_requant_q8_0": (I, [I, P, I64, I64, P, P, P]),
        "gguf_a8_linear": (I, [I, P, P, P, P, P, I64, I64, I64, P, P]),
        "svdq_prepare_subspace": (I64, [I64]),
        "svdq_prepare_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64]),
        "svdq_prepare": (I, [P, I64, I64, I64, P, I, P, P, P, P, P, P]),
        "w8a8_quant_act_rowwise_hadamard": (I, [I, P, I64, I64, I64, P, I64, P, P]),
        "w8a8_hadamard_rotate": (I, [P, I64, I64, I64, P, I64, P]),
        "lora_plan": (I, [P, P, I64, I64, P, I64, P]),
        "lora_forward_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
        "lora_forward": (I, [P, I64, I64, I64, P, P, I64, I64, I64, P, P, P, I64, P, I64, P, I64, P, P, P]),
        "lora_backward_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I64, I64, I64]),
        "lora_backward": (I, [P, I64, I64, I64, P, I64, I64, P, P, P, I64, I64, P, P, P, I64, P, I64, P, I64, P, P,
                              P, P]),
        "layer_norm_forward": (I, [I, P, I64, I64, I64, I, P, P, F, P, I64, P, P, P]),
        "layer_norm_backward_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
        "layer_norm_backward": (I, [I, P, I64, P, I64, P, P, I64, I64, I, P, P, I64, P, P, P, P]),
        "w8a8_quant_act_rowwise_layer_norm": (I, [I, I, P, I64, I64, I64, I, P, P, F, P, I64, P, P, P, P]),
        "w8a8_probe_sink_count": (I64, []),
        "w8a8_probe_mfma_i8": (I, [P, P, I64, P, P]),
        "w8a8_probe_cvt_e4m3": (I, [ctypes.c_uint32, I64, P, P]),
        "w8a8_probe_gemm_tile_n": (I, [I64, I64]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load_library()


def exported_names_in_header(path=HEADER):
    """Function names the C header declares (used to check the exports)."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    text = re.sub(r"^\s*#.*$", "", text, flags=re.M)   # preprocessor lines
    return sorted(set(re.findall(r"\b([A-Za-z_][A-Za-z0-9_]*)\s*\(", text)) -
                  {"if", "defined", "sizeof", "extern"})


def library():
    return _lib


def _check(status):
    if status != 0:
        raise W8A8Error(_lib.w8a8_status_str(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a torch.cuda.Stream (0.1 us against 2)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _qtype_of(codes):
    if codes.dtype == torch.int8:
        return INT8
    if codes.dtype == torch.float8_e4m3fn:
        return FP8_E4M3
    raise TypeError(f"codes must be torch.int8 or torch.float8_e4m3fn, got {codes.dtype}")


def _code_dtype(qtype):
    if qtype not in (INT8, FP8_E4M3):
        raise ValueError(f"qtype must be INT8 ({INT8}) or FP8_E4M3 ({FP8_E4M3}), got {qtype}")
    return torch.int8 if qtype == INT8 else torch.float8_e4m3fn


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _arg(t, dtype, name, device, min_numel=0):
    """An input tensor: dtype (None: any), on `device`, at least `min_numel`
    elements; returned contiguous (a copy only if it was not)."""
    _need(t, dtype, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs at least {min_numel}")
    return t.contiguous()


def _out(t, shape, dtype, device, name):
    """An output of exactly `shape`: allocated if None, else checked (dtype,
    device, shape, contiguous): the kernels write every element of it."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, dtype, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _buf(t, numel, dtype, device, name, alloc=None):
    """A flat output or workspace of at least `numel` elements: allocated
    (`alloc` elements, default numel) if None, else checked."""
    if t is None:
        return torch.empty(max(numel, alloc or 0, 1), dtype=dtype, device=device)
    _need(t, dtype, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs at least {numel}")
    return t


def _mat(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    return t


# ------------------------------------------------------------------ weights
def w8a8_weight_workspace_bytes(N, K):
    return int(_lib.w8a8_weight_workspace_bytes(N, K))


def w8a8_quant_weight_tensorwise(w, qtype=INT8, transposed=False, out=None, out_t=None, scale=None,
                                 workspace=None):
    """w: bf16 [N, K].  Returns (codes [N, K], codes^T [K, N] or None, scale f32 [1])."""
    cd = _code_dtype(qtype)
    _need(w, torch.bfloat16, "w")
    dev = w.device
    w = _mat(_arg(w, torch.bfloat16, "w", dev), "w")
    N, K = w.shape
    wq = _out(out, (N, K), cd, dev, "out")
    wq_t = _out(out_t, (K, N), cd, dev, "out_t") if (transposed or out_t is not None) else None
    s = _buf(scale, 1, torch.float32, dev, "scale", alloc=4)
    ws = _buf(workspace, w8a8_weight_workspace_bytes(N, K), torch.uint8, dev, "workspace")
    _check(_lib.w8a8_quant_weight_tensorwise(qtype, _ptr(w), N, K, _ptr(wq), _ptr(wq_t), _ptr(s), _ptr(ws),
                                             _stream(dev)))
    return wq, wq_t, s[:1]


# -------------------------------------------------------------- activations
def w8a8_quant_act_rowwise(x, qtype=INT8, ldq=None, out=None, scale=None):
    """x: bf16 [M, K] (row stride may exceed K).  Returns (codes [M, ldq], scales f32 [M])."""
    cd = _code_dtype(qtype)
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    ldx = x.stride(0)
    if M > 0 and (ldx % 8 != 0 or x.data_ptr() % 16 != 0):
        # no hidden copy: rows must start on 16-byte boundaries
        raise ValueError(f"x rows must start on 16-byte boundaries (row stride {ldx} must be a multiple of 8, "
                         "data 16-byte aligned); pass a [:, :K] view of a buffer with padded rows")
    if M > 0 and x.untyped_storage().nbytes() - 2 * x.storage_offset() < 2 * M * ldx:
        raise ValueError(f"x's storage must span M * row stride = {M * ldx} elements")
    ldq = ldq if ldq is not None else K + (-K) % 16
    dev = x.device
    xq = _out(out, (M, ldq), cd, dev, "out")
    s = _buf(scale, M, torch.float32, dev, "scale")
    _check(_lib.w8a8_quant_act_rowwise(qtype, _ptr(x), M, K, ldx, _ptr(xq), ldq, _ptr(s), _stream(dev)))
    return xq, s[:M]


def w8a8_quant_act_rowwise_hadamard(x, qtype=INT8, ldq=None, out=None, scale=None):
    """x: bf16 [M, K], K % 16 == 0.  Codes [M, ldq] and scales [M] of the Hadamard-rotated rows."""
    cd = _code_dtype(qtype)
    _need(x, torch.bfloat16, "x")
    dev = x.device
    x = _mat(_arg(x, torch.bfloat16, "x", dev), "x")
    M, K = x.shape
    ldq = ldq if ldq is not None else K
    xq = _out(out, (M, ldq), cd, dev, "out")
    s = _buf(scale, M, torch.float32, dev, "scale")
    _check(_lib.w8a8_quant_act_rowwise_hadamard(qtype, _ptr(x), M, K, K, _ptr(xq), ldq, _ptr(s), _stream(dev)))
    return xq, s[:M]


def w8a8_hadamard_rotate(x, out=None):
    """x: bf16 [M, K], K % 16 == 0 -> bf16 [M, K] rotated rows."""
    _need(x, torch.bfloat16, "x")
    dev = x.device
    x = _mat(_arg(x, torch.bfloat16, "x", dev), "x")
    M, K = x.shape
    y = _out(out, (M, K), torch.bfloat16, dev, "out")
    _check(_lib.w8a8_hadamard_rotate(_ptr(x), M, K, K, _ptr(y), K, _stream(dev)))
    return y


# --------------------------------------------------------------- the linear
def _product_args(xq, x_scale, wq, w_scale, w_scale_numel, bias):
    qt = _qtype_of(xq)
    if wq.dtype != xq.dtype:
        raise TypeError("xq and wq must hold the same code type")
    _need(xq, None, "xq")
    dev = xq.device
    xq = _mat(_arg(xq, None, "xq", dev), "xq")
    wq = _mat(_arg(wq, None, "wq", dev), "wq")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq must share K")
    x_scale = _arg(x_scale, torch.float32, "x_scale", dev, M)
    w_scale = _arg(w_scale, torch.float32, "w_scale", dev, w_scale_numel(N))
    if bias is not None:
        bias = _arg(bias, torch.bfloat16, "bias", dev, N)
    return qt, dev, xq, x_scale, wq, w_scale, bias, M, N, K


def w8a8_linear(xq, x_scale, wq, w_scale, bias=None, out=None):
    """Dequantized 8-bit linear.  xq [M, K], wq [N, K] codes (same dtype) -> bf16 [M, N]."""
    qt, dev, xq, x_scale, wq, w_scale, bias, M, N, K = _product_args(xq, x_scale, wq, w_scale, lambda n: 1, bias)
    y = _out(out, (M, N), torch.bfloat16, dev, "out")
    _check(_lib.w8a8_linear(qt, _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias), M, N, K, _ptr(y),
                            _stream(dev)))
    return y


def w8a8_linear_backward_dx(dyq, dy_scale, wq_t, w_scale, out=None):
    """dX = dY . W.  dyq [M, N] codes, wq_t [K, N] transposed weight codes -> bf16 [M, K]."""
    qt = _qtype_of(dyq)
    if wq_t.dtype != dyq.dtype:
        raise TypeError("dyq and wq_t must hold the same code type")
    _need(dyq, None, "dyq")
    dev = dyq.device
    dyq = _mat(_arg(dyq, None, "dyq", dev), "dyq")
    wq_t = _mat(_arg(wq_t, None, "wq_t", dev), "wq_t")
    M, N = dyq.shape
    K = wq_t.shape[0]
    if wq_t.shape[1] != N:
        raise ValueError("dyq and wq_t must share N")
    dy_scale = _arg(dy_scale, torch.float32, "dy_scale", dev, M)
    w_scale = _arg(w_scale, torch.float32, "w_scale", dev, 1)
    dx = _out(out, (M, K), torch.bfloat16, dev, "out")
    _check(_lib.w8a8_linear_backward_dx(qt, _ptr(dyq), _ptr(dy_scale), _ptr(wq_t), _ptr(w_scale), M, N, K,
                                        _ptr(dx), _stream(dev)))
    return dx


def w8a8_gemm_i32(xq, wq, out=None):
    """Raw int32 accumulators of the int8 product: xq [M, K] @ wq[N, K]^T."""
    _need(xq, torch.int8, "xq")
    dev = xq.device
    xq = _mat(_arg(xq, torch.int8, "xq", dev), "xq")
    wq = _mat(_arg(wq, torch.int8, "wq", dev), "wq")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq must share K")
    acc = _out(out, (M, N), torch.int32, dev, "out")
    _check(_lib.w8a8_gemm_i32(_ptr(xq), _ptr(wq), M, N, K, _ptr(acc), _stream(dev)))
    return acc


# ------------------------------------------------------------------ SVDQuant
def svdq_workspace_bytes(M, r):
    return int(_lib.svdq_workspace_bytes(M, r))


def _svdq_args(x, rq, r_scale, l1, l2, bias, out, xq_out, x_scale_out):
    qt = _qtype_of(rq)
    _need(x, torch.bfloat16, "x")
    dev = x.device
    x = _mat(_arg(x, torch.bfloat16, "x", dev), "x")
    rq = _mat(_arg(rq, None, "rq", dev), "rq")
    l1 = _mat(_arg(l1, torch.bfloat16, "l1", dev), "l1")
    l2 = _mat(_arg(l2, torch.bfloat16, "l2", dev), "l2")
    M, K = x.shape
    N = rq.shape[0]
    r = l1.shape[0]
    if rq.shape[1] != K or l1.shape[1] != K:
        raise ValueError("x, rq and l1 must share K")
    if tuple(l2.shape) != (N, r):
        raise ValueError(f"l2 must be [N, r] = [{N}, {r}], got {tuple(l2.shape)}")
    r_scale = _arg(r_scale, torch.float32, "r_scale", dev, 1)
    if bias is not None:
        bias = _arg(bias, torch.bfloat16, "bias", dev, N)
    y = _out(out, (M, N), torch.bfloat16, dev, "out")
    xq = _out(xq_out, (M, K), rq.dtype, dev, "xq_out")
    sx = _buf(x_scale_out, M, torch.float32, dev, "x_scale_out")
    return qt, dev, x, rq, r_scale, l1, l2, bias, M, N, K, r, y, xq, sx


def svdq_linear(x, rq, r_scale, l1, l2, bias=None, out=None, xq_out=None, x_scale_out=None, workspace=None):
    """x bf16 [M, K]; rq residual codes [N, K]; l1 bf16 [r, K]; l2 bf16 [N, r].
    Returns (y bf16 [M, N], xq [M, K], x_scale [M])."""
    qt, dev, x, rq, r_scale, l1, l2, bias, M, N, K, r, y, xq, sx = _svdq_args(x, rq, r_scale, l1, l2, bias, out,
                                                                             xq_out, x_scale_out)
    ws = _buf(workspace, svdq_workspace_bytes(M, r), torch.uint8, dev, "workspace", alloc=16)
    _check(_lib.svdq_linear(qt, _ptr(x), M, K, _ptr(rq), _ptr(r_scale), _ptr(l1), _ptr(l2), r, _ptr(bias), N,
                            _ptr(y), _ptr(xq), _ptr(sx), _ptr(ws), _stream(dev)))
    return y, xq, sx[:M]


def svdq_linear_noalloc(x, rq, r_scale, l1, l2, bias=None, out=None, xq_out=None, x_scale_out=None):
    """svdq_linear with its workspace in the library's fixed per-GPU scratch
    (W8A8_SVDQ_NOALLOC_SCRATCH_BYTES): the C call allocates nothing.  Pass
    `out`, `xq_out` and `x_scale_out` to allocate nothing here either."""
    qt, dev, x, rq, r_scale, l1, l2, bias, M, N, K, r, y, xq, sx = _svdq_args(x, rq, r_scale, l1, l2, bias, out,
                                                                             xq_out, x_scale_out)
    _check(_lib.svdq_linear_noalloc(qt, _ptr(x), M, K, _ptr(rq), _ptr(r_scale), _ptr(l1), _ptr(l2), r, _ptr(bias),
                                    N, _ptr(y), _ptr(xq), _ptr(sx), _stream(dev)))
    return y, xq, sx[:M]


SVDQ_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def svdq_prepare_subspace(r):
    return int(_lib.svdq_prepare_subspace(r))


def svdq_prepare_workspace_bytes(N, K, r):
    return int(_lib.svdq_prepare_workspace_bytes(N, K, r))


def svdq_prepare(w, r, omega, iters=2, l1=None, l2=None, residual=None, sigma=None, workspace=None):
    """w bf16 [N, K]; omega bf16 [svdq_prepare_subspace(r), K] (Gaussian).
    Returns (l1 bf16 [r, K], l2 bf16 [N, r], residual bf16 [N, K], sigma f32 [r])."""
    _need(w, torch.bfloat16, "w")
    dev = w.device
    w = _mat(_arg(w, torch.bfloat16, "w", dev), "w")
    omega = _arg(omega, torch.bfloat16, "omega", dev)
    N, K = w.shape
    if tuple(omega.shape) != (svdq_prepare_subspace(r), K):
        raise ValueError("omega must be [svdq_prepare_subspace(r), K]")
    l1 = _out(l1, (r, K), torch.bfloat16, dev, "l1")
    l2 = _out(l2, (N, r), torch.bfloat16, dev, "l2")
    res = _out(residual, (N, K), torch.bfloat16, dev, "residual")
    sg = _buf(sigma, r, torch.float32, dev, "sigma", alloc=4)
    ws = _buf(workspace, svdq_prepare_workspace_bytes(N, K, r), torch.uint8, dev, "workspace", alloc=16)
    _check(_lib.svdq_prepare(_ptr(w), N, K, r, _ptr(omega), iters, _ptr(l1), _ptr(l2), _ptr(res),
                             _ptr(sg), _ptr(ws), _stream(dev)))
    return l1, l2, res, sg[:r]


# ---------------------------------------------------------------------- Q8_0
def q8_0_nbytes(n):
    return int(_lib.q8_0_nbytes(n))


def q8_0_quantize(x, out=None):
    """x f32 (any shape, contiguous) -> uint8 [q8_0_nbytes(x.numel())] GGUF Q8_0 blocks."""
    _need(x, torch.float32, "x")
    dev = x.device
    x = _arg(x, torch.float32, "x", dev)
    n = x.numel()
    blocks = _buf(out, q8_0_nbytes(n), torch.uint8, dev, "out", alloc=16)
    _check(_lib.q8_0_quantize(_ptr(x), n, _ptr(blocks), _stream(dev)))
    return blocks[:q8_0_nbytes(n)]


def q8_0_dequantize(blocks, n, out=None):
    """blocks uint8 (>= q8_0_nbytes(n) bytes) -> f32 [n]."""
    _need(blocks, torch.uint8, "blocks")
    dev = blocks.device
    blocks = _arg(blocks, torch.uint8, "blocks", dev, q8_0_nbytes(n))
    y = _buf(out, n, torch.float32, dev, "out", alloc=4)
    _check(_lib.q8_0_dequantize(_ptr(blocks), n, _ptr(y), _stream(dev)))
    return y[:n]


# ------------------------------------------------------------------- GGUF A8
def gguf_a8_requant_q8_0(blocks, N, K, qtype=INT8, out=None, scale=None):
    """Q8_0 weight [N, K] (uint8 blocks, row n = K / 32 blocks) -> (codes [N, K], scales f32 [N])."""
    cd = _code_dtype(qtype)
    _need(blocks, torch.uint8, "blocks")
    dev = blocks.device
    blocks = _arg(blocks, torch.uint8, "blocks", dev, q8_0_nbytes(N * K) if K % 32 == 0 else 0)
    wq = _out(out, (N, K), cd, dev, "out")
    s = _buf(scale, N, torch.float32, dev, "scale", alloc=4)
    _check(_lib.gguf_a8_requant_q8_0(qtype, _ptr(blocks), N, K, _ptr(wq), _ptr(s), _stream(dev)))
    return wq, s[:N]


def gguf_a8_linear(xq, x_scale, wq, w_scale, bias=None, out=None):
    """8-bit linear with per-output-channel weight scales w_scale f32 [N] -> bf16 [M, N]."""
    qt, dev, xq, x_scale, wq, w_scale, bias, M, N, K = _product_args(xq, x_scale, wq, w_scale, lambda n: n, bias)
    y = _out(out, (M, N), torch.bfloat16, dev, "out")
    _check(_lib.gguf_a8_linear(qt, _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias), M, N, K, _ptr(y),
                               _stream(dev)))
    return y


# ------------------------------------------------------------------ adapters
_Tensor, _BF16, _F32, _I32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32


def _view(t, rows, cols, dtype, device, name, align=True):
    """A matrix operand that may be a view with a row stride, never copied:
    (data pointer, row stride in elements).  `align`: rows must start on
    16-byte boundaries."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    ptr, ld = t.data_ptr(), cols
    if not t.is_contiguous():
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit column stride")
        ld = t.stride(0) if rows > 1 else cols
        if ld < cols:
            raise ValueError(f"{name}'s rows overlap (row stride {ld} < {cols})")
    if rows > 0 and (ptr % 16 != 0 or (align and ld % 8 != 0)):
        raise ValueError(f"{name} must start on a 16-byte boundary" +
                         (f", its rows too (row stride {ld} must be a multiple of 8)" if align else ""))
    return ptr, ld


def _vec(t, n, dtype, device, name):
    """A contiguous operand of at least n elements, or None: its pointer."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != device or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, on {device}, of at least {n} elements")
    return t.data_ptr()


def _gpu_matrix(t, name):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    return t.device


class LoraPlan:
    """Which rows of a batch use which adapter of a pool (lora_plan).  Holds
    for one batch; every projection of every layer may share it."""

    __slots__ = ("rows", "adapters", "tiles", "data", "device")

    def __init__(self, rows, adapters, tiles, data):
        self.rows, self.adapters, self.tiles, self.data, self.device = rows, adapters, tiles, data, data.device


def lora_plan(lengths, adapters, num_adapters, device=None):
    """lengths: rows of each request, in the order of X's rows; adapters: the
    adapter of each request (0 .. num_adapters - 1, or -1 for none).  Copies
    the plan to `device` (default: the current GPU)."""
    lengths, adapters = [int(n) for n in lengths], [int(l) for l in adapters]
    if len(lengths) != len(adapters):
        raise ValueError(f"{len(lengths)} lengths, {len(adapters)} adapters")
    if any(not -1 <= l < num_adapters for l in adapters):
        raise ValueError(f"adapters must be -1 or in [0, {num_adapters})")
    S = len(lengths)
    cl, ca = (ctypes.c_int64 * S)(*lengths), (ctypes.c_int32 * S)(*adapters)
    tiles = ctypes.c_int64()
    _check(_lib.lora_plan(cl, ca, S, num_adapters, None, 0, ctypes.byref(tiles)))
    host = torch.empty(4 * tiles.value + num_adapters + 1, dtype=torch.int32)
    _check(_lib.lora_plan(cl, ca, S, num_adapters, _ptr(host), host.numel(), ctypes.byref(tiles)))
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return LoraPlan(sum(lengths), num_adapters, tiles.value, host.to(dev))


def lora_forward_workspace_bytes(M, R):
    return int(_lib.lora_forward_workspace_bytes(M, R))


def lora_backward_workspace_bytes(M, T, K, N, R, L):
    return int(_lib.lora_backward_workspace_bytes(M, T, K, N, R, L))


def _lora_args(rows, dev, a, b, plan, scale, ranks):
    if not isinstance(plan, LoraPlan):
        raise TypeError("plan must be a LoraPlan (lora_plan)")
    if not isinstance(a, _Tensor) or not isinstance(b, _Tensor):
        raise TypeError("a and b must be torch.Tensors")
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
        raise ValueError(f"a must be [L, R, K] and b [L, N, R], got {tuple(a.shape)} and {tuple(b.shape)}")
    L, R, K = a.shape
    if plan.rows != rows or plan.adapters != L or plan.device != dev:
        raise ValueError(f"the plan is for {plan.rows} rows and {plan.adapters} adapters on {plan.device}, "
                         f"the call has {rows} and {L} on {dev}")
    pa = _vec(a, 0, _BF16, dev, "a")
    pb = _vec(b, 0, _BF16, dev, "b")
    return L, R, K, b.shape[1], pa, pb, _vec(scale, L, _F32, dev, "scale"), _vec(ranks, L, _I32, dev,
                                                                                         "ranks")


def lora_forward(x, a, b, plan, scale=None, ranks=None, base=None, out=None, u=None, save_u=True, workspace=None):
    """Adapters added to a shared projection: x bf16 [M, K]; a bf16 [L, R, K]; b bf16 [L, N, R]; scale f32 [L];
    ranks int32 [L]; base bf16 [M, N] (the projection's output; `out` may be `base`).
    Returns (out bf16 [M, N], u f32 [M, R] for lora_backward, or None without save_u).
    x, base and out may be views with a row stride."""
    dev = _gpu_matrix(x, "x")
    M = x.shape[0]
    L, R, K, N, pa, pb, ps, pr = _lora_args(M, dev, a, b, plan, scale, ranks)
    px, ldx = _view(x, M, K, _BF16, dev, "x")
    pbase, ldbase = (None, 0) if base is None else _view(base, M, N, _BF16, dev, "base")
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=dev)
    po, ldo = _view(out, M, N, _BF16, dev, "out")
    if u is None and save_u:
        u = torch.empty((M, R), dtype=_F32, device=dev)
    pu = None if u is None else _vec(u, M * R, _F32, dev, "u")
    pws = None
    if u is None or workspace is not None:
        workspace = _buf(workspace, lora_forward_workspace_bytes(M, R), torch.uint8, dev, "workspace", alloc=16)
        pws = workspace.data_ptr()
    _check(_lib.lora_forward(px, M, K, ldx, pa, pb, L, N, R, ps, pr, plan.data.data_ptr(), plan.tiles, pbase, ldbase,
                             po, ldo, pu, pws, _stream(dev)))
    return out, u


def lora_backward(dy, x, u, a, b, plan, scale=None, ranks=None, base=None, out=None, da=None, db=None, need_dx=True,
                  need_weights=True, workspace=None):
    """Gradients of lora_forward: dy bf16 [M, N]; x, a, b, plan, scale, ranks of the forward call and its u;
    base bf16 [M, K]: the shared projection's input gradient (`out` may be `base`).
    Returns (dx bf16 [M, K], da f32 [L, R, K], db f32 [L, N, R]), None for what is not needed."""
    dev = _gpu_matrix(dy, "dy")
    M = dy.shape[0]
    L, R, K, N, pa, pb, ps, pr = _lora_args(M, dev, a, b, plan, scale, ranks)
    pdy, lddy = _view(dy, M, N, _BF16, dev, "dy")
    px, ldx = _view(x, M, K, _BF16, dev, "x")
    pu = _vec(u, M * R, _F32, dev, "u")
    pbase, ldbase = (None, 0) if base is None else _view(base, M, K, _BF16, dev, "base")
    dx, pdx, lddx = None, None, 0
    if need_dx:
        dx = _like(x) if out is None else out
        pdx, lddx = _view(dx, M, K, _BF16, dev, "out")
    if need_weights:
        if u is None:
            raise ValueError("u, as lora_forward returned it, is needed for the weights' gradients")
        da = _out(da, (L, R, K), _F32, dev, "da")
        db = _out(db, (L, N, R), _F32, dev, "db")
    else:
        da = db = None
    ws = _buf(workspace, lora_backward_workspace_bytes(M, plan.tiles, K, N, R, L), torch.uint8, dev,
              "workspace", alloc=16)
    _check(_lib.lora_backward(pdy, M, N, lddy, px, K, ldx, pu, pa, pb, L, R, ps, pr, plan.data.data_ptr(), plan.tiles,
                              pbase, ldbase, pdx, lddx, None if da is None else da.data_ptr(),
                              None if db is None else db.data_ptr(), ws.data_ptr(), _stream(dev)))
    return dx, da, db


# ---------------------------------------------------------------- layer norm
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _dtype_of(t, name):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _norm_args(x, weight, bias):
    dev = _gpu_matrix(x, "x")
    M, K = x.shape
    xt = _dtype_of(x, "x")
    px, ldx = _view(x, M, K, x.dtype, dev, "x", align=False)
    p = weight if weight is not None else bias
    if p is None:
        return dev, M, K, xt, px, ldx, xt, None, None
    wt = _dtype_of(p, "weight" if weight is not None else "bias")
    pw, pb = _vec(weight, K, p.dtype, dev, "weight"), _vec(bias, K, p.dtype, dev, "bias")
    return dev, M, K, xt, px, ldx, wt, pw, pb


def _like(x):
    """An uninitialized contiguous tensor of x's shape and type."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _first(t, n):
    return t if t.numel() == n else t[:n]


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None):
    """x bf16 or f32 [M, K] (may have a row stride, of any alignment); weight, bias [K] of one dtype (bf16 or f32)
    or None.  Returns (y like x, mean f32 [M], rstd f32 [M])."""
    dev, M, K, xt, px, ldx, wt, pw, pb = _norm_args(x, weight, bias)
    if out is None:
        out = _like(x)
    py, ldy = _view(out, M, K, x.dtype, dev, "out", align=False)
    if mean is None:
        mean = torch.empty(M, dtype=_F32, device=dev)
    if rstd is None:
        rstd = torch.empty_like(mean)
    pm, pr = _vec(mean, M, _F32, dev, "mean"), _vec(rstd, M, _F32, dev, "rstd")
    _check(_lib.layer_norm_forward(xt, px, M, K, ldx, wt, pw, pb, eps, py, ldy, pm, pr, _stream(dev)))
    return out, _first(mean, M), _first(rstd, M)


def layer_norm_backward_workspace_bytes(M, K):
    return int(_lib.layer_norm_backward_workspace_bytes(M, K))


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, dweight=None, dbias=None, need_dx=True,
                        need_params=None, workspace=None):
    """Gradients of layer_norm_forward from its x, mean, rstd and weight.  Returns (dx like x, dweight f32 [K],
    dbias f32 [K]), None for what is not needed (need_params: default, if there is a weight)."""
    dev, M, K, xt, px, ldx, wt, pw, _ = _norm_args(x, weight, None)
    pdy, lddy = _view(dy, M, K, x.dtype, dev, "dy", align=False)
    pm, pr = _vec(mean, M, _F32, dev, "mean"), _vec(rstd, M, _F32, dev, "rstd")
    dx, pdx, lddx = None, None, 0
    if need_dx:
        dx = _like(x) if out is None else out
        pdx, lddx = _view(dx, M, K, x.dtype, dev, "out", align=False)
    if weight is not None if need_params is None else need_params:
        dweight = _out(dweight, (K,), _F32, dev, "dweight")
        dbias = torch.empty_like(dweight) if dbias is None else _out(dbias, (K,), _F32, dev, "dbias")
        ws = _buf(workspace, layer_norm_backward_workspace_bytes(M, K), torch.uint8, dev, "workspace", alloc=16)
        args = dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr()
    else:
        dweight = dbias = None
        args = None, None, None
    _check(_lib.layer_norm_backward(xt, pdy, lddy, px, ldx, pm, pr, M, K, wt, pw, pdx, lddx, *args, _stream(dev)))
    return dx, dweight, dbias


def w8a8_quant_act_rowwise_layer_norm(x, weight=None, bias=None, eps=1e-5, qtype=INT8, ldq=None, out=None, scale=None,
                                      mean=None, rstd=None):
    """Row-wise quantization of layer_norm_forward's f32 values: (codes [M, ldq], scales f32 [M]).  `mean` and
    `rstd` f32 [M] are written if passed in."""
    cd = _code_dtype(qtype)
    dev, M, K, xt, px, ldx, wt, pw, pb = _norm_args(x, weight, bias)
    ldq = ldq if ldq is not None else K + (-K) % 16
    xq = _out(out, (M, ldq), cd, dev, "out")
    if scale is None:
        scale = torch.empty(M, dtype=_F32, device=dev)
    _check(_lib.w8a8_quant_act_rowwise_layer_norm(
        qtype, xt, px, M, K, ldx, wt, pw, pb, eps, xq.data_ptr(), ldq, _vec(scale, M, _F32, dev, "scale"),
        _vec(mean, M, _F32, dev, "mean"), _vec(rstd, M, _F32, dev, "rstd"), _stream(dev)))
    return xq, _first(scale, M)


# ---------------------------------------------------------------- diagnostics
def probe_mfma_i8(a, b, pairs, sink=None):
    """Sustained int8 MFMA loop on operand bytes `a`, `b` (device tensors of at
    least 65536 bytes each): `pairs` iterations of 64 v_mfma_i32_16x16x64_i8
    per wave, one workgroup of 4 waves per CU.  Returns the sink tensor; the
    integer operations are pairs * 32 * 2 * 32**3 * 4 * CUs."""
    import torch
    for t in (a, b):
        if t.numel() * t.element_size() < 65536 or not t.is_contiguous():
            raise ValueError("probe operands: contiguous, at least 65536 bytes")
    n = _lib.w8a8_probe_sink_count()
    sink = _buf(sink, n, torch.int32, a.device, "sink")
    _check(_lib.w8a8_probe_mfma_i8(_ptr(a), _ptr(b), int(pairs), _ptr(sink), _stream(a.device)))
    return sink


def probe_cvt_e4m3(first_bits, n, out=None, device=None):
    """e4m3 codes (uint8 [n], on the GPU) of the f32 values with bit patterns
    first_bits, first_bits + 1, ..., by the quantizers' clamp and conversion."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    codes = _buf(out, n, torch.uint8, dev, "out", alloc=16)
    _check(_lib.w8a8_probe_cvt_e4m3(ctypes.c_uint32(first_bits), n, _ptr(codes), _stream(dev)))
    return codes[:n]


def probe_gemm_tile_n(M, N):
    """Tile width along N (256 or 192) that w8a8_linear and
    w8a8_linear_backward_dx take for an M x N output on the current device."""
    return int(_lib.w8a8_probe_gemm_tile_n(int(M), int(N)))
