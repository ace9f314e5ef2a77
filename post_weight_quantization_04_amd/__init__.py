"""GPTQ layer quantizer for AMD MI355X (gfx950).

Thin Python binding over the C ABI of libgptq.so (include/gptq.h).  Every
stage of the method runs in the library's HIP kernels; this module only
allocates device memory and passes pointers and the current stream.  PyTorch
is used for device memory and streams only.

    H = torch.zeros(d_in, d_in, device="cuda")
    hessian_accumulate(X, H)                       # H += 2 X^T X
    q = quantize_layer(W, H, bits=4, group_size=128, block_size=128,
                       damp=0.01, act_order=False)
    q.qpacked, q.scales, q.zeros, q.perm
    Y = dequant_matmul(A, q)                       # A W_hat^T on the packed layer
    Y = dequant_linear(A, q, bias, "gelu", residual)   # the same with its epilogue fused
    h = dequant_gated(A, gate, up, "silu")         # act(A W_gate^T) * (A W_up^T)
    dA, _ = dequant_linear_backward(dY, q)         # gradients through packed layers
    w = mx_quantize(W, "fp4")                      # microscaled 4-bit weights
    x, S = rms_norm(X, weight, residual=R, format="fp8")   # the norm, its output in 8 bits
    Y = mx_linear(x, w, bias, "silu")              # on the scaled matrix cores

The library must have been built (python -m post_weight_quantization_04_amd.build);
the first call into it raises ImportError if libgptq.so is missing (there is
no fallback path).  The seeded input generator (.synth) does not need it.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from operator import attrgetter

__all__ = [
    "GptqError", "lib", "hessian_accumulate", "hessian_workspace_size", "quantize_layer",
    "quantize_layer_workspace_size", "inverse_factor", "packed_words", "num_groups", "QuantizedLayer",
    "LIB_PATH", "F32", "BF16", "profile_enable", "profile_read", "hessian_accumulate_noalloc",
    "hessian_noalloc_max_d_in", "dequant_matmul", "dequant_matmul_workspace_size", "quantize_layers",
    "ACTIVATIONS", "dequant_linear", "dequant_linear_workspace_size", "dequant_linear_backward",
    "dequant_linear_backward_workspace_size", "dequant_gated", "dequant_gated_workspace_size",
    "dequant_gated_backward", "dequant_gated_backward_workspace_size",
    "MX_FORMATS", "MxTensor", "mx_quantize", "mx_dequantize", "mx_linear", "mx_linear_workspace_size",
    "mx_linear_backward", "mx_linear_backward_workspace_size", "rms_norm", "rms_norm_backward",
    "rms_norm_backward_workspace_size",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgptq.so")
F32, BF16 = 0, 1
MX_FORMATS = {"fp8": 0, "fp4": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_STATUS = {0: "GPTQ_OK", 1: "GPTQ_EINVAL", 2: "GPTQ_ENOTSPD", 3: "GPTQ_EHIP", 4: "GPTQ_ENOMEM"}


class GptqError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = _STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libgptq.so not found at {LIB_PATH}; build it with "
            "`python -m post_weight_quantization_04_amd.build` (there is no fallback path)")
    L = ctypes.CDLL(LIB_PATH)
    c = ctypes
    L.gptq_hessian_workspace_size.argtypes = [c.c_int64, c.c_int64, c.c_int]
    L.gptq_hessian_workspace_size.restype = c.c_size_t
    L.gptq_hessian_accumulate.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_void_p,
                                          c.c_void_p, c.c_size_t, c.c_void_p]
    L.gptq_hessian_accumulate.restype = c.c_int
    L.gptq_hessian_accumulate_noalloc.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_void_p,
                                                  c.c_void_p]
    L.gptq_hessian_accumulate_noalloc.restype = c.c_int
    L.gptq_hessian_noalloc_max_d_in.argtypes = [c.c_int]
    L.gptq_hessian_noalloc_max_d_in.restype = c.c_int64
    L.gptq_quantize_layer_workspace_size.argtypes = [c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_int, c.c_int]
    L.gptq_quantize_layer_workspace_size.restype = c.c_size_t
    L.gptq_quantize_layer.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_void_p, c.c_int, c.c_int,
                                      c.c_int, c.c_float, c.c_int, c.c_void_p, c.c_void_p, c.c_void_p,
                                      c.c_void_p, c.c_void_p, c.c_size_t, c.c_void_p]
    L.gptq_quantize_layer.restype = c.c_int
    L.gptq_dequant_matmul_workspace_size.argtypes = [c.c_int64, c.c_int64, c.c_int64, c.c_int, c.c_int]
    L.gptq_dequant_matmul_workspace_size.restype = c.c_size_t
    L.gptq_dequant_matmul.argtypes = [c.c_void_p, c.c_int, c.c_int64, c.c_int64, c.c_void_p, c.c_void_p, c.c_void_p,
                                      c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_void_p, c.c_int, c.c_void_p,
                                      c.c_size_t, c.c_void_p]
    L.gptq_dequant_matmul.restype = c.c_int
    L.gptq_quantize_layers_workspace_size.argtypes = [c.c_int, c.c_void_p, c.c_int64, c.c_int, c.c_int, c.c_int,
                                                      c.c_int]
    L.gptq_quantize_layers_workspace_size.restype = c.c_size_t
    L.gptq_quantize_layers.argtypes = [c.c_int, c.c_void_p, c.c_int, c.c_void_p, c.c_int64, c.c_void_p, c.c_int,
                                       c.c_int, c.c_int, c.c_float, c.c_int, c.c_void_p, c.c_void_p, c.c_void_p,
                                       c.c_void_p, c.c_void_p, c.c_size_t, c.c_void_p]
    L.gptq_quantize_layers.restype = c.c_int
    i64, i32, ptr, size = c.c_int64, c.c_int, c.c_void_p, c.c_size_t
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        f = getattr(L, f"gptq_dequant_{name}_workspace_size")
        f.argtypes = [i64, i64, i64, i32, i32, i32, i32]
        f.restype = size
    L.gptq_dequant_linear.argtypes = [ptr, i32, i64, i64, ptr, ptr, ptr, ptr, i64, i32, i32, ptr, i32, i32, ptr,
                                      ptr, i32, ptr, ptr, size, ptr]
    L.gptq_dequant_linear_backward.argtypes = [ptr, i32, i64, i64, ptr, i32, ptr, ptr, ptr, ptr, i64, i32, i32, ptr,
                                               i32, ptr, ptr, size, ptr]
    L.gptq_dequant_gated.argtypes = [ptr, i32, i64, i64, ptr, ptr, ptr, ptr, ptr, ptr, ptr, i64, i32, i32, ptr, ptr,
                                     i32, i32, ptr, i32, ptr, ptr, ptr, size, ptr]
    L.gptq_dequant_gated_backward.argtypes = [ptr, i32, i64, i64, ptr, ptr, i32, ptr, ptr, ptr, ptr, ptr, ptr, ptr,
                                              i64, i32, i32, ptr, i32, ptr, ptr, ptr, size, ptr]
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        getattr(L, f"gptq_dequant_{name}").restype = i32
    f64 = c.c_double
    for name, args in {
            "mx_quantize": [ptr, i32, i64, i64, i32, ptr, ptr, ptr],
            "mx_dequantize": [ptr, ptr, i32, i64, i64, ptr, i32, ptr],
            "mx_linear": [ptr, i32, i64, i64, ptr, ptr, i64, ptr, i32, i32, ptr, ptr, i32, ptr, ptr, size, ptr],
            "mx_linear_mx": [ptr, ptr, i32, i64, i64, ptr, ptr, i64, ptr, i32, i32, ptr, ptr, i32, ptr, ptr, size, ptr],
            "mx_linear_backward": [ptr, i32, i64, i64, ptr, i32, ptr, ptr, i64, ptr, i32, ptr, ptr, size, ptr],
            "rms_norm": [ptr, ptr, ptr, i32, i64, i64, f64, ptr, ptr, ptr],
            "rms_norm_mx": [ptr, ptr, ptr, i32, i64, i64, f64, ptr, i32, ptr, ptr, ptr],
            "rms_norm_backward": [ptr, ptr, ptr, ptr, i32, i64, i64, f64, ptr, ptr, ptr, size, ptr]}.items():
        f = getattr(L, f"gptq_{name}")
        f.argtypes, f.restype = args, i32
    for name in ("mx_linear", "mx_linear_mx", "mx_linear_backward"):
        f = getattr(L, f"gptq_{name}_workspace_size")
        f.argtypes, f.restype = [i64, i64, i64, i32, i32], size
    L.gptq_rms_norm_backward_workspace_size.argtypes = [i64, i64]
    L.gptq_rms_norm_backward_workspace_size.restype = size
    L.gptq_mx_row_bytes.argtypes, L.gptq_mx_row_bytes.restype = [i64, i32], i64
    L.gptq_mx_steps.argtypes, L.gptq_mx_steps.restype = [i64], i64
    L.gptq_inverse_factor.argtypes = [c.c_void_p, c.c_int64, c.c_float, c.c_int, c.c_void_p, c.c_void_p,
                                      c.c_void_p, c.c_size_t, c.c_void_p]
    L.gptq_inverse_factor.restype = c.c_int
    L.gptq_packed_words.argtypes = [c.c_int64, c.c_int]
    L.gptq_packed_words.restype = c.c_int64
    L.gptq_num_groups.argtypes = [c.c_int64, c.c_int]
    L.gptq_num_groups.restype = c.c_int64
    L.gptq_status_string.argtypes = [c.c_int]
    L.gptq_status_string.restype = c.c_char_p
    L.gptq_last_error.argtypes = []
    L.gptq_last_error.restype = c.c_char_p
    L.gptq_version.argtypes = []
    L.gptq_version.restype = c.c_char_p
    L.gptq_profile_enable.argtypes = [c.c_int]
    L.gptq_profile_enable.restype = None
    L.gptq_profile_read.argtypes = [c.POINTER(_Profile), c.c_int]
    L.gptq_profile_read.restype = c.c_int
    L.gptq_profile_stage_name.argtypes = [c.c_int]
    L.gptq_profile_stage_name.restype = c.c_char_p
    return L


NUM_STAGES = 8


class _Profile(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * NUM_STAGES), ("launches", ctypes.c_int64 * NUM_STAGES)]


def profile_enable(on=True) -> None:
    """Record hipEvents around stage launches (see gptq_profile_enable): True
    times every stage, False none, an int is the stage bit mask."""
    if isinstance(on, bool):
        mask = (1 << NUM_STAGES) - 1 if on else 0
    else:
        mask = int(on)
    _lib().gptq_profile_enable(mask)


def profile_read(reset: bool = True) -> dict:
    """{stage name: (summed GPU ms, timed launch groups)} since the last reset."""
    p = _Profile()
    _check(_lib().gptq_profile_read(ctypes.byref(p), int(bool(reset))))
    return {_lib().gptq_profile_stage_name(i).decode(): (p.ms[i], int(p.launches[i])) for i in range(NUM_STAGES)}


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def _check(status: int) -> None:
    if status != 0:
        raise GptqError(status, _lib().gptq_last_error().decode(errors="replace"))


_TORCH = _FORWARD_AD = _RAW_STREAM = _CURRENT_DEVICE = None


def _torch():
    global _TORCH, _FORWARD_AD, _RAW_STREAM, _CURRENT_DEVICE
    if _TORCH is None:
        import torch  # memory and streams only
        # The current stream's handle without a Stream object around it, and the
        # current device without a check of the runtime: entry points that torch does
        # not promise, so that the public ones serve where they are missing.
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _TORCH, _FORWARD_AD = torch, torch.autograd.forward_ad
    return _TORCH


def _dual_level() -> bool:
    """Whether tensors may carry forward-mode tangents (yes where torch does not tell)."""
    return getattr(_FORWARD_AD, "_current_level", 0) >= 0


def _stream_ptr(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _require(t, name, dtype=None, ndim=None, device=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def packed_words(d_in: int, bits: int) -> int:
    return int(_lib().gptq_packed_words(d_in, bits))


def num_groups(d_in: int, group_size: int) -> int:
    return int(_lib().gptq_num_groups(d_in, group_size))


def hessian_workspace_size(n: int, d_in: int, dtype_code: int) -> int:
    return int(_lib().gptq_hessian_workspace_size(n, d_in, dtype_code))


def _workspace(nbytes: int, device, workspace=None):
    torch = _torch()
    if nbytes == 0:
        return None
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def hessian_accumulate(X, H, workspace=None, stream=None) -> None:
    """H += 2 X^T X.  X: [n, d_in] float32/bfloat16 (device); H: [d_in, d_in] float32."""
    torch = _torch()
    _require(X, "X", ndim=2)
    _require(H, "H", dtype=torch.float32, ndim=2)
    n, d = X.shape
    if H.shape != (d, d):
        raise ValueError(f"H must be [{d}, {d}]")
    code = _dtype_code(X)
    ws = _workspace(hessian_workspace_size(n, d, code), X.device, workspace)
    _check(_lib().gptq_hessian_accumulate(X.data_ptr() if n else None, code, n, d, H.data_ptr(),
                                       ws.data_ptr() if ws is not None else None,
                                       0 if ws is None else ws.numel(), _stream_ptr(stream)))


def hessian_accumulate_noalloc(X, H, stream=None) -> None:
    """H += 2 X^T X with the library's static scratch instead of a workspace
    (gptq_hessian_accumulate_noalloc: nothing is allocated; calls that overlap
    on one GPU race)."""
    torch = _torch()
    _require(X, "X", ndim=2)
    _require(H, "H", dtype=torch.float32, ndim=2)
    n, d = X.shape
    if H.shape != (d, d):
        raise ValueError(f"H must be [{d}, {d}]")
    _check(_lib().gptq_hessian_accumulate_noalloc(X.data_ptr() if n else None, _dtype_code(X), n, d, H.data_ptr(),
                                                  _stream_ptr(stream)))


def hessian_noalloc_max_d_in(dtype_code: int) -> int:
    return int(_lib().gptq_hessian_noalloc_max_d_in(dtype_code))


def quantize_layer_workspace_size(d_out, d_in, bits, group_size, block_size, act_order) -> int:
    return int(_lib().gptq_quantize_layer_workspace_size(d_out, d_in, bits, group_size, block_size, int(act_order)))


@dataclass
class QuantizedLayer:
    qpacked: "object"   # uint32 words, torch.int32 view [words, d_out]
    scales: "object"    # float32 [groups, d_out]
    zeros: "object"     # float32 [groups, d_out]
    perm: "object"      # int32 [d_in]
    bits: int
    group_size: int     # effective group size
    d_in: int
    act_order: bool = True   # False: perm is the identity (products then skip the gather)


def quantize_layer(W, H, bits: int = 4, group_size: int = 128, block_size: int = 128, damp: float = 0.01,
                   act_order: bool = False, workspace=None, stream=None) -> QuantizedLayer:
    """Quantize one layer.  W: [d_out, d_in] float32/bfloat16; H: [d_in, d_in] float32 (undamped)."""
    torch = _torch()
    _require(W, "W", ndim=2)
    _require(H, "H", dtype=torch.float32, ndim=2)
    d_out, d_in = W.shape
    if H.shape != (d_in, d_in):
        raise ValueError(f"H must be [{d_in}, {d_in}]")
    G = num_groups(d_in, group_size)
    nw = packed_words(d_in, bits)
    if G < 1 or nw < 0:
        raise GptqError(1, "invalid group_size or bits")
    dev = W.device
    q = torch.empty((max(nw, 0), d_out), dtype=torch.int32, device=dev)
    sc = torch.empty((G, d_out), dtype=torch.float32, device=dev)
    zr = torch.empty((G, d_out), dtype=torch.float32, device=dev)
    pm = torch.empty((d_in,), dtype=torch.int32, device=dev)
    need = quantize_layer_workspace_size(d_out, d_in, bits, group_size, block_size, act_order)
    ws = _workspace(need, dev, workspace)
    _check(_lib().gptq_quantize_layer(W.data_ptr(), _dtype_code(W), d_out, d_in, H.data_ptr(), bits, group_size,
                                   block_size, float(damp), int(bool(act_order)), q.data_ptr(), sc.data_ptr(),
                                   zr.data_ptr(), pm.data_ptr(), ws.data_ptr() if ws is not None else None,
                                   0 if ws is None else ws.numel(), _stream_ptr(stream)))
    g_eff = d_in if (group_size == -1 or group_size >= d_in) else group_size
    return QuantizedLayer(q, sc, zr, pm, bits, g_eff, d_in, bool(act_order))


def quantize_layers(Ws, H, bits: int = 4, group_size: int = 128, block_size: int = 128, damp: float = 0.01,
                    act_order: bool = False, workspace=None, stream=None):
    """Quantize several layers that share the input, hence H (gptq_quantize_layers):
    one factorization, then each W [d_out_l, d_in] as quantize_layer would.
    Returns a list of QuantizedLayer sharing one perm."""
    torch = _torch()
    Ws = list(Ws)
    if not Ws:
        raise ValueError("no layers")
    _require(H, "H", dtype=torch.float32, ndim=2)
    d_in = H.shape[0]
    code = None
    for W in Ws:
        _require(W, "W", ndim=2)
        if W.shape[1] != d_in:
            raise ValueError(f"every W must have {d_in} columns")
        c = _dtype_code(W)
        if code is not None and c != code:
            raise TypeError("every W must have the same dtype")
        code = c
    n = len(Ws)
    G = num_groups(d_in, group_size)
    nw = packed_words(d_in, bits)
    if G < 1 or nw < 0:
        raise GptqError(1, "invalid group_size or bits")
    dev = Ws[0].device
    d_outs = (ctypes.c_int64 * n)(*[W.shape[0] for W in Ws])
    outs = [(torch.empty((nw, W.shape[0]), dtype=torch.int32, device=dev),
             torch.empty((G, W.shape[0]), dtype=torch.float32, device=dev),
             torch.empty((G, W.shape[0]), dtype=torch.float32, device=dev)) for W in Ws]
    pm = torch.empty((d_in,), dtype=torch.int32, device=dev)
    ptrs = lambda xs: (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    need = int(_lib().gptq_quantize_layers_workspace_size(n, d_outs, d_in, bits, group_size, block_size,
                                                           int(act_order)))
    ws = _workspace(need, dev, workspace)
    _check(_lib().gptq_quantize_layers(n, ptrs(Ws), code, d_outs, d_in, H.data_ptr(), bits, group_size, block_size,
                                       float(damp), int(bool(act_order)), ptrs([o[0] for o in outs]),
                                       ptrs([o[1] for o in outs]), ptrs([o[2] for o in outs]), pm.data_ptr(),
                                       ws.data_ptr() if ws is not None else None, 0 if ws is None else ws.numel(),
                                       _stream_ptr(stream)))
    g_eff = d_in if (group_size == -1 or group_size >= d_in) else group_size
    return [QuantizedLayer(o[0], o[1], o[2], pm, bits, g_eff, d_in, bool(act_order)) for o in outs]


def dequant_matmul_workspace_size(m, d_out, d_in, bits, group_size) -> int:
    return int(_lib().gptq_dequant_matmul_workspace_size(m, d_out, d_in, bits, group_size))


def dequant_matmul(A, q: "QuantizedLayer", out_dtype=None, workspace=None, stream=None, use_perm=None):
    """Y = A W_hat^T on the packed layer q (gptq_dequant_matmul).  A: [m, d_in]
    bfloat16/float32 activations in the original column order; returns Y
    [m, d_out] in out_dtype (float32 by default, or bfloat16).  A workspace
    passed in must have been zeroed before its first use (calls leave it so).
    use_perm: gather A through q.perm (default: when q was quantized with
    act-order; otherwise perm is the identity and is not passed)."""
    torch = _torch()
    _require(A, "A", ndim=2)
    m, d_in = A.shape
    if d_in != q.d_in:
        raise ValueError(f"A has {d_in} columns, the layer {q.d_in}")
    d_out = q.scales.shape[1]
    out_dtype = out_dtype or torch.float32
    if use_perm is None:
        use_perm = q.act_order
    Y = torch.empty((m, d_out), dtype=out_dtype, device=A.device)
    need = dequant_matmul_workspace_size(m, d_out, d_in, q.bits, q.group_size)
    # zeroed before its first use (completion counters); calls leave it so
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        ws = workspace
    else:
        ws = torch.zeros(need, dtype=torch.uint8, device=A.device) if need else None
    _check(_lib().gptq_dequant_matmul(A.data_ptr() if m else None, _dtype_code(A), m, d_in, q.qpacked.data_ptr(),
                                      q.scales.data_ptr(), q.zeros.data_ptr(),
                                      q.perm.data_ptr() if use_perm else None, d_out, q.bits, q.group_size,
                                      Y.data_ptr(), _dtype_code(Y), ws.data_ptr() if ws is not None else None,
                                      0 if ws is None else ws.numel(), _stream_ptr(stream)))
    return Y


# ---------------------------------------------------------------------------
# fused products with packed layers, forward and backward
# ---------------------------------------------------------------------------
def dequant_linear_workspace_size(m, d_out, d_in, bits, group_size, a_dtype_code, y_dtype_code) -> int:
    return int(_lib().gptq_dequant_linear_workspace_size(m, d_out, d_in, bits, group_size, a_dtype_code,
                                                         y_dtype_code))


def dequant_linear_backward_workspace_size(m, d_out, d_in, bits, group_size, dy_dtype_code, da_dtype_code) -> int:
    return int(_lib().gptq_dequant_linear_backward_workspace_size(m, d_out, d_in, bits, group_size, dy_dtype_code,
                                                                  da_dtype_code))


def dequant_gated_workspace_size(m, d_ff, d_in, bits, group_size, a_dtype_code, y_dtype_code) -> int:
    return int(_lib().gptq_dequant_gated_workspace_size(m, d_ff, d_in, bits, group_size, a_dtype_code, y_dtype_code))


def dequant_gated_backward_workspace_size(m, d_ff, d_in, bits, group_size, dy_dtype_code, da_dtype_code) -> int:
    return int(_lib().gptq_dequant_gated_backward_workspace_size(m, d_ff, d_in, bits, group_size, dy_dtype_code,
                                                                 da_dtype_code))


def _operand(t, name, dtype, shape, device) -> int:
    """The device pointer of a packed tensor of this dtype and shape on `device`; raises otherwise."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _require(t, name, dtype=dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


class _FusedCall:
    """Checks and buffers of one fused call: operands on one device, a
    workspace and outputs that belong to the stream the work goes to."""
    __slots__ = ("device", "in_code", "act", "out_dtype", "out_code", "d_in", "d_out", "words", "groups", "perm",
                 "bits", "group", "stream", "given_ws", "guard")

    def __init__(self, x, name, q, activation, out_dtype, workspace, stream):
        torch = _torch()
        _require(x, name, ndim=2)
        self.in_code = _dtype_code(x)
        device = self.device = x.device
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}; got {activation!r}")
        self.act = ACTIVATIONS[activation]
        self.out_dtype = out_dtype or x.dtype
        if self.out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"unsupported out_dtype {self.out_dtype}; use float32 or bfloat16")
        self.out_code = F32 if self.out_dtype == torch.float32 else BF16
        self.d_in, self.d_out, self.bits, self.group = q.d_in, q.scales.shape[1], q.bits, q.group_size
        one = self.group == -1 or self.group >= self.d_in
        self.words = -(-self.bits * self.d_in // 32)
        self.groups = 1 if one or self.group < 1 else -(-self.d_in // self.group)
        self.perm = _operand(q.perm, "perm", torch.int32, (self.d_in,), device) if q.act_order else None
        self.guard = None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream belongs to {stream.device}, {name} to {device}")
            self.stream = stream.cuda_stream
            self.guard = torch.cuda.stream(stream)
        else:
            self.stream = _RAW_STREAM(device.index)
            if device.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(device)
        self.given_ws = workspace
        if workspace is not None:
            _operand(workspace, "workspace", workspace.dtype, workspace.shape, device)
        self.no_grad(x, q.scales, q.zeros)

    def layer(self, q):
        """A packed layer's pointers (codes, scales, zero points)."""
        torch = _torch()
        params = (self.groups, self.d_out)
        return (_operand(q.qpacked, "qpacked", torch.int32, (self.words, self.d_out), self.device),
                _operand(q.scales, "scales", torch.float32, params, self.device),
                _operand(q.zeros, "zeros", torch.float32, params, self.device))

    def pair(self, gate, up):
        if (up.d_in, up.bits, up.group_size, up.scales.shape[1]) != (self.d_in, self.bits, self.group, self.d_out):
            raise ValueError("the layers must have the same sizes, bits and group_size")
        if up.act_order != gate.act_order or (up.act_order and not self.same_order(gate.perm, up.perm)):
            raise ValueError("the layers must share one perm (quantize_layers gives them one)")
        self.no_grad(up.scales, up.zeros)

    def same_order(self, a, b):
        """One tensor, or two of equal values (compared on the call's stream, and waited for)."""
        if _operand(b, "perm", a.dtype, a.shape, self.device) == self.perm:
            return True
        torch = _torch()
        with self:
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("during a graph's capture the layers must share one perm tensor (two cannot be "
                                 "compared)")
            return torch.equal(a, b)

    def take(self, t, name, dtype, shape):
        """An optional operand's pointer."""
        if t is None:
            return None
        p = _operand(t, name, dtype, shape, self.device)
        self.no_grad(t)
        return p

    @staticmethod
    def no_grad(*tensors):
        """Raises for operands whose gradients, or forward-mode tangents, would be dropped."""
        if _TORCH.is_grad_enabled():
            for t in tensors:
                if t.requires_grad:
                    raise ValueError("autograd does not see through the fused products: call them under "
                                     "torch.no_grad() (or inside a torch.autograd.Function) and their _backward "
                                     "calls for the gradients")
        if _dual_level():
            for t in tensors:
                if _FORWARD_AD.unpack_dual(t).tangent is not None:
                    raise ValueError("forward-mode tangents do not pass through the fused products: give them the "
                                     "primals of dual tensors")

    def empty(self, shape, dtype=None):
        return _torch().empty(shape, dtype=dtype or self.out_dtype, device=self.device)

    def workspace(self, need):
        """(owner, pointer, bytes): the caller's when it suffices, otherwise allocated."""
        w = self.given_ws
        if w is not None and w.numel() * w.element_size() >= need:
            return w, w.data_ptr(), w.numel() * w.element_size()
        if need == 0:
            return None, None, 0
        w = self.empty((need,), dtype=_torch().uint8)
        return w, w.data_ptr(), need

    def __enter__(self):
        # allocations belong to the stream that uses them, on its own device
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def dequant_linear(A, q: "QuantizedLayer", bias=None, activation="none", residual=None, out_dtype=None,
                   save_preact=False, workspace=None, stream=None):
    """Y = act(A W_hat^T + bias) + residual on the packed layer q (gptq_dequant_linear).

    A: [m, d_in] bfloat16/float32; bias: [d_out] bfloat16/float32; residual:
    [m, d_out] of out_dtype (A's dtype by default); activation: one of
    ACTIVATIONS.  Returns Y, or (Y, Z) with the pre-activation Z = A W_hat^T +
    bias when save_preact.  workspace: any 256-byte aligned device tensor of at least
    dequant_linear_workspace_size bytes (allocated when absent or too small).
    With a bfloat16 result the weights, and float32 activations, may be rounded
    to 11 bits on the way; out_dtype=torch.float32 holds them to 22.
    Not differentiable by autograd: see dequant_linear_backward."""
    f = _FusedCall(A, "A", q, activation, out_dtype, workspace, stream)
    m, d_in = A.shape
    if d_in != f.d_in:
        raise ValueError(f"A has {d_in} columns, the layer {f.d_in}")
    Qp, Sp, Zp = f.layer(q)
    b = f.take(bias, "bias", bias.dtype, (f.d_out,)) if bias is not None else None
    bcode = _dtype_code(bias) if bias is not None else 0
    r = f.take(residual, "residual", f.out_dtype, (m, f.d_out))
    with f:
        Y = f.empty((m, f.d_out))
        Z = f.empty((m, f.d_out)) if save_preact else None
        _own, ws, wsb = f.workspace(dequant_linear_workspace_size(m, f.d_out, d_in, f.bits, f.group, f.in_code,
                                                                  f.out_code))
        _check(_lib().gptq_dequant_linear(A.data_ptr(), f.in_code, m, d_in, Qp, Sp, Zp, f.perm, f.d_out, f.bits,
                                          f.group, b, bcode, f.act, r, Y.data_ptr(), f.out_code,
                                          Z.data_ptr() if save_preact else None, ws, wsb, f.stream))
    return (Y, Z) if save_preact else Y


def dequant_linear_backward(dY, q: "QuantizedLayer", activation="none", preact=None, bias_grad=False, out_dtype=None,
                            workspace=None, stream=None):
    """(dA, dbias) of dequant_linear (gptq_dequant_linear_backward): dZ = dY act'(Z),
    dA = dZ W_hat, dbias the column sums of dZ.

    dY: [m, d_out] bfloat16/float32; preact: the saved Z of dY's dtype (may be
    None for activation "none").  dA: [m, d_in] in out_dtype (dY's dtype by
    default); dbias: [d_out] float32, or None unless bias_grad.  The residual's
    gradient is dY itself."""
    f = _FusedCall(dY, "dY", q, activation, out_dtype, workspace, stream)
    m, d_out = dY.shape
    if d_out != f.d_out:
        raise ValueError(f"dY has {d_out} columns, the layer {f.d_out} rows")
    if preact is None and f.act:
        raise ValueError("preact is required unless activation is 'none'")
    Qp, Sp, Zp = f.layer(q)
    z = f.take(preact, "preact", dY.dtype, (m, d_out))
    with f:
        dA = f.empty((m, f.d_in))
        db = f.empty((d_out,), dtype=_torch().float32) if bias_grad else None
        _own, ws, wsb = f.workspace(dequant_linear_backward_workspace_size(m, d_out, f.d_in, f.bits, f.group,
                                                                           f.in_code, f.out_code))
        _check(_lib().gptq_dequant_linear_backward(dY.data_ptr(), f.in_code, m, d_out, z, f.act, Qp, Sp, Zp, f.perm,
                                                   f.d_in, f.bits, f.group, dA.data_ptr(), f.out_code,
                                                   db.data_ptr() if bias_grad else None, ws, wsb, f.stream))
    return dA, db


def dequant_gated(A, gate: "QuantizedLayer", up: "QuantizedLayer", activation="silu", bias_gate=None, bias_up=None,
                  out_dtype=None, save_preact=False, workspace=None, stream=None):
    """H = act(A W_gate^T + bias_gate) * (A W_up^T + bias_up) (gptq_dequant_gated):
    the gated half of a feed-forward block in one call.

    gate, up: packed layers of the same sizes, bits and group_size sharing one
    perm (quantize_layers).  Equal perms in two tensors, as a reload gives, are
    taken too, but comparing them waits for the device at every call and cannot
    be captured: give both layers one tensor (up.perm = gate.perm).  Returns H [m, d_ff] in out_dtype (A's dtype by
    default), or (H, G, U) with both pre-activations when save_preact.  Other
    arguments as for dequant_linear."""
    f = _FusedCall(A, "A", gate, activation, out_dtype, workspace, stream)
    m, d_in = A.shape
    if d_in != f.d_in:
        raise ValueError(f"A has {d_in} columns, the layers {f.d_in}")
    f.pair(gate, up)
    Qg, Sg, Zg = f.layer(gate)
    Qu, Su, Zu = f.layer(up)
    biases = [b for b in (bias_gate, bias_up) if b is not None]
    if len(biases) == 2 and biases[0].dtype != biases[1].dtype:
        raise TypeError("both biases must have the same dtype")
    bdtype, bcode = (biases[0].dtype, _dtype_code(biases[0])) if biases else (None, 0)
    bg = f.take(bias_gate, "bias_gate", bdtype, (f.d_out,))
    bu = f.take(bias_up, "bias_up", bdtype, (f.d_out,))
    with f:
        H = f.empty((m, f.d_out))
        G, U = (f.empty((m, f.d_out)), f.empty((m, f.d_out))) if save_preact else (None, None)
        _own, ws, wsb = f.workspace(dequant_gated_workspace_size(m, f.d_out, d_in, f.bits, f.group, f.in_code,
                                                                 f.out_code))
        _check(_lib().gptq_dequant_gated(A.data_ptr(), f.in_code, m, d_in, Qg, Sg, Zg, Qu, Su, Zu, f.perm, f.d_out,
                                         f.bits, f.group, bg, bu, bcode, f.act, H.data_ptr(), f.out_code,
                                         G.data_ptr() if save_preact else None,
                                         U.data_ptr() if save_preact else None, ws, wsb, f.stream))
    return (H, G, U) if save_preact else H


def dequant_gated_backward(dH, gate: "QuantizedLayer", up: "QuantizedLayer", gate_pre, up_pre, activation="silu",
                           bias_grad=False, out_dtype=None, workspace=None, stream=None):
    """(dA, dbias_gate, dbias_up) of dequant_gated (gptq_dequant_gated_backward):
    dG = dH U act'(G), dU = dH act(G), dA = dG W_gate + dU W_up, and the column
    sums of dG and dU.

    dH, gate_pre (G), up_pre (U): [m, d_ff], one dtype (G and U as
    dequant_gated saved them).  dA: [m, d_in] in out_dtype (dH's dtype by
    default); the bias gradients: [d_ff] float32, or None unless bias_grad."""
    f = _FusedCall(dH, "dH", gate, activation, out_dtype, workspace, stream)
    m, d_ff = dH.shape
    if d_ff != f.d_out:
        raise ValueError(f"dH has {d_ff} columns, the layers {f.d_out} rows")
    if gate_pre is None or up_pre is None:
        raise ValueError("gate_pre and up_pre are required")
    f.pair(gate, up)
    Qg, Sg, Zg = f.layer(gate)
    Qu, Su, Zu = f.layer(up)
    g = f.take(gate_pre, "gate_pre", dH.dtype, (m, d_ff))
    u = f.take(up_pre, "up_pre", dH.dtype, (m, d_ff))
    with f:
        f32 = _torch().float32
        dA = f.empty((m, f.d_in))
        dbg, dbu = (f.empty((d_ff,), dtype=f32), f.empty((d_ff,), dtype=f32)) if bias_grad else (None, None)
        _own, ws, wsb = f.workspace(dequant_gated_backward_workspace_size(m, d_ff, f.d_in, f.bits, f.group,
                                                                          f.in_code, f.out_code))
        _check(_lib().gptq_dequant_gated_backward(dH.data_ptr(), f.in_code, m, d_ff, g, u, f.act, Qg, Sg, Zg, Qu, Su,
                                                  Zu, f.perm, f.d_in, f.bits, f.group, dA.data_ptr(), f.out_code,
                                                  dbg.data_ptr() if bias_grad else None,
                                                  dbu.data_ptr() if bias_grad else None, ws, wsb, f.stream))
    return dA, dbg, dbu


# ---------------------------------------------------------------------------
# microscaled (MX) formats, products with MX weights, and the norm before them
# ---------------------------------------------------------------------------
class MxTensor:
    """A matrix [rows, d] in blocks of 32 columns that share a power of two
    (gptq.h has the layout): codes uint8 [rows, row bytes], scales uint8
    [ceil(d / 128), rows, 4], format "fp8" (e4m3) or "fp4" (e2m1).

    Made from codes and scales of other origin, it needs zeros in what pads the
    columns to whole 128: codes 0 behind column d, scale bytes 0 of the blocks
    that lie behind it.  Sizes and types are checked at every call, this is
    not, and the products add whatever lies there."""
    __slots__ = ("_codes", "_scales", "_buffer", "_rows", "_format", "_d")
    # (what the kernels index by stays what the memory was laid out for)
    rows, format, d = (property(attrgetter(name)) for name in ("_rows", "_format", "_d"))

    def __init__(self, codes, scales, format, d):
        self._codes, self._scales, self._buffer = codes, scales, None
        self._rows, self._format, self._d = codes.shape[0], format, d

    @classmethod
    def _empty(cls, rows, d, format, device):
        """One allocation, codes before scales; its two views are made when asked for."""
        t = cls.__new__(cls)
        t._codes = t._scales = None
        t._rows, t._format, t._d = rows, format, d
        steps = -(-d // 128)
        t._buffer = _TORCH.empty_strided((rows * steps * (68 if format == "fp4" else 132),), (1,),
                                         dtype=_TORCH.uint8, device=device)
        return t

    def _split(self):
        row = _mx_row_bytes(self.d, self.format)
        n = self.rows * row
        self._codes = self._buffer[:n].view(self.rows, row)
        self._scales = self._buffer[n:].view(-(-self.d // 128), self.rows, 4)

    @property
    def codes(self):
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._split()
        return self._scales

    @property
    def shape(self):
        return (self.rows, self.d)

    @property
    def device(self):
        return (self._codes if self._buffer is None else self._buffer).device

    def _pointers(self, name, device):
        """The device pointers of codes and scales; raises if they do not fit the matrix."""
        b = self._buffer
        if b is not None and b.device == device:
            p = b.data_ptr()
            return p, p + self.rows * _mx_row_bytes(self.d, self.format)
        c, s, u8 = self.codes, self.scales, _TORCH.uint8
        codes = (self.rows, _mx_row_bytes(self.d, self.format))
        scales = (-(-self.d // 128), self.rows, 4)
        if (c.dtype is u8 and s.dtype is u8 and c.shape == codes and s.shape == scales and c.device == device
                and s.device == device and c.is_contiguous() and s.is_contiguous()):
            return c.data_ptr(), s.data_ptr()
        return _operand(c, f"{name}.codes", u8, codes, device), _operand(s, f"{name}.scales", u8, scales, device)


def _mx_row_bytes(d, format):
    return -(-d // 128) * (64 if format == "fp4" else 128)


def _mx_format(format) -> int:
    if format not in MX_FORMATS:
        raise ValueError(f"format must be one of {', '.join(MX_FORMATS)}; got {format!r}")
    return MX_FORMATS[format]


def _mx_tensor(t, name, format=None):
    if not isinstance(t, MxTensor):
        raise TypeError(f"{name} must be an MxTensor")
    if t.format not in MX_FORMATS:
        _mx_format(t.format)
    if format is not None and t.format != format:
        raise ValueError(f"{name} must be in {format}, got {t.format}")
    if t._buffer is None:
        _require(t._codes, f"{name}.codes", ndim=2)


class _Here:
    """No change of device or stream."""
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()


def _place(device, name, stream):
    """(stream handle, context that allocations belong into) of a call whose operand `name` is on `device`."""
    if stream is None:
        i = device.index
        return _RAW_STREAM(i), _HERE if i == _CURRENT_DEVICE() else _TORCH.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, {name} to {device}")
    return stream.cuda_stream, _TORCH.cuda.stream(stream)


def _no_grad(*tensors):
    """Raises for operands whose gradients, or forward-mode tangents, would be dropped (None: no operand)."""
    if _TORCH.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                _FusedCall.no_grad(t)
    if _dual_level():
        _FusedCall.no_grad(*[t for t in tensors if t is not None])


def _empty2(rows, cols, dtype, device):
    # (the strides given: a third less time than torch.empty takes)
    return _TORCH.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _scratch(workspace, need, device):
    """(owner, pointer, bytes) of a workspace: the caller's when it suffices, otherwise allocated."""
    if workspace is not None:
        _operand(workspace, "workspace", workspace.dtype, workspace.shape, device)
        n = workspace.numel() * workspace.element_size()
        if n >= need:
            return workspace, workspace.data_ptr(), n
    if need == 0:
        return None, None, 0
    w = _TORCH.empty_strided((need,), (1,), dtype=_TORCH.uint8, device=device)
    return w, w.data_ptr(), need


def _out_code(dtype, name="out_dtype") -> int:
    if dtype is _TORCH.bfloat16:
        return BF16
    if dtype is _TORCH.float32:
        return F32
    raise TypeError(f"unsupported {name} {dtype}; use float32 or bfloat16")


def _activation(activation) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}; got {activation!r}")
    return ACTIVATIONS[activation]


def mx_quantize(X, format="fp4", stream=None) -> MxTensor:
    """X [rows, d] bfloat16/float32 in an MX format (gptq_mx_quantize): "fp4"
    for weights, "fp8" or "fp4" for activations."""
    _require(X, "X", ndim=2)
    code, fmt = _dtype_code(X), _mx_format(format)
    _no_grad(X)
    device = X.device
    st, where = _place(device, "X", stream)
    rows, d = X.shape
    with where:
        t = MxTensor._empty(rows, d, format, device)
        codes, scales = t._pointers("t", device)
        _check(_lib().gptq_mx_quantize(X.data_ptr(), code, rows, d, fmt, codes, scales, st))
    return t


def mx_dequantize(t: MxTensor, dtype=None, stream=None):
    """The values [rows, d] of t in float32 (exact; the default) or bfloat16 (gptq_mx_dequantize)."""
    torch = _torch()
    _mx_tensor(t, "t")
    dtype = dtype or torch.float32
    code = _out_code(dtype, "dtype")
    device = t.device
    st, where = _place(device, "t", stream)
    codes, scales = t._pointers("t", device)
    with where:
        Y = _empty2(t.rows, t.d, dtype, device)
        _check(_lib().gptq_mx_dequantize(codes, scales, MX_FORMATS[t.format], t.rows, t.d, Y.data_ptr(), code, st))
    return Y


def mx_linear_workspace_size(m, d_out, d_in, a_kind, y_dtype_code) -> int:
    """a_kind: the activations' dtype code (F32, BF16) or MX format ("fp8", "fp4")."""
    if isinstance(a_kind, str):
        return _lib().gptq_mx_linear_mx_workspace_size(m, d_out, d_in, _mx_format(a_kind), y_dtype_code)
    return _lib().gptq_mx_linear_workspace_size(m, d_out, d_in, a_kind, y_dtype_code)


def mx_linear_backward_workspace_size(m, d_out, d_in, dy_dtype_code, da_dtype_code) -> int:
    return _lib().gptq_mx_linear_backward_workspace_size(m, d_out, d_in, dy_dtype_code, da_dtype_code)


def mx_linear(A, w: MxTensor, bias=None, activation="none", residual=None, out_dtype=None, save_preact=False,
              workspace=None, stream=None):
    """Y = act(A W^T + bias) + residual with MX weights w [d_out, d_in] in "fp4"
    (gptq_mx_linear, gptq_mx_linear_mx).

    A: [m, d_in], a bfloat16/float32 tensor (weights alone in 4 bits) or an
    MxTensor in "fp8" or "fp4" (both operands enter the scaled matrix cores as
    they are stored).  out_dtype: A's dtype by default, bfloat16 for an
    MxTensor.  Other arguments and the result as for dequant_linear.
    Not differentiable by autograd: see mx_linear_backward."""
    torch = _torch()
    _mx_tensor(w, "w", "fp4")
    mx = isinstance(A, MxTensor)
    if mx:
        _mx_tensor(A, "A")
        kind, dtype = A.format, out_dtype or torch.bfloat16
    else:
        _require(A, "A", ndim=2)
        kind, dtype = _dtype_code(A), out_dtype or A.dtype
    act, code, device = _activation(activation), _out_code(dtype), A.device
    st, where = _place(device, "A", stream)
    (m, d_in), d_out = A.shape, w.rows
    if d_in != w.d:
        raise ValueError(f"A has {d_in} columns, the layer {w.d}")
    codes, scales = w._pointers("w", device)
    b, bcode, r = None, 0, None
    if bias is not None:
        b, bcode = _operand(bias, "bias", bias.dtype, (d_out,), device), _dtype_code(bias)
    if residual is not None:
        r = _operand(residual, "residual", dtype, (m, d_out), device)
    _no_grad(None if mx else A, bias, residual)
    with where:
        Y = _empty2(m, d_out, dtype, device)
        Z = _empty2(m, d_out, dtype, device) if save_preact else None
        _own, ws, wsb = _scratch(workspace, mx_linear_workspace_size(m, d_out, d_in, kind, code), device)
        z = Z.data_ptr() if save_preact else None
        if mx:
            a, s = A._pointers("A", device)
            _check(_lib().gptq_mx_linear_mx(a, s, MX_FORMATS[kind], m, d_in, codes, scales, d_out, b, bcode, act, r,
                                            Y.data_ptr(), code, z, ws, wsb, st))
        else:
            _check(_lib().gptq_mx_linear(A.data_ptr(), kind, m, d_in, codes, scales, d_out, b, bcode, act, r,
                                         Y.data_ptr(), code, z, ws, wsb, st))
    return (Y, Z) if save_preact else Y


def mx_linear_backward(dY, w: MxTensor, activation="none", preact=None, bias_grad=False, out_dtype=None,
                       workspace=None, stream=None):
    """(dA, dbias) of mx_linear (gptq_mx_linear_backward): dZ = dY act'(Z),
    dA = dZ W, dbias the column sums of dZ.  Through quantized activations the
    gradient passes as through unquantized ones.  Arguments and results as for
    dequant_linear_backward."""
    _mx_tensor(w, "w", "fp4")
    _require(dY, "dY", ndim=2)
    dcode, act, dtype, device = _dtype_code(dY), _activation(activation), out_dtype or dY.dtype, dY.device
    code = _out_code(dtype)
    st, where = _place(device, "dY", stream)
    m, d_out = dY.shape
    if d_out != w.rows:
        raise ValueError(f"dY has {d_out} columns, the layer {w.rows} rows")
    if preact is None and act:
        raise ValueError("preact is required unless activation is 'none'")
    codes, scales = w._pointers("w", device)
    z = None if preact is None else _operand(preact, "preact", dY.dtype, (m, d_out), device)
    _no_grad(dY, preact)
    with where:
        dA = _empty2(m, w.d, dtype, device)
        db = _TORCH.empty_strided((d_out,), (1,), dtype=_TORCH.float32, device=device) if bias_grad else None
        _own, ws, wsb = _scratch(workspace, mx_linear_backward_workspace_size(m, d_out, w.d, dcode, code), device)
        _check(_lib().gptq_mx_linear_backward(dY.data_ptr(), dcode, m, d_out, z, act, codes, scales, w.d,
                                              dA.data_ptr(), code, db.data_ptr() if bias_grad else None, ws, wsb, st))
    return dA, db


def rms_norm(X, weight, residual=None, eps=1e-6, format=None, stream=None):
    """(Y, S): S = X + residual (rounded to X's dtype), Y = S / sqrt(mean(S^2) + eps) * weight
    (gptq_rms_norm, gptq_rms_norm_mx).

    X, residual: [m, d] bfloat16/float32; weight: [d] of X's dtype.  Y is a
    tensor of X's dtype, or an MxTensor when format is "fp8" or "fp4" (what
    mx_linear takes).  S is the residual stream behind the addition, X itself
    without a residual; rms_norm_backward takes it."""
    _require(X, "X", ndim=2)
    code, dtype, device = _dtype_code(X), X.dtype, X.device
    fmt = None if format is None else _mx_format(format)
    st, where = _place(device, "X", stream)
    m, d = shape = X.shape
    w = _operand(weight, "weight", dtype, (d,), device)
    r = None if residual is None else _operand(residual, "residual", dtype, shape, device)
    _no_grad(X, weight, residual)
    with where:
        S, s = X, None
        if residual is not None:
            S = _empty2(m, d, dtype, device)
            s = S.data_ptr()
        if fmt is None:
            Y = _empty2(m, d, dtype, device)
            _check(_lib().gptq_rms_norm(X.data_ptr(), r, w, code, m, d, float(eps), s, Y.data_ptr(), st))
        else:
            Y = MxTensor._empty(m, d, format, device)
            codes, scales = Y._pointers("Y", device)
            _check(_lib().gptq_rms_norm_mx(X.data_ptr(), r, w, code, m, d, float(eps), s, fmt, codes, scales,
                                           st))
    return Y, S


def rms_norm_backward_workspace_size(m, d) -> int:
    return _lib().gptq_rms_norm_backward_workspace_size(m, d)


def rms_norm_backward(dY, S, weight, eps=1e-6, dS=None, weight_grad=True, workspace=None, stream=None):
    """(dX, dweight) of rms_norm (gptq_rms_norm_backward) from the S that it
    returned; dX is the gradient of X and of the residual.

    dY, S, dS: [m, d], one dtype; dS: the gradient that reaches S by itself (the
    residual stream's), added to dX.  dX: of that dtype; dweight: [d] float32,
    or None unless weight_grad."""
    _require(dY, "dY", ndim=2)
    code, dtype, device = _dtype_code(dY), dY.dtype, dY.device
    st, where = _place(device, "dY", stream)
    m, d = shape = dY.shape
    s = _operand(S, "S", dtype, shape, device)
    w = _operand(weight, "weight", dtype, (d,), device)
    t = None if dS is None else _operand(dS, "dS", dtype, shape, device)
    _no_grad(dY, S, weight, dS)
    with where:
        dX = _empty2(m, d, dtype, device)
        dw = _TORCH.empty_strided((d,), (1,), dtype=_TORCH.float32, device=device) if weight_grad else None
        _own, ws, wsb = _scratch(workspace, rms_norm_backward_workspace_size(m, d), device)
        _check(_lib().gptq_rms_norm_backward(dY.data_ptr(), s, w, t, code, m, d, float(eps), dX.data_ptr(),
                                             dw.data_ptr() if weight_grad else None, ws, wsb, st))
    return dX, dw


def inverse_factor(H, damp: float = 0.01, act_order: bool = False, workspace=None, stream=None):
    """(perm, U) with (H[perm][:, perm] + lambda I)^-1 = U^T U, U upper (stage 2 alone)."""
    torch = _torch()
    _require(H, "H", dtype=torch.float32, ndim=2)
    d = H.shape[0]
    pm = torch.empty((d,), dtype=torch.int32, device=H.device)
    U = torch.empty((d, d), dtype=torch.float32, device=H.device)
    need = quantize_layer_workspace_size(1, d, 4, -1, 1, act_order)
    ws = _workspace(need, H.device, workspace)
    _check(_lib().gptq_inverse_factor(H.data_ptr(), d, float(damp), int(bool(act_order)), pm.data_ptr(),
                                   U.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
    return pm, U
