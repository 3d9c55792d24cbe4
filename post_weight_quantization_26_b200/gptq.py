"""Python binding of libgptq.so (the C ABI in include/gptq.h).

Each function has the name of the C entry point it wraps and only marshals
arguments: torch CUDA tensors become device pointers, the current torch
stream becomes the ``stream`` argument, and a non-OK status raises
:class:`GptqError`.  Every step of the path runs in the library's kernels;
there is no CPU or PyTorch fallback, and importing this module fails if the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgptq.so")

GPTQ_OK = 0
STATUS_NAMES = {0: "GPTQ_OK", 1: "GPTQ_ERR_INVALID", 2: "GPTQ_ERR_NOT_SPD",
                3: "GPTQ_ERR_NONFINITE", 4: "GPTQ_ERR_WORKSPACE",
                5: "GPTQ_ERR_CUDA", 6: "GPTQ_ERR_TIMEOUT"}

EXPORTED = ("gptq_workspace_size", "gptq_hessian_accumulate",
            "gptq_hessian_accumulate_ordered", "gptq_fault_inject", "gptq_prepare_hinv", "gptq_quantize_layer", "gptq_dequant_check",
            "gptq_prepare_factor", "gptq_quantize_layer_factor",
            "gptq_device_status", "gptq_status_string", "gptq_launch_count",
            "gptq_dequant_check_noalloc", "gptq_w4a16_matmul", "gptq_awq_channel_scale",
            "gptq_awq_workspace_size", "gptq_awq_search",
            "gptq_rmsnorm_quant8", "gptq_w4a8_matmul", "gptq_w4a8_workspace_size", "gptq_w4a8_gated")
NOALLOC_MAX_TILES = 65536  # GPTQ_NOALLOC_MAX_TILES in include/gptq.h
ACT_GROUP = 128  # columns that share an activation scale, where a token has several
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.int8: 2}  # gptq_dtype in include/gptq.h
FAULT_NONE, FAULT_SYRK_STALL, FAULT_TRAILING_STALL = 0, 1, 2  # GPTQ_FAULT_* in include/gptq.h
FAULT_W4A8_LOADS, FAULT_W4A8_STAGES = 4, 5


class GptqError(RuntimeError):
    def __init__(self, status: int, where: str, extra: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}{extra}")


class GptqConfig(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group_size", ctypes.c_int),
                ("sym", ctypes.c_int), ("block", ctypes.c_int),
                ("damp_rel", ctypes.c_double)]


def make_config(bits=4, group_size=0, sym=False, block=128, damp_rel=0.01):
    return GptqConfig(int(bits), int(group_size), int(bool(sym)), int(block),
                      float(damp_rel))


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgptq.so; raises if it is missing (no fallback path exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libgptq.so not found at {path}; build it with "
            "`python -m post_weight_quantization_26_b200.build`")
    lib = ctypes.CDLL(path)
    P, I64, SZ, I, D, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t,
                           ctypes.c_int, ctypes.c_double, ctypes.c_float)
    cfgp = ctypes.POINTER(GptqConfig)
    lib.gptq_workspace_size.argtypes = [I64, I64, cfgp]
    lib.gptq_workspace_size.restype = SZ
    lib.gptq_hessian_accumulate.argtypes = [P, P, I64, I64, I64, F, P]
    lib.gptq_hessian_accumulate.restype = I
    lib.gptq_hessian_accumulate_ordered.argtypes = [P, P, I64, I64, I64, F, P]
    lib.gptq_hessian_accumulate_ordered.restype = I
    lib.gptq_fault_inject.argtypes = [I, I64]
    lib.gptq_fault_inject.restype = I
    lib.gptq_prepare_hinv.argtypes = [P, I64, D, P, P, P, SZ,
                                      ctypes.POINTER(I64), P]
    lib.gptq_prepare_hinv.restype = I
    lib.gptq_quantize_layer.argtypes = [P, I64, I64, P, P, cfgp, P, P, P, P,
                                        SZ, P]
    lib.gptq_quantize_layer.restype = I
    lib.gptq_prepare_factor.argtypes = lib.gptq_prepare_hinv.argtypes
    lib.gptq_prepare_factor.restype = I
    lib.gptq_quantize_layer_factor.argtypes = lib.gptq_quantize_layer.argtypes
    lib.gptq_quantize_layer_factor.restype = I
    lib.gptq_dequant_check.argtypes = [P, P, P, P, P, I64, I64, cfgp, P,
                                       ctypes.POINTER(D), P, SZ, P]
    lib.gptq_dequant_check.restype = I
    lib.gptq_dequant_check_noalloc.argtypes = [P, P, P, P, P, I64, I64, cfgp, P,
                                               ctypes.POINTER(D), P]
    lib.gptq_dequant_check_noalloc.restype = I
    lib.gptq_w4a16_matmul.argtypes = [P, P, P, I64, I64, cfgp, P, I64, P, P]
    lib.gptq_w4a16_matmul.restype = I
    lib.gptq_rmsnorm_quant8.argtypes = [P, I, I64, P, I, I64, P, D, I64, I64, I, P, I64, P, I64,
                                        P, P]
    lib.gptq_rmsnorm_quant8.restype = I
    lib.gptq_w4a8_matmul.argtypes = [P, P, P, I64, I64, cfgp, P, I64, P, I, I64, P, I, I64, P]
    lib.gptq_w4a8_matmul.restype = I
    lib.gptq_w4a8_workspace_size.argtypes = [I64, I64, I]
    lib.gptq_w4a8_workspace_size.restype = SZ
    lib.gptq_w4a8_gated.argtypes = [P, P, P, P, P, P, I64, I64, cfgp, P, I64, P, I, I64, P, I,
                                    I64, P, P, SZ, P]
    lib.gptq_w4a8_gated.restype = I
    lib.gptq_awq_channel_scale.argtypes = [P, I64, I64, I64, P, P]
    lib.gptq_awq_channel_scale.restype = I
    lib.gptq_awq_workspace_size.argtypes = [I64, I64, cfgp]
    lib.gptq_awq_workspace_size.restype = SZ
    lib.gptq_awq_search.argtypes = [P, P, P, I64, I64, cfgp, I, P, P, P, P, P, P, P, SZ, P]
    lib.gptq_awq_search.restype = I
    lib.gptq_device_status.argtypes = [P]
    lib.gptq_device_status.restype = I
    lib.gptq_launch_count.argtypes = []
    lib.gptq_launch_count.restype = ctypes.c_uint64
    lib.gptq_status_string.argtypes = [I]
    lib.gptq_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st: int, where: str, extra: str = ""):
    if st != GPTQ_OK:
        raise GptqError(st, where, extra)


def gptq_workspace_size(d_row: int, d_col: int, cfg: GptqConfig) -> int:
    n = load_library().gptq_workspace_size(d_row, d_col, ctypes.byref(cfg))
    if n == 0:
        raise GptqError(1, "gptq_workspace_size")
    return int(n)


def alloc_workspace(d_row: int, d_col: int, cfg: GptqConfig, device=None):
    """A uint8 CUDA tensor of gptq_workspace_size bytes (256-byte aligned)."""
    n = gptq_workspace_size(d_row, d_col, cfg)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def gptq_hessian_accumulate(H: torch.Tensor, X: torch.Tensor,
                            scale: float = 2.0, stream=None) -> None:
    """H (fp32 d x d) += scale * X^T X for token-major bf16 X (n x d)."""
    _accumulate("gptq_hessian_accumulate", H, X, scale, stream)


def gptq_hessian_accumulate_ordered(H: torch.Tensor, X: torch.Tensor,
                                    scale: float = 2.0, stream=None) -> None:
    """gptq_hessian_accumulate with a fixed summation order (bitwise
    reproducible H)."""
    _accumulate("gptq_hessian_accumulate_ordered", H, X, scale, stream)


def _accumulate(name, H, X, scale, stream):
    assert H.dtype == torch.float32 and X.dtype == torch.bfloat16
    n, d = X.shape
    assert H.shape == (d, d) and H.is_contiguous() and X.stride(1) == 1
    st = getattr(load_library(), name)(
        _ptr(H), _ptr(X), n, d, X.stride(0), float(scale), _stream(stream))
    _check(st, name)


def gptq_fault_inject(where: int, wait_limit_ns: int = 0) -> None:
    """Set the fault injection of the failure-detection tests (FAULT_NONE
    and 0 restore normal operation)."""
    _check(load_library().gptq_fault_inject(int(where), int(wait_limit_ns)),
           "gptq_fault_inject")


def gptq_prepare_hinv(H: torch.Tensor, damp_rel: float, G: torch.Tensor,
                      dead_mask: torch.Tensor, ws: torch.Tensor,
                      stream=None) -> int:
    """G = upper U with U^T U = (H + damp)^-1.  Returns bad_pivot (-1 if SPD)."""
    d = H.shape[0]
    assert H.dtype == torch.float32 and H.shape == (d, d) and H.is_contiguous()
    assert G.dtype == torch.float32 and G.shape == (d, d) and G.is_contiguous()
    assert dead_mask.dtype == torch.uint8 and dead_mask.numel() == d
    piv = ctypes.c_int64(-1)
    st = load_library().gptq_prepare_hinv(
        _ptr(H), d, float(damp_rel), _ptr(G), _ptr(dead_mask), _ptr(ws),
        ws.numel(), ctypes.byref(piv), _stream(stream))
    _check(st, "gptq_prepare_hinv", f" (bad_pivot={piv.value})")
    return int(piv.value)


def gptq_prepare_factor(H: torch.Tensor, damp_rel: float, F: torch.Tensor,
                        dead_mask: torch.Tensor, ws: torch.Tensor,
                        stream=None) -> int:
    """F for gptq_quantize_layer_factor: G's 128x128 diagonal blocks and
    V_ab G_bb right of them (H + damp = V V^T).  Returns bad_pivot."""
    d = H.shape[0]
    assert H.dtype == torch.float32 and H.shape == (d, d) and H.is_contiguous()
    assert F.dtype == torch.float32 and F.shape == (d, d) and F.is_contiguous()
    assert dead_mask.dtype == torch.uint8 and dead_mask.numel() == d
    piv = ctypes.c_int64(-1)
    st = load_library().gptq_prepare_factor(
        _ptr(H), d, float(damp_rel), _ptr(F), _ptr(dead_mask), _ptr(ws),
        ws.numel(), ctypes.byref(piv), _stream(stream))
    _check(st, "gptq_prepare_factor", f" (bad_pivot={piv.value})")
    return int(piv.value)


def _quantize(name, W, G, dead_mask, cfg, qweight, scales, zeros, ws, stream):
    d_row, d_col = W.shape
    assert W.dtype == torch.float32 and W.is_contiguous()
    assert G.dtype == torch.float32 and G.shape == (d_col, d_col) and G.is_contiguous()
    assert qweight.dtype == torch.int32 or qweight.dtype == torch.uint32
    st = getattr(load_library(), name)(
        _ptr(W), d_row, d_col, _ptr(G), _ptr(dead_mask), ctypes.byref(cfg),
        _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(ws), ws.numel(),
        _stream(stream))
    _check(st, name)


def gptq_quantize_layer(W: torch.Tensor, G: torch.Tensor, dead_mask,
                        cfg: GptqConfig, qweight: torch.Tensor,
                        scales: torch.Tensor, zeros: torch.Tensor,
                        ws: torch.Tensor, stream=None) -> None:
    _quantize("gptq_quantize_layer", W, G, dead_mask, cfg, qweight, scales,
              zeros, ws, stream)


def gptq_quantize_layer_factor(W: torch.Tensor, F: torch.Tensor, dead_mask,
                               cfg: GptqConfig, qweight: torch.Tensor,
                               scales: torch.Tensor, zeros: torch.Tensor,
                               ws: torch.Tensor, stream=None) -> None:
    """The same layer from F (gptq_prepare_factor); block 128, group_size 0
    or a divisor of 128."""
    _quantize("gptq_quantize_layer_factor", W, F, dead_mask, cfg, qweight,
              scales, zeros, ws, stream)


def gptq_dequant_check(qweight, scales, zeros, W, H, cfg: GptqConfig,
                       W_hat=None, ws=None, want_loss: bool = True,
                       stream=None):
    """Returns the layer loss 1/2 sum_r dW_r H dW_r^T (or None)."""
    d_row, d_col = W.shape if W is not None else W_hat.shape
    loss = ctypes.c_double(float("nan"))
    st = load_library().gptq_dequant_check(
        _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(W), _ptr(H), d_row,
        d_col, ctypes.byref(cfg), _ptr(W_hat),
        ctypes.byref(loss) if want_loss else None, _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "gptq_dequant_check")
    return loss.value if want_loss else None


def gptq_dequant_check_noalloc(qweight, scales, zeros, W, H, cfg: GptqConfig,
                               W_hat=None, want_loss: bool = True, stream=None):
    """gptq_dequant_check for callers that cannot allocate device memory:
    no workspace argument; the library's fixed 512 KB device array serves as
    scratch (see include/gptq.h for the size limit and the rules on
    overlapping calls).  Returns the layer loss (or None)."""
    d_row, d_col = W.shape if W is not None else W_hat.shape
    loss = ctypes.c_double(float("nan"))
    st = load_library().gptq_dequant_check_noalloc(
        _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(W), _ptr(H), d_row,
        d_col, ctypes.byref(cfg), _ptr(W_hat),
        ctypes.byref(loss) if want_loss else None, _stream(stream))
    _check(st, "gptq_dequant_check_noalloc")
    return loss.value if want_loss else None


def gptq_w4a16_matmul(qweight, scales, zeros, cfg: GptqConfig, X, Y=None,
                      stream=None):
    """Y = X W^T for bf16 X (batch x d_col, batch 1..8) and the packed 4-bit
    layer (qweight, scales, zeros) as gptq_quantize_layer wrote it.  Y is fp32
    batch x d_row, allocated here when not given.  Returns Y."""
    assert X.dtype == torch.bfloat16 and X.dim() == 2 and X.is_contiguous()
    batch, d_col = X.shape
    d_row = scales.shape[0]
    if Y is None:
        Y = torch.empty(batch, d_row, dtype=torch.float32, device=X.device)
    assert Y.dtype == torch.float32 and Y.shape == (batch, d_row) and Y.is_contiguous()
    st = load_library().gptq_w4a16_matmul(
        _ptr(qweight), _ptr(scales), _ptr(zeros), d_row, d_col,
        ctypes.byref(cfg), _ptr(X), batch, _ptr(Y), _stream(stream))
    _check(st, "gptq_w4a16_matmul")
    return Y


def _elsewhere(t, stream):
    """None where a call on tensor t runs on the current stream of t's device
    and that device is current; else the context to make the call in.  Outputs
    that the call allocates then belong to the stream that it runs on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
        return torch.cuda.stream(stream)
    return None if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev)


def _rows(name, t, dtypes, n, d, dev):
    """The row stride of an n x d matrix on device `dev` whose rows are dense.
    (These checks run on every call of a generation's token, where they cost as
    much as the kernel, so they are kept short.)"""
    if t.dtype not in dtypes or t.shape != (n, d) or t.get_device() != dev:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected one of "
                         f"{dtypes} {(n, d)} on cuda:{dev}")
    s0, s1 = t.stride()
    if (s1 != 1 and d > 1) or (s0 < d and n > 1):
        raise ValueError(f"{name}: rows must be dense, strides {(s0, s1)}")
    return s0 if n > 1 else max(d, s0)


def _dense(name, t, dtypes, shape, dev):
    if (t.dtype not in dtypes or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected contiguous, "
                         f"one of {dtypes} {tuple(shape)} on cuda:{dev}")


def alloc_codes(n: int, d: int, group: int = ACT_GROUP, device="cuda"):
    """8-bit activations n x d: int8 codes (row stride a multiple of 16, as
    the products need it) and fp32 scales."""
    pitch = (d + 15) // 16 * 16
    codes = torch.empty((n, pitch), dtype=torch.int8, device=device)
    return (codes if pitch == d else codes[:, :d],
            torch.empty((n, -(-d // group) if group else 1), dtype=torch.float32, device=device))


_FLOATS, _F32 = (torch.float32, torch.bfloat16), (torch.float32,)
_I8, _U8, _WORDS = (torch.int8,), (torch.uint8,), (torch.int32, torch.uint32)


def gptq_rmsnorm_quant8(X, weight, eps: float = 1e-6, residual=None, group: int = ACT_GROUP,
                        residual_out=None, out=None, stream=None):
    """r = X + residual (stored in the residual's type), y = r / sqrt(mean r^2
    + eps) * weight, y as int8 codes and scales (one per token for group 0, one
    per token and 128 columns for group 128).  X and residual are n x d, fp32
    or bf16 each; weight is fp32[d] or None.  Returns (codes, scales), and r
    as a third where a residual is given; `out` = (codes, scales) and
    `residual_out` are allocated where they are not given, and residual_out
    may be the residual itself."""
    place = _elsewhere(X, stream)
    if place is not None:
        with place:
            return gptq_rmsnorm_quant8(X, weight, eps, residual, group, residual_out, out)
    if X.dim() != 2:
        raise ValueError("X must be n x d")
    n, d = X.shape
    dev = X.get_device()
    codes, scales = alloc_codes(n, d, group, X.device) if out is None else out
    ldx = _rows("X", X, _FLOATS, n, d, dev)
    ldq = _rows("codes", codes, _I8, n, d, dev)
    _dense("scales", scales, _F32, (n, -(-d // ACT_GROUP) if group else 1), dev)
    wp = rp = op = None
    r_type = ldr = ldo = 0
    if weight is not None:
        _dense("weight", weight, _F32, (d,), dev)
        wp = weight.data_ptr()
    if residual is not None:
        if residual_out is None:
            residual_out = torch.empty((n, d), dtype=residual.dtype, device=X.device)
        ldr = _rows("residual", residual, _FLOATS, n, d, dev)
        ldo = _rows("residual_out", residual_out, (residual.dtype,), n, d, dev)
        r_type, rp, op = DTYPES[residual.dtype], residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    st = (_lib or load_library()).gptq_rmsnorm_quant8(
        X.data_ptr(), DTYPES[X.dtype], ldx, rp, r_type, ldr, wp, eps, n, d, group, op, ldo,
        codes.data_ptr(), ldq, scales.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        raise GptqError(st, "gptq_rmsnorm_quant8")
    return (codes, scales) if residual is None else (codes, scales, residual_out)


def _layer_args(layer, cfg, d_row, d_col, dev):
    """Checks a packed layer; returns its three pointers."""
    qweight, scales, zeros = layer
    groups = (d_row, n_groups(d_col, cfg.group_size))
    _dense("qweight", qweight, _WORDS, (d_row, d_col // 8), dev)
    _dense("scales", scales, _F32, groups, dev)
    _dense("zeros", zeros, _U8, groups, dev)
    return qweight.data_ptr(), scales.data_ptr(), zeros.data_ptr()


def _codes_args(codes, x_scales, dev):
    """Checks 8-bit activations; returns (n, d_col, ldq, x_group)."""
    if codes.dim() != 2 or x_scales.dim() != 2:
        raise ValueError("codes must be n x d_col, x_scales n x blocks")
    n, d_col = codes.shape
    ldq = _rows("codes", codes, _I8, n, d_col, dev)
    if n <= 1:
        ldq = (ldq + 15) // 16 * 16  # the stride of one row is not used
    x_group = 0 if x_scales.shape[1] == 1 else ACT_GROUP
    _dense("x_scales", x_scales, _F32, (n, -(-d_col // ACT_GROUP) if x_group else 1), dev)
    return n, d_col, ldq, x_group


def gptq_w4a8_matmul(qweight, scales, zeros, cfg: GptqConfig, codes, x_scales, Y=None,
                     dtype=torch.float32, stream=None):
    """Y = X W^T for 8-bit activations (codes int8 n x d_col and x_scales, as
    gptq_rmsnorm_quant8 and gptq_w4a8_gated write them) and a packed 4-bit
    layer.  Y is n x d_row, fp32 or bf16, allocated in `dtype` when not given.
    Returns Y."""
    place = _elsewhere(codes, stream)
    if place is not None:
        with place:
            return gptq_w4a8_matmul(qweight, scales, zeros, cfg, codes, x_scales, Y, dtype)
    dev = codes.get_device()
    n, d_col, ldq, x_group = _codes_args(codes, x_scales, dev)
    d_row = scales.shape[0]
    qw, sc, ze = _layer_args((qweight, scales, zeros), cfg, d_row, d_col, dev)
    if Y is None:
        Y = torch.empty((n, d_row), dtype=dtype, device=codes.device)
    ldy = _rows("Y", Y, _FLOATS, n, d_row, dev)
    st = (_lib or load_library()).gptq_w4a8_matmul(
        qw, sc, ze, d_row, d_col, cfg, codes.data_ptr(), ldq, x_scales.data_ptr(), x_group, n,
        Y.data_ptr(), DTYPES[Y.dtype], ldy, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        raise GptqError(st, "gptq_w4a8_matmul")
    return Y


def gptq_w4a8_workspace_size(n: int, d_row: int, dtype) -> int:
    """Bytes of workspace of gptq_w4a8_gated for n tokens and an output type."""
    return int(load_library().gptq_w4a8_workspace_size(n, d_row, DTYPES[dtype]))


def gptq_w4a8_gated(gate, up, cfg: GptqConfig, codes, x_scales, out=None, dtype=torch.bfloat16,
                    ws=None, stream=None):
    """H = silu(X Wg^T) * (X Wu^T) for 8-bit activations and two packed 4-bit
    layers, each (qweight, scales, zeros).  dtype float32 or bfloat16: returns
    H (n x d_row), which `out` may give; int8: returns H as (codes, scales)
    with a scale per token and 128 columns, which `out` may give as a pair.
    `ws` (uint8, gptq_w4a8_workspace_size bytes) is allocated when not given."""
    place = _elsewhere(codes, stream)
    if place is not None:
        with place:
            return gptq_w4a8_gated(gate, up, cfg, codes, x_scales, out, dtype, ws)
    dev = codes.get_device()
    n, d_col, ldq, x_group = _codes_args(codes, x_scales, dev)
    d_row = gate[1].shape[0]
    layers = (*_layer_args(gate, cfg, d_row, d_col, dev), *_layer_args(up, cfg, d_row, d_col, dev))
    if out is None:
        out = (alloc_codes(n, d_row, ACT_GROUP, codes.device) if dtype == torch.int8 else
               torch.empty((n, d_row), dtype=dtype, device=codes.device))
    H, h_scales = out if isinstance(out, (tuple, list)) else (out, None)
    ldh = _rows("H", H, _FLOATS if h_scales is None else _I8, n, d_row, dev)
    hs = None
    if h_scales is not None:
        _dense("h_scales", h_scales, _F32, (n, -(-d_row // ACT_GROUP)), dev)
        hs = h_scales.data_ptr()
    h_type = DTYPES[H.dtype]
    lib = _lib or load_library()
    need = lib.gptq_w4a8_workspace_size(n, d_row, h_type)
    wp, ws_bytes = None, 0
    if need:
        if ws is None:
            ws = torch.empty(need, dtype=torch.uint8, device=codes.device)
        elif ws.dtype != torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous uint8 on the tensors' device")
        wp, ws_bytes = ws.data_ptr(), ws.numel()
    st = lib.gptq_w4a8_gated(
        *layers, d_row, d_col, cfg, codes.data_ptr(), ldq, x_scales.data_ptr(), x_group, n,
        H.data_ptr(), h_type, ldh, hs, wp, ws_bytes, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        raise GptqError(st, "gptq_w4a8_gated")
    return out


def gptq_awq_channel_scale(X, sx=None, stream=None):
    """sx[k] = mean_t |X[t][k]| (fp64) for token-major bf16 X (n x d)."""
    assert X.dtype == torch.bfloat16 and X.dim() == 2 and X.stride(1) == 1
    n, d = X.shape
    if sx is None:
        sx = torch.empty(d, dtype=torch.float64, device=X.device)
    st = load_library().gptq_awq_channel_scale(_ptr(X), n, d, X.stride(0), _ptr(sx),
                                               _stream(stream))
    _check(st, "gptq_awq_channel_scale")
    return sx


def gptq_awq_workspace_size(d_row: int, d_col: int, cfg: GptqConfig) -> int:
    n = load_library().gptq_awq_workspace_size(d_row, d_col, ctypes.byref(cfg))
    if n == 0:
        raise GptqError(1, "gptq_awq_workspace_size")
    return int(n)


def gptq_awq_search(W, H, sx, cfg: GptqConfig, n_grid: int = 20, ws=None, out=None,
                    stream=None):
    """The AWQ grid search over alpha; returns (losses fp64[n_grid], best
    int32[1], s fp32[d_col], qweight, scales, zeros), all on the device."""
    d_row, d_col = W.shape
    dev = W.device
    if ws is None:
        ws = torch.empty(gptq_awq_workspace_size(d_row, d_col, cfg), dtype=torch.uint8,
                         device=dev)
    if out is None:
        qw, sc, ze = alloc_outputs(d_row, d_col, cfg, device=dev)
        out = (torch.empty(n_grid, dtype=torch.float64, device=dev),
               torch.empty(1, dtype=torch.int32, device=dev),
               torch.empty(d_col, dtype=torch.float32, device=dev), qw, sc, ze)
    losses, best, s, qw, sc, ze = out
    st = load_library().gptq_awq_search(
        _ptr(W), _ptr(H), _ptr(sx), d_row, d_col, ctypes.byref(cfg), int(n_grid), _ptr(losses),
        _ptr(best), _ptr(s), _ptr(qw), _ptr(sc), _ptr(ze), _ptr(ws), ws.numel(),
        _stream(stream))
    _check(st, "gptq_awq_search")
    return out


def gptq_device_status(stream=None) -> int:
    return int(load_library().gptq_device_status(_stream(stream)))


def gptq_launch_count() -> int:
    return int(load_library().gptq_launch_count())


def gptq_status_string(status: int) -> str:
    return load_library().gptq_status_string(int(status)).decode()


def n_groups(d_col: int, group_size: int) -> int:
    return 1 if group_size == 0 else d_col // group_size


def alloc_outputs(d_row: int, d_col: int, cfg: GptqConfig, device="cuda"):
    """qweight (int32 words), scales (fp32), zeros (uint8) for one layer."""
    ng = n_groups(d_col, cfg.group_size)
    qweight = torch.empty((d_row, d_col * cfg.bits // 32), dtype=torch.int32,
                          device=device)
    scales = torch.empty((d_row, ng), dtype=torch.float32, device=device)
    zeros = torch.empty((d_row, ng), dtype=torch.uint8, device=device)
    return qweight, scales, zeros
