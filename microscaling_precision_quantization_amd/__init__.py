"""Python binding for libmx: microscaling (MX / NVFP4) quantization and the
block-scaled GEMM on AMD Instinct MI355X (gfx950).

Two layers:
  * mx_quantize, mx_dequantize, mx_gemm, ... : the C ABI (include/mx.h) under
    the same names, taking integers and raw device pointers;
  * quantize, dequantize, gemm, gemm_grouped, norm_quantize : torch conveniences that allocate outputs on
    the input's device and pass data_ptr() plus the current HIP stream.

Every step of the computation runs in libmx's HIP kernels. If libmx.so is not
built, loading fails with an error; there is no fallback path.
"""
import ctypes
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmx.so")

MX_FMT_BF16, MX_FMT_MXFP4, MX_FMT_MXFP8, MX_FMT_NVFP4 = 0, 1, 2, 3
MX_FMT_MXFP8_E5M2, MX_FMT_MXFP6_E3M2, MX_FMT_MXFP4_MBS, MX_FMT_MXFP4_MBS16 = 4, 5, 6, 7
MX_FMT_FP8_B128, MX_FMT_FP8_B128X128 = 8, 9
MX_ROUND_RNE = 0
MX_SCALE_CEIL, MX_SCALE_OAS = 0, 1
MX_ROTATE_NONE, MX_ROTATE_WHT32 = 0, 1
MX_OUT_F32, MX_OUT_BF16 = 0, 1
MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_HIP = 0, 1, 2, 3
MX_LAYOUT_ROWS, MX_LAYOUT_KPANEL = 0, 1

FORMATS = {"mxfp4": MX_FMT_MXFP4, "mxfp8": MX_FMT_MXFP8, "nvfp4": MX_FMT_NVFP4, "bf16": MX_FMT_BF16,
           "mxfp8_e5m2": MX_FMT_MXFP8_E5M2, "mxfp6_e3m2": MX_FMT_MXFP6_E3M2,
           "mxfp4_mbs": MX_FMT_MXFP4_MBS, "mxfp4_mbs16": MX_FMT_MXFP4_MBS16,
           "fp8_b128": MX_FMT_FP8_B128, "fp8_b128x128": MX_FMT_FP8_B128X128}
BLOCK = {MX_FMT_MXFP4: 32, MX_FMT_MXFP8: 32, MX_FMT_NVFP4: 16, MX_FMT_BF16: 32,
         MX_FMT_MXFP8_E5M2: 32, MX_FMT_MXFP6_E3M2: 32, MX_FMT_MXFP4_MBS: 32,
         MX_FMT_MXFP4_MBS16: 16, MX_FMT_FP8_B128: 128, MX_FMT_FP8_B128X128: 128}
MBS_FORMATS = (MX_FMT_MXFP4_MBS, MX_FMT_MXFP4_MBS16)
FP8_BLOCK_FORMATS = (MX_FMT_FP8_B128, MX_FMT_FP8_B128X128)  # fp32 scales
PAIRS = {MX_FMT_BF16: MX_FMT_MXFP4, MX_FMT_FP8_B128: MX_FMT_FP8_B128X128}  # a GEMM's b, where not a's format


def code_cols(fmt, cols):
    """Bytes of codes per row of `cols` elements."""
    if fmt in (MX_FMT_MXFP8, MX_FMT_MXFP8_E5M2) or fmt in FP8_BLOCK_FORMATS:
        return cols
    if fmt == MX_FMT_MXFP6_E3M2:
        return cols * 3 // 4
    return cols // 2

def scale_shape(fmt, rows, cols):
    """Shape of the scales tensor: [rows][cols/block]; for MXFP4-MBS (block 32)
    and MXFP4-MBS16 (block 16) one flat buffer, the E8M0 plane
    [rows][cols/block] followed by the macro mantissa plane [rows][cols/128];
    for FP8_B128X128 [ceil(rows/128)][cols/128]."""
    if fmt == MX_FMT_FP8_B128X128:
        return (-(-rows // 128), cols // 128)
    if fmt in MBS_FORMATS:
        return (rows * (cols // BLOCK[fmt]) + rows * (cols // 128),)
    return (rows, cols // BLOCK[fmt])


def mbs_planes(scales, rows, cols, block=32):
    """Views of an MXFP4-MBS (block 32) or MBS16 (block 16) scales buffer:
    (E8M0 [rows][cols/block], macro mantissas [rows][cols/128])."""
    n = rows * (cols // block)
    return scales[:n].view(rows, cols // block), scales[n:].view(rows, cols // 128)


# Symbols declared in include/mx.h.
EXPORTS = ("mx_quantize", "mx_quantize_workspace_bytes", "mx_quantize_ex", "mx_quantize_layout",
           "mx_dequantize",
           "mx_gemm", "mx_gemm_workspace_bytes", "mx_last_hip_error", "mx_status_string",
           "mx_pack", "mx_gemm_ex", "mx_gemm_noalloc", "mx_gemm_grouped", "mx_norm_quantize")

_lib = None


class MXError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = f"{what}: {status_string(status)}"
        if status == MX_ERR_HIP:
            msg += f" (hipError_t {mx_last_hip_error()})"
        super().__init__(msg)


def lib():
    """Load libmx.so (built by build.py). Raises if it is missing.
    MX_LIBRARY, if set, names another build of the same sources to load
    instead (the host-sanitizer build, in that CPU test's child process)."""
    global _lib
    if _lib is None:
        path = os.environ.get("MX_LIBRARY") or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run "
                               "microscaling_precision_quantization_amd.build.build()")
        L = ctypes.CDLL(path)
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.mx_quantize.restype = i32
        L.mx_quantize.argtypes = [i32, i32, i32, i64, i64, P, P, P, P, P, sz, P]
        L.mx_quantize_ex.restype = i32
        L.mx_quantize_ex.argtypes = [i32, i32, i32, i32, i32, i64, i64, P, P, P, P, i32]
        L.mx_quantize_layout.restype = i32
        L.mx_quantize_layout.argtypes = [i32, i32, i32, i64, i64, P, P, P, P, P, sz, P, i32]
        L.mx_quantize_workspace_bytes.restype = sz
        L.mx_quantize_workspace_bytes.argtypes = [i32, i64, i64]
        L.mx_dequantize.restype = i32
        L.mx_dequantize.argtypes = [i32, i32, i32, i64, i64, P, P, P, i32, P, P]
        L.mx_gemm.restype = i32
        L.mx_gemm.argtypes = [i32, i32, i32, i32, i64, i64, i64, P, P, P, P, P, P, i32, P, i64,
                              P, sz, P]
        L.mx_gemm_ex.restype = i32
        L.mx_gemm_ex.argtypes = [i32, i32, i32, i32, i64, i64, i64, P, P, P, P, P, P, i32, P, i64,
                                 P, sz, P, i32, i32]
        L.mx_gemm_noalloc.restype = i32
        L.mx_gemm_noalloc.argtypes = [i32, i32, i32, i32, i64, i64, i64, P, P, P, P, P, P, i32, P,
                                      i64, P]
        L.mx_gemm_grouped.restype = i32
        L.mx_gemm_grouped.argtypes = [i32, i32, i32, i32, i64, i64, i64, i64, P, P, P, P, P, i32, P,
                                      i64, P]
        L.mx_norm_quantize.restype = i32
        L.mx_norm_quantize.argtypes = [i32, i32, i32, i64, i64, P, i64, P, i64, P, i64, P,
                                       ctypes.c_float, P, ctypes.c_float, P, i64, P, P, P, i32]
        L.mx_pack.restype = i32
        L.mx_pack.argtypes = [i32, i32, i64, i64, P, P, P, P, P]
        L.mx_gemm_workspace_bytes.restype = sz
        L.mx_gemm_workspace_bytes.argtypes = [i32, i32, i64, i64, i64]
        L.mx_last_hip_error.restype = i32
        L.mx_last_hip_error.argtypes = []
        L.mx_status_string.restype = ctypes.c_char_p
        L.mx_status_string.argtypes = [i32]
        _lib = L
    return _lib


# ---- the C ABI, same names ---------------------------------------------------
def mx_quantize(fmt, block, rnd, rows, cols, x, codes, scales, tensor_scale, workspace,
                workspace_bytes, stream):
    return lib().mx_quantize(fmt, block, rnd, rows, cols, x, codes, scales, tensor_scale,
                             workspace, workspace_bytes, stream)


def mx_quantize_ex(fmt, block, rnd, rule, rot, rows, cols, x, codes, scales, stream, layout):
    return lib().mx_quantize_ex(fmt, block, rnd, rule, rot, rows, cols, x, codes, scales, stream,
                                layout)


def mx_quantize_layout(fmt, block, rnd, rows, cols, x, codes, scales, tensor_scale, workspace,
                       workspace_bytes, stream, layout):
    return lib().mx_quantize_layout(fmt, block, rnd, rows, cols, x, codes, scales, tensor_scale,
                                    workspace, workspace_bytes, stream, layout)


def mx_quantize_workspace_bytes(fmt, rows, cols):
    return lib().mx_quantize_workspace_bytes(fmt, rows, cols)


def mx_dequantize(fmt, block, rnd, rows, cols, codes, scales, tensor_scale, out_dtype, y, stream):
    return lib().mx_dequantize(fmt, block, rnd, rows, cols, codes, scales, tensor_scale,
                               out_dtype, y, stream)


def mx_gemm(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts, out_dtype,
            c, ldc, workspace, workspace_bytes, stream):
    return lib().mx_gemm(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                         out_dtype, c, ldc, workspace, workspace_bytes, stream)


def mx_gemm_ex(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts, out_dtype,
               c, ldc, workspace, workspace_bytes, stream, a_layout, b_layout):
    return lib().mx_gemm_ex(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales,
                            b_ts, out_dtype, c, ldc, workspace, workspace_bytes, stream, a_layout,
                            b_layout)


def mx_gemm_noalloc(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                    out_dtype, c, ldc, stream):
    return lib().mx_gemm_noalloc(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales,
                                 b_ts, out_dtype, c, ldc, stream)


def mx_gemm_grouped(fmt_a, fmt_b, block, rnd, groups, M, N, K, offsets, a, a_scales, b, b_scales,
                    out_dtype, c, ldc, stream):
    return lib().mx_gemm_grouped(fmt_a, fmt_b, block, rnd, groups, M, N, K, offsets, a, a_scales, b,
                                 b_scales, out_dtype, c, ldc, stream)


def mx_norm_quantize(fmt, block, rnd, rows, cols, x, ldx, residual, ldr, gate, gate_rows, post_weight,
                     alpha, weight, eps, h, ldh, codes, scales, stream, layout):
    return lib().mx_norm_quantize(fmt, block, rnd, rows, cols, x, ldx, residual, ldr, gate, gate_rows,
                                  post_weight, alpha, weight, eps, h, ldh, codes, scales, stream,
                                  layout)


def mx_pack(fmt, block, rows, cols, codes, scales, packed_codes, packed_scales, stream):
    return lib().mx_pack(fmt, block, rows, cols, codes, scales, packed_codes, packed_scales, stream)


def mx_gemm_workspace_bytes(fmt_a, fmt_b, M, N, K):
    return lib().mx_gemm_workspace_bytes(fmt_a, fmt_b, M, N, K)


def mx_last_hip_error():
    return lib().mx_last_hip_error()


def mx_status_string(status):
    return lib().mx_status_string(status).decode()


def status_string(status):
    return mx_status_string(status)


# ---- torch conveniences --------------------------------------------------------
@dataclass
class QTensor:
    """A block-quantized [rows][cols] tensor: codes, scales and (NVFP4) the
    fp32 tensor scale, all device tensors; layout MX_LAYOUT_KPANEL after pack().
    Scales are uint8, or float32 for the FP8 block formats. groups: a stack of
    that many [rows / groups][cols] weights, each quantized by itself (the b of
    gemm_grouped)."""
    fmt: int
    rows: int
    cols: int
    codes: "object"
    scales: "object"
    tensor_scale: "object" = None
    layout: int = MX_LAYOUT_ROWS
    groups: int = 1

    @property
    def block(self):
        return BLOCK[self.fmt]


def _check_qtensor(q, what):
    """The kernels read exactly the bytes a QTensor's shape implies: refuse
    buffers of another size, type or layout in memory."""
    import torch
    fmt, codes, scales = q.fmt, q.codes, q.scales
    if fmt not in BLOCK or fmt == MX_FMT_BF16 or q.cols % BLOCK[fmt] != 0:
        raise ValueError(f"{what}: not a quantized tensor of a supported format")
    if q.groups < 1 or q.rows % q.groups != 0:
        raise ValueError(f"{what}: {q.rows} rows are not a stack of {q.groups} weights")
    need_c = q.rows * code_cols(fmt, q.cols)
    if fmt == MX_FMT_FP8_B128X128 or fmt in MBS_FORMATS:
        need_s = q.groups
        for d in scale_shape(fmt, q.rows // q.groups, q.cols):
            need_s *= d
    else:
        need_s = q.rows * (q.cols // BLOCK[fmt])
    if codes.dtype != torch.uint8 or not codes.is_contiguous() or codes.numel() != need_c:
        raise ValueError(f"{what}: codes must be a contiguous uint8 tensor of {need_c} bytes")
    st, name = (torch.float32, "float32") if fmt in FP8_BLOCK_FORMATS else (torch.uint8, "uint8")
    if scales.dtype != st or not scales.is_contiguous() or scales.numel() != need_s:
        raise ValueError(f"{what}: scales must be a contiguous {name} tensor of {need_s} elements")
    if fmt == MX_FMT_NVFP4:
        ts = q.tensor_scale
        if ts is None or ts.dtype != torch.float32 or ts.numel() < 1:
            raise ValueError(f"{what}: NVFP4 needs a float32 tensor scale")


def _fmt_id(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _stream(torch, device, *tensors):
    """The current stream of `device`, after checking that the device is a GPU
    and that every tensor handed to the kernels lives on it (a host or
    foreign-device pointer must never reach a kernel)."""
    if device.type != "cuda":
        raise ValueError(f"libmx runs on GPU tensors; got a tensor on {device}")
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on {device}; got one on {t.device}")
    return torch._C._cuda_getCurrentRawStream(index)  # (1.8 us less than by a Stream object)


# (torch.empty below takes its sizes one by one: 0.7 us less than as a tuple.)
def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(status, what):
    if status != MX_OK:
        raise MXError(status, what)


def _on(device, call, *args):
    """call(*args) with `device` (the tensors' and the stream's) current: a
    kernel is launched on the current device."""
    import torch
    if device.index == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


SCALE_RULES = {"ceil": MX_SCALE_CEIL, "oas": MX_SCALE_OAS}
ROTATIONS = {None: MX_ROTATE_NONE, "none": MX_ROTATE_NONE, "wht32": MX_ROTATE_WHT32}


LAYOUTS = {"rows": MX_LAYOUT_ROWS, "kpanel": MX_LAYOUT_KPANEL}


def quantize(x, fmt, scale_rule="ceil", rotation=None, layout="rows"):
    """Quantize a contiguous bf16 [rows][cols] device tensor. scale_rule "oas"
    (MXFP4) and rotation "wht32" (MXFP4, MXFP8) select mx_quantize_ex, with
    the layout given; otherwise layout "kpanel" (MXFP4, MXFP8, E5M2, E3M2,
    NVFP4) selects mx_quantize_layout. A [groups][rows][cols] tensor ("mxfp4"
    or "fp8_b128x128", row layout) is a stack of weights for gemm_grouped, each
    quantized by itself. No rows give an empty QTensor, which dequantize, gemm and
    gemm_grouped take (not for NVFP4, whose scale is the tensor's, nor by mx_quantize_ex)."""
    import torch
    f = _fmt_id(fmt)
    lay = LAYOUTS[layout]
    if x.dim() == 3:
        if f not in (MX_FMT_MXFP4, MX_FMT_FP8_B128X128) or lay != MX_LAYOUT_ROWS:
            raise ValueError("a stack of weights is quantized to mxfp4 or fp8_b128x128 in the row layout")
        if f == MX_FMT_FP8_B128X128:
            return _quantize_tile_stack(x, scale_rule, rotation)
        if not x.is_contiguous():
            raise ValueError("quantize expects a contiguous bfloat16 tensor")
        q = quantize(x.view(-1, x.shape[2]), fmt, scale_rule, rotation)
        q.groups = x.shape[0]
        return q
    if scale_rule != "ceil" or rotation not in (None, "none"):
        if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
            raise ValueError("quantize expects a contiguous 2-D bfloat16 tensor")
        rows, cols = x.shape
        codes = torch.empty(rows, code_cols(f, cols), dtype=torch.uint8, device=x.device)
        scales = torch.empty(*scale_shape(f, rows, cols), dtype=torch.uint8, device=x.device)
        _check(_on(x.device, mx_quantize_ex, f, BLOCK[f], MX_ROUND_RNE, SCALE_RULES[scale_rule],
                   ROTATIONS[rotation], rows, cols, _ptr(x), _ptr(codes), _ptr(scales),
                   _stream(torch, x.device, x), lay), "mx_quantize_ex")
        return QTensor(f, rows, cols, codes, scales, None, lay)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("quantize expects a contiguous 2-D bfloat16 tensor")
    rows, cols = x.shape
    dev = x.device
    codes = torch.empty(rows, code_cols(f, cols), dtype=torch.uint8, device=dev)
    scales = torch.empty(*scale_shape(f, rows, cols), device=dev,
                         dtype=torch.float32 if f in FP8_BLOCK_FORMATS else torch.uint8)
    if rows == 0 and f != MX_FMT_NVFP4:
        return _empty(f, cols, codes, scales, lay, "mx_quantize", x)
    ts = ws = None
    wsb = 0
    if f == MX_FMT_NVFP4:
        ts = torch.empty(1, dtype=torch.float32, device=dev)
        wsb = mx_quantize_workspace_bytes(f, rows, cols)
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if lay == MX_LAYOUT_ROWS:
        _check(_on(dev, lib().mx_quantize, f, BLOCK[f], MX_ROUND_RNE, rows, cols, _ptr(x), _ptr(codes),
                   _ptr(scales), _ptr(ts), _ptr(ws), wsb, _stream(torch, dev, x)), "mx_quantize")
    else:
        _check(_on(dev, mx_quantize_layout, f, BLOCK[f], MX_ROUND_RNE, rows, cols, _ptr(x), _ptr(codes),
                   _ptr(scales), _ptr(ts), _ptr(ws), wsb, _stream(torch, dev, x), lay),
               "mx_quantize_layout")
    return QTensor(f, rows, cols, codes, scales, ts, lay)


def _empty(f, cols, codes, scales, layout, what, *inputs):
    """The QTensor of no rows (a rank that a router sent no tokens): nothing is launched."""
    import torch
    _stream(torch, codes.device, *inputs)
    granule = 128 if f in MBS_FORMATS else BLOCK[f]
    if f == MX_FMT_BF16 or cols == 0 or cols % granule != 0:
        raise MXError(MX_ERR_INVALID_ARG, what)
    return QTensor(f, 0, cols, codes, scales, None, layout)


def _quantize_tile_stack(x, scale_rule, rotation):
    """A [groups][rows][cols] stack to FP8_B128X128: one tall weight where no tile of
    it holds rows of two (64 x 2048 x 2048: 141 us, 633 by calls), else a call per weight."""
    import torch
    if scale_rule != "ceil" or rotation not in (None, "none"):
        raise ValueError("scale rules and rotations are not for fp8_b128x128")
    if x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise ValueError("quantize expects a contiguous bfloat16 tensor")
    g, rows, cols = x.shape
    f, dev = MX_FMT_FP8_B128X128, x.device
    if rows % 128 == 0 and x.numel() > 0:
        q = quantize(x.view(g * rows, cols), f)
        q.scales, q.groups = q.scales.view(g, *scale_shape(f, rows, cols)), g
        return q
    stream = _stream(torch, dev, x)
    codes = torch.empty((g * rows, cols), dtype=torch.uint8, device=dev)
    scales = torch.empty((g, *scale_shape(f, rows, cols)), dtype=torch.float32, device=dev)
    for i in range(g):
        _check(_on(dev, mx_quantize, f, BLOCK[f], MX_ROUND_RNE, rows, cols, _ptr(x[i]),
                   _ptr(codes[i * rows:]), _ptr(scales[i]), None, None, 0, stream), "mx_quantize")
    return QTensor(f, g * rows, cols, codes, scales, groups=g)


def dequantize(q, out_dtype=None):
    """Expand a QTensor (row layout) to float32 (default) or bfloat16."""
    import torch
    _check_qtensor(q, "dequantize")
    if q.layout != MX_LAYOUT_ROWS:
        raise ValueError("dequantize takes a tensor in the row layout")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    od = MX_OUT_F32 if out_dtype == torch.float32 else MX_OUT_BF16
    n = q.rows // q.groups
    if q.groups > 1 and q.fmt == MX_FMT_FP8_B128X128 and n % 128 != 0:  # each weight's last tiles are its own
        codes, scales = q.codes.view(q.groups, n, q.cols), q.scales.view(q.groups, -1)
        return torch.cat([dequantize(QTensor(q.fmt, n, q.cols, codes[i], scales[i]), out_dtype)
                          for i in range(q.groups)])
    y = torch.empty(q.rows, q.cols, dtype=out_dtype, device=q.codes.device)
    if q.rows == 0:
        _stream(torch, q.codes.device, q.codes, q.scales, q.tensor_scale)
        return y
    _check(_on(q.codes.device, mx_dequantize, q.fmt, q.block, MX_ROUND_RNE, q.rows, q.cols,
               _ptr(q.codes), _ptr(q.scales), _ptr(q.tensor_scale), od, _ptr(y),
               _stream(torch, q.codes.device, q.codes, q.scales, q.tensor_scale)), "mx_dequantize")
    return y


def pack(q):
    """A QTensor (MXFP4, MXFP8, E5M2, E3M2 or NVFP4) re-laid into the K-panel
    layout (mx_pack), for use as a gemm() operand."""
    import torch
    if q.layout != MX_LAYOUT_ROWS:
        raise ValueError("pack() takes a tensor in the row layout")
    _check_qtensor(q, "pack")
    if q.groups != 1:
        raise ValueError("pack() takes one weight, not a stack")
    codes = torch.empty_like(q.codes)
    scales = torch.empty_like(q.scales)
    _check(_on(q.codes.device, mx_pack, q.fmt, q.block, q.rows, q.cols, _ptr(q.codes), _ptr(q.scales),
               _ptr(codes), _ptr(scales), _stream(torch, q.codes.device, q.codes, q.scales)), "mx_pack")
    return QTensor(q.fmt, q.rows, q.cols, codes, scales, q.tensor_scale, MX_LAYOUT_KPANEL)


def gemm(a, b, out_dtype=None, out=None, workspace=None):
    """C = A * B^T. a: QTensor (any quantized format, M x K; b of the same format,
    or fp8_b128x128 for an fp8_b128 a) or a bf16 [M][K] tensor (with an MXFP4 b:
    W4A16); b: QTensor stored N x K (MXFP4: row or K-panel layout)."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    od = MX_OUT_F32 if out_dtype == torch.float32 else MX_OUT_BF16
    _check_qtensor(b, "gemm operand b")
    if b.groups != 1:
        raise ValueError("gemm takes one weight; a stack is gemm_grouped's")
    if isinstance(a, QTensor):
        _check_qtensor(a, "gemm operand a")
        fa, M, K = a.fmt, a.rows, a.cols
        pa, psa, pta = _ptr(a.codes), _ptr(a.scales), _ptr(a.tensor_scale)
        dev = a.codes.device
    else:
        if a.dtype != torch.bfloat16 or a.dim() != 2 or not a.is_contiguous():
            raise ValueError("bf16 activations must be a contiguous 2-D bfloat16 tensor")
        fa, (M, K) = MX_FMT_BF16, a.shape
        pa, psa, pta = _ptr(a), None, None
        dev = a.device
    N = b.rows
    if b.cols != K:
        raise ValueError(f"K mismatch: A has {K}, B has {b.cols}")
    if out is not None:
        if (out.dtype != out_dtype or out.dim() != 2 or tuple(out.shape) != (M, N)
                or out.stride(1) != 1):
            raise ValueError(f"out must be a [{M}][{N}] {out_dtype} tensor with unit column stride")
    c = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    wsb = mx_gemm_workspace_bytes(fa, b.fmt, M, N, K) if fa == MX_FMT_BF16 else 0  # (no other pair has one)
    if wsb and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        wsb = workspace.numel() * workspace.element_size()  # the C call checks it is enough
    ldc = c.stride(0) if M > 1 else N  # (the row stride of a single row says nothing)
    la = a.layout if isinstance(a, QTensor) else MX_LAYOUT_ROWS
    a_parts = (a.codes, a.scales, a.tensor_scale) if isinstance(a, QTensor) else (a,)
    stream = _stream(torch, dev, *a_parts, b.codes, b.scales, b.tensor_scale, c, workspace)
    if M == 0:
        _check(MX_OK if b.fmt == PAIRS.get(fa, fa) else MX_ERR_UNSUPPORTED, "mx_gemm")
        return c
    if la != MX_LAYOUT_ROWS or b.layout != MX_LAYOUT_ROWS:
        _check(_on(dev, lib().mx_gemm_ex, fa, b.fmt, b.block, MX_ROUND_RNE, M, N, K, pa, psa, pta,
                   _ptr(b.codes), _ptr(b.scales), _ptr(b.tensor_scale), od, _ptr(c), ldc,
                   _ptr(workspace), wsb, stream, la, b.layout), "mx_gemm_ex")
        return c
    _check(_on(dev, lib().mx_gemm, fa, b.fmt, b.block, MX_ROUND_RNE, M, N, K, pa, psa, pta, _ptr(b.codes),
               _ptr(b.scales), _ptr(b.tensor_scale), od, _ptr(c), ldc, _ptr(workspace), wsb,
               stream), "mx_gemm")
    return c


def gemm_grouped(a, b, offsets, out_dtype=None, out=None):
    """C = A * B_g^T by expert. a: QTensor [M][K] (mxfp4 or fp8_b128), rows
    sorted by expert; b: a stack of `groups` [N][K] weights (mxfp4 or
    fp8_b128x128; quantize of a 3-D tensor); offsets: int32 device tensor of
    groups + 1 nondecreasing row numbers, expert g's rows being offsets[g] ..
    offsets[g + 1] - 1. The offsets are read on the device only. Rows of no
    expert are left as `out` had them (undefined without `out`)."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    _check_qtensor(a, "gemm_grouped operand a")
    _check_qtensor(b, "gemm_grouped operand b")
    if a.layout != MX_LAYOUT_ROWS or b.layout != MX_LAYOUT_ROWS:
        raise ValueError("gemm_grouped takes operands in the row layout")
    if a.groups != 1:
        raise ValueError("gemm_grouped operand a is one [M][K] tensor")
    if b.cols != a.cols:
        raise ValueError(f"K mismatch: A has {a.cols}, B has {b.cols}")
    G, M, N, K = b.groups, a.rows, b.rows // b.groups, a.cols
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() != G + 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 tensor of {G + 1} row numbers")
    dev = a.codes.device
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
    elif out.dtype != out_dtype or out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError(f"out must be a [{M}][{N}] {out_dtype} tensor with unit column stride")
    stream = _stream(torch, dev, a.codes, a.scales, b.codes, b.scales, offsets, out)
    if M == 0:
        pair = a.fmt in (MX_FMT_MXFP4, MX_FMT_FP8_B128) and b.fmt == PAIRS.get(a.fmt, a.fmt)
        _check(MX_OK if pair else MX_ERR_UNSUPPORTED, "mx_gemm_grouped")
        return out
    _check(_on(dev, lib().mx_gemm_grouped, a.fmt, b.fmt, b.block, MX_ROUND_RNE, G, M, N, K, _ptr(offsets),
               _ptr(a.codes), _ptr(a.scales), _ptr(b.codes), _ptr(b.scales),
               MX_OUT_F32 if out_dtype == torch.float32 else MX_OUT_BF16, _ptr(out),
               out.stride(0) if M > 1 else N, stream), "mx_gemm_grouped")
    return out


def norm_quantize(x, weight, fmt, residual=None, gate=None, post_weight=None, alpha=1.0, eps=1e-6,
                  layout="rows", out=None):
    """The norms between two blocks, fused with the residual and the quantizer:
    y = x, or its RMS norm times post_weight; h = residual + alpha * gate * y;
    the RMS norm of h times weight, quantized to `fmt` (mxfp4, mxfp8 or
    fp8_b128). x, residual: bf16 [rows][cols] with unit column stride and rows
    that start on 16 bytes; weight,
    post_weight: bf16 [cols] (weight None: ones); gate: bf16 [cols] or [n][cols],
    each of its rows for rows / n rows of x. Returns the QTensor and h (bf16;
    `out` if given, which may be x or residual; None without a residual or out)."""
    import torch
    f = _fmt_id(fmt)
    if f not in (MX_FMT_MXFP4, MX_FMT_MXFP8, MX_FMT_FP8_B128):
        raise ValueError("norm_quantize gives mxfp4, mxfp8 or fp8_b128")
    if x.dim() != 2:
        raise ValueError("norm_quantize expects a 2-D bfloat16 tensor")
    rows, cols = shape = x.shape
    bf16 = torch.bfloat16
    for t, name in ((x, "x"), (residual, "residual"), (out, "out")):
        if t is not None and (t.dtype != bf16 or t.shape != shape or t.stride(1) != 1):
            raise ValueError(f"{name} must be a [{rows}][{cols}] bfloat16 tensor with unit column stride")
    for t, name in ((weight, "weight"), (post_weight, "post_weight")):
        if t is not None and (t.dtype != bf16 or t.dim() != 1 or t.numel() != cols or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor of {cols} elements")
    gate_rows = 0
    if gate is not None:
        if (gate.dtype != bf16 or gate.dim() not in (1, 2) or gate.shape[-1] != cols
                or not gate.is_contiguous()):
            raise ValueError(f"gate must be a contiguous bfloat16 tensor of rows of {cols}")
        n = 1 if gate.dim() == 1 else gate.shape[0]
        if n < 1 or rows % n != 0:
            raise ValueError(f"{rows} rows do not divide among {n} gates")
        gate_rows = rows // n
    dev = x.device
    if out is None and residual is not None:
        out = torch.empty(rows, cols, dtype=bf16, device=dev)
    codes = torch.empty(rows, code_cols(f, cols), dtype=torch.uint8, device=dev)
    scales = torch.empty(*scale_shape(f, rows, cols), device=dev,
                         dtype=torch.float32 if f == MX_FMT_FP8_B128 else torch.uint8)
    lay = LAYOUTS[layout]
    stream = _stream(torch, dev, x, residual, gate, post_weight, weight, out)
    if rows == 0:
        return _empty(f, cols, codes, scales, lay, "mx_norm_quantize"), out
    # (The row stride of a single row says nothing.)
    ldx = x.stride(0) if rows > 1 else cols
    ldr = residual.stride(0) if residual is not None and rows > 1 else cols
    ldh = out.stride(0) if out is not None and rows > 1 else cols
    _check(_on(dev, lib().mx_norm_quantize, f, BLOCK[f], MX_ROUND_RNE, rows, cols, _ptr(x), ldx,
               _ptr(residual), ldr, _ptr(gate), gate_rows, _ptr(post_weight), alpha, _ptr(weight), eps,
               _ptr(out), ldh, _ptr(codes), _ptr(scales), stream, lay),
           "mx_norm_quantize")
    return QTensor(f, rows, cols, codes, scales, None, lay), out
