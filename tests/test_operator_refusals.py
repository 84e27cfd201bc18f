"""Calls of the FP8 block formats, the GEMM by expert and norm + quantize that
are refused before anything is launched: the C calls' status, the Python
binding's errors. No GPU."""
import ctypes

import pytest
import torch

import microscaling_precision_quantization_amd as mx

P = ctypes.c_void_p(0x100000)
P2 = ctypes.c_void_p(0x200000)
P4 = ctypes.c_void_p(0x200004)   # aligned to 4
MIS = ctypes.c_void_p(0x100002)
INV, UNS = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED
A8, B8 = mx.MX_FMT_FP8_B128, mx.MX_FMT_FP8_B128X128


@pytest.mark.parametrize("fmt", [A8, B8])
def test_fp8_quantize_and_dequantize(fmt):
    def q(block=128, rnd=0, rows=4, cols=256, x=P, codes=P, scales=P4, ts=None, layout=mx.MX_LAYOUT_ROWS):
        return mx.mx_quantize_layout(fmt, block, rnd, rows, cols, x, codes, scales, ts, None, 0, None, layout)
    assert q(block=32) == UNS and q(rnd=1) == UNS and q(layout=mx.MX_LAYOUT_KPANEL) == UNS
    for kw in (dict(cols=192), dict(cols=64), dict(rows=0), dict(x=None), dict(codes=P4), dict(scales=MIS), dict(ts=P)):
        assert q(**kw) == INV, kw
    d = mx.mx_dequantize
    assert d(fmt, 32, 0, 4, 256, P, P4, None, 0, P2, None) == UNS
    assert d(fmt, 128, 0, 4, 192, P, P4, None, 0, P2, None) == INV
    assert d(fmt, 128, 0, 4, 256, P, MIS, None, 0, P2, None) == INV
    assert d(fmt, 128, 0, 4, 256, P, P4, P, 0, P2, None) == INV
    assert mx.mx_quantize_ex(fmt, 128, 0, 0, 0, 4, 256, P, P, P, None, 0) == UNS
    assert mx.mx_pack(fmt, 128, 4, 256, P, P, P2, P2, None) == UNS


@pytest.mark.parametrize("kw,status", [
    (dict(fa=B8), UNS), (dict(fb=A8), UNS), (dict(fa=mx.MX_FMT_MXFP8), UNS), (dict(block=32), UNS),
    (dict(K=192), INV), (dict(K=(1 << 22) + 128), INV), (dict(sa=MIS), INV), (dict(sb=MIS), INV),
    (dict(ts=P), INV), (dict(ldc=63), INV), (dict(a=P4), INV), (dict(sb=None), INV),
    (dict(M=1 << 23, N=1 << 30, ldc=1 << 30), INV),  # more tiles than a grid holds
    (dict(M=40, N=1 << 30, ldc=1 << 30), INV), (dict(M=65535 * 128, N=16512, ldc=16512), INV),
])
def test_fp8_gemm(kw, status):
    a = dict(fa=A8, fb=B8, block=128, M=64, N=64, K=256, a=P, sa=P4, ts=None, b=P, sb=P4, ldc=64)
    a.update(kw)
    assert mx.mx_gemm(a["fa"], a["fb"], a["block"], 0, a["M"], a["N"], a["K"], a["a"], a["sa"], a["ts"], a["b"], a["sb"],
                      None, 0, P2, a["ldc"], None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fa=1, fb=2), UNS), (dict(fa=2, fb=2), UNS), (dict(fa=0), UNS), (dict(block=16), UNS), (dict(rnd=1), UNS),
    (dict(od=2), UNS), (dict(fa=A8, fb=B8), UNS), (dict(fa=A8, fb=B8, block=128, K=160), INV),
    (dict(groups=0), INV), (dict(groups=65536), INV), (dict(M=0), INV), (dict(N=-1), INV), (dict(K=48), INV),
    (dict(K=(1 << 22) + 32), INV), (dict(groups=65535, N=1 << 20, K=1 << 20, ldc=1 << 20), INV),
    (dict(off=None), INV), (dict(off=MIS), INV), (dict(a=None), INV), (dict(sa=P4), INV), (dict(b=P4), INV),
    (dict(sb=None), INV), (dict(c=P4), INV), (dict(ldc=63), INV),
    (dict(M=1 << 30, N=1 << 30, ldc=1 << 30), INV),
    (dict(groups=65535, M=1 << 20, N=16384, ldc=16384, fa=A8, fb=B8, block=128), INV),  # mostly partly filled tiles
    (dict(groups=65535, M=1 << 21, N=12800, ldc=12800, fa=A8, fb=B8, block=128), INV),  # of 64 x 128
])
def test_grouped(kw, status):
    a = dict(fa=1, fb=1, block=32, rnd=0, groups=3, M=64, N=64, K=256, off=P4, a=P, sa=P, b=P, sb=P, od=0, c=P2, ldc=64)
    a.update(kw)
    assert mx.mx_gemm_grouped(a["fa"], a["fb"], a["block"], a["rnd"], a["groups"], a["M"], a["N"], a["K"], a["off"], a["a"],
                              a["sa"], a["b"], a["sb"], a["od"], a["c"], a["ldc"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=mx.MX_FMT_NVFP4, block=16), UNS), (dict(fmt=B8, block=128), UNS), (dict(fmt=mx.MX_FMT_BF16), UNS),
    (dict(block=128), UNS), (dict(rnd=1), UNS), (dict(layout=3), UNS),
    (dict(fmt=A8, block=128, layout=mx.MX_LAYOUT_KPANEL), UNS), (dict(layout=mx.MX_LAYOUT_KPANEL, cols=288, ldx=288, ldr=288, ldh=288), INV),
    (dict(rows=0), INV), (dict(cols=48), INV), (dict(fmt=A8, block=128, cols=192), INV),
    (dict(cols=32800, ldx=32800, ldr=32800, ldh=32800), INV), (dict(ldx=248), INV), (dict(ldx=260), INV), (dict(ldr=128), INV),
    (dict(ldh=264 + 4), INV), (dict(gate=P, gate_rows=0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(alpha=float("nan")), INV), (dict(alpha=float("inf")), INV), (dict(x=None), INV),
    (dict(x=P4), INV), (dict(residual=P4), INV), (dict(gate=P4), INV), (dict(post=P4), INV), (dict(weight=P4), INV),
    (dict(h=P4), INV), (dict(codes=None), INV), (dict(scales=P4), INV), (dict(fmt=A8, block=128, scales=MIS), INV),
])
def test_norm_quantize(kw, status):
    a = dict(fmt=1, block=32, rnd=0, rows=4, cols=256, x=P, ldx=256, residual=P, ldr=256, gate=None, gate_rows=1, post=None,
             alpha=1.0, weight=P, eps=1e-6, h=P, ldh=256, codes=P, scales=P, layout=0)
    a.update(kw)
    assert mx.mx_norm_quantize(a["fmt"], a["block"], a["rnd"], a["rows"], a["cols"], a["x"], a["ldx"], a["residual"], a["ldr"],
                               a["gate"], a["gate_rows"], a["post"], a["alpha"], a["weight"], a["eps"], a["h"], a["ldh"],
                               a["codes"], a["scales"], None, a["layout"]) == status


def test_launch_failure_is_reported():
    """Valid arguments and no GPU visible: MX_ERR_HIP from the launch itself."""
    hip = ctypes.CDLL("libamdhip64.so")
    n = ctypes.c_int(0)
    if hip.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
        pytest.skip("a GPU is visible: the launch would not fail")
    for call in (lambda: mx.mx_quantize(A8, 128, 0, 4, 256, P, P, P4, None, None, 0, None),
                 lambda: mx.mx_quantize(B8, 128, 0, 4, 256, P, P, P4, None, None, 0, None),
                 lambda: mx.mx_gemm(A8, B8, 128, 0, 4, 64, 256, P, P4, None, P, P4, None, 1, P2, 64, None, 0, None),
                 lambda: mx.mx_gemm_grouped(1, 1, 32, 0, 3, 64, 64, 256, P4, P, P, P, P, 1, P2, 64, None),
                 lambda: mx.mx_norm_quantize(1, 32, 0, 4, 256, P, 256, None, 0, None, 0, None, 1.0, None, 1e-6, None, 0, P, P, None, 0)):
        assert call() == mx.MX_ERR_HIP and mx.mx_last_hip_error() != 0


# ---- the Python binding ----------------------------------------------------------
def _q(fmt, rows, cols, groups=1):
    f = mx.FORMATS[fmt]
    s = mx.scale_shape(f, rows, cols)
    st = torch.float32 if f in mx.FP8_BLOCK_FORMATS else torch.uint8
    return mx.QTensor(f, groups * rows, cols, torch.zeros(groups * rows, mx.code_cols(f, cols), dtype=torch.uint8),
                      torch.zeros(groups, *s, dtype=st), groups=groups)


def test_python_quantize():
    w = torch.zeros(2, 4, 256, dtype=torch.bfloat16)
    for fmt in ("nvfp4", "mxfp8", "fp8_b128", "mxfp4_mbs"):
        with pytest.raises(ValueError, match="stack"):
            mx.quantize(w, fmt)
    with pytest.raises(ValueError, match="stack"):
        mx.quantize(w, "mxfp4", layout="kpanel")
    with pytest.raises(ValueError, match="not for"):
        mx.quantize(w, "fp8_b128x128", rotation="wht32")
    for fmt in ("mxfp4", "fp8_b128x128"):
        with pytest.raises(ValueError, match="contiguous"):
            mx.quantize(w.transpose(1, 2), fmt)
        with pytest.raises(ValueError, match="GPU tensors"):
            mx.quantize(w, fmt)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.quantize(w[0], "fp8_b128")
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.dequantize(_q("fp8_b128x128", 100, 256, groups=2))


def test_python_gemm():
    a, b = _q("fp8_b128", 4, 256), _q("fp8_b128x128", 100, 256)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.gemm(a, b)
    with pytest.raises(ValueError, match="stack"):
        mx.gemm(a, _q("fp8_b128x128", 100, 256, groups=2))
    with pytest.raises(ValueError, match="one weight"):
        mx.pack(_q("mxfp4", 100, 256, groups=2))
    b.scales = b.scales.to(torch.uint8)
    with pytest.raises(ValueError, match="scales must be a contiguous float32"):
        mx.gemm(a, b)
    c = _q("mxfp4", 4, 256)
    c.scales = c.scales.float()
    with pytest.raises(ValueError, match="scales must be a contiguous uint8"):
        mx.gemm(c, _q("mxfp4", 4, 256))


def test_python_grouped():
    a, b = _q("mxfp4", 8, 256), _q("mxfp4", 100, 256, groups=3)
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.gemm_grouped(a, b, off)
    for bad in (off[:3], off.long(), off.view(2, 2), torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="offsets"):
            mx.gemm_grouped(a, b, bad)
    with pytest.raises(ValueError, match="K mismatch"):
        mx.gemm_grouped(a, _q("mxfp4", 100, 128, groups=3), off)
    with pytest.raises(ValueError, match="out_dtype"):
        mx.gemm_grouped(a, b, off, torch.float16)
    with pytest.raises(ValueError, match="out must be"):
        mx.gemm_grouped(a, b, off, out=torch.zeros(8, 99, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="one \\[M\\]\\[K\\]"):
        mx.gemm_grouped(_q("mxfp4", 4, 256, groups=2), b, off)
    b.groups = 7
    with pytest.raises(ValueError, match="not a stack"):
        mx.gemm_grouped(a, b, off)
    a.layout = mx.MX_LAYOUT_KPANEL
    with pytest.raises(ValueError, match="row layout"):
        mx.gemm_grouped(a, _q("mxfp4", 100, 256, groups=3), off)


def test_python_norm_quantize():
    x, w = torch.zeros(6, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.norm_quantize(x, w, "mxfp4")
    for kw, match in ((dict(fmt="nvfp4"), "gives"), (dict(x=x[0]), "2-D"), (dict(x=x.float()), "x must be"),
                      (dict(x=x.t()), "x must be"), (dict(residual=x[:3]), "residual must be"),
                      (dict(out=x.float()), "out must be"), (dict(weight=w[:128]), "weight must be"),
                      (dict(post_weight=w.float()), "post_weight must be"), (dict(gate=w[:128]), "gate must be"),
                      (dict(gate=x.view(2, 3, 256)), "gate must be"), (dict(gate=w[0]), "gate must be"), (dict(gate=x[:4]), "do not divide"),
                      (dict(gate=x[:0]), "do not divide")):
        with pytest.raises(ValueError, match=match):
            mx.norm_quantize(**{**dict(x=x, weight=w, fmt="mxfp4"), **kw})
