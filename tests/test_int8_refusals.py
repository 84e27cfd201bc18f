"""Calls of the 8-bit integer format that are refused before anything is launched:
the C calls' status, the Python binding's errors. No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import int8_reference as ref
import microscaling_precision_quantization_amd as mx

P = ctypes.c_void_p(0x100000)
P2 = ctypes.c_void_p(0x200000)
P4 = ctypes.c_void_p(0x200004)   # aligned to 4
MIS = ctypes.c_void_p(0x100002)
INV, UNS = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED
I8 = mx.MX_FMT_INT8


def test_reference_against_fractions():
    """The reference's codes against exact rational arithmetic."""
    from fractions import Fraction
    r = np.random.RandomState(0)
    x = (r.randint(-255, 256, (40, 16)) * np.exp2(r.randint(-8, 1, (40, 16)))).astype(np.float32)
    x = torch.from_numpy(x).bfloat16().float().numpy().astype(np.float64)
    codes, scales = ref.quantize(x)
    for i in range(40):
        for k in range(16):
            assert codes[i, k] == round(Fraction(x[i, k]) / Fraction(float(scales[i])))


def test_quantize_and_dequantize():
    def q(block=0, rnd=0, rows=4, cols=256, x=P, codes=P, scales=P4, ts=None, layout=mx.MX_LAYOUT_ROWS):
        return mx.mx_quantize_layout(I8, block, rnd, rows, cols, x, codes, scales, ts, None, 0, None, layout)
    assert q(block=32) == UNS and q(block=128) == UNS and q(rnd=1) == UNS and q(layout=mx.MX_LAYOUT_KPANEL) == UNS
    for kw in (dict(cols=24), dict(cols=0), dict(rows=0), dict(x=None), dict(x=P4), dict(codes=P4), dict(scales=MIS), dict(ts=P),
               dict(rows=1 << 37)):
        assert q(**kw) == INV, kw
    d = mx.mx_dequantize
    assert d(I8, 16, 0, 4, 256, P, P4, None, 0, P2, None) == UNS
    assert d(I8, 0, 0, 4, 256, P, P4, None, 3, P2, None) == UNS
    assert d(I8, 0, 0, 4, 200, P, P4, None, 0, P2, None) == INV
    assert d(I8, 0, 0, 4, 256, P, MIS, None, 0, P2, None) == INV
    assert d(I8, 0, 0, 4, 256, P, P4, P, 0, P2, None) == INV
    assert mx.mx_quantize_ex(I8, 0, 0, 0, 0, 4, 256, P, P, P, None, 0) == UNS
    assert mx.mx_pack(I8, 0, 4, 256, P, P, P2, P2, None) == UNS
    assert mx.mx_norm_quantize(I8, 0, 0, 4, 256, P, 256, None, 0, None, 0, None, 1.0, None, 1e-6, None, 0, P, P, None, 0) == UNS


@pytest.mark.parametrize("kw,status", [
    (dict(fa=1), UNS), (dict(fb=1), UNS), (dict(fa=0), UNS), (dict(block=32), UNS), (dict(block=16), UNS), (dict(rnd=1), UNS), (dict(od=2), UNS),
    (dict(M=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=24), INV), (dict(K=1 << 17), INV), (dict(ldc=63), INV),
    (dict(a=P4), INV), (dict(b=P4), INV), (dict(c=P4), INV), (dict(sa=MIS), INV), (dict(sb=MIS), INV), (dict(sa=None), INV),
    (dict(sb=None), INV), (dict(ts=P), INV), (dict(M=1 << 23, N=1 << 30, ldc=1 << 30), INV), (dict(M=65535 * 128, N=16512, ldc=16512), INV),
])
def test_gemm(kw, status):
    a = dict(fa=I8, fb=I8, block=0, rnd=0, M=64, N=64, K=256, a=P, sa=P4, ts=None, b=P, sb=P4, od=0, c=P2, ldc=64)
    a.update(kw)
    args = (a["fa"], a["fb"], a["block"], a["rnd"], a["M"], a["N"], a["K"], a["a"], a["sa"], a["ts"], a["b"], a["sb"], None, a["od"],
            a["c"], a["ldc"])
    assert mx.mx_gemm(*args, None, 0, None) == status
    assert mx.mx_gemm_noalloc(*args, None) == status


def test_gemm_layouts():
    for la, lb in ((1, 0), (0, 1), (1, 1)):
        assert mx.mx_gemm_ex(I8, I8, 0, 0, 64, 64, 256, P, P4, None, P, P4, None, 0, P2, 64, None, 0, None, la, lb) == UNS


@pytest.mark.parametrize("kw,status", [
    (dict(fa=1), UNS), (dict(fb=1), UNS), (dict(block=32), UNS), (dict(rnd=1), UNS), (dict(od=2), UNS), (dict(groups=0), INV),
    (dict(groups=65536), INV), (dict(M=0), INV), (dict(K=24), INV), (dict(K=1 << 17), INV), (dict(off=None), INV), (dict(off=MIS), INV),
    (dict(a=P4), INV), (dict(sa=MIS), INV), (dict(sb=None), INV), (dict(ldc=63), INV), (dict(M=1 << 30, N=1 << 30, ldc=1 << 30), INV),
])
def test_grouped(kw, status):
    a = dict(fa=I8, fb=I8, block=0, rnd=0, groups=3, M=64, N=64, K=256, off=P4, a=P, sa=P4, b=P, sb=P4, od=0, c=P2, ldc=64)
    a.update(kw)
    assert mx.mx_gemm_grouped(a["fa"], a["fb"], a["block"], a["rnd"], a["groups"], a["M"], a["N"], a["K"], a["off"], a["a"],
                              a["sa"], a["b"], a["sb"], a["od"], a["c"], a["ldc"], None) == status


def test_launch_failure_is_reported():
    """Valid arguments and no GPU visible: MX_ERR_HIP from the launch itself."""
    hip = ctypes.CDLL("libamdhip64.so")
    n = ctypes.c_int(0)
    if hip.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
        pytest.skip("a GPU is visible: the launch would not fail")
    for call in (lambda: mx.mx_quantize(I8, 0, 0, 4, 256, P, P, P4, None, None, 0, None),
                 lambda: mx.mx_quantize(I8, 0, 0, 4, 65536, P, P, P4, None, None, 0, None),
                 lambda: mx.mx_dequantize(I8, 0, 0, 4, 256, P, P4, None, 1, P2, None),
                 lambda: mx.mx_gemm(I8, I8, 0, 0, 4, 64, 256, P, P4, None, P, P4, None, 1, P2, 64, None, 0, None),
                 lambda: mx.mx_gemm(I8, I8, 0, 0, 4000, 4000, 256, P, P4, None, P, P4, None, 1, P2, 4000, None, 0, None),
                 lambda: mx.mx_gemm_grouped(I8, I8, 0, 0, 3, 64, 64, 256, P4, P, P4, P, P4, 1, P2, 64, None)):
        assert call() == mx.MX_ERR_HIP and mx.mx_last_hip_error() != 0


# ---- the Python binding ----------------------------------------------------------
def _q(rows, cols, groups=1):
    return mx.QTensor(I8, groups * rows, cols, torch.zeros(groups * rows, cols, dtype=torch.uint8), torch.zeros(groups * rows), groups=groups)


def test_python():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for t in (x, x.view(2, 2, 256)):
        with pytest.raises(ValueError, match="GPU tensors"):
            mx.quantize(t, "int8")
    with pytest.raises(ValueError, match="2-D bfloat16"):
        mx.quantize(x.float(), "int8")
    with pytest.raises(ValueError, match="contiguous"):
        mx.quantize(x.t(), "int8")
    with pytest.raises(ValueError, match="gives"):
        mx.norm_quantize(x, None, "int8")
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.dequantize(_q(4, 256))
    a, b = _q(4, 256), _q(64, 256)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.gemm(a, b)
    with pytest.raises(ValueError, match="K mismatch"):
        mx.gemm(a, _q(64, 128))
    with pytest.raises(ValueError, match="stack"):
        mx.gemm(a, _q(64, 256, groups=2))
    with pytest.raises(ValueError, match="not a quantized tensor"):
        mx.gemm(_q(4, 24), _q(64, 24))
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensors"):
        mx.gemm_grouped(a, _q(64, 256, groups=3), off)
    for bad in (torch.zeros(5), torch.zeros(4, dtype=torch.uint8), torch.zeros(8)[::2]):
        with pytest.raises(ValueError, match="scales must be a contiguous float32"):
            mx.gemm(mx.QTensor(I8, 4, 256, a.codes, bad), b)
    with pytest.raises(ValueError, match="codes must be"):
        mx.gemm(mx.QTensor(I8, 4, 256, a.codes.view(torch.int8), a.scales), b)
