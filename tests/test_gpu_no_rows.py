"""Calls with no rows of activations, as a rank makes them that a router sent no tokens."""
import pytest
import torch

import microscaling_precision_quantization_amd as mx
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _zeros(*shape):
    return torch.zeros(*shape, dtype=BF16, device="cuda")


@pytest.mark.parametrize("act,weight", [("mxfp4", "mxfp4"), ("fp8_b128", "fp8_b128x128")])
def test_expert_layer_without_tokens(act, weight):
    require_gpu()
    K, N, G = 512, 256, 3
    w1, w2 = mx.quantize(_zeros(G, N, K), weight), mx.quantize(_zeros(K, N), weight)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    q, h = mx.norm_quantize(_zeros(0, K), _zeros(K), act, residual=_zeros(0, K), gate=_zeros(K))
    assert (q.rows, q.cols) == (0, K) and tuple(h.shape) == (0, K)
    up = mx.gemm_grouped(q, w1, offsets)
    assert tuple(up.shape) == (0, N) and up.dtype == BF16
    qu = mx.quantize(up, act)
    assert tuple(mx.gemm(qu, w2, F32).shape) == (0, K) and tuple(mx.dequantize(qu).shape) == (0, N)
    out = torch.empty(0, N, dtype=BF16, device="cuda")
    assert mx.gemm_grouped(q, w1, offsets, out=out) is out
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "mxfp8_e5m2", "mxfp6_e3m2", "mxfp4_mbs", "mxfp4_mbs16"])
def test_gemm_without_rows(fmt):
    require_gpu()
    b = mx.quantize(_zeros(64, 256), fmt)
    assert tuple(mx.gemm(mx.quantize(_zeros(0, 256), fmt), b).shape) == (0, 64)
    if fmt == "mxfp4":
        assert tuple(mx.gemm(_zeros(0, 256), b).shape) == (0, 64)


def test_refused_without_rows():
    """What is refused with rows is refused without."""
    require_gpu()
    b = mx.quantize(_zeros(2, 64, 256), "fp8_b128x128")
    one = mx.quantize(_zeros(64, 256), "fp8_b128x128")
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    mxfp4 = mx.quantize(_zeros(0, 256), "mxfp4")
    for call in (lambda: mx.quantize(_zeros(0, 192), "fp8_b128"), lambda: mx.quantize(_zeros(0, 256), "bf16"),
                 lambda: mx.norm_quantize(_zeros(0, 192), None, "fp8_b128"), lambda: mx.quantize(_zeros(0, 0), "mxfp4"),
                 lambda: mx.gemm(mxfp4, one), lambda: mx.gemm_grouped(mxfp4, b, offsets),
                 lambda: mx.quantize(_zeros(0, 256), "nvfp4")):
        with pytest.raises(mx.MXError):
            call()
    with pytest.raises(ValueError, match="K mismatch"):
        mx.gemm(mx.quantize(_zeros(0, 128), "fp8_b128"), one)
    with pytest.raises(ValueError, match="offsets"):
        mx.gemm_grouped(mx.quantize(_zeros(0, 256), "fp8_b128"), b, offsets[:2])
