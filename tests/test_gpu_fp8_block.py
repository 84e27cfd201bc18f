"""FP8 (E4M3) under fp32 scales per 1 x 128 and 128 x 128: codes and scales
equal the definition's bit for bit, dequantized values their fp32 rounding,
and every GEMM output lies within the bound of mx.h for its type."""
import numpy as np
import pytest
import torch

import llm_reference as ref
import microscaling_precision_quantization_amd as mx
from gpu_helpers import bf16_host_bits, dev_u8, host, require_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(BF16)


def _values(t):
    return t.float().numpy().astype(np.float64)


def _check_quantize(x, tall):
    """x: bf16 host tensor."""
    q = mx.quantize(x.cuda(), "fp8_b128x128" if tall else "fp8_b128")
    codes, scales = ref.quantize_fp8(_values(x), tall)
    assert q.scales.dtype == F32 and tuple(q.scales.shape) == scales.shape
    assert np.array_equal(host(q.scales), scales, equal_nan=True)
    assert np.array_equal(host(q.codes), codes)
    return q


def _mixed(rows, cols, seed):
    """Normal values with large and tiny entries, zeros of both signs."""
    r = np.random.RandomState(seed)
    x = r.standard_normal((rows, cols)) * np.exp2(r.randint(-12, 6, (rows, cols)))
    x[r.random_sample(x.shape) < 0.05] = 0.0
    x[r.random_sample(x.shape) < 0.02] = -0.0
    return _bf16(x)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 4096), (3, 256), (17, 1024), (127, 384), (128, 512),
                                       (129, 640), (300, 1152)])
def test_quantize_shapes(rows, cols, tall):
    require_gpu()
    _check_quantize(_mixed(rows, cols, rows + cols), tall)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("power", [-133, -130, -126, -100, -70, -61, -60, -52, 0, 100, 118])
def test_quantize_magnitudes(power, tall):
    """Scales from the fp32 subnormals to near overflow, both sides of 2^-60."""
    require_gpu()
    r = np.random.RandomState(power + 200)
    _check_quantize(_bf16(r.randint(-255, 256, (130, 256)) * 2.0**power), tall)


@pytest.mark.parametrize("tall", [False, True])
def test_quantize_ties(tall):
    """amax = 448 * 2^k makes s a power of two: every midpoint of two E4M3
    values is then an exact tie."""
    require_gpu()
    mid = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2
    row = np.concatenate([mid, [448.0, -448.0]])
    x = np.stack([row, -row, row * 2.0**-20, row * 2.0**30])
    _check_quantize(_bf16(x if not tall else np.concatenate([row[None], -row[None]])), tall)


def test_quantize_every_bf16_value():
    require_gpu()
    bits = np.arange(1 << 16, dtype=np.uint32)
    v = (bits << 16).astype(np.uint32).view(np.float32)
    v = v[np.isfinite(v)]  # 65280 values: 510 blocks
    _check_quantize(_bf16(v.reshape(-1, 128)), False)
    r = np.random.RandomState(1)
    _check_quantize(_bf16(r.permutation(v).reshape(-1, 128)), False)


@pytest.mark.parametrize("tall", [False, True])
def test_quantize_nonfinite_blocks(tall):
    """A block with Inf or NaN: NaN scale, zero codes; its neighbours are not touched."""
    require_gpu()
    x = _mixed(260, 384, 5)
    x[3, 130] = float("inf")
    x[140, 5] = float("nan")
    x[259, 383] = float("-inf")
    q = _check_quantize(x, tall)
    assert np.isnan(host(q.scales)).sum() == 3


@pytest.mark.parametrize("fmt", ["fp8_b128", "fp8_b128x128"])
@pytest.mark.parametrize("out", [F32, BF16])
def test_dequantize(fmt, out):
    require_gpu()
    tall = fmt == "fp8_b128x128"
    r = np.random.RandomState(3)
    rows, cols = 131, 256
    codes = r.randint(0, 256, (rows, cols)).astype(np.uint8)
    shape = (2, 2) if tall else (rows, 2)
    scales = np.exp2(r.uniform(-40, 40, shape)).astype(np.float32)
    scales[0, 0] = np.nan
    q = mx.QTensor(mx.FORMATS[fmt], rows, cols, dev_u8(codes), torch.from_numpy(scales).cuda())
    y = mx.dequantize(q, out)
    want = torch.from_numpy(ref.fp8_values(codes, scales, tall)).to(F32)
    if out == F32:
        assert np.array_equal(host(y), want.numpy(), equal_nan=True)
    else:
        w = want.to(BF16)
        same = bf16_host_bits(y) == bf16_host_bits(w)
        assert np.all(same | (np.isnan(want.numpy()) & np.isnan(host(y.float()))))


def test_dequantize_past_one_grid():
    """More chunks than threads of a grid, and byte offsets past 32 bits (52 GB)."""
    require_gpu()
    rows, cols = (1 << 17) + 128, 1 << 17
    codes = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.ones(rows // 128, cols // 128, device="cuda")
    for r, c in ((0, 5), (70000, 3), (1 << 17, 0), (rows - 1, cols - 1)):
        codes[r, c] = 0x38  # 1
    scales[-1, -1] = 3.0
    y = mx.dequantize(mx.QTensor(mx.MX_FMT_FP8_B128X128, rows, cols, codes, scales), BF16)
    assert y[0, 5] == 1 and y[70000, 3] == 1 and y[1 << 17, 0] == 1 and y[-1, -1] == 3
    assert y[-128:].float().sum().item() == 4 and y[:128].float().sum().item() == 1


def test_gemm_without_allocation():
    """mx_gemm_noalloc gives mx_gemm's bits: the pair needs no scratch."""
    require_gpu()
    a, b = _operands(20, 300, 512, 12)
    want = mx.gemm(a, b, BF16)
    got = torch.empty_like(want)
    assert mx.mx_gemm_noalloc(a.fmt, b.fmt, 128, 0, 20, 300, 512, a.codes.data_ptr(), a.scales.data_ptr(), None,
                              b.codes.data_ptr(), b.scales.data_ptr(), None, mx.MX_OUT_BF16, got.data_ptr(), 300,
                              torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(got, want)


def _operands(M, N, K, seed):
    r = np.random.RandomState(seed)
    a = _bf16(r.standard_normal((M, K)) * np.where(r.random_sample(K) < 0.01, 40, 1))
    b = _bf16(r.standard_normal((N, K)) * 0.02)
    return mx.quantize(a.cuda(), "fp8_b128"), mx.quantize(b.cuda(), "fp8_b128x128")


def _val(q):
    return ref.fp8_values(host(q.codes), host(q.scales), q.fmt == mx.MX_FMT_FP8_B128X128)


def tolerance(c, s, out):
    """mx.h: fp32 2^-18 sum|ab|; bf16 2^-10 sum|ab| from the FP8 MFMA, then half
    a bf16 step (at most 2^-8 of the rounded value)."""
    return 2.0**-18 * s if out == F32 else 2.0**-10 * s * (1 + 2.0**-8) + 2.0**-8 * np.abs(c)


def check(got, c, s, out):
    got = host(got.float()).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(c))
    bad = np.abs(got - c) > tolerance(c, s, out)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], c[bad][:4])


# Few rows (up to 16: few tiles, enough, long rows with 7 tiles a workgroup), then tiles
# of 32, 64, 128 and 256 square, each with ragged edges in M and N.
SHAPES = [(1, 1, 128), (1, 4096, 1024), (2, 17, 256), (7, 130, 640), (16, 512, 4096),
          (3, 8200, 2304), (5, 10300, 2176), (9, 29000, 6400), (16, 300, 14336),
          (9, 8300, 1024), (16, 6000, 2176), (11, 10100, 3200), (2, 16000, 2432), (3, 4200, 16512), (17, 129, 384), (33, 255, 1152), (700, 2100, 384), (64, 64, 128), (100, 1000, 2432), (129, 257, 512),
          (300, 513, 1024), (40, 13000, 256), (500, 1900, 640), (1000, 3300, 512), (130, 14300, 256),
          (1300, 5000, 384), (1290, 5100, 128), (2100, 2050, 640), (4000, 1500, 256)]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, out):
    require_gpu()
    a, b = _operands(M, N, K, M + N + K)
    check(mx.gemm(a, b, out), *ref.product(_val(a), _val(b)), out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M", [3, 40, 260])
def test_gemm_random_codes(M, out):
    """Codes of every exponent, where the FP8 MFMA drops the most."""
    require_gpu()
    r = np.random.RandomState(M)
    N, K = 150, 1024

    def rand(rows, tall):
        c = r.randint(0, 256, (rows, K)).astype(np.uint8)
        c[(c & 127) == 127] = 0
        s = np.exp2(r.uniform(-8, 8, (-(-rows // 128) if tall else rows, K // 128))).astype(np.float32)
        return mx.QTensor(mx.FORMATS["fp8_b128x128" if tall else "fp8_b128"], rows, K, dev_u8(c), torch.from_numpy(s).cuda())

    a, b = rand(M, False), rand(N, True)
    check(mx.gemm(a, b, out), *ref.product(_val(a), _val(b)), out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N", [(2, 200), (200, 200), (1500, 5000)])
def test_gemm_nan(M, N, out):
    """A NaN scale of A reaches its row, one of B its 128 columns, a NaN code its row or column."""
    require_gpu()
    a, b = _operands(M, N, 512, 9)
    a.scales[1, 2] = float("nan")
    b.scales[0, 3] = float("nan")
    b.codes[150, 7] = 0x7F
    c, s = ref.product(_val(a), _val(b))
    assert np.isnan(c[0, :128]).all() and np.isnan(c[1]).all() and np.isnan(c[0, 150]) and np.isfinite(c[0, 151])
    check(mx.gemm(a, b, out), c, s, out)


@pytest.mark.parametrize("M,N,ld", [(5, 100, 104), (5, 100, 101), (150, 200, 333), (300, 260, 264)])
def test_gemm_strided_out(M, N, ld):
    """Only the M x N outputs are written."""
    require_gpu()
    a, b = _operands(M, N, 256, 11)
    c, s = ref.product(_val(a), _val(b))
    for out in (F32, BF16):
        buf = torch.full((M + 2, ld), 7.0, dtype=out, device="cuda")
        check(mx.gemm(a, b, out, out=buf[:M, :N]), c, s, out)
        assert bool((buf[:, N:] == 7).all()) and bool((buf[M:] == 7).all())


def test_gemm_long_chain_f32():
    """Every product of one sign, K over one accumulation chain: still within 2^-18 sum|ab|."""
    require_gpu()
    r = np.random.RandomState(2)
    K = 128 * 100
    for M in (4, 140):
        a = mx.quantize(_bf16(np.abs(r.standard_normal((M, K)))).cuda(), "fp8_b128")
        b = mx.quantize(_bf16(np.abs(r.standard_normal((130, K)))).cuda(), "fp8_b128x128")
        check(mx.gemm(a, b, F32), *ref.product(_val(a), _val(b)), F32)


def test_gemm_repeats_and_streams():
    """The same bits on every call, on any stream, two calls at once among them."""
    require_gpu()
    for M in (9, 150):
        a, b = _operands(M, 300, 2048, 13)
        first = mx.gemm(a, b, BF16)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = []
        for s in streams:
            with torch.cuda.stream(s):
                outs += [mx.gemm(a, b, BF16) for _ in range(3)]
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, first)


def exact_tolerance(c, s):
    """A bf16 rounding of a result within 2^-18 sum|ab|."""
    return 2.0**-18 * s * (1 + 2.0**-8) + 2.0**-8 * np.abs(c)


def _cancelling(rows, K, tall, seed):
    """Codes 448 and, in b, -448 beside it, among values of 2 to 3.75: products of the first
    cancel, and what is left lies below 2^-13 of them, the last bits of the FP8 MFMA's sum."""
    r = np.random.RandomState(seed)
    c = r.randint(0x40, 0x48, (rows, K)).astype(np.uint8) | (r.randint(0, 2, (rows, K)) << 7).astype(np.uint8)
    c[:, 0::64], c[:, 1::64] = 0x7E, 0xFE if tall else 0x7E
    s = np.exp2(r.uniform(-8, 8, (-(-rows // 128) if tall else rows, K // 128))).astype(np.float32)
    return mx.QTensor(mx.FORMATS["fp8_b128x128" if tall else "fp8_b128"], rows, K, dev_u8(c), torch.from_numpy(s).cuda())


@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (16, 200, 1024), (16, 9000, 2176), (9, 10300, 2304), (5, 29000, 6400),
                                   (16, 300, 16512), (16, 6000, 2176), (7, 18500, 6272), (16, 28670, 6144)])
def test_gemm_few_rows_exact_before_rounding(M, N, K):
    """Up to 16 rows HBM is the bound and products are summed exactly: 2^-18 sum|ab| before
    a bf16 rounding, also where most of a sum cancels."""
    require_gpu()
    a, b = _cancelling(M, K, False, M), _cancelling(N, K, True, N)
    c, s = ref.product(_val(a), _val(b))
    got = host(mx.gemm(a, b, BF16).float()).astype(np.float64)
    bad = np.abs(got - c) > exact_tolerance(c, s)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4], got[bad][:4], c[bad][:4])


@pytest.mark.parametrize("sizes,N,K", [([3, 0, 17, 1], 300, 4096), ([1] * 8 + [0] * 24, 2048, 4224), ([2, 0, 5], 100, 2048)])
def test_grouped_few_rows_exact_before_rounding(sizes, N, K):
    require_gpu()
    G, M = len(sizes), sum(sizes)
    a = _cancelling(M, K, False, M)
    w = [_cancelling(N, K, True, 7 + g) for g in range(G)]
    b = mx.QTensor(w[0].fmt, G * N, K, torch.cat([x.codes for x in w]), torch.cat([x.scales for x in w]), groups=G)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    c, s = ref.grouped(_val(a), np.stack([_val(x) for x in w]), off)
    got = host(mx.gemm_grouped(a, b, torch.from_numpy(off).cuda(), BF16).float()).astype(np.float64)
    bad = np.abs(got - c) > exact_tolerance(c, s)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4], got[bad][:4], c[bad][:4])


def _uneven(q, seed):
    """Scales of q's 128-K blocks that differ 2^12-fold from one to the next."""
    r = np.random.RandomState(seed)
    f = np.exp2(r.randint(-6, 7, tuple(q.scales.shape))).astype(np.float32)
    q.scales = q.scales * torch.from_numpy(f).cuda()
    return q


def check_bf16(got, a, b):
    c, s = ref.product(a, b)
    bad = np.abs(host(got.float()).astype(np.float64) - c) > ref.fp8_mfma_tolerance(a, b, c, s)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4], c[bad][:4])


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[0] > 16] + [
    (9, 8300, 1024), (40, 1000, 4096), (300, 1000, 4096), (777, 2000, 2432), (150, 14300, 1664), (1300, 5000, 4096)])
def test_gemm_bf16_of_normal_values(M, N, K):
    """On each tile, long K among them: as near as sums of random signs are, which a lost or
    repeated chunk of a row is not."""
    require_gpu()
    a, b = _operands(M, N, K, M + N + K)
    check_bf16(mx.gemm(a, b, BF16), _val(a), _val(b))


@pytest.mark.parametrize("M,N,K", [(1300, 5000, 1152), (1281, 5100, 1280), (1400, 4500, 1408), (1500, 5000, 1664),
                                   (1536, 4096, 2048), (1300, 5000, 128), (1410, 5000, 2176)])
def test_gemm_large_tiles_uneven_scales(M, N, K):
    """256 x 256 tiles keep two groups of four steps' scales: from 9 steps on each is
    refilled and read again. Scales of neighbouring steps differ, so that a step under another one's
    shows (whole and partial groups, last row tiles of up to 64, 128 and 256 rows)."""
    require_gpu()
    a, b = _operands(M, N, K, M + K)
    _uneven(a, 1), _uneven(b, 2)
    check_bf16(mx.gemm(a, b, BF16), _val(a), _val(b))


@pytest.mark.parametrize("K", [1152, 1280, 1408, 1664, 2048])
def test_grouped_large_tiles_uneven_scales(K):
    """The same by expert, weights two steps ahead."""
    require_gpu()
    sizes, N = [257, 64, 0, 65, 128, 129, 1000], 4200
    G, M = len(sizes), sum(sizes)
    a = _uneven(_operands(M, 1, K, K)[0], 1)
    w = [_uneven(_operands(1, N, K, K + g)[1], 2 + g) for g in range(G)]
    b = mx.QTensor(w[0].fmt, G * N, K, torch.cat([x.codes for x in w]), torch.cat([x.scales for x in w]), groups=G)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    got = mx.gemm_grouped(a, b, torch.from_numpy(off).cuda(), BF16)
    values = _val(a)
    for g in range(G):
        rows = slice(off[g], off[g + 1])
        check_bf16(got[rows], values[rows], _val(w[g]))


@pytest.mark.parametrize("kind", ["fp8", "mxfp4", "mxfp8", "w4a16"])
def test_gemm_one_row_into_any_stride(kind):
    """The row stride of a single row says nothing."""
    require_gpu()
    N, K = 100, 256
    x, w = _mixed(1, K, 1).cuda(), _mixed(N, K, 2).cuda()
    if kind == "fp8":
        a, b = mx.quantize(x, "fp8_b128"), mx.quantize(w, "fp8_b128x128")
    else:
        a, b = x if kind == "w4a16" else mx.quantize(x, kind), mx.quantize(w, "mxfp4" if kind == "w4a16" else kind)
    out = torch.full((N, 1), 7.0, dtype=BF16, device="cuda").t()
    assert out.stride() == (1, 1)
    assert mx.gemm(a, b, BF16, out=out) is out
    assert torch.equal(out, mx.gemm(a, b, BF16))


@pytest.mark.parametrize("N", [1, 100, 128, 384])
def test_stack_is_each_weight_by_itself(N):
    """Codes, scales and dequantized values of a stack; weights of different magnitudes."""
    require_gpu()
    G, K = 5, 256
    x = torch.stack([_mixed(N, K, g) * 4.0**g for g in range(G)])
    q = mx.quantize(x.cuda(), "fp8_b128x128")
    assert q.groups == G and tuple(q.codes.shape) == (G * N, K) and tuple(q.scales.shape) == (G, -(-N // 128), K // 128)
    for out in (F32, BF16):
        y = mx.dequantize(q, out)
        assert tuple(y.shape) == (G * N, K)
        for g in range(G):
            codes, scales = ref.quantize_fp8(_values(x[g]), True)
            rows = slice(g * N, (g + 1) * N)
            assert np.array_equal(host(q.codes[rows]), codes) and np.array_equal(host(q.scales[g]), scales)
            assert torch.equal(y[rows].cpu(), torch.from_numpy(ref.fp8_values(codes, scales, True)).to(F32).to(out))
