"""GEMM by expert: every row against its expert's weight, within mx.h's bound;
rows of no expert are left as they were."""
import numpy as np
import pytest
import torch

import llm_reference as ref
import microscaling_precision_quantization_amd as mx
from gpu_helpers import dev_u8, host, require_gpu
from test_gpu_fp8_block import tolerance as fp8_tolerance

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _operands(fmt, M, G, N, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=gen, device="cuda").to(BF16)
    w = (torch.randn(G, N, K, generator=gen, device="cuda") * 0.02).to(BF16)
    if fmt == "mxfp4":
        return mx.quantize(x, "mxfp4"), mx.quantize(w, "mxfp4")
    return mx.quantize(x, "fp8_b128"), mx.quantize(w, "fp8_b128x128")


def _a_values(q):
    c, s = host(q.codes), host(q.scales)
    return ref.mxfp4_values(c, s) if q.fmt == mx.MX_FMT_MXFP4 else ref.fp8_values(c, s, False)


def _b_values(q):
    n = q.rows // q.groups
    c, s = host(q.codes).reshape(q.groups, n, -1), host(q.scales).reshape(q.groups, -1, host(q.scales).shape[-1])
    f = ref.mxfp4_values if q.fmt == mx.MX_FMT_MXFP4 else lambda c, s: ref.fp8_values(c, s, True)
    return np.stack([f(c[g], s[g]) for g in range(q.groups)])


def _tolerance(fmt, c, s, out):
    if fmt == "fp8":
        return fp8_tolerance(c, s, out)
    return 2.0**-18 * s * (1 if out == F32 else 1 + 2.0**-8) + (0 if out == F32 else 2.0**-8 * np.abs(c))


def _check(got, a, b, off, fmt, out):
    c, s = ref.grouped(_a_values(a), _b_values(b), off)
    rows = slice(off[0], off[-1])
    err = np.abs(host(got.float()).astype(np.float64) - c)[rows]
    bad = ~(err <= _tolerance(fmt, c, s, out)[rows])
    assert not bad.any(), (np.argwhere(bad)[:4], err[bad][:4])


def _offsets(sizes, start=0):
    off = np.concatenate([[start], start + np.cumsum(sizes)]).astype(np.int32)
    return off, torch.from_numpy(off).cuda()


CASES = [  # sizes of the groups, N, K
    ([1], 1, 128),
    ([1], 300, 512),
    ([0, 1, 0], 40, 256),
    ([3, 0, 5, 1], 100, 384),
    ([16, 17, 15, 0, 33], 130, 1024),
    ([0, 0, 130, 1], 257, 640),
    ([128, 129, 127], 128, 256),
    ([200, 0, 300], 385, 512),
    ([1] * 70, 48, 256),
    ([0, 2, 1] * 50, 33, 128),
    ([700], 260, 2048),
    # few rows per expert on average, more than 16 in one: further passes over its weight
    ([0, 40, 1, 0, 0, 0, 17, 0, 3, 0, 0, 0], 200, 4096),
    ([1] * 12 + [60] + [0] * 30, 2100, 2048),
    ([0, 3, 0, 0, 30, 0, 1, 0, 0], 330, 8192),
    ([2, 0, 20, 0], 100, 4480),
    ([1, 0, 2, 0, 0, 17, 0, 1], 2100, 4224),
    ([1, 3] * 10, 1800, 4224),
    # the same with short rows of weights: tiles
    ([0, 40, 1, 0, 0, 0, 17, 0, 3, 0], 200, 1024),
    ([1] * 12 + [60] + [0] * 30, 2100, 512),
    # enough for tiles of 64, of 128 and of 256 square
    ([33, 100, 1, 70], 2500, 256),
    ([130, 255, 3, 129, 400], 3300, 384),
    ([300, 511, 0, 700, 1], 4100, 512),
    ([257, 64, 65, 128, 129, 1000], 4200, 768),
]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("sizes,N,K", CASES)
def test_grouped(sizes, N, K, fmt, out):
    require_gpu()
    M = sum(sizes)
    a, b = _operands(fmt, M, len(sizes), N, K, M + N)
    off, d = _offsets(sizes)
    _check(mx.gemm_grouped(a, b, d, out), a, b, off, fmt, out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("sizes,N,K", [([20, 31, 0, 9] * 6, 1400, 384), ([20, 31, 0, 9] * 6, 1400, 416),
                                       ([100, 200], 6500, 640), ([100, 200], 6500, 32), ([40] * 5, 3400, 640),
                                       ([40] * 5, 3400, 672), ([350, 0, 90], 1790, 384), ([350, 0, 90], 1790, 288)])
def test_mxfp4_tiles(sizes, N, K, out):
    """MXFP4's steps of 256 K with an odd half at the end, on each tile: 128 square with
    few and with many rows an expert, 64 x 128 and 64 square."""
    require_gpu()
    a, b = _operands("mxfp4", sum(sizes), len(sizes), N, K, N)
    off, d = _offsets(sizes)
    _check(mx.gemm_grouped(a, b, d, out), a, b, off, "mxfp4", out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 288, 384, 736, 1056, 2880, 4128, 4256, 4480])
@pytest.mark.parametrize("sizes", [[2, 0, 3], [1, 18, 0, 0], [70, 150, 1], [300, 250, 600]])
def test_mxfp4_odd_k(K, sizes, out):
    """K that is no multiple of a step. Then every second row's first scale is made
    NaN: read past the end of the row before it, it would spread there."""
    require_gpu()
    a, b = _operands("mxfp4", sum(sizes), len(sizes), 90 if sum(sizes) < 1000 else 2000, K, K)
    off, d = _offsets(sizes)
    _check(mx.gemm_grouped(a, b, d, out), a, b, off, "mxfp4", out)
    a.scales[1::2, 0] = 255
    got = mx.gemm_grouped(a, b, d, out)
    assert bool(got[1::2].isnan().all()) and not bool(got[0::2].isnan().any())


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("start,tail,sizes", [(0, 5, [4, 9]), (3, 0, [6, 0, 2]), (130, 140, [200, 31]),
                                              (2, 300, [0, 0]), (0, 0, [300, 20])])
def test_rows_of_no_group_are_left(fmt, start, tail, sizes):
    require_gpu()
    M, N, K = start + sum(sizes) + tail, 200, 256
    a, b = _operands(fmt, M, len(sizes), N, K, 3)
    off, d = _offsets(sizes, start)
    for out, ld in ((F32, 200), (BF16, 203), (BF16, 208)):
        buf = torch.full((M + 1, ld), 7.0, dtype=out, device="cuda")
        got = mx.gemm_grouped(a, b, d, out, out=buf[:M, :N])
        _check(got, a, b, off, fmt, out)
        assert bool((buf[:start] == 7).all()) and bool((buf[start + sum(sizes):] == 7).all())
        assert bool((buf[:, N:] == 7).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_offsets_past_the_end_are_clamped(fmt):
    """Row numbers beyond [0, M] are read as 0 or M."""
    require_gpu()
    for M in (20, 400):
        a, b = _operands(fmt, M, 3, 64, 256, 4)
        d = torch.tensor([-5, M // 2, M // 2, M + 1000], dtype=torch.int32, device="cuda")
        off = np.array([0, M // 2, M // 2, M])
        _check(mx.gemm_grouped(a, b, d, BF16), a, b, off, fmt, BF16)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("M,N", [(20, 64), (400, 200), (1500, 2600), (3000, 4000)])
def test_offsets_out_of_order(M, N, fmt):
    """Undefined rows of C, but nothing outside C; and the next call is right."""
    require_gpu()
    a, b = _operands(fmt, M, 5, N, 256, 6)
    for bad in ([0, M, 0, M, 0, M], [M, 0, 0, M, 3, 1], [2**31 - 1, -2**31, 5, 4, 3, M]):
        d = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for out in (F32, BF16):
            buf = torch.full((M + 2, N + 8), 7.0, dtype=out, device="cuda")
            mx.gemm_grouped(a, b, d, out, out=buf[1:M + 1, :N])
            assert bool((buf[0] == 7).all()) and bool((buf[M + 1] == 7).all()) and bool((buf[:, N:] == 7).all())
    off, d = _offsets([M // 5] * 4 + [M - M // 5 * 4])
    _check(mx.gemm_grouped(a, b, d, BF16), a, b, off, fmt, BF16)


def test_one_row_into_any_stride():
    """The row stride of a single row says nothing."""
    require_gpu()
    a, b = _operands("fp8", 1, 2, 100, 256, 7)
    off, d = _offsets([0, 1])
    out = torch.empty(100, 1, dtype=BF16, device="cuda").t()
    assert out.stride() == (1, 1)
    _check(mx.gemm_grouped(a, b, d, BF16, out=out), a, b, off, "fp8", BF16)


@pytest.mark.parametrize("rows", [3, 200])
def test_stack_past_32_bits(rows):
    """A stack of more than 2^32 code bytes: the last expert is its own."""
    require_gpu()
    G, N, K = 17, 16384, 16384
    one = mx.quantize((torch.arange(N * K, device="cuda") % 251 - 125).to(BF16).view(N, K), "fp8_b128x128")
    codes = torch.zeros(G * N, K, dtype=torch.uint8, device="cuda")
    scales = torch.ones(G, N // 128, K // 128, device="cuda")
    codes[-N:].copy_(one.codes)
    scales[-1].copy_(one.scales)
    b = mx.QTensor(one.fmt, G * N, K, codes, scales, groups=G)
    a = mx.quantize((torch.arange(rows * K, device="cuda") % 127 - 63).to(BF16).view(rows, K), "fp8_b128")
    d = torch.tensor([0] * G + [rows], dtype=torch.int32, device="cuda")
    got, want = mx.gemm_grouped(a, b, d, F32), mx.gemm(a, one, F32)
    # Both are within 2^-18 sum|ab|, which Cauchy-Schwarz bounds by the rows' norms.
    bound = 2.0**-17 * mx.dequantize(a).norm(dim=1, keepdim=True) * mx.dequantize(one).norm(dim=1)[None, :]
    assert bool(((got - want).abs() <= bound).all()) and bool((want != 0).any())


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("sizes,N,K", [([3, 0, 2], 200, 3584), ([60, 80], 300, 6400), ([700, 0, 900], 3900, 3328)])
def test_long_chains_f32(sizes, N, K, fmt):
    """Every product of one sign and K over one accumulation chain: within 2^-18 sum|ab|."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.rand(sum(sizes), K, generator=gen, device="cuda").to(BF16)
    w = torch.rand(len(sizes), N, K, generator=gen, device="cuda").to(BF16)
    a = mx.quantize(x, "mxfp4" if fmt == "mxfp4" else "fp8_b128")
    b = mx.quantize(w, "mxfp4" if fmt == "mxfp4" else "fp8_b128x128")
    off, d = _offsets(sizes)
    _check(mx.gemm_grouped(a, b, d, F32), a, b, off, fmt, F32)


def test_more_groups_than_a_wave():
    """Row tiles are found by scanning the groups 64 at a time."""
    require_gpu()
    r = np.random.RandomState(0)
    for fmt in ("mxfp4", "fp8"):
        for G, M in ((64, 900), (65, 40), (200, 2000), (300, 7), (130, 9000)):
            sizes = r.multinomial(M, r.dirichlet(np.full(G, 0.3)))
            a, b = _operands(fmt, M, G, 64 if M < 9000 else 700, 128 if M < 9000 else 256, G)
            off, d = _offsets(sizes)
            _check(mx.gemm_grouped(a, b, d, BF16), a, b, off, fmt, BF16)


def test_equals_gemm_of_each_expert():
    """With every group a whole dense product, the same result within both bounds; FP8 weights
    whose rows are no multiple of 128 keep each expert's own tiles."""
    require_gpu()
    a, b = _operands("fp8", 96, 3, 100, 512, 8)
    assert tuple(b.scales.shape) == (3, 1, 4)
    off, d = _offsets([40, 30, 26])
    got = mx.gemm_grouped(a, b, d, F32)
    whole = mx.dequantize(b)
    for g in range(3):
        one = mx.QTensor(b.fmt, 100, 512, b.codes[100 * g:100 * (g + 1)], b.scales[g].contiguous())
        assert torch.equal(mx.dequantize(one), whole[100 * g:100 * (g + 1)])
        rows = slice(off[g], off[g + 1])
        ag = mx.QTensor(a.fmt, rows.stop - rows.start, 512, a.codes[rows], a.scales[rows])
        assert torch.allclose(mx.gemm(ag, one, F32), got[rows], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("M,N", [(150, 256), (40, 100), (2400, 2600)])
@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_captured_with_new_offsets(fmt, M, N):
    """A captured call follows the offsets of each replay: they are read on the device."""
    require_gpu()
    G, K = 6, 512
    a, b = _operands(fmt, M, G, N, K, 6)
    _, d = _offsets([M // 6] * 6)
    out = torch.zeros(M, N, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.gemm_grouped(a, b, d, BF16, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.gemm_grouped(a, b, d, BF16, out=out)
    for sizes in ([M, 0, 0, 0, 0, 0], [1, 2, 3, 4, 5, M - 15], [0, 0, M // 2, 0, M - M // 2, 0]):
        off, new = _offsets(sizes)
        d.copy_(new)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check(out, a, b, off, fmt, BF16)
        assert torch.equal(out, mx.gemm_grouped(a, b, new, BF16))


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_few_rows_skewed(fmt, out):
    """Few rows an expert on average (long rows of weights), most of them in one: its passes
    of 16 rows, found by scanning the groups 64 at a time."""
    require_gpu()
    for G, at, rows in ((64, 0, 384), (64, 63, 383), (65, 64, 200), (130, 70, 500), (200, 199, 17), (3, 1, 18)):
        sizes = [0] * G
        sizes[at] = rows - 2 if G > 3 else rows
        sizes[G // 2] += 1
        sizes[G - 1] += 1
        a, b = _operands(fmt, sum(sizes), G, 40, 4096, G + at)
        off, d = _offsets(sizes)
        _check(mx.gemm_grouped(a, b, d, out), a, b, off, fmt, out)


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_few_rows_offsets(fmt):
    """Few rows, long rows of weights: rows of no group are left, row numbers clamped to
    [0, M], and offsets out of order write nothing outside C."""
    require_gpu()
    M, G, N, K = 60, 70, 100, 4096
    a, b = _operands(fmt, M, G, N, K, 1)
    sizes = np.zeros(G, np.int64)
    sizes[[0, 3, 63, 64, 69]] = [2, 20, 1, 17, 3]
    off, d = _offsets(sizes, 5)
    buf = torch.full((M + 1, N + 4), 7.0, dtype=BF16, device="cuda")
    _check(mx.gemm_grouped(a, b, d, BF16, out=buf[:M, :N]), a, b, off, fmt, BF16)
    assert bool((buf[:5] == 7).all()) and bool((buf[off[-1]:] == 7).all()) and bool((buf[:, N:] == 7).all())
    wide = np.where(np.arange(G + 1) < 4, -9, np.where(np.arange(G + 1) < 66, 31, M + 99)).astype(np.int32)
    _check(mx.gemm_grouped(a, b, torch.from_numpy(wide).cuda(), BF16), a, b, np.clip(wide, 0, M), fmt, BF16)
    r = np.random.RandomState(0)
    for bad in (np.arange(G + 1) % 2 * M, r.randint(-50, 150, G + 1), M - np.arange(G + 1)):
        buf.fill_(7)
        mx.gemm_grouped(a, b, torch.from_numpy(bad.astype(np.int32)).cuda(), BF16, out=buf[:M, :N])
        assert bool((buf[M] == 7).all()) and bool((buf[:, N:] == 7).all())
