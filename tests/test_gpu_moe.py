"""The mixture-of-experts layer for a few tokens against its definition in 64
bits: layers whose every step is exact bit for bit, others within the roundings of
their steps."""
import pytest
import torch

import microscaling_precision_quantization_amd as mx
import moe_reference as ref
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FMTS = {"mxfp4": mx.MX_FMT_MXFP4, "fp8_b128x128": mx.MX_FMT_FP8_B128X128, "int8": mx.MX_FMT_INT8}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _whole(fmt, values):
    """A stack of whole numbers -2 .. 2 [E][rows][cols] in `fmt`, exactly (scales of 1)."""
    E, rows, cols = values.shape
    v = values.long()
    if fmt == "int8":
        return mx.QTensor(FMTS[fmt], E * rows, cols, (v & 255).to(torch.uint8).view(-1, cols), torch.ones(E * rows, device="cuda"), groups=E)
    if fmt == "fp8_b128x128":
        codes = values.float().to(torch.float8_e4m3fn).view(torch.uint8).view(-1, cols)
        return mx.QTensor(FMTS[fmt], E * rows, cols, codes, torch.ones(E, -(-rows // 128), cols // 128, device="cuda"), groups=E)
    code = torch.tensor([0, 2, 4], device="cuda")[v.abs()] | (v < 0) * 8
    code = code.view(E * rows, cols // 2, 2)
    codes = (code[..., 0] | code[..., 1] << 4).to(torch.uint8)
    return mx.QTensor(FMTS[fmt], E * rows, cols, codes, torch.full((E * rows, cols // 32), 127, dtype=torch.uint8, device="cuda"), groups=E)


def _exact_layer(fmt, T, E, H, I, seed):
    """x and weights whose gate is 64 (so that silu(gate) = gate in fp32: 1 + exp(-64) is 1),
    whose up projections are whole numbers of at most 18 and down's of at most 2: every step is
    exact. Three columns of x besides the first are not zero."""
    g = _gen(seed)
    up = torch.randint(-2, 3, (E, 2 * I, H), device="cuda", generator=g)
    up[:, :I] = 0
    up[:, :I, 0] = 1
    up[:, I:, 0] = 0
    down = torch.randint(-2, 3, (E, H, I), device="cuda", generator=g)
    x = torch.zeros(T, H, device="cuda")
    for _ in range(3):
        x[torch.arange(T), torch.randint(1, H, (T,), device="cuda", generator=g)] = torch.randint(1, 4, (T,), device="cuda", generator=g).float()
    x[:, 0] = 64
    return x.bfloat16(), _whole(fmt, up), _whole(fmt, down), up.double(), down.double()


def _exact(x, ids, weights, up, down):
    x, I = x.double(), down.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < up.shape[0]:
                both = up[e] @ x[t]
                y[t] += weights[t, j].double() * (down[e] @ (both[:I] * both[I:]))
    return y


def _ids(T, E, top, seed, kind="distinct"):
    g = _gen(seed)
    if kind == "distinct":
        ids = torch.rand(T, E, device="cuda", generator=g).argsort(1)[:, :top]
    elif kind == "any":  # the same expert twice, and none
        ids = torch.randint(-2, E + 2, (T, top), device="cuda", generator=g)
    elif kind == "one":  # all tokens to the last expert
        ids = torch.full((T, top), E - 1, device="cuda")
        ids[:, 1:] = -1
    elif kind == "none":
        ids = torch.full((T, top), -1, device="cuda")
        ids[::2] = E
    ids = ids.to(torch.int32).contiguous()
    weights = torch.exp2(torch.randint(-3, 2, (T, top), device="cuda", generator=g).float())
    return ids, weights


SIZES = {"mxfp4": [(64, 32), (256, 128), (288, 352), (1056, 416), (2880, 1440)],
         "fp8_b128x128": [(128, 128), (256, 384), (1408, 256), (2048, 1408)],
         "int8": [(16, 16), (128, 256), (144, 400), (1040, 336), (2064, 1424)]}


@pytest.mark.parametrize("T,E,top,kind", [(1, 1, 1, "distinct"), (1, 32, 8, "distinct"), (4, 64, 6, "distinct"), (17, 5, 2, "distinct"),
                                          (33, 9, 4, "any"), (64, 3, 3, "distinct"), (64, 70, 8, "any"), (64, 6, 2, "one"), (40, 4, 3, "none"),
                                          (3, 200, 32, "any")])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_exact_layers(fmt, T, E, top, kind):
    require_gpu()
    for H, I in SIZES[fmt]:
        if E * H * I > 1 << 27:
            continue
        x, up, down, vu, vd = _exact_layer(fmt, T, E, H, I, T + E + H)
        ids, weights = _ids(T, E, top, T * H + I, kind)
        y = _exact(x, ids, weights, vu, vd)
        # |up x| <= 18, so every sum is of multiples of 64 / 8 (the least weight) and of magnitudes below 2^24 of these.
        assert 64 * 18 * 2 * I * top * 2 < 2**24 * 8
        got = mx.moe(x, ids, weights, up, down, F32)
        assert torch.equal(got.double(), y), (H, I)
        assert torch.equal(mx.moe(x, ids, weights, up, down), y.float().bfloat16())


@pytest.mark.parametrize("fmt,H,I", [("mxfp4", 6176, 160), ("mxfp4", 8192, 96), ("mxfp4", 8224, 96), ("mxfp4", 96, 4224), ("mxfp4", 128, 8352),
                                     ("mxfp4", 18464, 32), ("fp8_b128x128", 2176, 128), ("fp8_b128x128", 4224, 256), ("fp8_b128x128", 128, 4096),
                                     ("fp8_b128x128", 256, 8576), ("int8", 2064, 48), ("int8", 4096, 16), ("int8", 4112, 80), ("int8", 16, 2192),
                                     ("int8", 176, 8240)])
def test_long_rows(fmt, H, I):
    """Rows of two to nine steps a wave, in one round of loads and in several, whole steps and parts of one."""
    require_gpu()
    for T, E, top, kind in ((1, 2, 1, "distinct"), (20, 3, 2, "any"), (64, 5, 2, "distinct")):
        x, up, down, vu, vd = _exact_layer(fmt, T, E, H, I, H + I)
        ids, weights = _ids(T, E, top, T + H, kind)
        assert 64 * 18 * 2 * I * top * 2 < 2**24 * 8  # (as above)
        assert torch.equal(mx.moe(x, ids, weights, up, down, F32).double(), _exact(x, ids, weights, vu, vd)), (T, kind)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("T,E,top,kind", [(64, 400, 6, "distinct"), (64, 1024, 32, "any"), (50, 1000, 8, "any")])
def test_more_passes_than_workgroups(fmt, T, E, top, kind):
    require_gpu()
    H, I = (288, 160) if fmt == "mxfp4" else (256, 128)
    x, up, down, vu, vd = _exact_layer(fmt, T, E, H, I, 4)
    ids, weights = _ids(T, E, top, T * H + I, kind)
    assert 64 * 18 * 2 * I * top * 2 < 2**24 * 8  # (as above)
    assert torch.equal(mx.moe(x, ids, weights, up, down, F32).double(), _exact(x, ids, weights, vu, vd))


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("T,E,top", [(1, 8, 2), (5, 12, 4), (31, 6, 3)])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_random_layers(fmt, T, E, top, out):
    require_gpu()
    for H, I in SIZES[fmt][1:]:
        g = _gen(H + I)
        x = torch.randn(T, H, device="cuda", generator=g)
        x[:, torch.rand(H, device="cuda", generator=g) < 0.01] *= 40
        x = x.bfloat16()
        up = mx.quantize((torch.randn(E, 2 * I, H, device="cuda", generator=g) * H**-0.5).bfloat16(), fmt)
        down = mx.quantize((torch.randn(E, H, I, device="cuda", generator=g) * 0.02).bfloat16(), fmt)
        ids, _ = _ids(T, E, top, H)
        weights = torch.softmax(torch.randn(T, top, device="cuda", generator=g), 1)
        y, tol = ref.layer(x, ids, weights, ref.stack_values(up, mx), ref.stack_values(down, mx))
        ref.check(mx.moe(x, ids, weights, up, down, out), y, tol, out)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_scales(fmt):
    """Scales that differ from block to block, row to row and expert to expert by powers of two up to 2^40."""
    require_gpu()
    T, E, top, H, I = 6, 5, 2, 512, 384
    x, up, down, _, _ = _exact_layer(fmt, T, E, H, I, 3)
    x = (x.float() * 2.0**-12).bfloat16()
    g = _gen(9)
    for q in (up, down):
        if fmt == "mxfp4":
            q.scales.copy_(127 + torch.randint(-20, 20, q.scales.shape, device="cuda", generator=g))
        else:
            q.scales.copy_(torch.exp2(torch.randint(-20, 20, q.scales.shape, device="cuda", generator=g).float()))
    ids, weights = _ids(T, E, top, 1)
    y, tol = ref.layer(x, ids, weights, ref.stack_values(up, mx), ref.stack_values(down, mx), random=False)
    for out in (F32, BF16):
        ref.check(mx.moe(x, ids, weights, up, down, out), y, tol, out)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_nan_stays_with_its_tokens(fmt):
    """NaN and Inf in a token reach no other; an expert with a NaN scale reaches its own tokens
    only; infinities next to columns that weights of zero meet give NaN, as 0 * Inf does."""
    require_gpu()
    T, E, top, H, I = 20, 4, 2, 288 if fmt == "mxfp4" else 256, 128
    x, up, down, vu, vd = _exact_layer(fmt, T, E, H, I, 5)
    ids, weights = _ids(T, E, top, 2)
    clean = mx.moe(x, ids, weights, up, down, F32)
    x[3, 7], x[11, H - 1] = float("nan"), float("inf")
    got = mx.moe(x, ids, weights, up, down, F32)
    keep = [t for t in range(T) if t not in (3, 11)]
    assert torch.isnan(got[3]).all() and torch.isnan(got[11]).all() and torch.equal(got[keep], clean[keep])
    x[3, 7], x[11, H - 1] = 0, 0
    for q in (up, down):
        s = q.scales.view(E, -1)
        old = s[2].clone()
        s[2] = 255 if fmt == "mxfp4" else float("nan")
        got = mx.moe(x, ids, weights, up, down, F32)
        s[2] = old
        hit = (ids == 2).any(1)
        again = mx.moe(x, ids, weights, up, down, F32)
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], again[~hit])


def test_extreme_gates():
    """Gates so large either way that exp overflows or vanishes."""
    require_gpu()
    H = I = 128
    up = torch.zeros(1, 2 * I, H, device="cuda")
    up[0, torch.arange(I), torch.arange(I)] = 1   # gate i = x_i
    up[0, I:, 0] = 1                              # up i = x_0
    down = torch.zeros(1, H, I, device="cuda")
    down[0, torch.arange(H), torch.arange(I)] = 1
    x = torch.zeros(2, H, device="cuda")
    x[:, 0] = 2
    x[0, 1:8] = torch.tensor([-1e4, 1e4, -88.5, -104.0, 88.5, -0.0, 1e37])
    x[1, 1:4] = torch.tensor([-3e38, -700.0, 0.25])
    x = x.bfloat16()
    got = mx.moe(x, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda"), _whole("int8", up), _whole("int8", down), F32)
    v = x.double()
    want = v * torch.sigmoid(v) * v[:, :1]
    # (an exponential of 88 has an argument rounded to 2^-18: h is within 2^-15 of itself, then bf16; tiny values to 0)
    assert ((got.double() - want).abs() <= want.abs() * (2.0**-8 + 2.0**-15) + 1e-37).all()


def test_strides_and_out():
    require_gpu()
    T, E, top, H, I = 7, 4, 2, 256, 128
    x, up, down, vu, vd = _exact_layer("mxfp4", T, E, H, I, 8)
    ids, weights = _ids(T, E, top, 4)
    y = _exact(x, ids, weights, vu, vd)
    wide = torch.full((T, H + 24), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:8 + H] = x
    for out in (F32, BF16):
        dst = torch.full((T + 2, H + 16), 5.0, dtype=out, device="cuda")
        got = mx.moe(wide[:, 8:8 + H], ids, weights, up, down, out, out=dst[1:1 + T, 4 if out == F32 else 8:][:, :H])
        assert torch.equal(got.double(), y.to(out).double())
        at = 4 if out == F32 else 8
        dst[1:1 + T, at:at + H] = 5
        assert (dst == 5).all()
    one = mx.moe(x[:1], ids[:1], weights[:1], up, down, F32, out=torch.zeros(1, H, device="cuda").as_strided((1, H), (3, 1)))
    assert torch.equal(one.double(), y[:1])
    with pytest.raises(mx.MXError):  # rows that do not start on 16 bytes
        mx.moe(torch.zeros(T, H + 4, dtype=BF16, device="cuda")[:, :H], ids, weights, up, down)
    with pytest.raises(mx.MXError):
        mx.moe(x, ids, weights, up, down, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mx.MXError):
        mx.moe(x, ids[:, :0].contiguous(), weights[:, :0].contiguous(), up, down)
    assert tuple(mx.moe(x[:0], ids[:0], weights[:0], up, down).shape) == (0, H)


def test_workspace():
    """Any contents of the workspace, and nothing written past it."""
    require_gpu()
    T, E, top, H, I = 30, 7, 4, 512, 256
    x, up, down, vu, vd = _exact_layer("int8", T, E, H, I, 8)
    n = mx.mx_moe_workspace_bytes(T, top, E, H, I)
    ws = torch.empty(n + 4096, dtype=torch.uint8, device="cuda")
    for seed, fill in ((1, 255), (2, 0), (3, 127)):
        ids, weights = _ids(T, E, top, seed, "any")
        ws.fill_(fill)
        got = mx.moe(x, ids, weights, up, down, F32, workspace=ws[:n])
        assert torch.equal(got.double(), _exact(x, ids, weights, vu, vd))
        assert (ws[n:] == fill).all()


@pytest.mark.parametrize("fmt", list(FMTS))
def test_captured(fmt):
    """Captured once, replayed with other tokens and ids between eager work: the eager result, bit for bit."""
    require_gpu()
    T, E, top, H, I = 24, 6, 3, 512, 384
    x, up, down, _, _ = _exact_layer(fmt, T, E, H, I, 8)
    ids, weights = _ids(T, E, top, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.moe(x, ids, weights, up, down)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mx.moe(x, ids, weights, up, down, F32)
    for i, kind in enumerate(("distinct", "any", "one", "none", "any")):
        a, b = _ids(T, E, top, 10 + i, kind)
        ids.copy_(a)
        weights.copy_(b * 0.3)
        x.copy_(torch.randn(T, H, device="cuda", generator=_gen(i)))
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, mx.moe(x, ids, weights, up, down, F32)), i
        again = mx.moe(x, ids, weights, up, down, F32)
        assert torch.equal(got, again)


def test_two_streams():
    """Two calls at once, each with its own workspace."""
    require_gpu()
    T, E, top, H, I = 16, 6, 3, 1024, 512
    x, up, down, _, _ = _exact_layer("mxfp4", T, E, H, I, 8)
    args = [(_ids(T, E, top, s)) for s in range(8)]
    want = [mx.moe(x, i, w, up, down, F32) for i, w in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for n, (i, w) in enumerate(args):
        with torch.cuda.stream(streams[n % 2]):
            got.append(mx.moe(x, i, w, up, down, F32))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_equals_the_products_by_expert():
    """The same layer by gemm_grouped: rows sorted by expert, the activations in the codes of int8
    (whole numbers below 128, so exactly), the result the same."""
    require_gpu()
    T, E, top, H, I = 48, 5, 2, 256, 160
    x, up, down, vu, vd = _exact_layer("int8", T, E, H, I, 21)
    x[:, 0], x[:, 1] = 64, 127   # (a scale of 1 for every row)
    ids, weights = _ids(T, E, top, 3)
    order = ids.flatten().long().argsort(stable=True)
    rows = order // top
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    both = mx.gemm_grouped(mx.quantize(x[rows].contiguous(), "int8"), up, offsets, F32)
    h = both[:, :I] * both[:, I:]  # (silu(64) = 64)
    q = mx.quantize((h / 64).bfloat16(), "int8")
    assert (both[:, :I] == 64).all()
    part = mx.gemm_grouped(q, down, offsets, F32) * 64 * weights.flatten()[order, None]
    y = torch.zeros(T, H, device="cuda").index_add_(0, rows, part)
    got = mx.moe(x, ids, weights, up, down, F32)
    # h here is rounded to int8's steps, half of amax / 127 each: within that times the weights' magnitudes.
    step = (h.abs().amax(1, keepdim=True) / 254).double()
    tol = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dmag = down.codes.view(torch.int8).double().view(E, H, I).abs().sum(2)
    tol.index_add_(0, rows, step * dmag[ids.flatten().long()[order]] * weights.flatten()[order, None].double())
    # (bf16 of h, both ways: 2^-8 of its terms, which are at most 254 of those half steps)
    assert ((got - y).double().abs() <= tol * 1.02 + 2 * 2.0**-8 * tol * 254).all()


def test_experts_past_32_bits():
    require_gpu()
    E, H, I = 40, 8192, 4096  # 2.7 GB of up, 1.3 of down
    g = _gen(0)
    up = mx.QTensor(mx.MX_FMT_INT8, E * 2 * I, H, torch.randint(0, 256, (E * 2 * I, H), dtype=torch.uint8, device="cuda", generator=g),
                    torch.full((E * 2 * I,), 1e-4, device="cuda"), groups=E)
    down = mx.QTensor(mx.MX_FMT_INT8, E * H, I, torch.randint(0, 256, (E * H, I), dtype=torch.uint8, device="cuda", generator=g),
                      torch.full((E * H,), 1e-4, device="cuda"), groups=E)
    x = torch.randn(2, H, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([[39, 0], [20, 39]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, 0.25], [0.75, 0.5]], device="cuda")
    got = mx.moe(x, ids, weights, up, down, F32)
    def one(e):
        a = mx.QTensor(mx.MX_FMT_INT8, 2 * I, H, up.codes[e * 2 * I:(e + 1) * 2 * I], up.scales[:2 * I])
        b = mx.QTensor(mx.MX_FMT_INT8, H, I, down.codes[e * H:(e + 1) * H], down.scales[:H])
        return ref.stack_values(a, mx), ref.stack_values(b, mx)
    us, ds = zip(*(one(e) for e in (0, 20, 39)))
    small = torch.tensor([[2, 0], [1, 2]], dtype=torch.int32, device="cuda")
    y, tol = ref.layer(x, small, weights, torch.cat(us), torch.cat(ds))
    ref.check(got, y, tol, F32)


@pytest.mark.parametrize("H,I", [(1 << 20, 1024), (1024, 1 << 20)])
@pytest.mark.parametrize("fmt", ["int8", "fp8_b128x128"])
def test_widest(fmt, H, I):
    """The largest widths and weights there may be; exact, as few values of x and of h are not zero."""
    require_gpu()
    T, g = 3, _gen(7)

    def stack(v):  # whole numbers -2 .. 2
        rows, cols = v.shape
        if fmt == "int8":
            return mx.QTensor(FMTS[fmt], rows, cols, v.view(torch.uint8), torch.ones(rows, device="cuda"))
        a = v.abs().view(torch.uint8)
        return mx.QTensor(FMTS[fmt], rows, cols, (a * 8 + 0x30) * (a > 0) | (v < 0) * torch.tensor(0x80, dtype=torch.uint8, device="cuda"),
                          torch.ones(-(-rows // 128), cols // 128, device="cuda"))
    up = torch.randint(-2, 3, (2 * I, H), dtype=torch.int8, device="cuda", generator=g)
    busy = torch.cat([torch.randint(0, I, (500,), device="cuda", generator=g), torch.tensor([0, I - 1], device="cuda")])
    idle = torch.ones(I, dtype=torch.bool, device="cuda")
    idle[busy] = False
    up[:I] = 0
    up[:I, 0] = 1
    up[I:][idle] = 0
    up[I:, 0] = 0
    down = torch.randint(-2, 3, (H, I), dtype=torch.int8, device="cuda", generator=g)
    x = torch.zeros(T, H, device="cuda")
    at = torch.cat([torch.randint(1, H - 1, (2,), device="cuda", generator=g), torch.tensor([0, H - 1], device="cuda")])
    x[:, at[:2]], x[:, H - 1], x[:, 0] = 2, 3, 64
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    weights = torch.tensor([[1.0], [0.5], [2.0]], device="cuda")
    lin = up[I:][:, at].double() @ x[:, at].double().t()
    assert len(set(at.tolist())) == 4 and lin.abs().max() <= 14  # so every sum is of multiples of 64, at most 64 * 14 * 2 * 502
    h = 64 * lin[busy.unique()]
    y = (down[:, busy.unique()].double() @ h).t() * weights.double()
    assert torch.equal(mx.moe(x.bfloat16(), ids, weights, stack(up), stack(down), F32).double(), y)


def _scaled(fmt, v, seed, rows_at_one=0):
    """A stack of whole numbers in `fmt` with scales of 1 and 2 (by block, INT8 by row; the first rows' 1), and its values."""
    q, (E, rows, cols) = _whole(fmt, v), v.shape
    two = torch.randint(0, 2, q.scales.shape, device="cuda", generator=_gen(seed))
    if fmt == "fp8_b128x128":
        two[:, :rows_at_one // 128] = 0
        by_row = two.repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)
    else:
        two.view(E, rows, -1)[:, :rows_at_one] = 0
        by_row = two.view(E, rows, -1).repeat_interleave(32 if fmt == "mxfp4" else cols, 2)
    q.scales += two.to(q.scales.dtype)
    return q, v.double() * (1 + by_row)


def _dense_layer(fmt, T, E, H, I, seed):
    """As _exact_layer, but a twelfth of x and two thirds of the up and down weights are not zero, so
    that a wrong code of any step changes a result."""
    g = _gen(seed)
    up = torch.randint(-1, 2, (E, 2 * I, H), dtype=torch.int8, device="cuda", generator=g)
    up[:, :I] = 0
    up[:, :I, 0] = 1
    up[:, I:, 0] = 0
    down = torch.randint(-1, 2, (E, H, I), dtype=torch.int8, device="cuda", generator=g)
    x = torch.randint(0, 2, (T, H), device="cuda", generator=g) * 2.0 - 1
    x *= torch.rand(T, H, device="cuda", generator=g) < 1 / 12
    x[:, 0] = 64
    up, vu = _scaled(fmt, up, seed + 1, I)
    down, vd = _scaled(fmt, down, seed + 2)
    return x.bfloat16(), up, down, vu, vd


@pytest.mark.parametrize("fmt,H,I", [("mxfp4", 8224, 8416), ("mxfp4", 8448, 8320), ("mxfp4", 4096, 14336), ("fp8_b128x128", 5120, 7168),
                                     ("fp8_b128x128", 7168, 5120), ("int8", 5120, 5136), ("int8", 7168, 4112)])
def test_dense_long_rows(fmt, H, I):
    """Rows of several rounds of loads, bit for bit, on weights larger than the last-level cache. Tiles of a
    workgroup that fill their groups and that do not."""
    require_gpu()
    E = 6
    x, up, down, vu, vd = _dense_layer(fmt, 40, E, H, I, H + I)
    # h is 64 times a whole number that bf16 holds; down's sums are of multiples of 64 and, weighted, of 64 / 8, all
    # below 2^24 of them.
    lin = torch.stack([vu[e, I:] @ x.double().t() for e in range(E)])
    assert lin.abs().max() <= 256 and vd.abs().sum(2).max() * 256 < 2**24
    assert max((vd[e] @ lin[e]).abs().max() for e in range(E)) * 64 * 2 * 3 < 2**24 * 8
    for T, top, kind in ((1, 1, "distinct"), (2, 2, "distinct"), (5, 3, "any"), (40, 2, "distinct")):
        ids, weights = _ids(T, E, top, T + H, kind)
        got = mx.moe(x[:T], ids, weights, up, down, F32)
        assert torch.equal(got.double(), _exact(x[:T], ids, weights, vu, vd)), (T, kind)


PARTED = {"mxfp4": [(256, 352), (256, 2176), (288, 4224), (256, 8352)], "fp8_b128x128": [(256, 384), (256, 1152), (128, 2176), (256, 4224)],
          "int8": [(144, 400), (176, 1040), (144, 2064), (208, 4112)]}


@pytest.mark.parametrize("T,E,top,kind", [(1, 3, 2, "distinct"), (8, 2, 1, "one"), (9, 2, 1, "one"), (7, 5, 3, "any"), (40, 4, 2, "distinct")])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_h_of_more_bits_than_bf16(fmt, T, E, top, kind):
    """h of whole numbers of up to 12 bits, which two bf16 numbers hold and one does not: bit for bit."""
    require_gpu()
    for H, I in PARTED[fmt]:
        g = _gen(H + I + T)
        _, up, down, vu, vd = _dense_layer(fmt, T, E, H, I, H + I)
        x = torch.randint(-50, 51, (T, H), device="cuda", generator=g).float()
        x[:, 0] = 64
        lin = torch.stack([vu[e, I:] @ x.double().t() for e in range(E)])
        out = torch.stack([vd[e] @ lin[e] for e in range(E)])
        # (sums of multiples of 64 and, weighted, of 64 / 8; the high part of a number is at most twice it)
        assert 256 < lin.abs().max() < 2**12 and max((vd[e].abs() @ lin[e].abs()).max() for e in range(E)) * 2 < 2**24
        assert out.abs().max() * 64 * 2 * top < 2**24 * 8
        ids, weights = _ids(T, E, top, T + H, kind)
        x = x.bfloat16()
        assert torch.equal(mx.moe(x, ids, weights, up, down, F32).double(), _exact(x, ids, weights, vu, vd)), (H, I)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("T,E,top", [(1, 8, 2), (8, 12, 4), (9, 3, 2), (31, 6, 3)])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_random_layers_in_32_bits(fmt, T, E, top, out):
    """Within the roundings of fp32 sums and of h's two parts, 2^-17: an fp32 result is one, and a bf16 one is rounded once."""
    require_gpu()
    for H, I in SIZES[fmt][1:] + PARTED[fmt][2:]:
        g = _gen(H * I + T)
        x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
        up = mx.quantize((torch.randn(E, 2 * I, H, device="cuda", generator=g) * H**-0.5).bfloat16(), fmt)
        down = mx.quantize((torch.randn(E, H, I, device="cuda", generator=g) * 0.02).bfloat16(), fmt)
        ids, _ = _ids(T, E, top, H)
        weights = torch.softmax(torch.randn(T, top, device="cuda", generator=g), 1)
        y, tol = ref.layer(x, ids, weights, ref.stack_values(up, mx), ref.stack_values(down, mx), parts=2)
        ref.check(mx.moe(x, ids, weights, up, down, out), y, tol, out)


@pytest.mark.parametrize("T", [2, 12])
def test_largest_h(T):
    """h past bf16's largest number but not fp32's, and infinite h, whose low part is none."""
    require_gpu()
    H = I = 128
    ones = torch.ones(1, 2 * I, H, device="cuda")
    up = _whole("int8", ones)
    up.scales[I:] = float.fromhex("0x1.ff8p121")
    down = _whole("int8", torch.eye(H, device="cuda")[None])
    down.scales[:] = 0.5
    x = torch.zeros(T, H, device="cuda")
    x[:, 0] = 1
    up.scales[:I] = 64  # gate 64, h = 64 * 0x1.ff8p121
    ids, weights = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    got = mx.moe(x.bfloat16(), ids, weights, up, down, F32)
    assert (got == float.fromhex("0x1.ff8p126")).all()
    up.scales[I:] = 1e37  # h = 6.4e38
    down = _whole("int8", ones[:, :I].contiguous())
    assert (mx.moe(x.bfloat16(), ids, weights, up, down, F32) == float("inf")).all()


@pytest.mark.parametrize("H", [256, 288])
@pytest.mark.parametrize("lo,hi,power", [(0, 3, 125), (124, 130, 0), (251, 254, -125)])
def test_mxfp4_scales_beside_any_others(H, lo, hi, power):
    """Blocks whose scales are the smallest and largest there are, next to scales of any kind: the
    expansion takes a scale with its neighbours' bits beside it."""
    require_gpu()
    T, E, top, I = 16, 3, 2, 128
    g = _gen(H + lo)
    # (codes of at most 1.5, so that a weight under the largest scale is finite)
    code = torch.randint(0, 4, (E * 2 * I, H), device="cuda", generator=g) | torch.randint(0, 2, (E * 2 * I, H), device="cuda", generator=g) * 8
    codes = (code[:, ::2] | code[:, 1::2] << 4).to(torch.uint8)
    scales = torch.randint(0, 255, (E * 2 * I, H // 32), device="cuda", generator=g)
    at = torch.randint(0, 2, (H // 32,), device="cuda", generator=g).bool()
    at[0], at[-1] = True, True
    scales[:, at] = torch.randint(lo, hi + 1, (E * 2 * I, int(at.sum())), device="cuda", generator=g)
    up = mx.QTensor(FMTS["mxfp4"], E * 2 * I, H, codes, scales.to(torch.uint8), groups=E)
    down = mx.quantize((torch.randn(E, H, I, device="cuda", generator=g) * 0.02).bfloat16(), "mxfp4")
    block = at.nonzero().flatten()[torch.randint(0, int(at.sum()), (T,), device="cuda", generator=g)]
    x = torch.zeros(T, H, device="cuda")
    x[torch.arange(T), block * 32 + torch.randint(0, 32, (T,), device="cuda", generator=g)] = 2.0**power
    x = x.bfloat16()
    ids, weights = _ids(T, E, top, H)
    y, tol = ref.layer(x, ids, weights, ref.stack_values(up, mx), ref.stack_values(down, mx), random=False, parts=2)
    assert (y != 0).any(1).sum() > T // 2
    ref.check(mx.moe(x, ids, weights, up, down, F32), y, tol, F32)


@pytest.mark.parametrize("fmt", list(FMTS))
def test_at_most_eight_tokens(fmt):
    """Where the low parts of h are rows of the matrix instructions: NaN and Inf reach their own tokens only, an expert
    of NaN its own, and a captured call follows its inputs, beside eager ones on another stream."""
    require_gpu()
    T, E, top, H, I = 8, 3, 2, 256, 1152
    x, up, down, vu, vd = _dense_layer(fmt, T, E, H, I, 12)
    ids, weights = _ids(T, E, top, 3)
    clean = mx.moe(x, ids, weights, up, down, F32)
    assert torch.equal(clean.double(), _exact(x, ids, weights, vu, vd))
    bad = x.clone()
    bad[1, 7], bad[6, H - 1] = float("nan"), float("inf")
    keep = [0, 2, 3, 4, 5, 7]
    got = mx.moe(bad, ids, weights, up, down, F32)
    assert torch.isnan(got[[1, 6]]).all() and torch.equal(got[keep], clean[keep])
    s = down.scales.view(E, -1)
    old = s[1].clone()
    s[1] = 255 if fmt == "mxfp4" else float("nan")
    got = mx.moe(x, ids, weights, up, down, F32)
    s[1] = old
    hit = (ids == 1).any(1)
    assert 0 < hit.sum() < T and torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.moe(x, ids, weights, up, down)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mx.moe(x, ids, weights, up, down, F32)
    for i, kind in enumerate(("any", "one", "none", "distinct")):
        a, b = _ids(T, E, top, 20 + i, kind)
        ids.copy_(a)
        weights.copy_(b)
        want = _exact(x, ids, weights, vu, vd)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            eager = mx.moe(x, ids, weights, up, down, F32)
        torch.cuda.synchronize()
        assert torch.equal(y.double(), want) and torch.equal(eager, y), kind
