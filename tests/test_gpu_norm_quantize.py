"""The fused norms, residual, gate and quantizer against 64 bits. n has fp32
rounding errors before it is quantized, so a code may be any that the formula
gives for a value within n's error; scales likewise."""
import numpy as np
import pytest
import torch

import llm_reference as ref
import microscaling_precision_quantization_amd as mx
from gpu_helpers import host, require_gpu
from test_gpu_fp8_block import check as check_fp8_gemm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# A sum of squares over a thread's 32 elements at most, a wave's 6 steps and 16
# waves' parts, its mean, root and inverse, and the products: under 64
# roundings of 2^-24 in all.
REL = 64 * 2.0**-24


def _t(r, *shape, scale=1.0, add=0.0):
    return torch.from_numpy((r.standard_normal(shape) * scale + add).astype(np.float32)).to(BF16)


def _v(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _dev(t):
    return None if t is None else t.cuda()


def _inputs(rows, cols, seed, residual=True, gates=0, post=False, big=True):
    r = np.random.RandomState(seed)
    x = _t(r, rows, cols)
    if big:
        x[:, r.random_sample(cols) < 0.01] *= 40
    return {"x": x, "weight": _t(r, cols, scale=0.1, add=1.0), "residual": _t(r, rows, cols, scale=2.0) if residual else None,
            "gate": _t(r, gates, cols, scale=0.5) if gates else None, "post_weight": _t(r, cols, scale=0.1, add=1.0) if post else None}


def _check(q, h, d, fmt, alpha=1.0, eps=1e-6):
    rows, cols = d["x"].shape
    hv, n = ref.norm_quantize_parts(_v(d["x"]), _v(d["weight"]), _v(d["residual"]), _v(d["gate"]), _v(d["post_weight"]), alpha, eps)
    # h's error, before its rounding to bf16: relative to its terms.
    terms = np.abs(hv) if d["residual"] is None else np.abs(_v(d["residual"])) + np.abs(hv - _v(d["residual"]))
    eh = REL * terms
    if h is not None:
        assert np.all(np.abs(_v(h) - hv) <= 2.0**-8 * np.abs(hv) + 2 * eh)
    w = 1.0 if d["weight"] is None else np.abs(_v(d["weight"]))
    # n moves with h itself and, through the norm, with all of its row's h.
    rms = np.sqrt((hv * hv).mean(1, keepdims=True) + eps)
    en = eh * w / rms + np.abs(n) * (REL + np.sqrt((eh * eh).mean(1, keepdims=True)) / rms)
    size = 128 if fmt == "fp8_b128" else 32
    nb, eb = n.reshape(rows, -1, size), en.reshape(rows, -1, size)
    lo, hi = (np.abs(nb) - eb).clip(0).max(2), (np.abs(nb) + eb).max(2)
    codes, scales = host(q.codes), host(q.scales)
    if fmt == "fp8_b128":
        assert np.all(scales >= lo / 448 * (1 - 2.0**-23)) and np.all(scales <= np.where(hi == 0, 1, hi / 448 * (1 + 2.0**-23)))
        s, table, got = scales.astype(np.float64), ref.E4M3, codes
    else:
        emax = 6 if fmt == "mxfp4" else 448

        def e8(a):
            with np.errstate(divide="ignore"):
                return np.clip(np.ceil(np.log2(a / emax)) + 127, 0, 254)
        assert np.all(scales >= e8(lo)) and np.all(scales <= e8(hi))
        s = 2.0 ** (scales.astype(np.float64) - 127)
        table, got = (ref.E2M1, np.stack([codes & 15, codes >> 4], -1)) if fmt == "mxfp4" else (ref.E4M3, codes)
    top = 8 if fmt == "mxfp4" else 127

    def rounded(v):
        c, neg = ref.nearest_code(v / s[..., None], table[:top])
        return np.where(neg, -table[c], table[c])
    value = table[got.reshape(nb.shape)]
    assert np.all(value >= rounded(nb - eb)) and np.all(value <= rounded(nb + eb))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "fp8_b128"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (5, 512), (2, 640), (3, 2048), (1, 2176), (4, 4096), (2, 4224), (1, 8192),
                                       (3, 8320), (1, 16384), (2, 16512), (1, 32768)])
def test_shapes(rows, cols, fmt):
    require_gpu()
    d = _inputs(rows, cols, rows + cols)
    q, h = mx.norm_quantize(**{k: _dev(v) for k, v in d.items()}, fmt=fmt)
    _check(q, h, d, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("cols", [32, 96, 544, 2080])
def test_mx_odd_cols(cols, fmt):
    require_gpu()
    d = _inputs(7, cols, cols, big=False)
    q, h = mx.norm_quantize(**{k: _dev(v) for k, v in d.items()}, fmt=fmt)
    _check(q, h, d, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "fp8_b128"])
@pytest.mark.parametrize("residual,gates,post,alpha,eps", [(False, 0, False, 1.0, 1e-6), (True, 1, False, 0.25, 1e-5),
                                                           (True, 3, True, -1.5, 1e-6), (False, 2, True, 1.0, 0.0),
                                                           (True, 0, True, 0.0, 1e-2)])
def test_options(residual, gates, post, alpha, eps, fmt):
    require_gpu()
    d = _inputs(6, 768, 21, residual, gates, post)
    q, h = mx.norm_quantize(**{k: _dev(v) for k, v in d.items()}, fmt=fmt, alpha=alpha, eps=eps)
    assert (h is not None) == residual
    _check(q, h, d, fmt, alpha, eps)


def test_many_rows_and_gates():
    """More rows than workgroups: each takes several, and the gate changes between them."""
    require_gpu()
    for cols, rows in ((128, 9000), (1024, 4200)):
        d = _inputs(rows, cols, 2, gates=300, post=True)
        q, h = mx.norm_quantize(**{k: _dev(v) for k, v in d.items()}, fmt="mxfp8")
        _check(q, h, d, "mxfp8")


def test_weight_none_and_one_gate_row():
    require_gpu()
    d = _inputs(4, 256, 1, gates=1)
    d["weight"] = None
    q, h = mx.norm_quantize(d["x"].cuda(), None, "fp8_b128", residual=d["residual"].cuda(), gate=d["gate"][0].cuda())
    _check(q, h, d, "fp8_b128")


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "fp8_b128"])
def test_zero_tiny_and_nonfinite_rows(fmt):
    """A row of zeros gives zero codes; the smallest values survive; Inf makes its own element's
    block NaN and the rest of the row 0 / inf = 0 codes; NaN makes every block of its row NaN."""
    require_gpu()
    cols = 512
    x = torch.zeros(5, cols, dtype=BF16)
    x[1] = _t(np.random.RandomState(0), cols, scale=2.0**-120)
    x[2] = _t(np.random.RandomState(1), cols)
    x[2, 130] = float("inf")
    x[3] = _t(np.random.RandomState(2), cols)
    x[3, 3] = float("nan")
    x[4] = _t(np.random.RandomState(3), cols)
    q, h = mx.norm_quantize(x.cuda(), torch.ones(cols, dtype=BF16, device="cuda"), fmt, eps=1e-6)
    assert h is None
    size = 128 if fmt == "fp8_b128" else 32
    scales = host(q.scales)
    nan = np.isnan(scales) if fmt == "fp8_b128" else scales == 255
    assert not nan[0].any() and not nan[1].any() and not nan[4].any() and nan[3].all()
    assert nan[2].sum() == 1 and nan[2, 130 // size]
    codes = host(q.codes)
    assert not codes[0].any() and not codes[3].any() and not (codes[2] & (0x77 if fmt == "mxfp4" else 0x7F)).any()
    one = {"x": x[1:2], "weight": None, "residual": None, "gate": None, "post_weight": None}
    q1, _ = mx.norm_quantize(x[1:2].cuda(), None, fmt)
    _check(q1, None, one, fmt)


@pytest.mark.parametrize("where", ["residual", "x", "new"])
def test_strides_and_in_place(where):
    """Rows of wider buffers; h may replace the residual or x."""
    require_gpu()
    d = _inputs(9, 384, 4)
    wide = torch.full((3, 9, 640), 7.0, dtype=BF16, device="cuda")
    x, r, h = wide[0][:, 128:512], wide[1][:, 64:448], wide[2][:, :384]
    x.copy_(d["x"])
    r.copy_(d["residual"])
    out = {"residual": r, "x": x, "new": h}[where]
    q, got = mx.norm_quantize(x, d["weight"].cuda(), "mxfp4", residual=r, out=out)
    assert got is out
    _check(q, got, d, "mxfp4")
    assert bool((wide[0][:, :128] == 7).all()) and bool((wide[1][:, 448:] == 7).all()) and bool((wide[2][:, 384:] == 7).all())


@pytest.mark.parametrize("fmt,cols", [("mxfp4", 1024), ("mxfp8", 640)])
def test_kpanel_is_the_packed_row_layout(fmt, cols):
    require_gpu()
    d = _inputs(37, cols, 8)
    args = {k: _dev(v) for k, v in d.items()}
    q, _ = mx.norm_quantize(**args, fmt=fmt)
    k, _ = mx.norm_quantize(**args, fmt=fmt, layout="kpanel")
    p = mx.pack(q)
    assert k.layout == p.layout
    assert torch.equal(k.codes.flatten(), p.codes.flatten()) and torch.equal(k.scales.flatten(), p.scales.flatten())


def test_captured_and_on_another_stream():
    require_gpu()
    d = {k: _dev(v) for k, v in _inputs(20, 1024, 3, gates=2, post=True).items()}
    x = d["x"].clone()
    args = {**d, "x": x, "fmt": "fp8_b128"}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.norm_quantize(**args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, h = mx.norm_quantize(**args)
    for k in range(3):
        x.copy_(d["x"] * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        q1, h1 = mx.norm_quantize(**{**args, "x": d["x"] * (k + 1)})
        assert torch.equal(q.codes, q1.codes) and torch.equal(q.scales, q1.scales) and torch.equal(h, h1)


@pytest.mark.parametrize("kind", ["fp8", "mxfp4"])
@pytest.mark.parametrize("tokens", [1, 9, 200])
def test_expert_layer(tokens, kind):
    """As they are used together: norm + quantize, the experts' products of the
    tokens sorted by expert, the dense projection after them."""
    require_gpu()
    K, N, G = 512, 256, 5
    act, wt = ("fp8_b128", "fp8_b128x128") if kind == "fp8" else ("mxfp4", "mxfp4")
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    rand = lambda *s, k=1.0: (torch.randn(*s, generator=gen, device="cuda") * k).to(BF16)  # noqa: E731
    w1, w2 = mx.quantize(rand(G, N, K, k=0.05), wt), mx.quantize(rand(K, N, k=0.05), wt)
    x, res = rand(tokens, K), rand(tokens, K)
    expert = torch.randint(0, G, (tokens,), generator=gen, device="cuda")
    order = torch.argsort(expert, stable=True)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(expert, minlength=G).cumsum(0)
    q, h = mx.norm_quantize(x, rand(K, k=0.1) + 1, act, residual=res)
    qs = mx.QTensor(q.fmt, tokens, K, q.codes[order], q.scales[order])
    up = mx.gemm_grouped(qs, w1, offsets)
    qu = mx.quantize(up, act)
    down = mx.gemm(qu, w2, F32)
    # Each stage from the stage before it, in 64 bits.
    val = lambda q: (ref.fp8_values(host(q.codes), host(q.scales), False) if kind == "fp8"  # noqa: E731
                     else ref.mxfp4_values(host(q.codes), host(q.scales)))
    e = host(expert[order])
    wv = (np.stack([ref.fp8_values(c, s, True) for c, s in zip(host(w1.codes).reshape(G, N, K), host(w1.scales))]) if kind == "fp8"
          else ref.mxfp4_values(host(w1.codes), host(w1.scales)).reshape(G, N, K))
    c = np.stack([wv[g] @ row for g, row in zip(e, val(qs))])
    s = np.stack([np.abs(wv[g]) @ np.abs(row) for g, row in zip(e, val(qs))])
    if kind == "fp8":
        check_fp8_gemm(up, c, s, BF16)
    else:
        assert np.all(np.abs(_v(up) - c) <= 2.0**-18 * s * (1 + 2.0**-8) + 2.0**-8 * np.abs(c))
    w2v = ref.fp8_values(host(w2.codes), host(w2.scales), True) if kind == "fp8" else ref.mxfp4_values(host(w2.codes), host(w2.scales))
    check_fp8_gemm(down, *ref.product(val(qu), w2v), F32)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "fp8_b128"])
@pytest.mark.parametrize("power", [-18, -4])
@pytest.mark.parametrize("beside", [False, True])
def test_blocks_of_subnormals(fmt, power, beside):
    """Blocks of n from one fp32 subnormal step (2^-149) up, alone and beside a block of
    normal size: an FP8 scale that would be zero is 1, under one too coarse (few steps of
    2^-149) codes saturate, and nothing becomes NaN. mean(h^2) + eps is 1 or 4 without error,
    so n, its codes and scales are exactly known."""
    require_gpu()
    r = np.random.RandomState(power + 50)
    tops, cols = (1, 2, 3, 100, 127, 200, 225, 255), 2048
    x = np.stack([r.randint(-k, k + 1, cols) * 2.0**-133 for k in tops])
    x[:, 0::128], x[:, 1::128], x[:, 2::128] = np.array(tops)[:, None] * 2.0**-133, 0.0, -0.0
    x[:, 3::32] = -x[:, 0:1]  # (every 32-element block has the row's largest)
    w = np.repeat(2.0 ** (power + np.arange(16)), 128)
    if beside:
        x[:, 256:384], w[256:384] = r.choice([-4.0, 4.0], (len(tops), 128)), 1.0
    x, w = _bf16_exact(x), _bf16_exact(w)
    q, _ = mx.norm_quantize(x.cuda(), w.cuda(), fmt, eps=3.0 if beside else 1.0)
    with np.errstate(under="ignore"):
        h = np.float32(0) + x.float().numpy()  # (no residual: 0, so that -0 becomes 0)
        n = (h * w.float().numpy()) * np.float32(0.5 if beside else 1.0)
    size = 128 if fmt == "fp8_b128" else 32
    nb = n.astype(np.float64).reshape(len(tops), -1, size)
    amax = np.abs(nb).max(2)
    if fmt == "fp8_b128":
        scales = (amax.astype(np.float32) / np.float32(448)).astype(np.float32)
        scales = np.where(scales == 0, np.float32(1), scales)
        s = scales.astype(np.float64)
        if power == -18:  # both kinds are there
            assert (amax[(s == 1) & (amax > 0)] > 0).any() and ((amax / s > 464) & (s < 1)).any()
    else:
        with np.errstate(divide="ignore"):
            scales = np.clip(np.ceil(np.log2(amax / (6 if fmt == "mxfp4" else 448))) + 127, 0, 254).astype(np.uint8)
        s = 2.0 ** (scales.astype(np.float64) - 127)
    table = ref.E2M1[:8] if fmt == "mxfp4" else ref.E4M3[:127]
    code, neg = ref.nearest_code(nb / s[..., None], table)
    want = (code + (8 if fmt == "mxfp4" else 128) * neg).astype(np.uint8).reshape(n.shape)
    got = host(q.codes)
    if fmt == "mxfp4":
        got = np.stack([got & 15, got >> 4], -1).reshape(n.shape)
    assert np.array_equal(host(q.scales), scales)
    assert np.array_equal(got, want)


def _bf16_exact(v):
    t = torch.from_numpy(v.astype(np.float32)).to(BF16)
    assert np.array_equal(_v(t), v)
    return t
