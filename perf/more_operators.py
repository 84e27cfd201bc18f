"""Operators of a quantized language model's linear layers, second part: the cases
they are measured on, their inputs, and their plain forms.

  quantize  bf16 to 8-bit integers with an fp32 scale per row: a token of the
            activations, an output channel of a weight
  gemm      the product over those codes and scales, C = A B^T
  grouped   the same product by expert: rows of A sorted by expert, ragged and
            possibly empty groups, one weight per expert
  moe       a whole mixture-of-experts layer for a few tokens: each token through
            the experts a router chose for it, y = sum of w down(silu(gate x) up x)

`own` false: elementary torch operations in 32 bits (64 next to a rounding
border); true: the library's calls.
"""
import math

import numpy as np
import torch

own = False

INT8_MAX = 127.0
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # a decode step's activations, 16 sequences
        {"name": "quant_act_step", "op": "quantize", "rows": 16, "cols": 8192},
        # a decode MLP weight, once when the model is loaded or updated
        {"name": "quant_weights", "op": "quantize", "rows": 28672, "cols": 8192},
        # one decode step of 16 sequences against that weight: bound by the weight's bytes
        {"name": "gemm_decode", "op": "gemm", "M": 16, "N": 28672, "K": 8192, "out": "bf16"},
        # a short prompt against a narrow projection, odd sizes, fp32 result
        {"name": "gemm_ragged_f32", "op": "gemm", "M": 777, "N": 2000, "K": 2448, "out": "f32"},
        # a long prompt (rows not a multiple of a tile): bound by the matrix cores
        {"name": "gemm_prefill", "op": "gemm", "M": 6000, "N": 8192, "K": 8192, "out": "bf16"},
        # a decode step of 32 sequences, 4 experts each, 64 experts
        {"name": "grouped_step", "op": "grouped", "M": 128, "G": 64, "N": 2048, "K": 4096, "out": "bf16"},
        # long prompts through 16 experts
        {"name": "grouped_prefill", "op": "grouped", "M": 8192, "G": 16, "N": 4096, "K": 4096, "out": "bf16"},
        # one token, 8 of 32 experts
        {"name": "moe_token_mxfp4", "op": "moe", "fmt": "mxfp4", "T": 1, "E": 32, "top": 8, "H": 4096, "I": 2048},
        # a decode step of 4 sequences through many small experts
        {"name": "moe_step_fp8", "op": "moe", "fmt": "fp8", "T": 4, "E": 64, "top": 6, "H": 2048, "I": 1408},
        # 17 sequences, few experts (some with more rows than a matrix instruction has), odd sizes
        {"name": "moe_ragged_mxfp4", "op": "moe", "fmt": "mxfp4", "T": 17, "E": 5, "top": 2, "H": 2880, "I": 1440},
        # a decode step of 32 sequences, 4 experts each, 64 experts
        {"name": "moe_batch_int8", "op": "moe", "fmt": "int8", "T": 32, "E": 64, "top": 4, "H": 4096, "I": 2048},
        # the most tokens that count as a few, nearly every expert busy
        {"name": "moe_full_mxfp4", "op": "moe", "fmt": "mxfp4", "T": 64, "E": 64, "top": 8, "H": 4096, "I": 2048},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "grouped", "moe", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16000), "cols": 16 * _log(rng, 8, 896)}
    if op == "moe":
        fmt = rng.choice(["mxfp4", "fp8", "int8"])
        step = {"mxfp4": 32, "fp8": 128, "int8": 16}[fmt]
        E = _log(rng, 2, 128)
        H, I = step * _log(rng, 512 // step, 5120 // step), step * _log(rng, 256 // step, 2048 // step)
        return {"op": op, "fmt": fmt, "T": _log(rng, 1, 64), "E": max(2, min(E, (3 << 28) // (H * I))),
                "top": min(E, rng.choice([1, 2, 4, 6, 8]), max(2, min(E, (3 << 28) // (H * I)))), "H": H, "I": I}
    out = "f32" if rng.random() < 0.25 else "bf16"
    M, N = _log(rng, 1, 8192), _log(rng, 256, 8192)
    if op == "gemm":
        return {"op": op, "M": M, "N": N, "K": 16 * _log(rng, 32, 512), "out": out}
    K = 16 * _log(rng, 32, 256)
    return {"op": op, "M": M, "G": max(1, min(_log(rng, 2, 64), (1 << 29) // (N * K))), "N": N, "K": K, "out": out}


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 2 * n}
    if op == "moe":
        T, E, top, H, I = (case[k] for k in ("T", "E", "top", "H", "I"))
        used = E * (1 - (1 - top / E) ** T)  # experts that a token chose, on average
        per = {"mxfp4": 0.5 + 1 / 32, "fp8": 1 + 4 / 128 / 128, "int8": 1}[case["fmt"]]
        scales = 4 * (2 * I + H) if case["fmt"] == "int8" else 0
        return {"bytes": used * (3 * H * I * per + scales) + 2 * T * H * 2 + 8 * T * top, "flops": 2 * T * top * 3 * H * I}
    M, N, K = case["M"], case["N"], case["K"]
    c = M * N * (4 if case["out"] == "f32" else 2)
    used = min(case["G"], M) if op == "grouped" else 1
    offsets = 4 * (case["G"] + 1) if op == "grouped" else 0
    return {"bytes": M * (K + 4) + used * N * (K + 4) + c + offsets, "flops": 2 * M * N * K}


# ---- inputs ------------------------------------------------------------------
def _randn(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(gen, rows, cols):
    """Normal values with one channel in 200 forty times as large, as hidden
    states have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32)
    big = torch.rand(cols, generator=gen, device="cuda") < 0.005
    return (x * torch.where(big, 40.0, 1.0)).to(torch.bfloat16)


def _as_int8(x):
    """Codes (int8 in uint8) and fp32 scales of rows."""
    v = x.float()
    s = v.abs().amax(-1) / INT8_MAX
    s = torch.where(s == 0, 1.0, s)
    return torch.round(v / s[..., None]).to(torch.int8).view(torch.uint8), s


def _as_fp8_tiles(w):
    """Codes and fp32 scales of 128 x 128 tiles of a [N, K] weight."""
    n, k = w.shape
    pad = torch.nn.functional.pad(w, (0, 0, 0, -n % 128)).float().view(-1, 128, k // 128, 128)
    s = pad.abs().amax((1, 3)) / E4M3_MAX
    s = torch.where(s == 0, 1.0, s)
    codes = (pad / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, k)
    return codes[:n], s


def _as_mxfp4(x):
    """Codes (two per byte) and E8M0 scales of 32-element blocks of a [rows, K] matrix."""
    v = x.float().view(x.shape[0], -1, 32)
    amax = v.abs().amax(2)
    m, e = torch.frexp(amax / 6.0)  # 2^(e-1) <= amax / 6 < 2^e
    e = torch.where(m == 0.5, e - 1, e)
    e8 = torch.where(amax == 0, 0, (e + 127).clamp(0, 254))
    q = v * torch.exp2((127 - e8).double()).float()[..., None]
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(q.abs(), border, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    c = c.view(x.shape[0], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), e8.to(torch.uint8)


def _stack(gen, fmt, E, rows, cols):
    """Codes and scales of E weights, one at a time."""
    form = {"mxfp4": _as_mxfp4, "fp8": _as_fp8_tiles, "int8": _as_int8}[fmt]
    parts = [form(_randn(gen, rows, cols, scale=0.02)) for _ in range(E)]
    return torch.stack([c for c, _ in parts]), torch.stack([s for _, s in parts])


def _group_sizes(case, seed):
    """Rows per expert: a skewed router's choice. One token's experts are all different."""
    r = np.random.RandomState(seed % (2**32))
    M, G = case["M"], case["G"]
    if M <= G:
        sizes = np.zeros(G, np.int64)
        sizes[r.permutation(G)[:M]] = 1
        return sizes
    return r.multinomial(M, r.dirichlet(np.full(G, 2.0)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(gen, rows, cols)
        return s
    if op == "moe":
        T, E, top, H, I = (case[k] for k in ("T", "E", "top", "H", "I"))
        s["x"] = _activations(gen, T, H)
        # a router's choice: its probabilities, the largest `top` of each token, made to sum to 1
        logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
        p, ids = torch.topk(torch.softmax(logits, 1), top, dim=1)
        s["weights"], s["ids"] = (p / p.sum(1, keepdim=True)).contiguous(), ids.to(torch.int32).contiguous()
        s["used"] = torch.unique(ids).tolist()  # the plain form's: experts that a token chose
        s["up"] = _stack(gen, case["fmt"], E, 2 * I, H)
        s["down"] = _stack(gen, case["fmt"], E, H, I)
        return s
    M, N, K, G = case["M"], case["N"], case["K"], case.get("G", 1)
    s["a"], s["a_scales"] = _as_int8(_activations(gen, M, K))
    s["b"], s["b_scales"] = _stack(gen, "int8", G, N, K)
    if op == "grouped":
        sizes = _group_sizes(case, seed)
        used = np.flatnonzero(sizes)
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        s["used"] = torch.from_numpy(used).cuda()  # the plain form's: experts with rows, the longest group
        s["longest"] = int(sizes.max())
    else:
        s["b"], s["b_scales"] = s["b"][0], s["b_scales"][0]
    return s


# ---- plain forms -------------------------------------------------------------
def _plain_quantize(x):
    v = x.float()
    amax = v.abs().amax(1)
    s = amax / torch.full_like(amax, INT8_MAX)  # a quotient: a number would become a product with its inverse
    s = torch.where(s == 0, 1.0, s)
    q = torch.round(v.double() / s.double()[:, None]).clamp(-INT8_MAX, INT8_MAX)
    return q.to(torch.int8), s


def _mxfp4_values(codes, scales):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).view(*scales.shape, 32)
    return (v * torch.exp2(scales.double() - 127).float()[..., None]).flatten(-2)


def _int8_values(codes, scales):
    return codes.view(torch.int8).float() * scales[..., None]


def _fp8_values(codes, scales):
    s = scales.repeat_interleave(128, -1).repeat_interleave(128, -2)[..., : codes.shape[-2], :]
    return codes.view(torch.float8_e4m3fn).float() * s


def _plain_grouped(s):
    case = s["case"]
    a = _int8_values(s["a"], s["a_scales"])
    b = _int8_values(s["b"][s["used"]], s["b_scales"][s["used"]])
    row = torch.arange(case["M"], device=a.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    slot = torch.searchsorted(s["used"], expert)  # the expert's place among those with rows
    place = row - s["offsets"].long()[expert]
    padded = torch.zeros(b.shape[0], s["longest"], case["K"], device=a.device)
    padded[slot, place] = a
    return torch.bmm(padded, b.transpose(1, 2).contiguous())[slot, place]


def _plain_moe(s):
    """Expert by expert, all tokens through each under the weight that they give it (0: none)."""
    case = s["case"]
    values = {"mxfp4": _mxfp4_values, "fp8": _fp8_values, "int8": _int8_values}[case["fmt"]]
    x, I = s["x"].float(), case["I"]
    share = torch.zeros(case["T"], case["E"], device=x.device).scatter_add_(1, s["ids"].long(), s["weights"])
    y = torch.zeros_like(x)
    for e in s["used"]:
        both = x @ values(s["up"][0][e], s["up"][1][e]).T
        gate, up = both[:, :I], both[:, I:]
        h = gate / (1 + torch.exp(-gate)) * up
        y += share[:, e, None] * (h @ values(s["down"][0][e], s["down"][1][e]).T)
    return y.bfloat16()


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        q, sc = _plain_quantize(s["x"])
        return {"codes": q, "scales": sc}
    if op == "moe":
        return _plain_moe(s)
    if op == "gemm":
        c = _int8_values(s["a"], s["a_scales"]) @ _int8_values(s["b"], s["b_scales"]).T
    else:
        c = _plain_grouped(s)
    return c if case["out"] == "f32" else c.bfloat16()


# ---- the library's calls -----------------------------------------------------
def _run_own(s):
    import microscaling_precision_quantization_amd as mx

    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        q = mx.quantize(s["x"], "int8")
        return {"codes": q.codes.view(torch.int8), "scales": q.scales}
    if op == "moe":
        fmt = {"mxfp4": mx.MX_FMT_MXFP4, "fp8": mx.MX_FMT_FP8_B128X128, "int8": mx.MX_FMT_INT8}[case["fmt"]]
        E, H, I = case["E"], case["H"], case["I"]
        up = mx.QTensor(fmt, E * 2 * I, H, *s["up"], groups=E)
        down = mx.QTensor(fmt, E * H, I, *s["down"], groups=E)
        return mx.moe(s["x"], s["ids"], s["weights"], up, down)
    M, N, K = case["M"], case["N"], case["K"]
    out = torch.float32 if case["out"] == "f32" else torch.bfloat16
    G = case.get("G", 1)
    a = mx.QTensor(mx.MX_FMT_INT8, M, K, s["a"], s["a_scales"])
    b = mx.QTensor(mx.MX_FMT_INT8, G * N, K, s["b"], s["b_scales"], groups=G)
    return mx.gemm(a, b, out) if op == "gemm" else mx.gemm_grouped(a, b, s["offsets"], out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- from the definitions, in 64 bits ----------------------------------------
def _exact_values(fmt, codes, scales):
    """float64 values of one [rows][...] weight."""
    if fmt == "int8":
        c = codes.long()
        return torch.where(c > 127, c - 256, c).double() * scales.double().reshape(-1, 1)
    if fmt == "fp8":
        c = np.arange(256)
        e, m = (c >> 3) & 15, c & 7
        v = np.where(e == 0, m * 2.0**-9, (8 + m) * 2.0 ** (e - 10.0))
        table = torch.from_numpy(np.where(c & 128, -v, v)).cuda()
        at = torch.arange(codes.shape[0], device="cuda") // 128
        return table[codes.long()] * scales.double()[at][:, torch.arange(codes.shape[1], device="cuda") // 128]
    K = 2 * codes.shape[1]
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    nib = torch.stack((codes % 16, codes // 16), 2).reshape(codes.shape[0], K).long()
    power = torch.exp2(scales.double() - 127)[:, torch.arange(K, device="cuda") // 32]
    return torch.where(nib > 7, -1.0, 1.0) * mag[nib % 8] * power


def _exact_quantize(x):
    v = x.double()
    amax = v.abs().max(1, keepdim=True).values
    s = torch.where(amax == 0, 1.0, amax / INT8_MAX).float()  # the scale is the fp32 value
    a = v.abs() / s.double()
    low = torch.floor(a)
    up = (a - low > 0.5) | ((a - low == 0.5) & (low % 2 == 1))
    q = torch.minimum(low + up, torch.full_like(low, INT8_MAX))
    return torch.where(v < 0, -q, q).to(torch.int8), s[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        parts = [_exact_quantize(p) for p in s["x"].split(8192)]
        return {"codes": torch.cat([c for c, _ in parts]), "scales": torch.cat([v for _, v in parts])}
    if op == "moe":
        x, I = s["x"].double(), case["I"]
        y = torch.zeros_like(x)
        for e in torch.unique(s["ids"]).tolist():
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            both = x[t] @ _exact_values(case["fmt"], s["up"][0][e], s["up"][1][e]).T
            h = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
            out = h @ _exact_values(case["fmt"], s["down"][0][e], s["down"][1][e]).T
            y.index_add_(0, t, out * s["weights"].double()[t, j, None])
        return y
    if op == "gemm":
        return _exact_values("int8", s["a"], s["a_scales"]) @ _exact_values("int8", s["b"], s["b_scales"]).T
    off = s["offsets"].tolist()
    c = torch.zeros(case["M"], case["N"], device="cuda", dtype=torch.float64)
    for g in range(case["G"]):
        lo, hi = off[g], off[g + 1]
        if lo < hi:
            a = _exact_values("int8", s["a"][lo:hi], s["a_scales"][lo:hi])
            c[lo:hi] = a @ _exact_values("int8", s["b"][g], s["b_scales"][g]).T
    return c
