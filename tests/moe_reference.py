"""A mixture-of-experts layer in 64 bits, from its definition, with how far a
result may be from it."""
import math

import torch

U = 2.0**-24


def stack_values(q, mx):
    """float64 [groups][rows][cols] values of a quantized stack, decoded here from its bytes."""
    g, rows, cols = q.groups, q.rows // q.groups, q.cols
    if q.fmt == mx.MX_FMT_INT8:
        return q.codes.view(torch.int8).double().view(g, rows, cols) * q.scales.double().view(g, rows, 1)
    if q.fmt == mx.MX_FMT_FP8_B128X128:
        c = torch.arange(256, device=q.codes.device)
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e == 0, m * 2.0**-9, (8 + m) * torch.exp2(e.double() - 10))
        v = torch.where(c & 127 == 127, float("nan"), torch.where(c >= 128, -v, v))
        s = q.scales.double().view(g, -(-rows // 128), cols // 128).repeat_interleave(128, 1).repeat_interleave(128, 2)
        return v[q.codes.long()].view(g, rows, cols) * s[:, :rows]
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=q.codes.device)
    lut = torch.cat([lut, -lut])
    b = q.codes.long().view(-1)
    v = torch.stack([lut[b & 15], lut[b >> 4]], 1).view(g, rows, cols // 32, 32)
    s = q.scales.view(g, rows, cols // 32, 1).long()
    return (v * torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))).view(g, rows, cols)


def layer(x, ids, weights, up, down, random=True, parts=1):
    """(y, tolerance before the result's own rounding) in 64 bits; up, down: values.
    Errors, u = 2^-24: a product's sums (K / 16 + 12) u of their terms' magnitudes; the
    silu, whose slope is at most 1.1, and the product after it 16 u (1 + |gate|) of h
    (a division, an exponential of a few ulps whose argument may be rounded, two
    products); h's rounding to bf16 2^-8 of it, or 2^-134 among the subnormals; the weighted sum (top + 1) u of its
    terms. With `random` the roundings of h, each within its bound b_i = 2^-8 |h_i d_i| of a
    term and of either sign as likely, add up to at most sqrt(2 ln(2 n / 1e-9) sum of b_i^2), but
    for a probability of 1e-9 that one of n outputs passes it (Hoeffding's inequality); otherwise to
    the sum of the b_i. With h in two `parts`, the nearest bf16 number and what is left of it, in bf16: of h in
    [1, 2) at most 2^-8 is left, exactly, and rounded by at most 2^-17 (below 2^-8 its steps are 2^-16 at most); the
    products are twice as many, and so are the roundings of their sums."""
    T, H = x.shape
    E, I = up.shape[0], down.shape[2]
    x, w = x.double(), weights.double()
    y, tol, size = (torch.zeros(T, H, dtype=torch.float64, device=x.device) for _ in range(3))
    var = torch.zeros_like(y)
    for t, j in ((t, j) for t in range(T) for j in range(ids.shape[1])):
        e = int(ids[t, j])
        if not 0 <= e < E:
            continue
        both, mag = up[e] @ x[t], up[e].abs() @ x[t].abs()
        gate, lin = both[:I], both[I:]
        dg, dl = ((H / 16 + 12) * U * mag).split(I)
        h = gate * torch.sigmoid(gate) * lin
        dh = 1.1 * dg * (lin.abs() + dl) + (gate * torch.sigmoid(gate)).abs() * dl + 16 * U * (1 + gate.abs()) * h.abs() + 2.0**-130
        b = (2.0**-8 if parts == 1 else 2.0**-17) * (h.abs() + dh) + 2.0**-134
        d, aw = down[e].abs(), w[t, j].abs()
        out = down[e] @ h
        y[t] += w[t, j] * out
        tol[t] += aw * (d @ dh + (parts * I / 16 + 12) * U * (d @ (h.abs() + dh + b)))
        if random:
            var[t] += aw**2 * ((d * d) @ (b * b))
        else:
            tol[t] += aw * (d @ b)
        size[t] += aw * (out.abs() + d @ (dh + b))
    tol += (ids.shape[1] + 1) * U * size
    return y, tol + torch.sqrt(2 * math.log(2 * y.numel() / 1e-9) * var)


def check(got, y, tol, out):
    assert got.dtype == out and got.shape == y.shape
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan)
    if out == torch.bfloat16:
        tol = tol * (1 + 2.0**-8) + 2.0**-8 * y.abs() + 2.0**-134
    worst = ((got.double() - y).abs() - tol)[~nan]
    assert worst.numel() == 0 or worst.max() <= 0, (worst.max(), tol.max())
