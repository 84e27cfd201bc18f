"""Plain 64-bit forms of the 8-bit integer format (a scale per row) and its
products, from their definitions."""
import numpy as np
import torch


def quantize(x):
    """Codes (int8) and fp32 scales of float64 [rows][cols] holding bf16 values."""
    with np.errstate(invalid="ignore"):
        amax = np.abs(x).max(1)
        bad = ~np.isfinite(amax)
        s = (np.where(bad, 0, amax).astype(np.float32) / np.float32(127)).astype(np.float32)
        s = np.where(s == 0, np.float32(1), s)
        # |x / s| in 64 bits tells a quotient next to a border from one on it (they are
        # at least 2^-33 apart: x has 8 significant bits, s 24, the border 9).
        q = np.rint(np.where(bad[:, None], 0.0, x) / s[:, None].astype(np.float64))
    assert np.abs(q).max() <= 127
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s)


def sums(a, b):
    """Exact sums of products of int8 codes [M][K], [N][K], on their device (float64
    holds them: K 2^14 < 2^53)."""
    return a.view(torch.int8).double() @ b.view(torch.int8).double().T


def product(a, sa, b, sb):
    """C of device codes and scales in 64 bits."""
    return sums(a, b) * sa.double()[:, None] * sb.double()[None, :]


def tolerance(c, out):
    """The sum's conversion to fp32, the product of the scales' significands and the result
    round once each, by half a step (2^-24), and again below 2^-126 by at most
    2^-150; a bf16 result then by half a step of its own (2^-8; below 2^-126 by 2^-134)."""
    t = 3.01 * 2.0**-24 * c.abs() + 2.0**-149
    if out == torch.float32:
        return t
    return t * (1 + 2.0**-8) + 2.0**-8 * c.abs() + 2.0**-134


def check(got, c, out):
    assert got.dtype == out and got.shape == c.shape
    nan = torch.isnan(c)
    assert torch.equal(torch.isnan(got), nan)
    worst = ((got.double() - c).abs() - tolerance(c, out))[~nan]
    assert worst.numel() == 0 or worst.max() <= 0, worst.max()
