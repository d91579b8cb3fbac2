"""Rotary positions and paged appending by their definitions, in 64 bits, and
the bound their outputs have to keep."""
import math

import torch

# half a step of the type, relative to the value, and the smallest absolute half step
HALF_STEP = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 0.0)}


def rotate(x, positions, inv_freq, interleaved=False, mscale=1.0):
    """float64 rotation of x [T, H, d] (CPU), pair by pair."""
    r = 2 * inv_freq.numel()
    y = x.double().clone()
    angle = positions.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = mscale * angle.cos(), mscale * angle.sin()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = cos[:, i, None], sin[:, i, None]
        xa, xb = x[:, :, a].double(), x[:, :, b].double()
        y[:, :, a] = xa * c - xb * s
        y[:, :, b] = xb * c + xa * s
    return y


def bound(x, want, inv_freq, interleaved, mscale):
    """Largest error of a rotated tensor: one rounding to its type, and fp32 inside.

    The angle's remainder is rounded to fp32 in turns (2^-25 turn = 1.9e-7 rad), cos
    and sin are a few ulp off (2.4e-7), and the two products and the sum round three
    times at 2^-24 (1.8e-7): each of the pair's inputs carries at most 6.1e-7 of its
    size; 8e-7 is allowed.  Copied elements are exact."""
    r = 2 * inv_freq.numel()
    half, least = HALF_STEP[x.dtype]
    x64 = x.double().abs()
    inside = torch.zeros_like(x64)
    if interleaved:
        size = x64[..., 0:r:2] + x64[..., 1:r:2]
        inside[..., 0:r:2] = size
        inside[..., 1:r:2] = size
    else:
        size = x64[..., :r // 2] + x64[..., r // 2:r]
        inside[..., :r // 2] = size
        inside[..., r // 2:r] = size
    inside *= abs(mscale) * 8e-7
    out = inside + half * (want.abs() + inside) + least
    out[..., r:] = 0.0
    return out


def assert_rotated(got, x, positions, inv_freq, interleaved=False, mscale=1.0):
    x, got = x.cpu(), got.cpu()
    want = rotate(x, positions.cpu(), inv_freq.cpu(), interleaved, mscale)
    excess = (got.double() - want).abs() - bound(x, want, inv_freq.cpu(), interleaved, mscale)
    assert got.shape == x.shape and got.dtype == x.dtype
    assert excess.max() <= 0, f"off by {float(excess.max())} over the bound"


def frequencies(rotary, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rotary) for i in range(rotary // 2)],
                        dtype=torch.float64)


def turns_of_table(inv_freq, length):
    return length * inv_freq / (2.0 * math.pi)
