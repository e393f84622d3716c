"""64-bit references and bounds for what a dense layer does around its
products: the norm, products with bias, activation and residual, 8-bit values
with scales, and the gradients.

Bounds, fixed before the first run. An FP32 sum is off by at most 1e-5 of the
sum of magnitudes (routed_ref.REL). A rounding is off by half a step: 2^-11 of
an FP16 value (2^-25 below the smallest normal), 2^-24 of an FP32 value, 2^-4 of
an E4M3 and 2^-3 of an E5M2 code (2^-10 and 2^-17 below the smallest normal
code). An activation of z in FP32 is a product of z and a factor in [0, 1] that
comes from one exponential, whose argument's rounding adds its size times 2^-24
(|z| and z^2 / 2 at most, with the cubic of the tanh form 2 |z|^3 where the
factor is not 0 or 1), and either from a reciprocal and, for GELU, a fitted
polynomial of 2.7e-7 or less (FP32 results, derivatives) or, for GELU into FP16 and
FP8, from a polynomial in the exponent, off by 1.4e-6 of the factor up to |z| = 3 and
5.2e-6 up to 7: off by at most 2^-19 (1 + z^2) of the value, and 2^-33 |z| where the
factor is below that polynomial's range. A derivative is that factor and z times its slope: off by at
most 2^-19 (1 + |z| + z^2) absolutely, the slope being at most 1.13."""
import math

import torch

from routed_ref import REL, half_step_f16

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF_CODE = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}
STEEPEST = 1.13


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def act_error(z, name):
    """How far FP32 may be from act(z)."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    return act(z, name).abs() * 2.0 ** -19 * (1 + z * z) + z.abs() * 2.0 ** -33


def slope_error(z, name):
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    return 2.0 ** -19 * (1 + z.abs() + z * z)


def stored(v, dtype):
    """Half a step of a stored value."""
    return half_step_f16(v) if dtype == torch.float16 else v.abs() * 2.0 ** -24 + 2.0 ** -149


def code_step(v, scale, fmt):
    """Half a step of v held as a code times scale."""
    rel, least = HALF_CODE[fmt]
    return torch.maximum(v.abs() * rel, scale * least)


def spread(scale, cols):
    """Scales of blocks of 32 values for every column."""
    return scale.repeat_interleave(32, dim=1)[:, :cols]


def powers(scale):
    """2^(e - 127) of scale bytes e, exactly (exp2 is not), NaN for 255."""
    return scale.view(torch.uint8).view(torch.float8_e8m0fnu).double()


def mx_scale(amax, fmt):
    """The least power of two with amax / scale <= the format's largest, 1 for 0 (64-bit)."""
    m = torch.where(amax > 0, amax, torch.full_like(amax, FP8_MAX[fmt]))
    f, e = torch.frexp(m)
    p = e - {"e4m3": 9, "e5m2": 16}[fmt] + (f > 0.875)
    return powers((p.clamp(min=-127) + 127).to(torch.uint8))


def mx_pack(x, fmt, half=False):
    """(codes as values, scales) of x in 64 bits."""
    rows, cols = x.shape
    x = x.double()
    if half:
        top = {"e4m3": 61440.0, "e5m2": 57344.0}[fmt]
        x = torch.where(x.isfinite(), x.clamp(-top, top), x)
    fin = torch.where(x.isfinite(), x, torch.zeros_like(x))
    blocks = torch.nn.functional.pad(fin, (0, -cols % 32)).reshape(rows, -1, 32)
    s = mx_scale(blocks.abs().amax(dim=2), fmt)
    u = x / spread(s, cols)
    return u, s


def codes_of(u, fmt):
    """FP8 codes of 64-bit values in range: nearest even (through FP32, which holds a code's ties exactly)."""
    return u.float().to(CODE[fmt])


def as_bytes(t):
    return t.view(torch.uint8)


def scale_bytes(s):
    return (torch.log2(s).round() + 127).to(torch.uint8)


def values(q, scale, fmt):
    """What codes and scale bytes stand for, 64 bits."""
    s = powers(scale)
    return q.view(torch.uint8).view(CODE[fmt]).double() * spread(s, q.shape[1])


def norm(h, w, eps):
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + eps)
    return h * rstd[:, None] * w, rstd


def norm_backward(dy, h, w, rstd, dh):
    """(dx, dweight, sums of magnitudes of both)."""
    n, g = h * rstd[:, None], dy * w
    gn = g * n
    dx = rstd[:, None] * (g - n * gn.mean(dim=1, keepdim=True))
    mag = rstd[:, None] * (g.abs() + n.abs() * gn.abs().mean(dim=1, keepdim=True))
    if dh is not None:
        dx, mag = dx + dh, mag + dh.abs()
    return dx, (dy * n).sum(dim=0), mag, (dy * n).abs().sum(dim=0)
