"""What the 8-bit operators compute, in 64 bits and written apart from the library, and how far its
arithmetic may be off."""
import math

import torch

TOP, LEAST = 448.0, 2.0 ** -100
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24  # half a step, relative


def e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, and half of its step there."""
    e = torch.frexp(x).exponent.clamp(min=-5).double()  # |x| in [2^(e-1), 2^e), or subnormal
    step = torch.exp2(e - 4)
    return (torch.round(x / step) * step).clamp(-TOP, TOP), step / 2


def norm(x, weight, eps, residual=None):
    """(y, h) of rows."""
    h = x.double() if residual is None else x.double() + residual.double()
    return weight.double() * h / torch.sqrt(h.square().mean(1, keepdim=True) + eps), h


def check_rows8(codes, scale, y, rel):
    """Codes and scales of rows y (fp64) that the library knows to `rel` of themselves: the scale is as
    near as that, and a code times its scale is within half a step of y and what y and the scale are off."""
    want = (y.abs().amax(1) / TOP).clamp(min=LEAST)
    assert ((scale.double() - want).abs() <= (rel + HALF_F32) * want).all()
    q, s = codes.double(), scale.double()[:, None]
    _, half = e4m3(y / s)
    # a value near a border of two steps' ranges may round by the wider one
    assert ((q * s - y).abs() <= half * s * (1 + 2.0 ** -18) + 4 * rel * y.abs()).all()


def activation(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def linear(w, x, bias, act, residual, w_scale, x_scale, out_dtype):
    """(y, tol).  tol, from the library's arithmetic:
      sums        K products, exact in fp32 but for their sum: each addition off by at most 2^-23 of the sum
                  of magnitudes A (accumulation that truncates), and as much for each of up to 16 partial
                  sums: (K + 16) 2^-23 A
      scales      two products and the bias: 3 x 2^-24 of |z| + |bias|
      activation  its slope is at most 1.13 (silu 1.1, gelu 1.13); the exponential, the quotient and erf are
                  good to 2^-19 of the result's operands
      swiglu      the errors of both factors
      residual    one rounding, the output one more: 2^-24, and half a step of the output's type"""
    K = x.shape[1]
    xd, wd = x.double(), w.double()
    if w_scale is not None:
        xd, wd = xd * x_scale.double()[:, None], wd * w_scale.double()[:, None]
    z, size = xd @ wd.T, xd.abs() @ wd.abs().T
    d = (K + 16) * 2.0 ** -23 * size
    if bias is not None:
        z = z + bias.double()
    d = d + 3 * HALF_F32 * (z.abs() + (0 if bias is None else bias.double().abs()))
    if act == "swiglu":
        (g, u), (dg, du) = z.chunk(2, 1), d.chunk(2, 1)
        a = activation(g, "silu")
        da = 1.13 * dg + 2.0 ** -19 * g.abs()
        y, d = a * u, da * u.abs() + (a.abs() + da) * du
    elif act in ("silu", "gelu"):
        y, d = activation(z, act), 1.13 * d + 2.0 ** -19 * z.abs()
    else:
        y = z
    if residual is not None:
        y = y + residual.double()
    half = HALF_BF16 if out_dtype is torch.bfloat16 else HALF_F32
    return y, (d + HALF_F32 * y.abs()) * (1 + half) + half * y.abs() + 1e-37


def turned(x, pos, theta):
    """x [..., n, heads, D] turned at pos [..., n], fp64, and the magnitudes that its rounding errors go by."""
    D = x.shape[-1]
    f = torch.tensor([math.pow(theta, -2.0 * j / D) for j in range(D // 2)], dtype=torch.float64, device=x.device)
    ang = pos.double()[..., None, None] * f
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
    size = (a.abs() + b.abs()).repeat_interleave(1, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)
