"""Plain forms of the int8 path, with bounds on what the library's results may
differ from them (see expert_reference.py for the manner)."""
import torch

import expert_reference as R

HALF = 2.0 ** -24  # half a unit in the last place of fp32, relative


def quantise(v):
    """Scales and codes of each row (last axis): fp32 s = amax/127 and RNE(v/s); an all-zero row
    has zeros, one with an infinity or a NaN has that as its scale and zero codes."""
    v = v.float()
    amax = v.abs().amax(-1)  # a NaN wins
    # (a quotient of tensors: by a number, torch multiplies by the rounded reciprocal)
    s = torch.where(amax.isfinite(), amax / torch.full_like(amax, 127.0), amax)
    fine = (amax.isfinite() & (s > 0))[..., None]
    q = torch.where(fine, v / torch.where(fine, s[..., None], 1.0), 0.0)
    return torch.round(q).to(torch.int8), s


def dequantise(codes, scale):
    return codes.double() * scale.double()[..., None]


def rows_times(a, a_scale, w, w_scale, counts):
    """Products of codes and then the scales, with their bound: the sums are exact in fp32 while
    the magnitudes of their products stay below 2^24 together (whatever the order), else within
    K 2^-23 of those; two multiplications by scales round."""
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device=a.device)
    err = torch.zeros_like(out)
    for e, lo, hi in R.segments(counts):
        x, m = a[lo:hi].double(), w[e].double().T
        scale = a_scale[lo:hi, None].double().abs() * w_scale[e][None, :].double().abs()
        whole, size = x @ m, x.abs() @ m.abs()
        out[lo:hi] = whole * a_scale[lo:hi, None].double() * w_scale[e][None, :].double()
        off = torch.where(size < 2.0 ** 24, torch.zeros_like(size),
                          size * (a.shape[1] + 8) * 2.0 ** -23)
        err[lo:hi] = (off + (whole.abs() + off) * 2.02 * HALF) * scale
    return out, err + R.TINY


def gated(a, a_scale, w, w_scale, counts):
    """h before its quantisation, and its bound."""
    F = w.shape[1] // 2
    both, err = rows_times(a, a_scale, w, w_scale, counts)
    return R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])


def check_quantised(codes, scale, value, err):
    """Codes and scales of rows known to within err: s is amax/127 to within the largest error and
    a rounding, and a value is within half a step of its code (and the quotient's rounding)."""
    amax, e_max = value.abs().amax(1), err.amax(1)
    R.check("scale", scale, amax / 127, (e_max + amax * 2 * HALF) / 127 + 2.0 ** -149)
    step = scale.double()[:, None]
    R.check("codes", dequantise(codes, scale), value, err + step * (0.5 + 127 * 2 * HALF))
    full = codes.int().abs().amax(1)
    assert ((full == 127) | (scale == 0)).all() and (codes != -128).all()
