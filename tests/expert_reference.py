"""Plain 64-bit forms of the expert operators, with bounds on what fp32 sums
and the final roundings may differ from them.

Every function returns (value, bound): a kernel's result r must satisfy
|r - value| <= bound element by element. The bounds follow from the formats:
bf16 (8 significant bits) rounds to within 2^-8 of a value; a sum of n products in fp32, in any
order and with truncating additions, is within n * 2^-23 of the sum of the
products' magnitudes.
"""
import torch

BF16 = 2.0 ** -8  # half a unit in the last of 8 significant bits, relative
TINY = 2.0 ** -126


def segments(counts):
    lo = 0
    for e, n in enumerate(counts):
        yield e, lo, lo + n
        lo += n


def dequant_rows(codes, scale):
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    return v * scale.double().repeat_interleave(128, dim=-1)


def dequant_weights(codes, scale):
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    return v * scale.double().repeat_interleave(128, dim=-1).repeat_interleave(128, dim=-2)


def rows_times(a, w, counts, transpose=True, a_err=None):
    """a_r w[e]^T (or a_r w[e]) for each row; a_err: elementwise error of a."""
    n = w.shape[1] if transpose else w.shape[2]
    out = torch.zeros(a.shape[0], n, dtype=torch.float64, device=a.device)
    err = torch.zeros_like(out)
    K = a.shape[1]
    for e, lo, hi in segments(counts):
        m = w[e].T if transpose else w[e]
        out[lo:hi] = a[lo:hi] @ m
        err[lo:hi] = (a[lo:hi].abs() @ m.abs()) * (K + 8) * 2.0 ** -23
        if a_err is not None:
            err[lo:hi] += a_err[lo:hi] @ m.abs()
    return out, err + TINY


def outer(a, b, counts, a_err=None):
    E = len(counts)
    out = torch.zeros(E, a.shape[1], b.shape[1], dtype=torch.float64, device=a.device)
    err = torch.zeros_like(out)
    for e, lo, hi in segments(counts):
        out[e] = a[lo:hi].T @ b[lo:hi]
        err[e] = (a[lo:hi].abs().T @ b[lo:hi].abs()) * (hi - lo + 8) * 2.0 ** -23
        if a_err is not None:
            err[e] += a_err[lo:hi].T @ b[lo:hi].abs()
    return out, err


def silu_product(g, u, g_err, u_err):
    """silu(g) u. |silu'| <= 1.1; the kernel's exponential and quotient are
    within 2^-20 of the value (2 ulp each, and the rounding of g log2 e in an
    argument of magnitude below 32; past that both sides are below 2^-40)."""
    s = torch.sigmoid(g)
    h = g * s * u
    err = 1.1 * g_err * (u.abs() + u_err) + (g * s).abs() * u_err + 2.0 ** -18 * h.abs() \
        + 2.0 ** -38 * u.abs()
    return h, err


def bf16_out(value, err):
    return value, err + BF16 * (value.abs() + err) + TINY


def backward(x, gu, hid, dy, w13, w2, counts):
    """dx, dw13, dw2 from the inputs in 64 bits, each with its bound; dg and du
    are rounded to bf16 on the way."""
    F = hid.shape[1]
    dh, dh_err = rows_times(dy, w2, counts, transpose=False)
    g, u = gu[:, :F], gu[:, F:]
    s = torch.sigmoid(g)
    dsilu = s * (1 + g * (1 - s))
    dgu = torch.cat([dh * u * dsilu, dh * g * s], 1)
    # (1 + g (1 - s)) cancels: its error is absolute, about |g| 2^-20
    part = torch.cat([u.abs() * (dsilu.abs() + 2.0 ** -18 * s * (1 + g.abs())), (g * s).abs()], 1)
    dh2, e2 = torch.cat([dh, dh], 1).abs(), torch.cat([dh_err, dh_err], 1)
    d_err = e2 * part * 1.01 + dh2 * part * 2.0 ** -18 \
        + dh2 * torch.cat([u.abs() * 2.0 ** -18 * (1 + g.abs()), 2.0 ** -38 * g.abs()], 1)
    d_err = d_err + BF16 * (dgu.abs() + d_err) + TINY
    dx = rows_times(dgu, w13, counts, transpose=False, a_err=d_err)
    dw13 = outer(dgu, x, counts, a_err=d_err)
    dw2 = outer(dy, hid, counts)
    return bf16_out(*dx), bf16_out(*dw13), bf16_out(*dw2)


def check(name, got, value, bound):
    got = got.double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    off = (got - value).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int((off / bound.clamp_min(1e-300)).nan_to_num(nan=float("inf")).argmax())
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} outside the bound; worst at {i}: got "
            f"{got.flatten()[i].item()!r}, expected {value.flatten()[i].item()!r} +- "
            f"{bound.flatten()[i].item()!r}")
