"""The experts' e4m3 quotient h / s, emulated operation for operation in fp_emulation.c:
two corrections of h * RN(1/s) against the IEEE quotient, for fp32 h (no GPU)."""
import numpy as np

from test_fp_emulation import emu, _f32p  # noqa: F401


def quotients(emu, x, s):  # noqa: F811
    import ctypes
    emu.two_step_quotient_many.restype = None
    emu.two_step_quotient_many.argtypes = [ctypes.c_int64, _f32p, _f32p, _f32p]
    q = np.empty(x.size, np.float32)
    emu.two_step_quotient_many(x.size, x, s, q)
    return q


def same(q, ref):
    """Equal with their signs, or both so small that the code is a zero of the same sign."""
    return (q.view(np.uint32) == ref.view(np.uint32)) | (
        (np.abs(ref) < 2.0 ** -39) & (np.abs(q) < 2.0 ** -38) & (np.signbit(q) == np.signbit(ref)))


def scales(rng, n):
    s = (rng.uniform(1, 2, n) * 2.0 ** rng.integers(-64, 64, n)).astype(np.float32)
    s[:4] = np.float32(2.0 ** -64), np.float32(2.0 ** 64), np.nextafter(
        np.float32(1), np.float32(2)), np.nextafter(np.float32(2), np.float32(1))
    return s


def test_quotients_of_random_values(emu):  # noqa: F811
    rng = np.random.default_rng(31)
    n = 8_000_000
    s = scales(rng, n)
    share = rng.uniform(-448, 448, n) * 2.0 ** -np.abs(rng.normal(0, 8, n))
    x = (share * s).astype(np.float32)
    x[1000:1100], x[1100:1200] = 0.0, -0.0
    assert same(quotients(emu, x, s), x / s).all()


def test_quotients_beside_the_ties_of_e4m3(emu):  # noqa: F811
    """Values within a few units of s times a midpoint of two neighbouring e4m3 values, where one
    unit in the quotient decides the code."""
    rng = np.random.default_rng(32)
    grid = [m * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8, 16)]  # normal values
    grid = sorted([m * 2.0 ** -9 for m in range(8)] + grid)
    grid = [v for v in grid if v <= 448]
    ties = np.array([(a + b) / 2 for a, b in zip(grid, grid[1:])])
    n = 200_000
    for _ in range(30):
        s = scales(rng, n)
        x = (rng.choice(ties, n) * s.astype(np.float64)).astype(np.float32)
        x = (x.view(np.uint32) + rng.integers(-2, 3, n)).astype(np.uint32).view(np.float32)
        x *= rng.choice(np.float32([-1, 1]), n)
        assert (quotients(emu, x, s) == x / s).all()
