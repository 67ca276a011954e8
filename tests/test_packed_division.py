"""The rotated append's division on the CPU: one product with the rounded reciprocal and one correction, emulated exactly,
gives the correctly rounded quotient for every scale and value where an E4M3FN code could depend on it."""
import numpy as np

F4, F8 = np.float32, np.float64


def corrected(x, s):
    """RN(q - RN(q s - x) RN(1 / s)) with q = RN(x RN(1 / s)); every fused step rounded once."""
    inv = (F4(1) / s).astype(F4)
    q = (x * inv).astype(F4)
    r = (q.astype(F8) * s.astype(F8) - x.astype(F8)).astype(F4)   # 48 bits less a near neighbour: exact before rounding
    t = -(r.astype(F8) * inv.astype(F8))                          # exact
    whole = q.astype(F8) + t
    rest = t - (whole - q.astype(F8))                             # |t| < |q|: exact
    c = whole.astype(F4)
    # where the double sum is the middle of two floats its own rounding error decides
    below, above = np.nextafter(c, F4(-np.inf)), np.nextafter(c, F4(np.inf))
    c = np.where((whole == (c.astype(F8) + above) / 2) & (rest > 0), above, c)
    return np.where((whole == (c.astype(F8) + below) / 2) & (rest < 0), below, c), q


def test_quotients_next_to_the_borders_of_codes():
    """Significands within 64 of a multiple of 2^19 (12 of 2^20 would do), every border of 5 bits, values around it."""
    S = ((np.arange(16, 33) << 19)[:, None] + np.arange(-64, 65)[None]).ravel()
    S = S[(S >= 1 << 23) & (S < 1 << 24)].astype(F8)
    far = 0
    for t in range(16, 32):
        unit = 2.0 ** (np.floor(np.log2(S * t)) - 23)
        for d in range(-6, 7):
            x, s = (np.rint(S * t / unit) + d).astype(F4), S.astype(F4)
            c, q = corrected(x, s)
            assert np.array_equal(c, (x / s).astype(F4))
            far += int((np.abs(q.astype(F8) - x.astype(F8) / s) > np.spacing(c)).sum())
    assert far > 0      # first quotients more than one ulp off are among them


def test_random_quotients():
    g = np.random.default_rng(1)
    x, s = (g.integers(1 << 23, 1 << 24, 2_000_000).astype(F4) for _ in range(2))
    assert np.array_equal(corrected(x, s)[0], (x / s).astype(F4))
