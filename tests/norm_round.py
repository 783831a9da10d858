"""64-bit numbers rounded once to fewer bits, in plain numpy, for the tests of the norm's outputs. Shares
nothing with the library."""
import numpy as np

# significant bits, exponent of the smallest normal number, largest number
KINDS = {"f32": (24, -126, float(np.finfo(np.float32).max)), "f16": (11, -14, 65504.0),
         "bf16": (8, -126, (2.0 - 2.0 ** -7) * 2.0 ** 127)}


def step(v, kind):
    """Distance of the neighbours of `kind` that v lies between."""
    bits, low, _ = KINDS[kind]
    with np.errstate(invalid="ignore"):
        e = np.frexp(np.where(np.isfinite(v), v, 1.0))[1] - 1  # 2^e <= |v| < 2^(e + 1)
    return 2.0 ** (np.maximum(np.where(v == 0, low, e), low) - (bits - 1))


def once(v, kind):
    """v to the nearest number of `kind`, ties to the even one, as 64-bit numbers."""
    v = np.asarray(v, np.float64)
    s = step(v, kind)
    with np.errstate(invalid="ignore"):
        q = np.rint(v / s) * s
        return np.where(np.abs(q) > KINDS[kind][2], np.copysign(np.inf, v), q)


def off(got, v, kind, room=2.0 ** -45):
    """How many of `got` are not v rounded once. Where v lies within `room` of itself from the middle of
    two neighbours, either of them will do."""
    v = np.asarray(v, np.float64)
    top = KINDS[kind][2]
    want = once(v, kind)
    with np.errstate(invalid="ignore"):
        s = step(v, kind)
        low = np.floor(v / s)
        middle = np.abs((v / s - low - 0.5) * s) <= room * np.abs(v)
        either = middle & ((got == low * s) | (got == (low + 1) * s)
                           | (((low + 1) * s > top) & (got == np.inf)) | ((low * s < -top) & (got == -np.inf)))
    return int((~((got == want) | either | (np.isnan(got) & np.isnan(v)))).sum())


def beside_middles(kind, rng, n):
    """(w, y): 32-bit numbers w whose product y = 1.5 w, exact in 64 bits, lies beside the middle of two
    neighbours of `kind` by less than 32 bits tell: n middles, of all sizes of `kind`, the smallest and
    largest among them."""
    bits, low, top = KINDS[kind]
    high = int(np.frexp(top)[1]) - 1
    s = rng.integers(2 ** (bits - 1), 2 ** bits, n) + 0.5
    e = rng.integers(low - (bits - 1), high - (bits - 1) + 1, n)
    m = s * 2.0 ** e.astype(np.float64)
    m[: n // 4] = (rng.integers(0, 2 ** (bits - 1), n // 4) + 0.5) * 2.0 ** (low - bits + 1)  # below the normal ones
    m[n // 4] = (2.0 ** bits - 0.5) * 2.0 ** (high - bits + 1)  # the border of infinity
    at = (m / 1.5).astype(np.float32)
    w = np.concatenate([at, np.nextafter(at, np.float32(np.inf)), np.nextafter(at, np.float32(0))])
    w *= rng.choice(np.array([-1, 1], np.float32), len(w))
    return w, 1.5 * w.astype(np.float64)
