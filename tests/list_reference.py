"""Plain references for the tests of the update over a list of tensors: the
float32 operation sequence of one update, the 64-bit definition beside it, and
the 8-bit form of the moments, in numpy, one tensor at a time."""
import numpy as np

BLOCK = 128
LOW = {"m": 18, "v": 33}       # lowest biased block exponents
UNITS = {"m": 127, "v": 255}   # codes above zero
M32 = 0xFFFFFFFF


def mixed(x):
    x = np.asarray(x, dtype=np.uint64) & np.uint64(M32)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x5BD9E4B5)) & np.uint64(M32)
    return x ^ (x >> np.uint64(15))


def random_bits(seed, t, first, n):
    """32 bits for each of the list's elements first .. first + n - 1."""
    key = int(mixed(int(mixed((seed * 0x9E3779B1 + t * 0xC2A3F1D7) & M32)) + 0x7F4A7C15))
    i = np.arange(first, first + n, dtype=np.uint64)
    lo, hi = i & np.uint64(M32), i >> np.uint64(32)
    return mixed(lo * np.uint64(0x9E3779B1) + hi * np.uint64(0xC2A3F1D7) + np.uint64(key))


def _blocks(mag):
    return np.pad(mag, (0, -mag.size % BLOCK)).reshape(-1, BLOCK)


def exponents(x, which):
    """Biased exponent of each block of the float32 vector x."""
    top = _blocks(x.view(np.uint32) & np.uint32(0x7FFFFFFF)).max(1).astype(np.int64)
    return np.clip((top + 0x7FFFFF) >> 23, LOW[which], 255)


def encode(x, which, add=None):
    """(codes filled up to whole blocks, block exponents) of the float32 vector
    x; add: what is added below the third mantissa bit (None: the nearest)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    e = exponents(x, which)
    base = np.repeat(8 * e - UNITS[which], BLOCK)[:x.size]
    mag = (x.view(np.uint32) & np.uint32(0x7FFFFFFF)).astype(np.int64)
    add = 0x7FFFF + ((mag >> 20) & 1) if add is None else np.asarray(add).astype(np.int64)
    low = 0 if which == "v" else ((base + 1) << 20) - (1 << 23)
    k = np.clip(np.maximum(((mag + add) >> 20) - base, (mag > low).astype(np.int64)), 0,
                UNITS[which])
    if which == "m":
        k |= ((x.view(np.uint32) >> 24) & 0x80).astype(np.int64)
    out = np.zeros(e.size * BLOCK, np.uint8)
    out[:x.size] = k
    return out, e.astype(np.uint8)


def decode(codes, e, which, n):
    base = np.repeat(8 * e.astype(np.int64) - UNITS[which], BLOCK)
    k = codes.astype(np.int64)
    sign = k >> 7 if which == "m" else np.zeros_like(k)
    k = k & 0x7F if which == "m" else k
    bits = np.where(k > 0, ((k + base) << 20) | (sign << 31), 0).astype(np.uint32)
    return bits.view(np.float32)[:n]


def clip_scale(norm, clip):
    return np.float32(clip / norm) if norm > clip else np.float32(1.0)


def update32(w, g, m, v, norm, t, lr, wd, clip, scale=1.0, b1=0.9, b2=0.999, eps=1e-8):
    """One update in float32, each operation rounded on its own; w, m and v
    come back as float32 (weights not yet rounded to their type)."""
    f = np.float32
    if not np.isfinite(norm):
        return w.copy(), m.copy(), v.copy()
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        gp = (g * f(scale)) * clip_scale(norm, clip)
        m1 = f(b1) * m + f(1.0 - b1) * gp
        v1 = f(b2) * v + f(1.0 - b2) * (gp * gp)
        mh = m1 / f(1.0 - b1 ** t)
        vh = v1 / f(1.0 - b2 ** t)
        den = np.sqrt(vh) + f(eps)
        w1 = w * f(1.0 - float(f(lr)) * float(f(wd))) - (f(lr) * mh) / den
    return w1, m1, v1


def weights64(w, m1, v1, t, lr, wd, b1=0.9, b2=0.999, eps=1e-8):
    """The weights in 64 bits, from the update's own float32 moments, and the
    size of its largest term (what rounding errors are relative to)."""
    f = np.float32
    w, m1, v1 = (x.astype(np.float64) for x in (w, m1, v1))
    keep = w * float(f(1.0 - float(f(lr)) * float(f(wd))))
    step = float(f(lr)) * (m1 / float(f(1.0 - b1 ** t))) / (
        np.sqrt(v1 / float(f(1.0 - b2 ** t))) + float(f(eps)))
    return keep - step, np.maximum(np.abs(keep), np.abs(step))
