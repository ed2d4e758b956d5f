"""Plain references for the calls over lists of tensors (test code only).

The 8-bit moments follow include/zshard_tensors.h word for word in numpy, in
binary32 where the header says so; the AdamW update is in binary64.
"""
import numpy as np

GOLDEN, M32 = 0x9E3779B9, 0xFFFFFFFF
TOP = {"m": 15, "v": 31}
BLOCK = 256


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & M32
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def key_of(seed, step):
    return int(mix((int(mix(seed)) + (step & M32)) & M32))


def words(n, index, key, first=0):
    """The dither word of elements [first, first + n) of tensor `index`."""
    i = np.arange(first, first + n, dtype=np.uint64)
    group = i >> np.uint64(2)
    key_k = mix((key + index * GOLDEN) & M32)
    h = mix((group & np.uint64(M32)) + (group >> np.uint64(32)) * np.uint64(GOLDEN) + key_k)
    return (h + (i & np.uint64(3)) * np.uint64(GOLDEN)) & np.uint64(M32)


def encode(x, name, word):
    """fp32 values -> (codes uint8, one scale byte per block)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    n, top = x.size, TOP[name]
    r = (word >> np.uint64(12) if name == "m" else word & np.uint64(0xFFFFF)).astype(np.int64)
    bits = x.view(np.uint32).astype(np.int64)
    size = bits & 0x7FFFFFFF
    blocks = -(-n // BLOCK)
    most = np.zeros(blocks * BLOCK, np.int64)
    most[:n] = size
    e = np.minimum((most.reshape(blocks, BLOCK).max(axis=1) + 0x0FFFFF) >> 23, 255)
    k = top - np.repeat(e, BLOCK)[:n]
    with np.errstate(all="ignore"):
        s = np.ldexp(size.astype(np.uint32).view(np.float32).astype(np.float64), k).astype(np.float32)
    code = (s.view(np.uint32).astype(np.int64) + r) >> 20
    bad = np.repeat(e, BLOCK)[:n] == 255
    if name == "m":
        assert (code[~bad] <= 0x7F).all()
        code = (code & 0x7F) | (bits >> 31) << 7
    else:
        assert (code[~bad] <= 0xFF).all()
        code = np.where((code & 0xFF == 0) & (x > 0), 1, code & 0xFF)
    return code.astype(np.uint8), e.astype(np.uint8)


def decode(codes, e, name):
    c = codes.astype(np.uint32)
    body = (c & 0x7F if name == "m" else c) << 20
    each = np.repeat(e.astype(np.int64), BLOCK)[:codes.size]
    with np.errstate(all="ignore"):
        x = np.ldexp(body.astype(np.uint32).view(np.float32).astype(np.float64), each - TOP[name]).astype(np.float32)
    if name == "m":
        x = np.where(c & 0x80, -x, x)
    return np.where(each == 255, np.float32(np.nan), x).astype(np.float32)


def stored(x, name, index, key):
    """The values that x is stored as."""
    return decode(*encode(x, name, words(x.size, index, key)), name)


def new_moments(g, m, v, s, coef):
    """binary32, one rounding per operation; s: adamw_scalars' fields."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = (g.astype(f) * f(s.grad_scale)) * f(coef)
        m = (f(s.beta1) * m) + (f(s.one_minus_beta1) * g)
        v = (f(s.beta2) * v) + (f(s.one_minus_beta2) * (g * g))
    return m.astype(f), v.astype(f)


def update64(p, m, v, s):
    """The parameter after the step and the step itself, in binary64, from the
    new moments and the step's binary32 scalars."""
    with np.errstate(all="ignore"):
        u = m.astype(np.float64) / (np.sqrt(v.astype(np.float64)) / np.float64(np.float32(s.bias_correction2_sqrt))
                                    + np.float64(np.float32(s.eps))) * np.float64(np.float32(s.step_size))
        return p.astype(np.float64) * np.float64(np.float32(s.decay)) - u, u
