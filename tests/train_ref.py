"""Plain 64-bit forms of the gated feed-forward block and of the AdamW step
(NumPy, CPU), and the rounding-error bounds that the GPU tests hold their
outputs to.

U is the unit roundoff of FP32, UB that of BF16, as in layer_ref.py.  E4M3 codes
have three stored significand bits: a value rounded to the nearest one is off by
at most 2^-4 of itself, or 2^-10 below 2^-6; rounded at random by twice that.
"""
import numpy as np

from tests.layer_ref import U, UB


def decode(q):
    """E4M3 codes (uint8) as FP64."""
    q = np.asarray(q).astype(np.int64)
    e, m = (q >> 3) & 15, q & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((q & 0x7F) == 0x7F, np.nan, v)
    return np.where(q & 0x80, -v, v)


def spread(s, n):
    return np.repeat(np.asarray(s, np.float64), 128)[:n]


def group_max(x):
    n = x.size
    return np.pad(np.abs(x), (0, -n % 128)).reshape(-1, 128).max(1)


def adamw(p, g, m, v, lr, step, b1, b2, eps, decay, clip=1.0):
    """{name: (value, error bound before storage)} of one step in FP64.  m, v:
    moments as stored (FP64 of what is decoded; for codes the decoded product is
    off by U, its square by 3 U in all).

    Bounds: b, 1 - b, lr and the correction terms are rounded once each (U), the
    clipping factor takes three operations (4 U with its inputs), every product,
    sum, root and quotient one U of its result; the sum of these U per term is
    charged twice."""
    gc = g * clip
    m1, v1 = b1 * m + (1 - b1) * gc, b2 * v + (1 - b2) * gc * gc
    v1 = np.where(v1 < 2.0 ** -150, 0.0, v1)  # below half the smallest FP32 value: zero there
    em = 2 * U * (3 * np.abs(b1 * m) + 8 * np.abs((1 - b1) * gc) + np.abs(m1)) + 2.0 ** -149
    ev = 2 * U * (6 * b2 * v + 14 * (1 - b2) * gc * gc + v1) + 2.0 ** -149
    r = np.sqrt(v1)
    with np.errstate(divide="ignore", invalid="ignore"):
        er = np.where(v1 > 0, np.minimum(ev / np.maximum(r, 1e-300), np.sqrt(ev)), np.sqrt(ev)) + 2 * U * r
    root = 1 / np.sqrt(1 - b2 ** step)
    den = r * root + eps
    size = lr / (1 - b1 ** step)
    with np.errstate(divide="ignore", invalid="ignore"):
        upd = size * m1 / den
        eu = size * em / den + np.abs(upd) * (er * root / den + 2 * U * 8)
    p1 = p * (1 - lr * decay) - upd
    ep = 2 * U * (2 * np.abs(p) + np.abs(p1)) + 2 * eu
    return {"p": (p1, ep), "m": (m1, em), "v": (v1, ev), "r": (r, er)}


def bf16_bound(x, e, random):
    """Storage in BF16: half a step to nearest, a whole one at random (2^-133 where BF16 is subnormal)."""
    k = 2 if random else 1
    return e + k * UB * (np.abs(x) + e) + k * 2.0 ** -134


def code_bounds(x, e, random, floor):
    """(scale, its bound, bound of code times scale) of values x, off by e, in groups of 128."""
    n = x.size
    top, et = group_max(x), group_max(e)
    s = np.where(top == 0, 1.0, top / 448)
    es = np.where(top == 0, 0.0, et / 448 + 3 * U * s)  # 1 / 448 and the product are rounded: 2 U and their product
    S = spread(s + es, n)
    k = 2 if random else 1
    # the quotient is within one unit in the last place, and what saturates at 448 is off by the scale's error
    b = e + k * np.maximum(2.0 ** -4 * (np.abs(x) + e), 2.0 ** -10 * S) + 8 * U * np.abs(x) + spread(es, n) * 448
    if floor:
        b = np.maximum(b, 2.0 ** -9 * S)
    return s, es, b


M32 = 0xFFFFFFFF


def random_bits(key, place):
    """The 32 random bits of an element, as the header defines them."""
    i = np.asarray(place, dtype=np.uint64)
    h = ((i * np.uint64(0x9E3779B1)) ^ (i >> np.uint64(32))) + np.uint64(key & M32) & np.uint64(M32)
    h = (h ^ (h >> np.uint64(16))) * np.uint64(0x85EBCA6B) & np.uint64(M32)
    h = (h ^ (h >> np.uint64(13))) * np.uint64(0xC2B2AE35) & np.uint64(M32)
    return (h ^ (h >> np.uint64(16))).astype(np.int64)


def key_of(seed, index=0):
    return (seed + index * 0x27D4EB2F) & M32


def drop(x, bits, r):
    """FP32 x without its lowest bits after r was added there (exact integer arithmetic)."""
    w = np.asarray(x, np.float32).view(np.uint32).astype(np.int64)
    w = ((w + r) >> bits) << bits
    return (w & M32).astype(np.uint32).view(np.float32)


# --- the gated feed-forward block ------------------------------------------

def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def act(g, kind):
    """(z, dz/dg) of act(g) = g sigmoid(z)."""
    if kind == "silu":
        return g, np.ones_like(g)
    k = np.sqrt(8 / np.pi)
    return k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g ** 2)


def _sigmoid_bound(z, p):
    """FP32 error of p: z is off by at most 6 U of itself (GELU: five operations and a constant), its product with
    log2 e and that constant by 2 U more, each of which e^-z multiplies by |z|; 2^x one unit in the last place (2 U),
    the sum U, the reciprocal 2 U.  Below 2^-126 it may be zero."""
    return p * U * ((1 - p) * (8 * np.abs(z) + 2) + 4) + 2.0 ** -125


def gated(g, v, kind):
    """(h, FP32 error bound) in FP64."""
    z, _ = act(g, kind)
    p = _sigmoid(z)
    h = g * p * v
    return h, np.abs(g * v) * _sigmoid_bound(z, p) + 3 * U * np.abs(h) + 2.0 ** -140


def gated_slope(g, v, kind, eg, ev):
    """How far h moves when g and v are off by eg and ev: |act'| <= 1.13, |act| <= |g|."""
    return 1.13 * np.abs(v) * eg + np.abs(g) * ev + 1.13 * eg * ev


def gated_grad(dh, g, v, kind):
    """{name: (value, FP32 error bound)} for dg, dv and h in FP64."""
    z, dz = act(g, kind)
    p = _sigmoid(z)
    ep = _sigmoid_bound(z, p)
    a, q = g * p, 1 - p
    ea = np.abs(g) * ep + U * np.abs(a)
    t = a * q
    et = ea * q + np.abs(a) * (ep + U * q) + U * np.abs(t)
    slope = t * dz + p
    es = et * np.abs(dz) + 5 * U * np.abs(t * dz) + ep + U * np.abs(slope)
    h, eh = gated(g, v, kind)
    return {"dg": (dh * v * slope, np.abs(dh * v) * es + 3 * U * np.abs(dh * v * slope) + 2.0 ** -140),
            "dv": (dh * a, np.abs(dh) * ea + 2 * U * np.abs(dh * a) + 2.0 ** -140), "h": (h, eh)}
