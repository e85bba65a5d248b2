"""Models of the step by orthogonalised momentum.

exact(): the orthogonalisation in float64 from its definition.  rounded(): the
same with the iterate and the two symmetric matrices rounded to fp16 between
products where the header says so, sums in float64.

bound(): how far a result may be from exact() in the Frobenius norm.  A kernel
makes the roundings of rounded() up to the order of its float32 sums, so its
error is that model's error again, taken twice for the freedom of which way each
rounding falls; a sum that lands on the other side of a middle moves X by one
more half step of fp16, which a step passes on at most 5 times larger (its
slope |a + 3 b x^2 + 5 c x^4| and its gain a stay below 4.3 on [0, 1.21]); and
the stored result is off by half a step of its type."""
import math

import numpy as np

COEFS = ((3.4445, -4.7750, 2.0315),) * 5
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}                             # half a step relative to the value, at most


def _start(u, eps):
    x = np.asarray(u, dtype=np.float64)
    norm = math.sqrt(float(np.sum(x * x)))
    by = max(norm, eps)
    return x / by if by > 0 else x * 0.0


def exact(u, coefs=COEFS, eps=1e-7):
    x = _start(u, eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coefs:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _half(x, scale):
    return (x * scale).astype(np.float32).astype(np.float16).astype(np.float64) / scale


def rounded(u, coefs=COEFS, eps=1e-7):
    x = _start(u, eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    k = 0
    while k < 12 and 4 << 2 * k <= x.shape[1]:
        k += 1
    x = _half(x, 2.0 ** k)
    for i, (a, b, c) in enumerate(coefs):
        g = _half(x @ x.T, 1024.0)
        x = _half(a * np.eye(len(g)) + b * g + c * (g @ g), 1024.0) @ x
        if i + 1 < len(coefs):
            x = _half(x, 2.0 ** k)
    return x.T if tall else x


def bound(u, out_type, coefs=COEFS, eps=1e-7):
    """(exact result, the largest Frobenius distance from it)."""
    ref = exact(u, coefs, eps)
    off = float(np.linalg.norm(rounded(u, coefs, eps) - ref))
    return ref, 2.0 * off + (UNIT[out_type] + 5 * 2.0 ** -11) * float(np.linalg.norm(ref))


def momentum32(m, g, gscale, mu, nesterov):
    """The momentum pass in float32, in its order: (m, u)."""
    f = np.float32
    g = f(1.0 - mu) * (g.astype(f) * f(gscale))
    mu = f(mu)
    m = fma32(mu, m, g)
    return m, (fma32(mu, m, g) if nesterov else m)


def update32(p, o, lr, scale, wd):
    f = np.float32
    return fma32(f(1.0 - lr * wd), p, -(f(lr * scale) * o.astype(f)))


def fma32(a, b, c):
    """round32(a b + c): the product is exact in float64, and the sum is taken
    to odd there (its last bit set where it is inexact), so that rounding it to
    float32 rounds the exact sum."""
    a, b, c = (np.asarray(x, dtype=np.float32).astype(np.float64) for x in (a, b, c))
    p = a * b
    p, c = np.broadcast_arrays(p, c)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)                     # the sum's exact rounding error
    bits = s.view(np.int64).copy()
    even = (bits & 1) == 0
    with np.errstate(invalid="ignore"):
        toward = np.where(err != 0, np.where((err > 0) == (s > 0), 1, -1), 0)
    bits = np.where((err != 0) & even & np.isfinite(s), np.where(toward > 0, bits + 1, bits - 1), bits)
    return bits.view(np.float64).astype(np.float32)
