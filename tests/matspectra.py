"""Matrices whose singular values fall, and the model of the roundings that the
orthogonalisation states, for tests of how far its results are off.

rounded(): the iteration in float64 with the roundings of a short side above 128:
the iterate begins as U times a power of two, the first step takes the rest of the
factor, and X, X X^T and the polynomial are fp16 between products.
short(): one run of steps with a short side up to 128: X X^T and the polynomials
carried as float32, and as two fp16 into products, of which the lower halves' own
is left out; float32 sums, eight products at a time.  What limits it where values
fall are those sums: they know X X^T to 2^-24 of its largest entries, and small
singular values by their squares.

A rounding of X leaves something in the place of a zero singular value, which each
later step multiplies by a.  determined() is what a matrix of low rank determines
all the same: the result between its own singular directions."""
import math

import numpy as np

import matmodel as M

FEW = 1e-4                                         # relative: see bound()
HALF = 2.0 ** -11                                  # half a step of fp16, relative

KINDS = ("noise", "k1", "k1.5", "k2", "exp", "rank3", "rank16")


def draw(kind, shape, seed):
    """float64; of low rank: small whole numbers, exact in fp16 and bf16."""
    rng = np.random.default_rng(seed)
    s, l = min(shape), max(shape)
    if kind == "noise":
        return rng.normal(size=shape)
    if kind.startswith("rank"):
        r = min(int(kind[4:]), s)
        return rng.integers(-2, 3, (shape[0], r)) @ rng.integers(-2, 3, (r, shape[1])).astype(float)
    k = np.arange(1.0, s + 1)
    values = np.exp(-8.0 * k / s) if kind == "exp" else k ** -float(kind[1:])
    u = np.linalg.qr(rng.normal(size=(s, s)))[0]
    v = np.linalg.qr(rng.normal(size=(l, s)))[0]
    x = (u * values) @ v.T
    x = x * (8.0 / np.abs(x).max())
    return x if shape[0] <= shape[1] else x.T


def rounded(u, coefs):
    u = np.asarray(u, dtype=np.float64)
    tall = u.shape[0] > u.shape[1]
    u = u.T if tall else u
    k = 0
    while k < 12 and 4 << 2 * k <= u.shape[1]:
        k += 1
    rest, up = math.frexp(math.sqrt(float(np.sum(u * u))))
    rest = 1.0 / rest
    x = M._half(u * 2.0 ** -up, 2.0 ** k)
    for i, (a, b, c) in enumerate(coefs):
        g = M._half((x @ x.T) * (rest * rest), 1024.0)
        x = (M._half(a * np.eye(len(g)) + b * g + c * (g @ g), 1024.0) @ x) * rest
        rest = 1.0
        if i + 1 < len(coefs):
            x = M._half(x, 2.0 ** k)
    return x.T if tall else x


def _two(x, scale):
    y = (x * scale).astype(np.float32)
    high = y.astype(np.float16)
    return high.astype(np.float64), (y - high.astype(np.float32)).astype(np.float16).astype(np.float64)


def _sum(products):
    """Of a b over products of halves, in float32, eight inner elements at a time."""
    total = np.zeros((products[0][0].shape[0], products[0][1].shape[1]), np.float32)
    for k in range(0, products[0][0].shape[1], 8):
        for a, b in products:
            total = (total + a[:, k:k + 8] @ b[k:k + 8]).astype(np.float32)
    return total.astype(np.float64)


def short(u, coefs, low=True):
    """low=False: with the lower halves left out altogether."""
    u = np.asarray(u, dtype=np.float64)
    tall = u.shape[0] > u.shape[1]
    u = u.T if tall else u

    def product(x, y, scale_x=1024.0, scale_y=1024.0):
        (xh, xl), (yh, yl) = _two(x, scale_x), _two(y, scale_y)
        return _sum([(xh, yh), (xh, yl), (xl, yh)] if low else [(xh, yh)]) / (scale_x * scale_y)

    def symmetric(x):
        x = x.astype(np.float32).astype(np.float64)
        return np.tril(x) + np.tril(x, -1).T

    k = 0
    while k < 12 and 4 << 2 * k <= u.shape[1]:
        k += 1
    scale = 2.0 ** (14 - math.floor(math.log2(float(np.abs(u).max()))))
    h, l = _two(u, scale)
    g = _sum([(h, h.T), (h, l.T), (l, h.T)] if l.any() else [(h, h.T)]) / scale ** 2
    norm = math.sqrt(float(np.trace(g)))
    g, p = symmetric(g / norm ** 2), None
    for i, (a, b, c) in enumerate(coefs):
        q = symmetric(b * g + c * product(g, g))
        p = symmetric(q + a * np.eye(len(g)) if i == 0 else a * p + product(q, p, 1024.0, 16.0))
        for _ in range(2 if i + 1 < len(coefs) else 0):
            g = symmetric(a * g + product(q, g))
    x = product(p, u / norm, 16.0, 2.0 ** k)
    return x.T if tall else x


def stored(ref, out_type):
    """What the result's own rounding costs: its error on the exact result.  A
    kernel's values differ from those by less than a step, so that their roundings
    fall as these do: the same norm to within 1 / sqrt(elements)."""
    if out_type == "f16":
        return float(np.linalg.norm(ref.astype(np.float16).astype(np.float64) - ref))
    bits = ref.astype(np.float32).view(np.uint32)
    near = ((bits + 0x7FFF + (bits >> 16 & 1)) & np.uint32(0xFFFF0000)).view(np.float32)
    return float(np.linalg.norm(near.astype(np.float64) - ref))


def bound(u, out_type, coefs):
    """(exact result, the largest Frobenius distance from it).  Above 128: the
    model's error half again, since a norm over tens of thousands of independent
    roundings varies by a few percent, and float32 sums, 2^-24 of each, do not
    show beside fp16's 2^-11.  Up to 128: the model's error twice, and FEW, since
    in a small matrix few roundings make the error and fall otherwise.  Then the
    result's own rounding, a tenth more of it."""
    ref = M.exact(u, coefs)
    if min(u.shape) > 128:
        off = 1.5 * float(np.linalg.norm(rounded(u, coefs) - ref))
    else:
        off = 2.0 * float(np.linalg.norm(short(u, coefs) - ref)) + FEW * float(np.linalg.norm(ref))
    return ref, off + 1.1 * stored(ref, out_type)


def directions(u, rank):
    p, _, q = np.linalg.svd(np.asarray(u, dtype=np.float64), full_matrices=False)
    return p[:, :rank], q[:rank].T


def determined(u, rank, coefs):
    """(the exact result between the matrix's singular directions, how far a result
    may be from it there): twice the model's error there, and half a step of fp16
    for each step's X, X X^T and polynomial and for the result: what any of them
    rounds, it rounds between these few directions by less than that."""
    p, q = directions(u, rank)
    core = p.T @ M.exact(u, coefs) @ q
    off = float(np.linalg.norm(p.T @ rounded(u, coefs) @ q - core)) if min(u.shape) > 128 else 0.0
    return core, 2.0 * off + (3 * len(coefs) + 1) * HALF * float(np.linalg.norm(core))
