"""Moments in 8 bits, in float64: the format (blocks of 32 elements, OCP e4m3
codes times one power of two per block), the random words that round the step's
moments, and both roundings.

The e4m3 code is decoded from its fields as the OCP 8-bit floating point
specification defines them (1 sign, 4 exponent bits with bias 7, 3 fraction
bits, no infinities, 0x7F and 0xFF NaN).  Stochastic rounding: a value between
two codes goes to the upper one with the probability of its distance from the
lower one, here by adding a random fraction of the spacing and truncating.
"""
import numpy as np

BLOCK = 32


def e4m3_values() -> np.ndarray:
    """float64 value of each of the 256 codes."""
    c = np.arange(256)
    e, f = c >> 3 & 15, c & 7
    mag = np.where(e == 0, np.ldexp(f.astype(np.float64), -9), np.ldexp(8.0 + f, e - 10))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag)


_VALUE = e4m3_values()


def split(moments8: np.ndarray, scales8: np.ndarray, n: int):
    """(codes, exponent bytes) of each moment: two arrays [2, n] of uint8."""
    codes = np.asarray(moments8, np.uint8)[:8 * -(-n // 4)].reshape(-1, 2, 4).transpose(1, 0, 2).reshape(2, -1)[:, :n]
    scales = np.asarray(scales8, np.uint8)[:2 * -(-n // BLOCK)].reshape(-1, 2).T
    return codes, np.repeat(scales, BLOCK, axis=1)[:, :n]


def decode(moments8: np.ndarray, scales8: np.ndarray, n: int):
    """(exp_avg, root of exp_avg_sq), float64, exact."""
    codes, scales = split(moments8, scales8, n)
    x = _VALUE[codes] * np.ldexp(1.0, scales.astype(np.int64) - 127)
    return x[0], x[1]


def exponent_bytes(x: np.ndarray) -> np.ndarray:
    """k + 127 of each block of 32 of x: k = max(floor(log2 max|x|) - 7, -126)."""
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = np.abs(x)
    top = pad.reshape(-1, BLOCK).max(1)
    _, e = np.frexp(top)                                   # top in [2^(e-1), 2^e)
    return np.where(top > 0, np.maximum(e - 1 - 7, -126), -126) + 127


def encode(x: np.ndarray, scale_byte: np.ndarray, words=None, root: bool = False) -> np.ndarray:
    """Code of each x given its block's exponent byte (per element).  words: 32
    random bits per element (stochastic); None: to nearest even.  root: a
    positive x is at least the smallest code.  In the blocks of float32's last
    binade (2^120, roots: 2^56) no code is above 240: 256 * 2^120 and the square
    of 256 * 2^56 are not float32 numbers."""
    y = np.asarray(x, np.float64) * np.ldexp(1.0, 127 - scale_byte.astype(np.int64))
    mag = np.abs(y)
    if root:
        mag = np.where((mag > 0) & (mag < 2.0 ** -9), 2.0 ** -9, mag)
    last = np.asarray(scale_byte) == 127 + (56 if root else 120)
    mag = np.where(last & (mag < 256), np.minimum(mag, 240.0), mag)
    _, e = np.frexp(mag)
    q = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)           # spacing of the codes at this magnitude
    steps = mag / q
    if words is None:
        steps = np.rint(steps)
    else:
        steps = np.floor(steps + (np.asarray(words, np.int64) >> 12) / 2.0 ** 20)
    mag = np.minimum(steps * q, 448.0)                     # beyond the format's largest value
    # back to fields
    _, e = np.frexp(mag)
    e = np.maximum(e - 1, -6)
    f = np.rint(mag / np.ldexp(1.0, e - 3)).astype(np.int64)
    code = np.where(f < 8, f, (e + 7) * 8 + (f - 8))
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def join(m_codes, s_codes, m_bytes, s_bytes):
    """(moments8, scales8) from codes per element and exponent bytes per block."""
    n = m_codes.size
    c = np.zeros((2, -(-n // 4) * 4), np.uint8)
    c[0, :n], c[1, :n] = m_codes, s_codes
    return (c.reshape(2, -1, 4).transpose(1, 0, 2).reshape(-1),
            np.stack([m_bytes, s_bytes], 1).astype(np.uint8).reshape(-1))


def pack(exp_avg: np.ndarray, exp_avg_sq: np.ndarray):
    """(moments8, scales8), each moment rounded to nearest even."""
    x = [np.asarray(exp_avg, np.float64), np.sqrt(np.asarray(exp_avg_sq, np.float64))]
    b = [exponent_bytes(v) for v in x]
    n = x[0].size
    per = [np.repeat(v, BLOCK)[:n] for v in b]
    return join(encode(x[0], per[0]), encode(x[1], per[1], root=True), *b)


def words(seed: int, step: int, n: int, tensor: int = 0, first: int = 0):
    """(word for exp_avg, word for the root) of elements first .. first + n."""
    m64, m32 = (1 << 64) - 1, 0xFFFFFFFF
    k = (seed * 0x9E3779B97F4A7C15 + step * 0xBB67AE8584CAA73B) & m64
    k = (k ^ k >> 32) * 0x6A09E667F3BCC909 & m64
    key = (k ^ k >> 32) & m32
    e = np.arange(first, first + n, dtype=np.int64).astype(np.uint64)
    a = (np.uint64(key + tensor * 0x3C6EF373 & m32) + (e >> np.uint64(32)) * np.uint64(0xA54FF53B)) & np.uint64(m32)
    x = (e & np.uint64(m32)) ^ a
    x = (x ^ x >> np.uint64(16)) * np.uint64(0x9E3779B9) & np.uint64(m32)
    x = (x ^ x >> np.uint64(13)) * np.uint64(0xBB67AE85) & np.uint64(m32)
    x = x ^ x >> np.uint64(16)
    return x, (x << np.uint64(16) | x >> np.uint64(16)) & np.uint64(m32)
