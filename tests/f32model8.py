"""A float32 model of the update with 8-bit moments, written from the operation
order that include/zero_shard.h documents, on top of tests/f32model.py; and the
check of stored codes against the float64 oracle."""
import numpy as np

import oracle.moments8 as O8
from f32model import F32, _fma, coefficients, gradient_factor


def adam8_update(p, moments8, scales8, g_values, global_sq, seed, tensor=0, **hp):
    """(p, moments8, scales8) after one step, bit for bit."""
    n = np.asarray(p).size
    c = coefficients(**hp)
    gscale = gradient_factor(hp["inv_loss_scale"], hp["max_grad_norm"], global_sq)
    m, s = (x.astype(F32) for x in O8.decode(moments8, scales8, n))
    g = (np.asarray(g_values, F32) * gscale).astype(F32)
    m = _fma(c["B1"], m, (c["O1"] * g).astype(F32))
    v = _fma(c["B2"], (s * s).astype(F32), ((c["O2"] * g).astype(F32) * g).astype(F32))
    s = np.sqrt(v).astype(F32)
    d = _fma(s, c["RB"], c["E"])
    with np.errstate(invalid="ignore", divide="ignore"):
        p = _fma(p, c["D"], -((c["SS"] * m).astype(F32) / d).astype(F32))
    w = O8.words(seed, hp["step"], n, tensor)
    b = [O8.exponent_bytes(x.astype(np.float64)) for x in (m, s)]
    per = [np.repeat(x, O8.BLOCK)[:n] for x in b]
    codes = O8.join(O8.encode(m, per[0], w[0]), O8.encode(s, per[1], w[1], root=True), *b)
    return p, codes[0], codes[1]


def check_codes(name, moments8, scales8, n, m, s, dm, ds, words):
    """The stored moments against float64 ones known to within dm and ds: each
    exponent byte and each code is one that some value within the bound gives
    (both are monotone in the value)."""
    codes, _ = O8.split(moments8, scales8, n)
    nb = -(-n // O8.BLOCK)
    got = np.asarray(scales8, np.uint8)[:2 * nb].reshape(-1, 2).T.astype(np.int64)
    value = O8.e4m3_values()
    for k, (x, dx, w) in enumerate(((m, dm, words and words[0]), (s, ds, words and words[1]))):
        lo = O8.exponent_bytes(np.maximum(np.abs(x) - dx, 0))
        hi = O8.exponent_bytes(np.abs(x) + dx)
        assert ((got[k] >= lo) & (got[k] <= hi)).all(), f"{name}: exponent bytes of moment {k}"
        per = np.repeat(got[k], O8.BLOCK)[:n]
        # a root is not negative
        a = value[O8.encode(np.maximum(x - dx, 0) if k else x - dx, per, w, root=k == 1)]
        b = value[O8.encode(x + dx, per, w, root=k == 1)]
        have = value[codes[k]]
        low, high = np.minimum(a, b), np.maximum(a, b)
        bad = ~((have >= low) & (have <= high))
        assert not bad.any(), (f"{name}: {bad.sum()} codes of moment {k}; idx {np.flatnonzero(bad)[:5].tolist()} have "
                               f"{have[bad][:5]} between {low[bad][:5]} and {high[bad][:5]}")
    pad = np.asarray(moments8, np.uint8)[:8 * -(-n // 4)].reshape(-1, 2, 4).transpose(1, 0, 2).reshape(2, -1)[:, n:]
    assert not pad.any(), f"{name}: codes past the last element"
