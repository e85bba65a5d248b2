"""8-bit moments at float32's upper end (no GPU): a finite moment is stored as a
finite one, whose square is finite where the format squares it."""
import numpy as np
import pytest

import oracle.moments8 as O8
from f32model8 import adam8_update

FLT_MAX = float(np.finfo(np.float32).max)
HP = dict(lr=1e-3, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0, step=1, inv_loss_scale=1.0, max_grad_norm=0.0)


def upper_values():
    """exp_avg and exp_avg_sq whose codes reach the last binade's upper end."""
    y = np.array([128, 200, 239.9, 240, 241, 247.9, 248, 250, 255.99])
    m = np.ldexp(np.concatenate([y, -y]), 120)
    return np.append(m, [FLT_MAX, -FLT_MAX]), np.append(np.ldexp(np.concatenate([y, y]), 56) ** 2, [FLT_MAX, FLT_MAX])


def finite32(m, s):
    with np.errstate(over="ignore"):
        m, s = m.astype(np.float32), s.astype(np.float32)
        return np.isfinite(m).all() and np.isfinite(s * s).all()


def test_packed_moments_stay_finite():
    m, v = upper_values()
    dm, ds = O8.decode(*O8.pack(m, v), m.size)
    assert finite32(dm, ds)
    # to nearest, and from 240 on to 240, the largest code of these blocks
    for x, d, k in ((np.abs(m), np.abs(dm), 120), (np.sqrt(v), ds, 56)):
        y = np.ldexp(x, -k)
        assert (np.abs(np.ldexp(d, -k) - np.minimum(y, 240)) <= 8).all() and (d[y >= 240] == np.ldexp(240, k)).all()


@pytest.mark.parametrize("seed", range(4))
def test_stepped_moments_stay_finite(seed):
    """With beta2 = 0 the root is the gradient's magnitude."""
    n = 64
    g = np.ldexp(np.linspace(200, 255.999, n), 56).astype(np.float32)
    c, s = np.zeros(8 * n // 4, np.uint8), np.zeros(2 * n // 32, np.uint8)
    _, c, s = adam8_update(np.zeros(n, np.float32), c, s, g, 0.0, seed, **HP)
    m, root = O8.decode(c, s, n)
    assert finite32(m, root) and (root[g >= np.ldexp(240.0, 56)] == np.ldexp(240.0, 56)).all()
    # exp_avg has room above: it still rounds up
    assert (np.abs(m) == np.ldexp(256.0, 56)).any()


def test_other_blocks_round_up_to_256():
    """One binade lower nothing overflows, and nothing is held back."""
    dm, ds = O8.decode(*O8.pack(np.array([np.ldexp(250.0, 119)]), np.array([np.ldexp(250.0, 55) ** 2])), 1)
    assert dm[0] == np.ldexp(256.0, 119) and ds[0] == np.ldexp(256.0, 55)
