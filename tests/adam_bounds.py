"""How far float32 arithmetic in the documented operation order may be from
the formulas of AdamW in float64, element by element, counted in half steps
u = 2^-24 of float32 before any run:

  g = raw * gscale            gscale is rounded once, the product once: 2u
  m = fma(B1, m0, O1*g)       first term: B1, the final rounding: 2u; second:
                              g 2u, O1, the product, the final one: 5u
  v = fma(B2, v0, (O2*g)*g)   first term: B2, the final rounding: 2u (v0
                              itself is given); second: g twice 4u, O2, two
                              products, the final one: 8u
  s = sqrt(v)                 half of v's relative error and u
  d = fma(s, RB, E)           all terms positive: s's, RB or E, the final one
  p = fma(p0, D, -(SS*m)/d)   p0*D: D 1u; the quotient: SS, product,
                              division 3u and d's, plus m's own absolute error
                              times SS/d; the final rounding: u of the result

Products of the errors are covered by a factor 1.01.  `floor` covers results
near float32's smallest values."""
import math

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -148


def adam64(p, m, v, g_raw, global_sq, *, lr, beta1, beta2, eps, weight_decay, step, inv_loss_scale, max_grad_norm):
    """((p, m, v), (bound on p, m, v)) in float64 from the definition."""
    p, m, v, g = (np.asarray(x, np.float64) for x in (p, m, v, g_raw))
    coef = inv_loss_scale
    if max_grad_norm > 0:
        coef *= min(1.0, max_grad_norm / (math.sqrt(global_sq) + 1e-6))
    g = g * coef
    m1, m2 = beta1 * m, (1 - beta1) * g
    v1, v2 = beta2 * v, (1 - beta2) * g * g
    mn, vn = m1 + m2, v1 + v2
    # sums and products of zeros are exact
    dm = 1.01 * U * (2 * np.abs(m1) + 5 * np.abs(m2)) + TINY * ((m1 != 0) | (m2 != 0))
    dv = 1.01 * U * (2 * v1 + 8 * v2) + TINY * ((v1 != 0) | (v2 != 0))
    bc1, bc2 = 1 - beta1 ** step, 1 - beta2 ** step
    s = np.sqrt(vn)
    # the root's relative error; where v is tiny its floor may be all of it
    rel_s = np.where(vn > 0, np.sqrt(1 + dv / np.maximum(vn, TINY)) - 1, 0.0) + U
    d = s / math.sqrt(bc2) + eps
    with np.errstate(divide="ignore", invalid="ignore"):
        upd = np.where(mn == 0, 0.0, lr / bc1 * mn / d)
        rel_d = rel_s + 2 * U
        du = np.where(d > 0, np.abs(upd) * (rel_d + 3 * U) + lr / bc1 * dm / d, 0.0)
    decay = 1 - lr * weight_decay
    pn = p * decay - upd
    dp = 1.01 * (U * np.abs(p * decay) + du * 1.01 + U * np.abs(pn)) + TINY
    return (pn, mn, vn), (dp, dm, dv)


def assert_within(name, got, want, bound):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = np.flatnonzero(bad)[:5]
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of bounds; idx {i.tolist()} got {got[i].tolist()} "
                             f"want {want[i].tolist()} bound {np.broadcast_to(bound, want.shape)[i].tolist()}")
