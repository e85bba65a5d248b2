"""The float64 oracle of the 8-bit moments: the format against torch's e4m3
type and closed forms, the random words' distribution, and the float32 model
against the oracle."""
import numpy as np
import pytest

import oracle.moments8 as O8
from adam_bounds import U, adam64
from f32model8 import adam8_update, check_codes

torch = pytest.importorskip("torch")


def test_values_are_torchs_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O8.e4m3_values(), want, equal_nan=True)


def test_nearest_encoding_is_torchs():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-256, 256, 20000), np.ldexp(rng.uniform(-1, 1, 20000), rng.integers(-12, 8, 20000)),
                        O8.e4m3_values()[np.abs(O8.e4m3_values()) <= 256]]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O8.encode(y, np.full(y.size, 127)), want)


@pytest.mark.parametrize("n", [1, 3, 4, 31, 32, 33, 1000])
def test_pack_decodes_to_within_half_a_step(n):
    rng = np.random.default_rng(n)
    m = rng.normal(0, 1, n) * np.exp(rng.normal(0, 2, n))
    v = (rng.normal(0, 1, n) * np.exp(rng.normal(0, 2, n))) ** 2
    c, s = O8.pack(m, v)
    assert c.size == 8 * -(-n // 4) and s.size == 2 * -(-n // 32)
    dm, ds = O8.decode(c, s, n)
    root = np.sqrt(v)
    # codes below the normal range are 2^(k-9) apart: half of that for exp_avg;
    # a root between 0 and 2^(k-9) becomes 2^(k-9), so up to all of it there
    for x, d, b, low in ((m, dm, s[::2], -10), (root, ds, s[1::2], -9)):
        k = np.repeat(b.astype(int) - 127, 32)[:n]
        assert (np.abs(x - d) <= np.maximum(np.abs(x) * 2.0 ** -4, np.ldexp(1.0, k + low))).all()
    assert (ds > 0).all()                                  # a positive root is never stored as zero
    assert (np.abs(np.abs(dm).reshape(-1)).max() > 0)


def test_scale_puts_the_largest_value_in_the_top_binade():
    for top in (1.0, 0.75, 255.9, 1e-30, 3e38, 2.0 ** -126, 1e-45):
        x = np.zeros(40)
        x[35] = top
        b = O8.exponent_bytes(x)
        assert b[0] == 1
        y = top * 2.0 ** (127.0 - b[1])
        assert 128 <= y < 256 or (b[1] == 1 and y < 256)


def test_zero_state_is_all_zero_bytes():
    m, s = O8.decode(np.zeros(8 * 25, np.uint8), np.zeros(2 * 4, np.uint8), 100)
    assert not m.any() and not s.any()


def test_stochastic_rounding_is_unbiased():
    """The mean over all 2^20 random fractions is the value itself, to within
    the fraction's own resolution, for normal and subnormal codes."""
    w = np.arange(1 << 20, dtype=np.int64) << 12
    for y, q in ((1.3, 2.0 ** -3), (200.7, 16.0), (2.0 ** -8 * 1.37, 2.0 ** -9), (2.0 ** -9 * 0.2, 2.0 ** -9),
                 (-17.1, 2.0)):
        code = O8.encode(np.full(w.size, y), np.full(w.size, 127), w)
        x = O8.e4m3_values()[code]
        assert len(np.unique(x)) == 2 and np.ptp(x) == q
        assert abs(x.mean() - y) <= q * 2.0 ** -20


def test_words_are_uniform_and_differ_by_key():
    n = 1 << 16
    a, b = O8.words(7, 3, n)
    for w in (a, b):
        counts = np.bincount((w >> np.uint64(24)).astype(int), minlength=256)
        # chi-squared over 255 degrees of freedom: mean 255, standard deviation 22.6; six of them
        assert ((counts - n / 256) ** 2 / (n / 256)).sum() < 255 + 6 * 22.6
    for other in (O8.words(8, 3, n), O8.words(7, 4, n), O8.words(7, 3, n, tensor=1), O8.words(7, 3, n, first=1 << 32)):
        same = np.mean(a == other[0])
        assert same < 1e-3
        u, v = (a >> np.uint64(12)) / 2.0 ** 20, (other[0] >> np.uint64(12)) / 2.0 ** 20
        assert abs(np.corrcoef(u, v)[0, 1]) < 6 / np.sqrt(n)
    u, v = (a >> np.uint64(12)) / 2.0 ** 20, (b >> np.uint64(12)) / 2.0 ** 20
    assert abs(np.corrcoef(u, v)[0, 1]) < 6 / np.sqrt(n)


@pytest.mark.parametrize("seed", range(4))
def test_float32_model_is_within_the_bounds_of_the_formulas(seed):
    rng = np.random.default_rng(seed)
    n = 1000 + seed
    spread = np.exp(rng.normal(0, 1.5, n)) * 1e-3
    c, s = O8.pack(rng.normal(0, 1, n) * spread, (rng.uniform(0.2, 1, n) * spread) ** 2)
    p = rng.normal(0, 0.02, n).astype(np.float32)
    g = (rng.normal(0, 1, n) * spread).astype(np.float32)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=7, inv_loss_scale=0.5,
              max_grad_norm=1.0)
    pn, cn, sn = adam8_update(p, c, s, g, 4.0, seed, **hp)
    m0, s0 = O8.decode(c, s, n)
    (p64, m64, v64), (dp, dm, dv) = adam64(p, m0, s0 * s0, g, 4.0, **hp)
    assert (np.abs(pn - p64) <= dp).all()
    root = np.sqrt(v64)
    check_codes("model", cn, sn, n, m64, root, dm, np.sqrt(v64 + dv) - root + U * root, O8.words(seed, 7, n))


def test_second_moment_follows_a_change_of_scale_on_average():
    """Why the step rounds stochastically: with beta2 = 0.999 a block of equal
    gradients keeps its root when rounding to nearest, and follows the exact
    recurrence on average when rounding stochastically."""
    n, beta2 = 3200, 0.999
    g = np.full(n, 0.25)
    g[::32] = 1.0                                          # sets each block's scale
    root = np.sqrt(0.5) * g                                # v at half of its limit
    exact = np.sqrt(0.5 * beta2 ** 100 + (1 - beta2 ** 100)) * g
    for stochastic in (False, True):
        s = root.copy()
        for t in range(100):
            v = beta2 * s * s + (1 - beta2) * g * g
            b = np.repeat(O8.exponent_bytes(np.sqrt(v)), 32)
            code = O8.encode(np.sqrt(v), b, O8.words(1, t, n)[1] if stochastic else None, root=True)
            s = O8.e4m3_values()[code] * np.ldexp(1.0, b - 127)
        mean = (s / exact).mean()
        # 3,200 elements, each off by at most one code (12.5%): the mean's spread is below 0.3%
        assert abs(mean - 1) < 0.02 if stochastic else mean < 0.99
