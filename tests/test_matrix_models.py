"""The models and bounds that the GPU tests of the orthogonalisation's accuracy
compare with (no GPU): what they give, and that a wrong result does not meet them."""
import numpy as np
import pytest

import matmodel as M
import matspectra as S


def off(x, ref):
    return float(np.linalg.norm(x - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("kind", S.KINDS)
@pytest.mark.parametrize("shape", [(16, 16), (30, 300), (500, 50), (64, 64), (127, 300)], ids=lambda s: "x".join(map(str, s)))
def test_short_sides(shape, kind):
    """The model is as near as the header says; without the lower halves the bound is missed."""
    u = S.draw(kind, shape, 1).astype(np.float16).astype(np.float64)
    ref, most = S.bound(u, "f16", M.COEFS)
    assert off(S.short(u, M.COEFS), ref) <= (5e-5 if kind == "noise" else 7e-4)
    assert np.linalg.norm(S.short(u, M.COEFS).astype(np.float16) - ref) <= most < 0.2 * np.linalg.norm(ref)
    assert np.linalg.norm(S.short(u, M.COEFS, low=False).astype(np.float16) - ref) > most


@pytest.mark.parametrize("kind", S.KINDS)
def test_long_sides(kind):
    """Rounding U once more, as a start from U / |U| in fp16 does, costs two to three
    times the error where values fall by k^1.5 and more, and misses the bound."""
    u = S.draw(kind, (200, 210), 1).astype(np.float16).astype(np.float64)
    ref, most = S.bound(u, "f16", M.COEFS)
    now, before = off(S.rounded(u, M.COEFS), ref), off(M.rounded(u, M.COEFS), ref)
    assert now * np.linalg.norm(ref) < most < 0.2 * np.linalg.norm(ref)
    assert now < 1.05 * before
    if kind in ("k1.5", "k2", "rank3"):
        assert before * np.linalg.norm(ref) > most
    for wrong in (np.zeros_like(u), 0.97 * ref) if not kind.startswith("rank") else (np.zeros_like(u),):
        assert np.linalg.norm(wrong - ref) > most


@pytest.mark.parametrize("n", [5, 7, 12])
def test_low_rank(n):
    """Zeros and noise of the right size are not what a low rank determines."""
    u = S.draw("rank3", (64, 90), 2)
    core, most = S.determined(u, 3, M.COEFS[:1] * n)
    p, q = S.directions(u, 3)
    noise = np.random.default_rng(3).normal(size=u.shape)
    noise *= np.sqrt(3) / np.linalg.norm(noise)
    for wrong in (0 * u, noise, u / np.linalg.norm(u)):
        assert np.linalg.norm(p.T @ wrong @ q - core) > 5 * most
    assert most < 0.05 * np.linalg.norm(core) and np.linalg.svd(core, compute_uv=False)[-1] > 0.66
