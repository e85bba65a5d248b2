"""GPU: the shard's step with 8-bit moments and the conversions, against the
float64 oracle within bounds counted beforehand (adam_bounds), and bit for bit
against the float32 model of the documented operation order."""
import numpy as np
import pytest

import oracle.moments8 as O8
from adam_bounds import U, adam64, assert_within
from f32model8 import adam8_update, check_codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=100, inv_loss_scale=0.5,
          max_grad_norm=1.0)


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def inputs(n, seed, gdt):
    rng = np.random.default_rng(seed)
    spread = np.exp(rng.normal(0, 1.5, n)) * 1e-3
    c, s = O8.pack(rng.normal(0, 0.3, n) * spread, (rng.uniform(0.3, 1.2, n) * spread) ** 2)
    p = rng.normal(0, 0.02, n).astype(np.float32)
    g = torch.from_numpy((rng.normal(0, 1, n) * spread * 2).astype(np.float32)).to(DT[gdt])
    return p, c, s, g


def run(Z, p, c, s, g, pdt, hp, sq=4.0, ovf=0, seed=11, stream=None, **kw):
    P, C, S, G = cuda(p), cuda(c), cuda(s), g.cuda()
    out = None if pdt is None else torch.full((P.numel(),), 7.0, dtype=DT[pdt], device="cuda")
    sq = torch.tensor([sq], dtype=torch.float64, device="cuda")
    ovf = torch.tensor([ovf], dtype=torch.int32, device="cuda")
    Z.zero_shard_adam8_step(P, C, S, G, out, Z.AdamHyper(**hp), sq, ovf, seed=seed, **kw)
    torch.cuda.synchronize()
    return P, C, S, out


def check(name, p, c, s, g, got, hp, sq=4.0, seed=11, model=True):
    n = p.size
    P, C, S, out = got
    P, C, S = P.cpu().numpy(), C.cpu().numpy(), S.cpu().numpy()
    gv = g.float().numpy()
    m0, s0 = O8.decode(c, s, n)
    (p64, m64, v64), (dp, dm, dv) = adam64(p, m0, s0 * s0, gv, sq, **hp)
    assert_within(f"{name} master", P, p64, dp)
    root = np.sqrt(v64)
    check_codes(name, C, S, n, m64, root, dm, np.sqrt(v64 + dv) - root + U * root, O8.words(seed, hp["step"], n))
    if out is not None:
        assert torch.equal(out.cpu(), torch.from_numpy(P).to(out.dtype)), f"{name}: the copy is not the rounded master"
    if model:
        pm, cm, sm = adam8_update(p, c, s, gv, sq, seed, **hp)
        assert np.array_equal(P.view(np.int32), pm.view(np.int32)), f"{name}: master differs from the float32 model"
        assert np.array_equal(C, cm) and np.array_equal(S, sm), f"{name}: codes differ from the float32 model"


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 32, 33, 63, 255, 256, 257, 1021, 8192, 100_003])
@pytest.mark.parametrize("gdt,pdt", [("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", None), ("f32", "f16")])
def test_step(Z, n, gdt, pdt):
    p, c, s, g = inputs(n, n, gdt)
    check(f"{n} {gdt} {pdt}", p, c, s, g, run(Z, p, c, s, g, pdt, HP), HP)


@pytest.mark.parametrize("over", [dict(step=1), dict(beta1=0.0, beta2=0.0, step=3), dict(beta1=0.95, beta2=0.9999),
                                  dict(eps=0.0), dict(weight_decay=0.0, max_grad_norm=0.0), dict(inv_loss_scale=2.0 ** -16),
                                  dict(lr=0.0), dict(step=10 ** 6, eps=1e-3)])
def test_hyperparameters(Z, over):
    hp = dict(HP, **over)
    p, c, s, g = inputs(5003, 3, "bf16")
    check(str(over), p, c, s, g, run(Z, p, c, s, g, "bf16", hp), hp)


def test_from_zero_state(Z):
    """All-zero bytes are moments of zero; elements that never had a gradient
    stay exactly where they are."""
    n = 1003
    p, _, _, g = inputs(n, 5, "bf16")
    g[100:200] = 0
    g[960:] = 0
    c, s = np.zeros(Z.zero_moments8_bytes(n), np.uint8), np.zeros(Z.zero_scales8_bytes(n), np.uint8)
    hp = dict(HP, step=1, weight_decay=0.0)
    got = run(Z, p, c, s, g, "bf16", hp)
    check("zero state", p, c, s, g, got, hp)
    P = got[0].cpu().numpy()
    assert np.array_equal(P[100:200], p[100:200]) and np.array_equal(P[960:], p[960:])


def test_extreme_values(Z):
    """Blocks whose values span more than the codes do, float32's smallest and
    largest finite moments, and gradients that vanish beside their block."""
    n = 32 * 6
    p, c, s, g = inputs(n, 6, "f32")
    rng = np.random.default_rng(6)
    g = torch.from_numpy(np.concatenate([np.ldexp(rng.uniform(0.5, 1, 32), np.arange(32)),
                                         np.ldexp(rng.uniform(0.5, 1, 32), -3 * np.arange(32)),
                                         rng.uniform(1, 2, 32) * 1e-38, rng.uniform(1, 2, 32) * 1e18,
                                         rng.uniform(1, 2, 32) * 1e-22, rng.uniform(-1, 1, 32)]).astype(np.float32))
    c[:] = 0
    hp = dict(HP, inv_loss_scale=1.0, max_grad_norm=0.0)
    got = run(Z, p, c, s, g, "bf16", hp)
    check("extreme", p, c, s, g, got, hp)
    root = O8.decode(got[1].cpu().numpy(), got[2].cpu().numpy(), n)[1]
    v = (1 - 0.999) * g.double().numpy() ** 2
    assert (root[v > 1e-44] > 0).all()                     # a positive second moment never becomes zero


def test_skipped_step_writes_nothing(Z):
    p, c, s, g = inputs(1000, 8, "f16")
    P, C, S, out = run(Z, p, c, s, g, "f16", HP, ovf=1)
    assert np.array_equal(P.cpu().numpy(), p) and np.array_equal(C.cpu().numpy(), c)
    assert np.array_equal(S.cpu().numpy(), s) and (out == 7).all()


def test_nonfinite_moments_are_nan(Z):
    n = 128
    p, c, s, g = inputs(n, 9, "f32")
    g[5], g[70] = float("inf"), float("nan")
    hp = dict(HP, max_grad_norm=0.0)
    P, C, S, _ = run(Z, p, c, s, g, "bf16", hp)
    m, root = O8.decode(C.cpu().numpy(), S.cpu().numpy(), n)
    assert np.isnan(m[[5, 70]]).all() and np.isnan(root[[5, 70]]).all()
    ok = np.ones(n, bool)
    ok[[5, 70]] = False
    keep = ok.copy()
    keep[0:32] = keep[64:96] = False                       # the blocks that hold one are unspecified
    pm, cm, sm = adam8_update(p, c, s, np.where(np.isfinite(g.numpy()), g.numpy(), 0), 4.0, 11, **hp)
    mm, rm = O8.decode(cm, sm, n)
    assert np.array_equal(m[keep], mm[keep]) and np.array_equal(root[keep], rm[keep])
    assert np.array_equal(P.cpu().numpy()[ok], pm[ok])


def test_guard_bytes_stay(Z):
    """Nothing past the last element's quad, block and copy is written."""
    for n in (1, 30, 257, 4097):
        p, c, s, g = inputs(n, n, "bf16")
        bufs = []
        for a in (p, c, s):
            t = torch.from_numpy(np.concatenate([a, np.full(64, 85, a.dtype)])).cuda()
            bufs.append((t, a.size))
        out = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        G = torch.cat([g, torch.full((64,), float("nan"), dtype=g.dtype)]).cuda()
        sq = torch.tensor([4.0], dtype=torch.float64, device="cuda")
        Z.zero_shard_adam8_step(bufs[0][0][:n], bufs[1][0], bufs[2][0], G[:n], out[:n], Z.AdamHyper(**HP), sq, None,
                                seed=11)
        for t, k in bufs:
            assert (t[k:] == 85).all()
        assert (out[n:] == 3).all()
        check(f"guard {n}", p, c, s, g, (bufs[0][0][:n], bufs[1][0][:c.size], bufs[2][0][:s.size], out[:n]), HP)


def test_device_coefficients_equal_host_ones(Z):
    p, c, s, g = inputs(10_007, 12, "bf16")
    want = run(Z, p, c, s, g, "bf16", HP)
    P, C, S, G = cuda(p), cuda(c), cuda(s), g.cuda()
    out = torch.empty(P.numel(), dtype=torch.bfloat16, device="cuda")
    blk = torch.empty(Z.zero_adam_coef_bytes(), dtype=torch.uint8)
    Z.zero_adam_prepare(Z.AdamHyper(**HP), blk)
    sq = torch.tensor([4.0], dtype=torch.float64, device="cuda")
    t = torch.tensor([HP["step"]], dtype=torch.int64, device="cuda")
    Z.zero_shard_adam8_step_coef(P, C, S, G, out, blk.cuda(), t, sq, None, seed=11)
    for a, b in zip((P, C, S, out), want):
        assert torch.equal(a, b)


def test_seed_and_step_change_the_rounding_only(Z):
    p, c, s, g = inputs(4096, 13, "bf16")
    a = run(Z, p, c, s, g, "bf16", HP, seed=1)
    b = run(Z, p, c, s, g, "bf16", HP, seed=2)
    d = run(Z, p, c, s, g, "bf16", HP, seed=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])       # master and scales come before the rounding
    assert not torch.equal(a[1], b[1])
    assert torch.equal(a[1], d[1])


def test_rounding_is_unbiased_over_seeds(Z):
    """The stored moments' mean over 200 seeds is within six standard errors
    (of a rounding between two codes one step apart: at most half a step) of
    the values before rounding."""
    n, seeds = 256, 200
    p, c, s, g = inputs(n, 14, "f32")
    m0, s0 = O8.decode(c, s, n)
    (_, m64, v64), _ = adam64(p, m0, s0 * s0, g.numpy(), 4.0, **HP)
    total = np.zeros((2, n))
    for k in range(seeds):
        _, C, S, _ = run(Z, p, c, s, g, None, HP, seed=k)
        total += np.stack(O8.decode(C.cpu().numpy(), S.cpu().numpy(), n))
    b = S.cpu().numpy().reshape(-1, 2).T.astype(int)
    for k, x in enumerate((m64, np.sqrt(v64))):
        unit = np.ldexp(1.0, np.repeat(b[k] - 127, 32))
        _, e = np.frexp(np.abs(x) / unit)
        q = np.ldexp(unit, np.maximum(e - 1, -6) - 3)
        keep = np.abs(x) >= unit * 2.0 ** -9 if k else np.ones(n, bool)   # below it the root is raised
        off = np.abs(total[k] / seeds - x)
        assert (off <= 6 * 0.5 * q / np.sqrt(seeds) + 1e-6 * np.abs(x))[keep].all()


@pytest.mark.parametrize("n", [1, 3, 4, 31, 33, 256, 1000, 100_003])
def test_pack_and_unpack(Z, n):
    rng = np.random.default_rng(n)
    spread = np.exp(rng.normal(0, 2, n)) * 1e-3
    m = (rng.normal(0, 1, n) * spread).astype(np.float32)
    v = (rng.uniform(0, 1, n) * spread ** 2).astype(np.float32)
    m[:: 7] = 0
    v[::11] = 0
    C = torch.full((Z.zero_moments8_bytes(n) + 8,), 9, dtype=torch.uint8, device="cuda")
    S = torch.full((Z.zero_scales8_bytes(n) + 8,), 9, dtype=torch.uint8, device="cuda")
    Z.zero_moments8_pack(C, S, cuda(m), cuda(v))
    # the root is rounded to float32 before its code is
    root = np.sqrt(v)
    b = O8.exponent_bytes(root.astype(np.float64))
    want_c = O8.join(O8.encode(m, np.repeat(O8.exponent_bytes(m.astype(np.float64)), 32)[:n]),
                     O8.encode(root, np.repeat(b, 32)[:n], root=True), O8.exponent_bytes(m.astype(np.float64)), b)
    assert np.array_equal(C.cpu().numpy()[:-8], want_c[0]) and np.array_equal(S.cpu().numpy()[:-8], want_c[1])
    assert (C[-8:] == 9).all() and (S[-8:] == 9).all()
    M, V = torch.full((n + 4,), 5.0, device="cuda"), torch.full((n + 4,), 5.0, device="cuda")
    Z.zero_moments8_unpack(M[:n], V[:n], C, S)
    dm, ds = O8.decode(want_c[0], want_c[1], n)
    assert np.array_equal(M[:n].cpu().numpy(), dm.astype(np.float32))
    assert np.array_equal(V[:n].cpu().numpy(), (ds * ds).astype(np.float32))
    assert (M[n:] == 5).all() and (V[n:] == 5).all()


def test_unpacked_codes_pack_to_themselves(Z):
    """Codes are numbers of the format: going to fp32 and back changes nothing
    where the block's largest code is below 256 (there the exponent moves)."""
    n = 4096
    _, c, s, _ = inputs(n, 15, "f32")
    M, V = _unpack(Z, cuda(c), cuda(s), n)
    C, S = torch.empty_like(cuda(c)), torch.empty_like(cuda(s))
    Z.zero_moments8_pack(C, S, M, V)
    codes, _ = O8.split(c, s, n)
    top = np.abs(O8.e4m3_values()[codes]).reshape(2, -1, 32).max(2)
    keep = torch.from_numpy(np.repeat(top < 256, 32, axis=1)).cuda()
    assert keep.float().mean() > 0.5
    assert torch.equal(torch.stack([M, V])[keep], torch.stack(_unpack(Z, C, S, n))[keep])


def _unpack(Z, C, S, n):
    M, V = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    Z.zero_moments8_unpack(M, V, C, S)
    return M, V


def test_empty_shard_and_other_stream(Z):
    e = torch.empty(0, device="cuda")
    b = torch.empty(0, dtype=torch.uint8, device="cuda")
    Z.zero_shard_adam8_step(e, b, b, e.half(), None, Z.AdamHyper(step=1))
    Z.zero_moments8_pack(b, b, e, e)
    Z.zero_moments8_unpack(e, e, b, b)
    p, c, s, g = inputs(50_001, 16, "f16")
    want = run(Z, p, c, s, g, "f16", HP)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(Z, p, c, s, g, "f16", HP)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
