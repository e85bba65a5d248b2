"""GPU: the calls over a list of matrices: the orthogonalisation against its
definition in float64, the momentum pass and the update bit for bit against
float32 models, skipped steps, streams, graphs, and what they must not touch."""
import math

import numpy as np
import pytest

import matmodel as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def draw(shape, seed, kind="noise", size=1e-3):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape)
    if kind == "spread":                                   # rows, columns and a low-rank part of different size
        r, c = shape[-2:]
        rank = max(1, min(r, c) // 16)
        x += rng.normal(size=shape[:-1] + (rank,)) @ rng.normal(size=shape[:-2] + (rank, c)) / math.sqrt(rank)
        x *= np.exp(0.4 * rng.normal(size=shape[:-1] + (1,))) * np.exp(0.4 * rng.normal(size=shape[:-2] + (1, c)))
    return x * size


def place(x, dtype, offset=0):
    """x on the GPU in this type, `offset` elements into an allocation whose rest
    holds 7, and that allocation."""
    flat = torch.full((x.size + offset + 64,), 7.0, dtype=TYPE[dtype], device="cuda")
    view = flat[offset:offset + x.size].view(x.shape)
    view.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return view, flat


def untouched(flat, offset, n):
    return bool((flat[:offset] == 7).all()) and bool((flat[offset + n:] == 7).all())


def workspace(Z, table, fill=255):
    # bytes 0xff are NaN in every format: nothing may be read before it is written
    return torch.full((max(1, Z.zero_multi_orthogonalize_workspace_bytes(table)),), fill, dtype=torch.uint8, device="cuda")


def orthogonalize(Z, table, **kw):
    Z.zero_multi_orthogonalize(table, workspace(Z, table), **kw)


def bits(x):
    return x.reshape(-1).view(torch.uint8) if x.numel() else torch.empty(0, dtype=torch.uint8, device=x.device)


def check(got, u, out, **kw):
    """One matrix against the definition; u as the kernel saw it."""
    ref, most = M.bound(u.cpu().double().numpy(), out, **kw)
    off = float(np.linalg.norm(got.cpu().double().numpy() - ref))
    assert off <= most, (tuple(got.shape), off, most, float(np.linalg.norm(ref)))


SHAPES = [(1, 1), (1, 2), (2, 1), (2, 2), (1, 1000), (1000, 1), (3, 5), (7, 7), (15, 17), (16, 4096), (4096, 16), (31, 33),
          (32, 32), (33, 65), (63, 64), (64, 64), (65, 64), (64, 65), (100, 1), (127, 300), (128, 128), (128, 1000),
          (129, 128), (129, 131), (255, 257), (256, 256), (257, 256), (300, 700), (331, 881), (881, 331), (512, 512),
          (1023, 1025), (1024, 1024), (1025, 1030), (1030, 2050), (1500, 1100)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_one_matrix(Z, shape):
    for k, (ut, ot, kind) in enumerate((("bf16", "bf16", "noise"), ("f32", "f16", "spread"), ("f16", "bf16", "spread"))):
        u, _ = place(draw(shape, 10 + k, kind, 1.0 if ut == "f16" else 1e-3), ut, offset=k)
        o, flat = place(np.full(shape, 7.0), ot, offset=3 * k)
        before = bits(u).clone()
        orthogonalize(Z, Z.MatrixTable([u], [o]))
        check(o, u, ot)
        assert untouched(flat, 3 * k, u.numel()) and torch.equal(bits(u), before)


def test_lists_batches_and_places_do_not_matter(Z):
    """A list of many shapes, in place, batches among them: each matrix ends as it
    does alone, bit for bit, and what lies between them stays."""
    shapes = [(3, 40, 70), (331, 200), (2, 200, 331), (1, 64, 64), (0, 5), (700, 300), (5, 16, 33), (1040, 1030), (2, 0, 3)]
    flat = torch.full((sum(math.prod(s) + 5 for s in shapes),), 7.0, dtype=torch.bfloat16, device="cuda")
    at, us, gaps = 1, [], []
    for k, s in enumerate(shapes):
        us.append(flat[at:at + math.prod(s)].view(s))
        us[-1].copy_(torch.from_numpy(draw(s, 50 + k, "spread") if math.prod(s) else np.zeros(s)))
        gaps.append(flat[at + math.prod(s):at + math.prod(s) + 4])
        at += math.prod(s) + 5
    alone = []
    for u in us:
        for m in u.reshape(-1, *u.shape[-2:]) if u.numel() else []:
            o = torch.empty(m.shape, dtype=torch.bfloat16, device="cuda")
            orthogonalize(Z, Z.MatrixTable([m.clone()], [o]))
            alone.append(o)
    table = Z.MatrixTable(us)
    orthogonalize(Z, table)
    got = [m for u in us if u.numel() for m in u.reshape(-1, *u.shape[-2:])]
    assert len(got) == len(alone)
    for a, b in zip(got, alone):
        assert torch.equal(bits(a), bits(b)), a.shape
    assert all(bool((g == 7).all()) for g in gaps)


@pytest.mark.parametrize("shape", [(5, 9), (64, 64), (200, 130), (300, 513), (1100, 1030)], ids=lambda s: "x".join(map(str, s)))
def test_sizes_of_values(Z, shape):
    """Scaling U by a power of two changes nothing, up to the ends of the types;
    zero gives zero, whatever eps; a norm below eps divides by eps."""
    x = draw(shape, 3, size=1.0)
    base = None
    for e in (0, 40, -40, 100, -100):
        u, _ = place(x.astype(np.float32) * np.float32(2.0) ** e, "f32")
        o = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        orthogonalize(Z, Z.MatrixTable([u], [o]), eps=0.0)
        if base is None:
            base = o
            check(o, u, "bf16", eps=0.0)
        assert torch.equal(bits(o), bits(base)), e
    u, _ = place(np.zeros(shape), "f32")
    for eps in (0.0, 1e-7, 1e-320, 1e300):
        o = torch.full(shape, 7.0, dtype=torch.float16, device="cuda")
        orthogonalize(Z, Z.MatrixTable([u], [o]), eps=eps)
        assert not o.any()
    u, _ = place(x * 1e-6, "f32")
    o = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    orthogonalize(Z, Z.MatrixTable([u], [o]), eps=0.5)
    check(o, u, "bf16", eps=0.5)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_matrix_that_is_not_finite_becomes_nan_alone(Z, bad):
    for shape in ((20, 30), (200, 140), (300, 520), (1030, 1100)):
        for dt in ("bf16", "f32"):
            x = draw((3,) + shape, 4)
            x[1, shape[0] // 2, shape[1] - 1] = bad
            u, _ = place(x, dt)
            o = torch.empty(u.shape, dtype=torch.bfloat16, device="cuda")
            orthogonalize(Z, Z.MatrixTable([u], [o]))
            assert bool(o[1].isnan().all()), shape
            for k in (0, 2):
                check(o[k], u[k], "bf16")


@pytest.mark.parametrize("n", [1, 2, 3, 6, 8])
def test_steps_and_coefficients(Z, n):
    """Odd and even numbers of steps, coefficients that differ from step to step."""
    coefs = tuple(((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375))[k % 3] for k in range(n))
    for shape in ((30, 20), (140, 150), (300, 700), (1030, 1100)):
        u, _ = place(draw(shape, 5, "spread"), "bf16")
        o = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        orthogonalize(Z, Z.MatrixTable([u], [o]), coefs=coefs)
        check(o, u, "bf16", coefs=coefs)


@pytest.mark.parametrize("n", [7, 12, 32])
@pytest.mark.parametrize("shape", [(2, 2), (16, 16), (30, 300), (64, 64), (500, 50), (128, 128), (128, 2000), (200, 210)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_steps(Z, shape, n):
    """Nothing that a step leaves grows in the next ones: five of the usual steps,
    then ones that converge; all of them the usual ones."""
    after = (1.875, -1.25, 0.375)
    for k, (kind, ut) in enumerate((("noise", "bf16"), ("spread", "f16"))):
        u, _ = place(draw(shape, 40 + k, kind, 1.0), ut)
        for coefs in (M.COEFS[:5] + (after,) * (n - 5), M.COEFS[:1] * n):
            o = torch.empty(shape, dtype=torch.float16, device="cuda")
            orthogonalize(Z, Z.MatrixTable([u], [o]), coefs=coefs)
            if coefs[-1] == after:
                check(o, u, "f16", coefs=coefs)
            else:                                            # no limit, but a band: [0.68, 1.21]
                s = torch.linalg.svdvals(o.cpu().double())
                assert 0.66 < float(s[-1]) <= float(s[0]) < 1.23, s


@pytest.mark.parametrize("n", [5, 7, 12])
@pytest.mark.parametrize("shape", [(4, 4), (16, 16), (30, 300), (300, 60), (128, 300), (200, 210)], ids=lambda s: "x".join(map(str, s)))
def test_rank_three(Z, shape, n):
    """Most singular values are exactly 0: what rounding leaves in their place may
    not grow beyond what the model of the roundings gives."""
    rng = np.random.default_rng(7)
    u, _ = place(rng.integers(-3, 4, (shape[0], 3)) @ rng.integers(-3, 4, (3, shape[1])).astype(float), "bf16")
    o = torch.empty(shape, dtype=torch.float16, device="cuda")
    orthogonalize(Z, Z.MatrixTable([u], [o]), coefs=M.COEFS[:1] * n)
    check(o, u, "f16", coefs=M.COEFS[:1] * n)
    assert float(torch.linalg.svdvals(o.cpu().double())[0]) < 1.23


def test_many_steps_in_place_and_recorded(Z):
    """Steps that take several runs, in the update's place, in batches and in a
    graph: as out of place and alone."""
    shapes = [(3, 20, 300), (4, 500, 40), (2, 128, 260), (90, 90), (150, 140)]
    coefs = M.COEFS[:1] * 12
    us = [place(draw(s, 60 + k, "spread"), "f16")[0] for k, s in enumerate(shapes)]
    alone = []
    for u in us:
        for m in u.reshape(-1, *u.shape[-2:]):
            o = torch.empty(m.shape, dtype=torch.float16, device="cuda")
            orthogonalize(Z, Z.MatrixTable([m.clone()], [o]), coefs=coefs)
            alone.append(o)
    table, kept = Z.MatrixTable(us), [u.clone() for u in us]
    ws = workspace(Z, table)
    Z.zero_multi_orthogonalize(table, ws, coefs)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    for k in range(3):
        got = [m for u in us for m in u.reshape(-1, *u.shape[-2:])]
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, alone)), k
        for u, x in zip(us, kept):
            u.copy_(x)
        if k == 0:
            with torch.cuda.graph(graph):
                Z.zero_multi_orthogonalize(table, ws, coefs)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()


def test_one_step_that_keeps_x(Z):
    """(1, 0, 0) returns U over its norm: X's rounding and the result's remain."""
    u, _ = place(draw((150, 90), 6), "f32")
    o = torch.empty(150, 90, dtype=torch.float16, device="cuda")
    orthogonalize(Z, Z.MatrixTable([u], [o]), coefs=((1.0, 0.0, 0.0),))
    x = u.cpu().double().numpy()
    x /= np.linalg.norm(x)
    # two roundings to fp16, one of them where the result may be subnormal
    assert (np.abs(o.cpu().double().numpy() - x) <= 2 * 2.0 ** -11 * np.abs(x) + 2.0 ** -24).all()


def test_a_skipped_step_writes_nothing(Z):
    shapes = [(40, 50), (300, 200), (1030, 1030)]
    ms = [torch.randn(s, device="cuda") for s in shapes]
    ps = [torch.randn(s, device="cuda") for s in shapes]
    gs = [torch.randn(s, device="cuda").half() for s in shapes]
    us = [torch.randn(s, device="cuda").bfloat16() for s in shapes]
    os_ = [torch.randn(s, device="cuda").bfloat16() for s in shapes]
    outs = [torch.randn(s, device="cuda").half() for s in shapes]
    table = Z.MatrixTable(us, os_, ms, gs, ps, outs)
    before = [bits(x).clone() for x in ms + ps + gs + us + os_ + outs]
    flag = torch.ones(1, dtype=torch.int32, device="cuda")
    sq = torch.ones(1, dtype=torch.float64, device="cuda")
    Z.zero_multi_momentum_step(table, [Z.MuonHyper()], 1.0, 1.0, sq, flag)
    orthogonalize(Z, table, global_overflow=flag)
    Z.zero_multi_muon_update(table, [Z.MuonHyper()], flag)
    assert all(torch.equal(bits(x), b) for x, b in zip(ms + ps + gs + us + os_ + outs, before))
    flag.zero_()
    Z.zero_multi_momentum_step(table, [Z.MuonHyper()], 1.0, 1.0, sq, flag)
    orthogonalize(Z, table, global_overflow=flag)
    Z.zero_multi_muon_update(table, [Z.MuonHyper()], flag)
    for x, b in zip(ms + ps + us + os_ + outs, before[:6] + before[9:]):
        assert not torch.equal(bits(x), b)


# ---------------------------------------------------------------- momentum and update

SIZES = [(1, 1), (3, 5), (16, 16), (17, 15), (1, 257), (64, 64), (100, 333), (2, 31, 33), (0, 4)]


@pytest.mark.parametrize("grad", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("update", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_momentum_bit_for_bit(Z, grad, update, offset):
    hps = [Z.MuonHyper(momentum=0.95), Z.MuonHyper(momentum=0.9, nesterov=False)]
    rows = [(place(draw(s, 20 + k, size=8.0), grad, offset), place(draw(s, 40 + k), "f32", offset),
             place(np.zeros(s), update, offset)) for k, s in enumerate(SIZES)]
    gs, ms, us = ([r[j][0] for r in rows] for j in range(3))
    groups = [k % 2 for k in range(len(SIZES))]
    sq = torch.full((1,), 9.0, dtype=torch.float64, device="cuda")
    inv, clip = 1.0 / 64, 0.75
    factor = np.float32(inv * (clip / (3.0 + 1e-6)))
    want = [M.momentum32(m.cpu().numpy(), g.cpu().float().numpy(), factor, hps[k].momentum, hps[k].nesterov)
            for m, g, k in zip(ms, gs, groups)]
    table = Z.MatrixTable(us, None if update != "f32" else [torch.empty(s, dtype=torch.half, device="cuda") for s in SIZES],
                          ms, gs, groups=groups)
    Z.zero_multi_momentum_step(table, hps, inv, clip, sq)
    for (wm, wu), m, u, r in zip(want, ms, us, rows):
        assert np.array_equal(wm.view(np.int32), m.cpu().numpy().view(np.int32)), m.shape
        assert torch.equal(bits(torch.from_numpy(wu).to(TYPE[update])), bits(u.cpu())), u.shape
        assert all(untouched(flat, offset, v.numel()) for v, flat in r)


@pytest.mark.parametrize("param", ["f16", "bf16", None])
@pytest.mark.parametrize("ortho", ["f16", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_update_bit_for_bit(Z, param, ortho, offset):
    hps = [Z.MuonHyper(lr=0.02, weight_decay=0.1), Z.MuonHyper(lr=0.5)]
    rows = [(place(draw(s, 20 + k, size=0.02), "f32", offset), place(draw(s, 40 + k, size=0.1), ortho, offset),
             place(np.zeros(s), param or "f16", offset)) for k, s in enumerate(SIZES)]
    ps, os_, outs = ([r[j][0] for r in rows] for j in range(3))
    groups, scales = [k % 2 for k in range(len(SIZES))], [0.3 + k for k in range(len(SIZES))]
    want = [M.update32(p.cpu().numpy(), o.cpu().float().numpy(), hps[k].lr, x, hps[k].weight_decay)
            for p, o, k, x in zip(ps, os_, groups, scales)]
    # an entry without a copy among others
    copies = None if param is None else [None if k == 3 else x for k, x in enumerate(outs)]
    Z.zero_multi_muon_update(Z.MatrixTable(None, os_, masters=ps, params_out=copies, scales=scales, groups=groups), hps)
    for k, (w, p, r) in enumerate(zip(want, ps, rows)):
        assert np.array_equal(w.view(np.int32), p.cpu().numpy().view(np.int32)), p.shape
        if param is not None and k != 3:
            assert torch.equal(bits(torch.from_numpy(w).to(TYPE[param])), bits(outs[k].cpu())), p.shape
        else:
            assert not outs[k].any()
        assert all(untouched(flat, offset, v.numel()) for v, flat in r)


def test_momentum_with_a_device_block(Z):
    """The block that the decision forms gives the host's factor."""
    g = torch.randn(90, 70, device="cuda").half()
    scaler = Z.LossScaler(scale=512.0)
    state, sq, flag = Z.StepState(scaler, 0, g.device), torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    norms = Z.TensorTable.of_grads([g])
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(norms), dtype=torch.uint8, device="cuda")
    block = torch.empty(Z.zero_adam_coef_bytes(), dtype=torch.uint8, device="cuda")
    Z.zero_multi_norm_decide_dev(norms, [Z.AdamHyper(max_grad_norm=0.1)], state, sq, flag, block, ws)
    got = []
    for coef in (True, False):
        m, u = torch.ones(90, 70, device="cuda"), torch.empty(90, 70, dtype=torch.bfloat16, device="cuda")
        table = Z.MatrixTable([u], None, [m], [g])
        if coef:
            Z.zero_multi_momentum_step_coef(table, [Z.MuonHyper()], block, sq, flag)
        else:
            Z.zero_multi_momentum_step(table, [Z.MuonHyper()], 1.0 / 512, 0.1, sq, flag)
        got.append((bits(m).clone(), bits(u).clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------- streams, graphs, sizes

def test_other_streams_and_repeats(Z):
    """Two lists at the same time on two streams, each with its workspace: as alone."""
    us = [[torch.from_numpy(draw(s, k + 9)).cuda().bfloat16() for s in ((300, 200), (64, 900), (1030, 1030))] for k in range(2)]
    os_ = [[torch.empty_like(u) for u in x] for x in us]
    tables = [Z.MatrixTable(u, o) for u, o in zip(us, os_)]
    spaces = [workspace(Z, t) for t in tables]
    for t, w in zip(tables, spaces):
        Z.zero_multi_orthogonalize(t, w)
    torch.cuda.synchronize()
    alone = [[bits(o).clone() for o in x] for x in os_]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for x in os_:
            for o in x:
                o.fill_(7.0)
        torch.cuda.synchronize()
        for t, w, s in zip(tables, spaces, streams):
            with torch.cuda.stream(s):
                Z.zero_multi_orthogonalize(t, w)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(o), b) for x, y in zip(os_, alone) for o, b in zip(x, y))


def test_recorded_in_a_graph(Z):
    """Recorded once and replayed on new values, with eager work between."""
    shapes = [(30, 200), (300, 150), (1030, 1040)]
    us = [torch.empty(s, dtype=torch.float32, device="cuda") for s in shapes]
    os_ = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
    table = Z.MatrixTable(us, os_)
    ws = workspace(Z, table)
    for u in us:
        u.normal_()
    Z.zero_multi_orthogonalize(table, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_multi_orthogonalize(table, ws)
    for k in range(3):
        for u in us:
            u.normal_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [bits(o).clone() for o in os_]
        for o in os_:
            o.fill_(7.0)
        Z.zero_multi_orthogonalize(table, ws)
        assert all(torch.equal(bits(o), b) for o, b in zip(os_, got)), k


def test_a_list_in_several_parts(Z):
    """A list beyond one part's workspace, and past 2^32 elements in one batch:
    first, last and middle matrices as alone."""
    batch = 16390
    u = torch.empty(batch, 512, 513, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in range(0, batch, 1024):
        part = u[k:k + 1024]
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen))
    probe = [0, 1, 1023, batch // 2, batch - 2, batch - 1]
    alone = []
    for k in probe:
        o = torch.empty(512, 513, dtype=torch.bfloat16, device="cuda")
        orthogonalize(Z, Z.MatrixTable([u[k].clone()], [o]))
        alone.append(o)
    table = Z.MatrixTable([u])
    assert Z.zero_multi_orthogonalize_workspace_bytes(table) <= 4 << 30
    orthogonalize(Z, table)
    for k, o in zip(probe, alone):
        assert torch.equal(bits(u[k]), bits(o)), k


@pytest.mark.parametrize("shape", [(130, 1 << 21), ((1 << 22) - 3, 5), (70, 1 << 22), (1 << 20, 300)], ids=lambda s: "x".join(map(str, s)))
def test_long_sides(Z, shape):
    """Up to the longest side: against the definition in float64 on the device."""
    u = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    for k in range(0, shape[0], 1 << 16):
        part = u[k:k + (1 << 16)]
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen))
    o = torch.empty_like(u)
    orthogonalize(Z, Z.MatrixTable([u], [o]))
    tall = shape[0] > shape[1]
    x = (u.T if tall else u).double()
    x /= x.norm()
    for a, b, c in M.COEFS:
        g = x @ x.T
        x = (a * torch.eye(len(g), dtype=torch.float64, device="cuda") + b * g + c * (g @ g)) @ x
    off = float(((o.T if tall else o).double() - x).norm() / x.norm())
    # bf16's half step, at most 2^-8 of each value, and twice what the model of the
    # roundings gives where all singular values are alike, as here (1.2e-3)
    assert off <= 2.0 ** -8 + 2 * 1.2e-3, off


def test_device_of_the_table(Z):
    u = torch.zeros(4, 6, dtype=torch.bfloat16, device="cuda")
    table = Z.MatrixTable([u])
    with pytest.raises(ValueError, match="device tensor expected"):
        Z.zero_multi_orthogonalize(table, torch.empty(4096, dtype=torch.uint8))
    with pytest.raises(Z.ZeroShardError, match="lack"):
        Z.zero_multi_muon_update(table, [Z.MuonHyper()])
    with pytest.raises(Z.ZeroShardError, match="workspace"):
        Z.zero_multi_orthogonalize(table, torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="without gradients"):
        table.set_grads([u])
    table.release_grads()
    orthogonalize(Z, table)
