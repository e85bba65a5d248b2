"""GPU: the norm pass and the update over a list of tensors.  Every tensor of a
list ends bit for bit as the shard's own calls leave it (the 32-bit update) or
as the float32 model says (8 bits), and within bounds counted beforehand of the
float64 formulas; the norms against exact sums."""
import math

import numpy as np
import pytest

import oracle
import oracle.moments8 as O8
from adam_bounds import U, adam64, assert_within
from f32model import adam_update
from f32model8 import adam8_update, check_codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GROUPS = [dict(lr=1e-3, weight_decay=0.1), dict(lr=1e-3, weight_decay=0.0), dict(lr=2e-4, weight_decay=0.3, beta2=0.95)]
COMMON = dict(beta1=0.9, beta2=0.999, eps=1e-8, step=100, inv_loss_scale=0.5, max_grad_norm=1.0)
HPS = [dict(COMMON, **g) for g in GROUPS]
SQ = 4.0


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def scalar(x, dtype):
    return torch.tensor([x], dtype=dtype, device="cuda")


class List:
    """Host inputs of a list and its device buffers.  gap: elements between
    the tensors of each flat buffer (all kinds of alignment), None: separate
    allocations.  Guard values stand before, between and behind."""

    def __init__(self, Z, sizes, seed, gdts, pdts, bits=32, gap=None, groups=None):
        rng = np.random.default_rng(seed)
        self.bits, self.sizes = bits, sizes
        k = len(sizes)
        self.gdt = [gdts[i % len(gdts)] for i in range(k)]
        self.pdt = [pdts[i % len(pdts)] for i in range(k)]
        self.groups = groups if groups is not None else [i % 3 for i in range(k)]
        self.p, self.g, self.a, self.b = [], [], [], []
        for i, n in enumerate(sizes):
            spread = np.exp(rng.normal(0, 1.5, n)) * 1e-3
            m, v = rng.normal(0, 0.3, n) * spread, (rng.uniform(0.3, 1.2, n) * spread) ** 2
            self.p.append(rng.normal(0, 0.02, n).astype(np.float32))
            self.g.append(torch.from_numpy((rng.normal(0, 1, n) * spread * 2).astype(np.float32)).to(DT[self.gdt[i]]))
            if bits == 8:
                c, s = O8.pack(m, v)
                self.a.append(c)
                self.b.append(s)
            else:
                self.a.append(m.astype(np.float32))
                self.b.append(v.astype(np.float32))
        dev = lambda cols, gap: self._place(cols, gap)  # noqa: E731
        self.P, self.A, self.B = dev(self.p, gap), dev(self.a, gap if bits == 32 else None), dev(self.b, None if bits == 8 else gap)
        self.G = dev([g for g in self.g], gap)
        self.O = dev([None if d is None else torch.full((n,), 7.0, dtype=DT[d]) for d, n in zip(self.pdt, sizes)], gap)
        self.table = Z.TensorTable(self.P, self.A, self.B, self.G, self.O, groups=self.groups, state_bits=bits)

    def _place(self, cols, gap):
        out = []
        flats = {}
        for x in cols:
            if x is None:
                out.append(None)
                continue
            t = torch.from_numpy(x) if isinstance(x, np.ndarray) else x
            if gap is None:
                # room for 8 guard elements behind
                buf = torch.full((t.numel() + 8,), 85, dtype=t.dtype, device="cuda")
                buf[:t.numel()] = t
                out.append(buf[:t.numel()])
                self.guards = getattr(self, "guards", []) + [buf[t.numel():]]
            else:
                total = sum(y.size if isinstance(y, np.ndarray) else y.numel() for y in cols if y is not None)
                flat, at = flats.setdefault(t.dtype, (torch.full((total + gap * (len(cols) + 1),), 85, dtype=t.dtype,
                                                                 device="cuda"), [gap]))
                flat[at[0]:at[0] + t.numel()] = t
                out.append(flat[at[0]:at[0] + t.numel()])
                if gap:
                    self.guards = getattr(self, "guards", []) + [flat[at[0] - gap:at[0]],
                                                                 flat[at[0] + t.numel():at[0] + t.numel() + gap]]
                at[0] += t.numel() + gap
        return out

    def step(self, Z, hps=HPS, seed=11, sq=SQ, ovf=0, table=None):
        Z.zero_multi_adam_step(self.table if table is None else table, [Z.AdamHyper(**h) for h in hps],
                               scalar(sq, torch.float64), scalar(ovf, torch.int32), seed=seed)
        torch.cuda.synchronize()

    def check(self, hps=HPS, seed=11, sq=SQ):
        for i, n in enumerate(self.sizes):
            hp, name = hps[self.groups[i]], f"tensor {i} ({n}, {self.gdt[i]}, {self.pdt[i]})"
            gv = self.g[i].float().numpy()
            P, A, B = (x.cpu().numpy() for x in (self.P[i], self.A[i], self.B[i]))
            if self.bits == 8:
                m0, s0 = O8.decode(self.a[i], self.b[i], n)
                v0 = s0 * s0
                want = adam8_update(self.p[i], self.a[i], self.b[i], gv, sq, seed, tensor=i, **hp)
            else:
                m0, v0 = self.a[i], self.b[i]
                want = adam_update(self.p[i], m0, v0, gv, sq, **hp)
            for what, x, y in zip(("master", "exp_avg", "exp_avg_sq"), (P, A, B), want):
                assert np.array_equal(x.view(np.uint8), np.asarray(y).view(np.uint8)), f"{name}: {what} differs from the model"
            (p64, m64, v64), (dp, dm, dv) = adam64(self.p[i], m0, v0, gv, sq, **hp)
            assert_within(f"{name} master", P, p64, dp)
            if self.bits == 8:
                root = np.sqrt(v64)
                check_codes(name, A, B, n, m64, root, dm, np.sqrt(v64 + dv) - root + U * root,
                            O8.words(seed, hp["step"], n, i))
            else:
                assert_within(f"{name} exp_avg", A, m64, dm)
                assert_within(f"{name} exp_avg_sq", B, v64, dv)
            if self.O[i] is not None:
                assert torch.equal(self.O[i].cpu(), torch.from_numpy(P).to(self.O[i].dtype)), f"{name}: copy"
        self.check_guards()

    def check_guards(self):
        for x in getattr(self, "guards", []):
            assert (x == 85).all()

    def unchanged(self):
        for i in range(len(self.sizes)):
            for t, x in ((self.P, self.p), (self.A, self.a), (self.B, self.b)):
                assert np.array_equal(t[i].cpu().numpy(), x[i])
            if self.O[i] is not None:
                assert (self.O[i] == 7).all()


SIZES = [1, 0, 5, 255, 256, 257, 8191, 8192, 8193, 3, 20000, 0, 64, 100_003]
MIXED = dict(gdts=["bf16", "f32", "f16"], pdts=["bf16", None, "f16", "bf16"])


@pytest.mark.parametrize("gap", [None, 0, 1, 3, 8])
def test_update_32(Z, gap):
    x = List(Z, SIZES, 1, gap=gap, **MIXED)
    x.step(Z)
    x.check()


@pytest.mark.parametrize("gap", [None, 0, 1, 3, 8])
def test_update_8(Z, gap):
    x = List(Z, SIZES, 2, bits=8, gap=gap, **MIXED)
    x.step(Z)
    x.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_types(Z, bits):
    """Every pair of gradient and copy types."""
    sizes = [300, 5] * 9
    gd, pd = ["f16", "bf16", "f32"], ["f16", "bf16", None]
    x = List(Z, sizes, 3, gdts=[gd[i // 3 % 3] for i in range(18)], pdts=[pd[i % 3] for i in range(18)], bits=bits)
    assert len({(a, b) for a, b in zip(x.gdt, x.pdt)}) == 9
    x.step(Z)
    x.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_skip_and_empty(Z, bits):
    x = List(Z, SIZES, 4, bits=bits, **MIXED)
    x.step(Z, ovf=1)
    x.unchanged()
    for t in (Z.TensorTable([], [], [], [], state_bits=bits), List(Z, [0, 0], 5, bits=bits, **MIXED).table):
        Z.zero_multi_adam_step(t, [Z.AdamHyper(**h) for h in HPS], scalar(SQ, torch.float64))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_of_one_is_the_shard(Z, bits):
    n = 70_001
    x = List(Z, [n], 6, gdts=["bf16"], pdts=["bf16"], bits=bits)
    P, A, B, O = (torch.empty_like(t[0]).copy_(t[0]) for t in (x.P, x.A, x.B, x.O))
    hp, sq = Z.AdamHyper(**HPS[0]), scalar(SQ, torch.float64)
    if bits == 8:
        Z.zero_shard_adam8_step(P, A, B, x.G[0], O, hp, sq, None, seed=11)
    else:
        Z.zero_shard_adam_step(P, A, B, x.G[0], O, hp, sq, None)
    x.step(Z)
    for a, b in ((P, x.P), (A, x.A), (B, x.B), (O, x.O)):
        assert torch.equal(a, b[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_sixteen_groups(Z, bits):
    rng = np.random.default_rng(7)
    sizes = [int(n) for n in rng.integers(0, 700, 1500)]
    hps = [dict(COMMON, lr=1e-4 * (g + 1), weight_decay=0.01 * g, step=1 + 7 * g) for g in range(16)]
    x = List(Z, sizes, 7, bits=bits, groups=[int(g) for g in rng.integers(0, 16, 1500)], **MIXED)
    x.step(Z, hps)
    x.check(hps)


@pytest.mark.parametrize("bits", [32, 8])
def test_device_coefficients(Z, bits):
    x, y = (List(Z, SIZES, 8, bits=bits, **MIXED) for _ in range(2))
    x.step(Z)
    nb = Z.zero_adam_coef_bytes()
    blk = torch.empty(3 * nb, dtype=torch.uint8)
    for i, h in enumerate(HPS):
        Z.zero_adam_prepare(Z.AdamHyper(**h), blk[i * nb:(i + 1) * nb])
    Z.zero_multi_adam_step_coef(y.table, blk.cuda(), 3, scalar(SQ, torch.float64), None,
                                scalar(100, torch.int64) if bits == 8 else None, seed=11)
    for a, b in zip(x.P + x.A + x.B, y.P + y.A + y.B):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- the norm pass

def norm(Z, grads, inv=1.0, per=True, table=None):
    t = Z.TensorTable.of_grads(grads) if table is None else table
    nb = Z.zero_multi_norm_workspace_bytes(t)
    ws = torch.full((nb + 64,), 255, dtype=torch.uint8, device="cuda")        # NaN everywhere
    sq, ov = scalar(-1.0, torch.float64), scalar(-1, torch.int32)
    out = torch.full((t.n_tensors + 1,), -1.0, dtype=torch.float64, device="cuda")
    Z.zero_multi_unscale_norm_overflow(t, inv, sq, ov, ws[:nb], out[:t.n_tensors] if per else None)
    torch.cuda.synchronize()
    assert (ws[nb:] == 255).all() and out[t.n_tensors] == -1
    return sq.item(), int(ov.item()), out[:t.n_tensors].cpu().numpy()


def grads_of(sizes, seed, dts=("bf16", "f32", "f16"), offset=0):
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.from_numpy((rng.normal(0, 1, n) * 10.0 ** rng.uniform(-4, 1)).astype(np.float32)).to(DT[dts[i % len(dts)]])
        buf = torch.full((n + offset + 8,), float("nan"), dtype=t.dtype, device="cuda")
        buf[offset:offset + n] = t
        out.append(buf[offset:offset + n])
    return out


def exact(grads, inv):
    """Exact sums of squares (float64 squares of at most 24-bit values are exact), rounded once."""
    return [math.fsum((g.double().cpu().numpy() ** 2).tolist()) * inv * inv for g in grads]


def check_norm(Z, grads, inv):
    sq, ov, per = norm(Z, grads, inv)
    want = exact(grads, inv)
    # sums of n positive terms in float64: every partial sum is off by at most
    # the depth of the additions (here below 400) times 2^-53, and the factor
    # inv^2 (rounded once) and its product by 2 more
    rel = 402 * 2.0 ** -53
    assert ov == 0
    for i, w in enumerate(want):
        assert abs(per[i] - w) <= rel * w, (i, per[i], w)
    total = math.fsum(want)
    assert abs(sq - total) <= 2 * rel * total
    assert norm(Z, grads, inv, per=False)[0] == sq
    again = norm(Z, grads, inv)
    assert again[0] == sq and np.array_equal(again[2], per)


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_of_a_mixed_list(Z, offset):
    check_norm(Z, grads_of(SIZES, 20, offset=offset), 1.0 / 1024)


@pytest.mark.parametrize("sizes", [[1], [0], [], [8192 * 3], [8192] * 5, [8193, 1, 8191], [100] * 3000,
                                   [8192 * 1100 + 5, 7, 8192 * 40], [7, 8192 * 1024, 9], [3] * 1023 + [20000]])
def test_norm_layouts(Z, sizes):
    """Fewer chunks than blocks, exactly as many, more; tensors that end with a
    block's run and ones that span many blocks."""
    check_norm(Z, grads_of(sizes, 21, dts=("bf16", "f16")), 0.25)


@pytest.mark.parametrize("where", [0, 1, -1, 12345])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_norm_flag(Z, where, value, dt):
    grads = grads_of([5, 20_001, 8192, 31], 22, dts=(dt,))
    clean = norm(Z, grads)
    for k in range(4):
        n = grads[k].numel()
        g = [x.clone() for x in grads]
        g[k][where % n] = value
        sq, ov, per = norm(Z, g)
        assert ov == 1
        assert math.isnan(sq) if math.isnan(value) else sq == math.inf
        assert [i for i in range(4) if not math.isfinite(per[i])] == [k]
        assert all(per[i] == clean[2][i] for i in range(4) if i != k)


def test_norm_of_huge_finite_values_is_no_overflow(Z):
    g = torch.full((1000,), 3e38, dtype=torch.bfloat16, device="cuda")
    sq, ov, _ = norm(Z, [g, torch.full((9,), 65504.0, dtype=torch.float16, device="cuda")])
    assert ov == 0 and sq > 1e79


def test_shared_gradients(Z):
    g = grads_of([5000], 23)[0]
    one, two = norm(Z, [g]), norm(Z, [g, g])
    assert two[2][0] == two[2][1] == one[2][0]
    assert abs(two[0] - 2 * one[0]) <= 4 * 2.0 ** -53 * two[0]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("bits", [32, 8])
def test_whole_steps_on_the_device(Z, bits):
    """Norm, decision and update over a list, three steps without the host: the
    middle one overflows.  Against the host-scaled calls, bit for bit."""
    x, y = (List(Z, [300, 9000, 77], 30, gdts=["f16"], pdts=["f16"], bits=bits) for _ in range(2))
    hps = [Z.AdamHyper(**{k: v for k, v in h.items() if k != "step"}) for h in HPS]
    scaler = Z.LossScaler(scale=1024.0, growth_interval=2)
    st = Z.StepState(Z.LossScaler(scale=1024.0, growth_interval=2))
    d_step = st.tensor.view(torch.int64)[6:7]                 # zero_step_state.applied, after the 48-byte scaler
    sq, ov = scalar(0.0, torch.float64), scalar(0, torch.int32)
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(x.table), dtype=torch.uint8, device="cuda")
    coefs = torch.empty(3 * Z.zero_adam_coef_bytes(), dtype=torch.uint8, device="cuda")
    per = torch.empty(3, dtype=torch.float64, device="cuda")
    applied = 0
    for step in range(4):
        for L in (x, y):
            torch.manual_seed(step)
            for g in L.G:
                g.copy_(torch.randn(g.numel()) * 0.5)
            if step == 1:
                L.G[1][5] = float("inf")
        Z.zero_multi_norm_decide_dev(x.table, hps, st, sq, ov, coefs, ws, per)
        Z.zero_multi_adam_step_coef(x.table, coefs, 3, sq, ov, d_step if bits == 8 else None, seed=3)
        dev_per, dev_sq = per.clone(), sq.clone()
        inv = 1.0 / scaler.scale
        Z.zero_multi_unscale_norm_overflow(y.table, inv, sq, ov, ws, per)
        assert torch.equal(sq.view(torch.int64), dev_sq.view(torch.int64)) and torch.equal(
            per.view(torch.int64), dev_per.view(torch.int64))
        Z.zero_multi_adam_step(y.table, [Z.AdamHyper(**dict(h, step=applied + 1, inv_loss_scale=inv)) for h in HPS],
                               sq, ov, seed=3)
        if not Z.zero_loss_scaler_update(scaler, bool(ov.item())):
            applied += 1
        now = st.read()
        assert now.applied == applied and now.scaler.scale == scaler.scale and now.last_overflow == int(step == 1)
    assert applied == 3
    for a, b in zip(x.P + x.A + x.B + x.O, y.P + y.A + y.B + y.O):
        assert torch.equal(a, b)


def test_decision_alone_equals_the_folded_one(Z):
    grads = grads_of([1000, 50], 31, dts=("f16",))
    t = Z.TensorTable.of_grads(grads)
    hps = [Z.AdamHyper(**{k: v for k, v in h.items() if k != "step"}) for h in HPS]
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(t), dtype=torch.uint8, device="cuda")
    for unscaled in (False, True):
        out = []
        for folded in (True, False):
            st = Z.StepState(Z.LossScaler(scale=64.0))
            sq, ov = scalar(0.0, torch.float64), scalar(0, torch.int32)
            coefs = torch.zeros(3 * Z.zero_adam_coef_bytes(), dtype=torch.uint8, device="cuda")
            if folded:
                Z.zero_multi_norm_decide_dev(t, hps, st, sq, ov, coefs, ws, unscaled=unscaled)
            else:
                Z.zero_multi_unscale_norm_overflow_dev(t, st, sq, ov, ws, unscaled=unscaled)
                Z.zero_multi_decide_dev(hps, st, ov, coefs, unscaled=unscaled)
            out.append((sq, ov, coefs, st.tensor))
        for a, b in zip(*out):
            assert torch.equal(a, b)
        blk = torch.empty(Z.zero_adam_coef_bytes(), dtype=torch.uint8)
        Z.zero_adam_prepare(Z.AdamHyper(**dict(HPS[2], step=1, inv_loss_scale=1.0 if unscaled else 1.0 / 64.0)), blk)
        assert torch.equal(out[0][2][-blk.numel():].cpu(), blk)
        want = math.fsum(exact(grads, 1.0 if unscaled else 1.0 / 64.0))
        assert abs(out[0][0].item() - want) <= 804 * 2.0 ** -53 * want


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_replay(Z, bits):
    """Norm, decision and update in a captured graph, replayed with the same
    program's eager steps on another list and synchronizations between; and two
    graphs that share a workspace, replayed in turn."""
    lists = [List(Z, [300, 9000, 8192, 77], 40 + k, gdts=["bf16"], pdts=["bf16"], bits=bits) for k in (0, 0, 1, 1)]
    hps = [Z.AdamHyper(**{k: v for k, v in h.items() if k != "step"}) for h in HPS]
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(lists[0].table), dtype=torch.uint8, device="cuda")
    own = []
    for x in lists:
        st = Z.StepState(Z.LossScaler.static(1.0))
        own.append((st, scalar(0.0, torch.float64), scalar(0, torch.int32),
                    torch.empty(3 * Z.zero_adam_coef_bytes(), dtype=torch.uint8, device="cuda"),
                    st.tensor.view(torch.int64)[6:7]))

    def step(i):
        st, sq, ov, coefs, t = own[i]
        Z.zero_multi_norm_decide_dev(lists[i].table, hps, st, sq, ov, coefs, ws)
        Z.zero_multi_adam_step_coef(lists[i].table, coefs, 3, sq, ov, t if bits == 8 else None, seed=5)

    graphs = []
    for i in (0, 2):                                          # captured: nothing runs yet
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i)
        graphs.append(g)
    for _ in range(4):
        graphs[0].replay()
        graphs[1].replay()
        step(1)
        torch.cuda.synchronize()
        step(3)
        torch.cuda.synchronize()
        for i in (0, 2):
            a, b = lists[i], lists[i + 1]
            for u, v in zip(a.P + a.A + a.B + a.O, b.P + b.A + b.B + b.O):
                assert torch.equal(u, v)
    assert own[0][0].read().applied == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_table_with_moved_gradients(Z, bits):
    x, y = (List(Z, [300, 9000], 50, gdts=["bf16"], pdts=["bf16"], bits=bits) for _ in range(2))
    moved = [g.clone() for g in x.G]
    for g in x.G:
        g.fill_(float("nan"))
    x.table.set_grads(moved)
    x.step(Z)
    y.step(Z)
    for a, b in zip(x.P + x.A, y.P + y.A):
        assert torch.equal(a, b)
    other = [g.clone() for g in y.G]
    with pytest.raises(RuntimeError, match="graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            x.table.set_grads(other)


def test_another_stream(Z):
    x, y = (List(Z, SIZES, 60, bits=8, **MIXED) for _ in range(2))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        x.step(Z)
    y.step(Z)
    for a, b in zip(x.P + x.A, y.P + y.A):
        assert torch.equal(a, b)


def test_a_replaced_table_outlives_its_readers_on_another_stream(Z):
    """The memory of the device copy that a stream still has to read is not
    handed out again when the gradients move."""
    x, y = (List(Z, SIZES, 62, bits=8, **MIXED) for _ in range(2))
    moved = [g.clone() for g in x.G]
    big, sq = torch.empty(1 << 28, device="cuda"), scalar(SQ, torch.float64)
    torch.cuda.synchronize()
    old, st = x.table.device.data_ptr(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(100):                             # 17 ms or more of writes before the step's reads
            big.zero_()
        Z.zero_multi_adam_step(x.table, [Z.AdamHyper(**h) for h in HPS], sq, seed=11)
    x.table.set_grads(moved)
    again = [torch.empty_like(x.table.device) for _ in range(4)]
    if not st.query():                                   # else there is nothing to show
        assert old not in [t.data_ptr() for t in again]
    torch.cuda.synchronize()
    y.step(Z)
    for a, b in zip(x.P + x.A, y.P + y.A):
        assert torch.equal(a, b)


def test_norm_matches_the_shard_pass(Z):
    """One tensor: the same exact squares as the shard's norm pass, against
    the oracle's exact sum."""
    g = grads_of([1_000_003], 61, dts=("f16",))[0]
    want, _ = oracle.shard_sqnorm_overflow(g.view(torch.int16).cpu().numpy().view(np.uint16), "f16", 0.5)
    sq, ov, per = norm(Z, [g], 0.5)
    assert ov == 0 and abs(sq - want) <= 402 * 2.0 ** -53 * want and per[0] == sq
