"""Host-side tests of the calls over a list of matrices (no GPU): the table,
every refusal of the library and of the binding before anything is enqueued, and
the models that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import matmodel as M  # noqa: E402
import zero_sharded_mixed_partition_amd as Z  # noqa: E402
from zero_sharded_mixed_partition_amd import _lib as L  # noqa: E402

AL = 1 << 40                        # a plausible, 16-byte aligned device address
STEP = 1 << 24
FIELDS = ("master", "momentum", "grad", "update", "ortho", "param_out")


def matrix(base=AL, rows=30, cols=50, batch=1, **over):
    """A zero_matrix with its buffers 16 MiB apart."""
    t = L.zero_matrix(*[base + k * STEP for k in range(6)], rows, cols, batch, 1.0, L.ZERO_BF16, L.ZERO_BF16, L.ZERO_BF16,
                      L.ZERO_BF16, 0, 0)
    for k, v in over.items():
        setattr(t, k, v)
    return t


def build(matrices, capacity=None):
    lib = L.lib()
    arr = (L.zero_matrix * max(1, len(matrices)))(*matrices)
    size, dev = ctypes.c_size_t(), ctypes.c_size_t()
    st = lib.zero_matrix_table_build(arr, len(matrices), None, 0, ctypes.byref(size), ctypes.byref(dev))
    if st != L.ZERO_ENOSPC:
        return st, None
    buf = ctypes.create_string_buffer(size.value + 16)
    st = lib.zero_matrix_table_build(arr, len(matrices), buf, size.value if capacity is None else capacity,
                                     ctypes.byref(size), ctypes.byref(dev))
    assert dev.value <= size.value
    return st, buf


def hyper(n=1, **over):
    kw = dict(lr=0.1, momentum=0.9, weight_decay=0.0, nesterov=1, reserved=0)
    kw.update(over)
    return (L.zero_muon_params * n)(*[L.zero_muon_params(**kw) for _ in range(n)])


COEFS = (ctypes.c_double * 15)(*[x for step in Z.ORTHO_COEFS for x in step])


def test_table_refusals():
    assert build([matrix()])[0] == L.ZERO_OK
    assert build([])[0] == L.ZERO_OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(batch=-1), dict(grad_dtype=4), dict(update_dtype=0), dict(group=-1),
                dict(group=16), dict(ortho_dtype=L.ZERO_F32), dict(param_dtype=L.ZERO_F32), dict(scale=math.nan),
                dict(scale=math.inf), dict(ortho=AL + 3 * STEP, ortho_dtype=L.ZERO_F16)):
        assert build([matrix(**bad)])[0] == L.ZERO_EINVAL, bad
    for k, name in enumerate(FIELDS):
        assert build([matrix(**{name: AL + k * STEP + 1})])[0] == L.ZERO_EALIGN, name
    for k, name in ((0, "master"), (1, "momentum")):
        assert build([matrix(**{name: AL + k * STEP + 2})])[0] == L.ZERO_EALIGN, name
    assert build([matrix(update=AL + 3 * STEP + 2, update_dtype=L.ZERO_F32)])[0] == L.ZERO_EALIGN
    assert build([matrix(grad=AL + 2 * STEP + 2, grad_dtype=L.ZERO_F32)])[0] == L.ZERO_EALIGN
    for bad in (dict(rows=(1 << 22) + 1), dict(cols=(1 << 22) + 1), dict(rows=1 << 22, cols=1 << 22, batch=1 << 20),
                dict(rows=1 << 22, cols=1 << 22, batch=1 << 62), dict(rows=1 << 22, cols=1 << 22), dict(rows=1, cols=1, batch=1 << 25),
                dict(rows=1 << 21, cols=1 << 20)):
        assert build([matrix(**bad)])[0] == L.ZERO_ERANGE, bad
    assert build([matrix()], capacity=10)[0] == L.ZERO_ENOSPC
    lib, s = L.lib(), ctypes.c_size_t()
    assert lib.zero_matrix_table_build(None, 1, None, 0, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EINVAL
    assert lib.zero_matrix_table_build(None, -1, None, 0, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EINVAL
    assert lib.zero_matrix_table_build(None, 0, None, 0, None, ctypes.byref(s)) == L.ZERO_EINVAL
    odd = ctypes.addressof(ctypes.create_string_buffer(4096)) // 8 * 8 + 4
    assert lib.zero_matrix_table_build(None, 0, odd, 4096, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EALIGN
    assert lib.zero_multi_muon_update(odd, None, hyper(), 1, None, None) == L.ZERO_EALIGN


def test_table_refuses_overlaps():
    a, far = matrix(), AL + (1 << 30)
    assert build([a, a])[0] == L.ZERO_EINVAL                                  # the same matrix twice
    n = 30 * 50
    for over in (dict(master=AL + 4 * n - 4), dict(momentum=AL), dict(update=AL + 4 * STEP), dict(ortho=AL + 5 * STEP + 2),
                 dict(param_out=AL + STEP), dict(grad=AL), dict(grad=AL + 3 * STEP + 2 * n - 2)):
        assert build([a, matrix(far, **over)])[0] == L.ZERO_EINVAL, over
    assert build([a, matrix(far, grad=a.grad)])[0] == L.ZERO_OK                # gradients may be shared
    assert build([a, matrix(far, master=AL + 4 * n)])[0] == L.ZERO_OK          # end to end
    assert build([matrix(ortho=AL + 3 * STEP)])[0] == L.ZERO_OK                # in the update's place
    assert build([matrix(ortho=AL + 3 * STEP + 2)])[0] == L.ZERO_EINVAL        # but nowhere else in it
    assert build([matrix(batch=0), matrix(batch=0)])[0] == L.ZERO_OK           # empty ones have no buffers


def test_calls_need_their_buffers():
    lib, d = L.lib(), AL - (1 << 30)

    def momentum(buf, hp=None, n=1, inv=1.0, clip=0.0, sq=None, ovf=None):
        return lib.zero_multi_momentum_step(buf, d, hyper(n) if hp is None else hp, n, inv, clip, sq, ovf, None)

    def coef(buf, block=AL - STEP, sq=AL - STEP + 256):
        return lib.zero_multi_momentum_step_coef(buf, d, hyper(), 1, block, sq, None, None)

    def ortho(buf, coefs=COEFS, steps=5, eps=1e-7, ovf=None, ws=AL - (1 << 29), room=1 << 28, table=d):
        return lib.zero_multi_orthogonalize(buf, table, coefs, steps, eps, ovf, ws, room, None)

    def update(buf, hp=None, n=1, ovf=None):
        return lib.zero_multi_muon_update(buf, d, hyper(n) if hp is None else hp, n, ovf, None)

    for call, names in ((momentum, ("momentum", "grad", "update")), (coef, ("momentum", "grad", "update")),
                        (ortho, ("update", "ortho")), (update, ("master", "ortho"))):
        for name in names:
            _, buf = build([matrix(), matrix(AL + (1 << 30), **{name: None})])
            assert call(buf) == L.ZERO_EINVAL, (call, name)
            assert b"lack" in lib.zero_last_error()
        junk = ctypes.create_string_buffer(4096)
        assert call(junk) == L.ZERO_EINVAL and call(None) == L.ZERO_EINVAL
    _, buf = build([matrix(group=2)])
    for bad in (dict(lr=-1.0), dict(lr=math.nan), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=math.nan),
                dict(weight_decay=-1.0), dict(weight_decay=math.inf)):
        assert momentum(buf, hyper(3, **bad), 3) == L.ZERO_EINVAL, bad
        assert update(buf, hyper(3, **bad), 3) == L.ZERO_EINVAL, bad
    assert momentum(buf, None, 2) == L.ZERO_EINVAL                              # the table names group 2
    assert update(buf, None, 17) == L.ZERO_EINVAL and update(buf, None, 0) == L.ZERO_EINVAL
    assert lib.zero_multi_muon_update(buf, d, None, 3, None, None) == L.ZERO_EINVAL
    for inv in (0.0, -1.0, math.nan, math.inf):
        assert momentum(buf, None, 3, inv) == L.ZERO_EINVAL
    assert momentum(buf, None, 3, 1.0, math.nan) == L.ZERO_EINVAL
    assert momentum(buf, None, 3, 1.0, math.inf) == L.ZERO_EINVAL
    assert momentum(buf, None, 3, 1.0, 1.0) == L.ZERO_EINVAL                    # clipping needs the norm
    assert momentum(buf, None, 3, 1.0, 1.0, d + 4) == L.ZERO_EALIGN
    assert momentum(buf, None, 3, 1.0, 1.0, AL + 8) == L.ZERO_EINVAL            # the norm in the master
    assert momentum(buf, None, 3, ovf=AL + STEP) == L.ZERO_EINVAL               # the flag in the momentum
    assert update(buf, None, 3, ovf=AL + 4) == L.ZERO_EINVAL and update(buf, None, 3, ovf=d + 2) == L.ZERO_EALIGN
    _, buf = build([matrix()])
    assert coef(buf, block=None) == L.ZERO_EINVAL and coef(buf, sq=None) == L.ZERO_EINVAL
    assert coef(buf, block=AL - STEP + 4) == L.ZERO_EALIGN and coef(buf, block=AL + 64) == L.ZERO_EINVAL
    for table in (None, AL + 4096):
        assert ortho(buf, table=table) == L.ZERO_EINVAL
    assert ortho(buf, table=d + 8) == L.ZERO_EALIGN
    assert ortho(buf, None) == L.ZERO_EINVAL and ortho(buf, steps=0) == L.ZERO_EINVAL and ortho(buf, steps=33) == L.ZERO_EINVAL
    assert ortho(buf, eps=-1.0) == L.ZERO_EINVAL and ortho(buf, eps=math.nan) == L.ZERO_EINVAL
    assert ortho(buf, ws=None) == L.ZERO_EINVAL and ortho(buf, ws=AL - (1 << 29) + 16) == L.ZERO_EALIGN
    need = lib.zero_multi_orthogonalize_workspace_bytes(buf)
    assert need > 0 and ortho(buf, room=need - 1) == L.ZERO_ENOSPC
    assert ortho(buf, ovf=AL + 4 * STEP) == L.ZERO_EINVAL and ortho(buf, ovf=d + 2) == L.ZERO_EALIGN
    for where in (AL - 256, AL + 2 * STEP, AL + 4 * STEP, d):
        assert ortho(buf, ws=where, room=need) == L.ZERO_EINVAL, where
    assert ortho(buf, ws=AL - (1 << 29), ovf=AL - (1 << 29) + need - 4) == L.ZERO_EINVAL
    assert lib.zero_multi_orthogonalize_workspace_bytes(None) == 0
    assert lib.zero_multi_orthogonalize_workspace_bytes(ctypes.create_string_buffer(4096)) == 0


def test_coefficients_that_leave_fp16_are_refused():
    lib, d = L.lib(), AL - (1 << 30)
    _, buf = build([matrix()])

    def status(*steps):
        flat = [x for s in steps for x in s]
        # a workspace too small: what passes the coefficients' check ends there
        return lib.zero_multi_orthogonalize(buf, d, (ctypes.c_double * len(flat))(*flat), len(steps), 1e-7, None, d, 0, None)

    fine = ((1.5, -0.5, 0.0),) * 12, ((3.4445, -4.7750, 2.0315),) * 8, ((8.28721, -23.59588, 17.30038), (4.10706, -2.94785, 0.544843))
    for steps in fine:
        assert status(*steps) == L.ZERO_ENOSPC, steps
    for steps in (((5.0, 0.0, 0.0),), ((2.0, 0.0, 0.0),) * 3, ((1.0, 33.0, -33.0),), ((1.0, 40.0, -40.0),)):
        assert status(*steps) == L.ZERO_ERANGE, steps
    # and those that leave nothing at fp16's small end
    assert status(*((0.9, 0.0, 0.0),) * 26) == L.ZERO_ENOSPC
    for steps in (((0.9, 0.0, 0.0),) * 27, ((0.0, 0.0, 0.0),), ((0.06, 0.0, 0.0),)):
        assert status(*steps) == L.ZERO_ERANGE, steps
    for bad in (math.nan, math.inf):
        assert status((bad, 0.0, 0.0)) == L.ZERO_EINVAL


def test_empty_lists_do_nothing():
    lib = L.lib()
    for entries in ([], [matrix(rows=0)], [matrix(cols=0), matrix(batch=0)]):
        for m in entries:
            for name in FIELDS:
                setattr(m, name, None)
        st, buf = build(entries)
        assert st == L.ZERO_OK
        assert lib.zero_multi_momentum_step(buf, None, hyper(), 1, 1.0, 0.0, None, None, None) == L.ZERO_OK
        assert lib.zero_multi_orthogonalize(buf, None, COEFS, 5, 0.0, None, None, 0, None) == L.ZERO_OK
        assert lib.zero_multi_muon_update(buf, None, hyper(), 1, None, None) == L.ZERO_OK
        assert lib.zero_multi_orthogonalize_workspace_bytes(buf) == 0


def test_workspace_is_bounded():
    """A long list is worked off in parts: the workspace stays near 4 GiB, however
    long the list, unless one matrix alone needs more."""
    lib, n = L.lib(), 4096 * 4096
    def entry(k, **kw):
        return matrix(AL, 4096, 4096, master=None, momentum=None, grad=None, param_out=None, update=AL + 4 * n * k,
                      ortho=AL + 4 * n * k + 2 * n, **kw)
    one = lib.zero_multi_orthogonalize_workspace_bytes(build([entry(0)])[1])
    assert 8 * n <= one <= 8 * n + (1 << 20)
    many = lib.zero_multi_orthogonalize_workspace_bytes(build([entry(k) for k in range(200)])[1])
    assert 1 << 31 < many <= 4 << 30
    wide = build([matrix(AL, 8192, 1 << 19, master=None, momentum=None, grad=None, param_out=None, update=AL,
                         ortho=AL + (1 << 36))])[1]
    assert lib.zero_multi_orthogonalize_workspace_bytes(wide) >= 2 * 2 * 8192 << 19


# ---------------------------------------------------------------- the binding

class Fake:
    """A device tensor as far as the binding's checks can tell."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.bfloat16, addr=AL, contiguous=True):
        self.shape, self.dtype, self._addr, self._contiguous = torch.Size(shape), dtype, addr, contiguous
        self.device = "cuda:0"

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self._contiguous

    def get_device(self):
        return 0

    def data_ptr(self):
        return self._addr


def test_binding_checks_shapes_and_types():
    u = Fake((4, 6))
    with pytest.raises(ValueError, match="expected"):
        Z.MatrixTable()
    with pytest.raises(ValueError, match="orthos has 2"):
        Z.MatrixTable([u], [u, u])
    for shape in ((24,), (2, 2, 2, 3), ()):
        with pytest.raises(ValueError, match="a matrix or a batch"):
            Z.MatrixTable([Fake(shape)])
    with pytest.raises(ValueError, match=r"momentums\[0\]: shape"):
        Z.MatrixTable([u], momentums=[Fake((6, 4), torch.float32)], grads=[u])
    with pytest.raises(ValueError, match=r"masters\[0\]: torch.float32"):
        Z.MatrixTable([u], masters=[Fake((4, 6), torch.float64)])
    with pytest.raises(ValueError, match="contiguous"):
        Z.MatrixTable([Fake((4, 6), contiguous=False)])
    with pytest.raises(ValueError, match="dtype"):
        Z.MatrixTable([Fake((4, 6), torch.float64)])
    with pytest.raises(ValueError, match="device tensor expected|current device"):
        Z.MatrixTable([torch.zeros(4, 6)])
    hp = Z.MuonHyper()
    with pytest.raises(ValueError, match="sets expected"):
        Z.zero_multi_muon_update(None, [])
    with pytest.raises(ValueError, match="sets expected"):
        Z.zero_multi_momentum_step(None, [hp] * 17)
    with pytest.raises(ValueError, match="three numbers"):
        Z.zero_multi_orthogonalize(None, None, coefs=((1.0, 2.0),))


def test_muon_refuses_before_it_allocates():
    with pytest.raises(ValueError, match="empty list"):
        Z.MultiMuon([], [])
    x = torch.zeros(4, 6)
    for kw, why in ((dict(update_dtype=torch.float32), "update_dtype"), (dict(hyper=()), "groups expected"),
                    (dict(hyper=({"beta1": 0.9},)), "unknown"), (dict(groups=[1]), "groups must lie")):
        with pytest.raises(ValueError, match=why):
            Z.MultiMuon([x], [x], **kw)
    with pytest.raises(ValueError, match="differ in their shapes"):
        Z.MultiMuon([x], [torch.zeros(4, 5)])
    with pytest.raises(ValueError, match="adjust"):
        Z.muon_scale((4, 6), "wide")
    assert Z.muon_scale((4, 9), "rms") == pytest.approx(0.6) and Z.muon_scale((8, 2), "spectral") == 2.0
    assert Z.muon_scale((2, 8), "spectral") == 1.0 and Z.muon_scale((2, 8), None) == 1.0
    assert Z.muon_scale((5, 16, 9), "rms") == pytest.approx(0.8)


# ---------------------------------------------------------------- the models

def test_exact_against_singular_values():
    """The iteration acts on the singular values alone."""
    rng = np.random.default_rng(0)
    for shape in ((5, 9), (9, 5), (8, 8)):
        x = rng.normal(size=shape)
        u, s, v = np.linalg.svd(x / np.linalg.norm(x), full_matrices=False)
        for a, b, c in M.COEFS:
            s = a * s + b * s ** 3 + c * s ** 5
        assert np.allclose(M.exact(x), (u * s) @ v, atol=1e-12)
    assert not M.exact(np.zeros((3, 4))).any() and not M.exact(np.zeros((3, 4)), eps=0.0).any()


def test_the_roundings_cost_what_the_header_says():
    rng = np.random.default_rng(1)
    for shape in ((256, 256), (128, 512)):
        x = rng.normal(size=shape)
        ref = M.exact(x)
        off = np.linalg.norm(M.rounded(x) - ref) / np.linalg.norm(ref)
        assert 2.0 ** -12 < off < 2.5e-3, off


def test_fused_model():
    """fma32 rounds once: against integers' exact arithmetic."""
    from fractions import Fraction
    rng = np.random.default_rng(2)
    a, b = rng.normal(size=(2, 2000)).astype(np.float32)
    c = (-a.astype(np.float64) * b * (1 + rng.integers(-2, 3, 2000) * 2.0 ** -24)).astype(np.float32)
    c[::2] = rng.normal(size=1000).astype(np.float32) * np.float32(1e-3)
    got = M.fma32(a, b, c)
    for x, y, z, g in zip(a, b, c, got):
        want = Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))
        lo, hi = np.nextafter(g, np.float32(-np.inf)), np.nextafter(g, np.float32(np.inf))
        err = abs(Fraction(float(g)) - want)
        assert err <= abs(Fraction(float(lo)) - want) and err <= abs(Fraction(float(hi)) - want)
