"""GPU: how far the orthogonalisation is from its definition where singular values
fall or are zero, within bounds that a result of zeros or of noise does not meet."""
import numpy as np
import pytest

import matmodel as M
import matspectra as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SHORT = [(16, 16), (30, 300), (500, 50), (64, 64), (127, 300), (128, 1000)]
LONG = [(129, 200), (200, 210), (300, 140), (512, 512), (520, 1000)]


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def ident(x):
    return "x".join(map(str, x)) if isinstance(x, tuple) else None


def result(Z, x, update, out, coefs):
    """(U as the call sees it, its result), in float64."""
    u = torch.from_numpy(np.ascontiguousarray(x)).to(TYPE[update]).cuda()
    o = torch.empty(u.shape, dtype=TYPE[out], device="cuda")
    table = Z.MatrixTable([u], [o])
    ws = torch.full((Z.zero_multi_orthogonalize_workspace_bytes(table),), 255, dtype=torch.uint8, device="cuda")
    Z.zero_multi_orthogonalize(table, ws, coefs)
    return u.cpu().double().numpy(), o.cpu().double().numpy()


def check(u, got, out, coefs):
    ref, most = S.bound(u, out, coefs)
    norm, off = float(np.linalg.norm(ref)), float(np.linalg.norm(got - ref))
    assert most < 0.2 * norm, "a bound that says nothing"
    assert off <= most, (u.shape, off / norm, most / norm)


@pytest.mark.parametrize("update", ["f16", "f32"])
@pytest.mark.parametrize("kind", S.KINDS)
@pytest.mark.parametrize("shape", SHORT + LONG, ids=ident)
def test_five_steps(Z, shape, kind, update):
    u, got = result(Z, S.draw(kind, shape, 1), update, "f16", M.COEFS)
    check(u, got, "f16", M.COEFS)


# the header's figures for five steps and short sides above 128: 16-bit updates, fp32
STATED = {"noise": (1.2e-3, 1.3e-3), "k1": (2.5e-3, 4.2e-3), "k2": (7.5e-3, 2.1e-2), "rank16": (3.3e-2, 3.4e-2), "rank3": (5e-2, 5e-2)}


@pytest.mark.parametrize("kind", sorted(STATED))
@pytest.mark.parametrize("shape", [(200, 210), (512, 512), (520, 1000), (2048, 1024)], ids=ident)
def test_the_header_says_how_far(Z, shape, kind):
    """A tenth for matrices other than those measured, and the result's own rounding."""
    for k, update in ((0, "f16"), (0, "bf16"), (1, "f32")):
        u, got = result(Z, S.draw(kind, shape, 7), update, "f16", M.COEFS)
        ref = M.exact(u)
        norm = float(np.linalg.norm(ref))
        assert float(np.linalg.norm(got - ref)) <= 1.1 * (STATED[kind][k] * norm + S.stored(ref, "f16")), update


@pytest.mark.parametrize("kind", ["noise", "k2", "rank16"])
@pytest.mark.parametrize("shape", [(64, 300), (200, 210), (512, 512)], ids=ident)
def test_bf16(Z, shape, kind):
    u, got = result(Z, S.draw(kind, shape, 2), "bf16", "bf16", M.COEFS)
    check(u, got, "bf16", M.COEFS)


@pytest.mark.parametrize("kind", ["noise", "k1", "k1.5", "k2", "exp"])
@pytest.mark.parametrize("shape", LONG, ids=ident)
def test_seven_steps(Z, shape, kind):
    coefs = M.COEFS[:1] * 7
    u, got = result(Z, S.draw(kind, shape, 3), "f16", "f16", coefs)
    check(u, got, "f16", coefs)


@pytest.mark.parametrize("n", [5, 7, 12])
@pytest.mark.parametrize("rank", [1, 3, 16])
@pytest.mark.parametrize("shape", [(4, 4), (16, 16), (30, 300), (300, 60), (128, 300)] + LONG, ids=ident)
def test_low_rank_is_orthogonalised(Z, shape, rank, n):
    """Whatever grows in the place of the zeros: between the matrix's own singular
    directions the result is the definition's, and nothing leaves the steps' band."""
    rank = min(rank, min(shape) - 1)
    coefs = M.COEFS[:1] * n
    u, got = result(Z, S.draw(f"rank{rank}", shape, 4), "f16", "f16", coefs)
    core, most = S.determined(u, rank, coefs)
    p, q = S.directions(u, rank)
    off = float(np.linalg.norm(p.T @ got @ q - core))
    assert off <= most < 0.05 * float(np.linalg.norm(core)), (off, most)
    values = np.linalg.svd(got, compute_uv=False)
    assert values[0] < 1.23 and values[rank - 1] > 0.66, values[:rank + 1]


def test_tile_sizes_do_not_matter(Z):
    """The same matrices in lists whose products take tiles of 64, 128 and 256: the
    first step's factor, no power of two, is rounded alike in all of them."""
    us = [torch.from_numpy(np.ascontiguousarray(S.draw("k1", s, 5))).half().cuda() for s in ((300, 200), (512, 640))]
    others = ([], [(1024, 1024)] * 8, [(4096, 4096)] * 4)
    for coefs in (M.COEFS, M.COEFS[:1]):
        got = []
        for shapes in others:
            ins = us + [torch.randn(s, device="cuda").half() for s in shapes]
            outs = [torch.empty_like(u) for u in ins]
            table = Z.MatrixTable(ins, outs)
            ws = torch.full((Z.zero_multi_orthogonalize_workspace_bytes(table),), 255, dtype=torch.uint8, device="cuda")
            Z.zero_multi_orthogonalize(table, ws, coefs)
            got.append([o.view(torch.int16).cpu() for o in outs[:2]])
        assert all(torch.equal(a, b) for one in got[1:] for a, b in zip(one, got[0]))


@pytest.mark.parametrize("power", [-120, -60, -15, 0, 40, 100])
def test_the_start_covers_the_types_range(Z, power):
    """U times a power of two has the same result, and norms on both sides of one."""
    u = torch.from_numpy(S.draw("k2", (200, 210), 6)).half().float().cuda()
    for factor in (1.0, 1.999, 1.001):
        ins = [(u * factor).half().float(), (u * factor).half().float() * 2.0 ** power]
        outs = [torch.empty(u.shape, dtype=torch.float16, device="cuda") for _ in ins]
        table = Z.MatrixTable(ins, outs)
        ws = torch.full((Z.zero_multi_orthogonalize_workspace_bytes(table),), 255, dtype=torch.uint8, device="cuda")
        Z.zero_multi_orthogonalize(table, ws, eps=0.0)
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
        check(ins[0].cpu().double().numpy(), outs[0].cpu().double().numpy(), "f16", M.COEFS)
