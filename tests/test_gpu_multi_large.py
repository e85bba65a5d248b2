"""GPU: the 8-bit and list calls past 32-bit element counts, and past one
launch's workgroups (2^34 elements), where every workgroup takes a second
task.  Everything is zero but a few places whose results are checked against
the float32 model; the rest has to stay zero."""
import math

import numpy as np
import pytest

import oracle.moments8 as O8
from f32model import adam_update
from f32model8 import adam8_update

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=3, inv_loss_scale=1.0, max_grad_norm=0.0)


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    free, _ = torch.cuda.mem_get_info()
    if free < 200e9:
        pytest.skip("needs about 150 GB of free device memory")
    yield Z
    torch.cuda.empty_cache()


def places(n):
    """(begin, end) of a few runs, at multiples of 32."""
    spots = [0, (1 << 31) - 64, 1 << 32, (1 << 32) + 4096, (1 << 34) - 256, 1 << 34, n // 32 * 32 - 64]
    return [(a, min(a + 160, n)) for a in spots if 0 <= a < n]


@pytest.fixture(scope="module", params=[(1 << 32) + 8192 + 5, (1 << 34) + 1000 + 3], ids=["2^32", "2^34"])
def data(Z, request):
    n = request.param
    torch.cuda.empty_cache()
    P = torch.zeros(n, device="cuda")
    G = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    C = torch.zeros(Z.zero_moments8_bytes(n), dtype=torch.uint8, device="cuda")
    S = torch.zeros(Z.zero_scales8_bytes(n), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    want = {}
    for a, b in places(n):
        p = rng.normal(0, 0.02, b - a).astype(np.float32)
        g = torch.from_numpy(rng.normal(0, 1e-3, b - a).astype(np.float32)).bfloat16()
        P[a:b], G[a:b] = torch.from_numpy(p).cuda(), g.cuda()
        want[a, b] = p, g
    yield n, P, G, C, S, want
    del P, G, C, S
    torch.cuda.empty_cache()


def model8(want, tensor):
    out = {}
    for (a, b), (p, g) in want.items():
        k = b - a
        hi, lo = a >> 32, a & 0xFFFFFFFF
        assert lo + k <= 1 << 32
        c = np.zeros(8 * -(-k // 4), np.uint8), np.zeros(2 * -(-k // 32), np.uint8)
        words = O8.words(5, HP["step"], k, tensor, first=a)
        real = O8.words
        O8.words = lambda seed, step, n, t=0, first=0: words
        try:
            out[a, b] = adam8_update(p, *c, g.float().numpy(), 0.0, 5, tensor, **HP)
        finally:
            O8.words = real
    return out


def check(n, P, C, S, want, name):
    for (a, b), (p, c, s) in want.items():
        assert np.array_equal(P[a:b].cpu().numpy(), p), f"{name}: master at {a}"
        assert np.array_equal(C[2 * a:2 * a + c.size].cpu().numpy(), c), f"{name}: codes at {a}"
        assert np.array_equal(S[a // 16:a // 16 + s.size].cpu().numpy(), s), f"{name}: scales at {a}"
    used = sum(int((p != 0).sum()) for p, _, _ in want.values())
    assert sum(int(torch.count_nonzero(x)) for x in P.split(1 << 30)) == used, f"{name}: an element elsewhere moved"
    used = sum(int((c != 0).sum()) for _, c, _ in want.values())
    assert sum(int(torch.count_nonzero(x)) for x in C.split(1 << 30)) == used, f"{name}: codes elsewhere"


def reset(P, C, S, want):
    P.zero_(), C.zero_(), S.zero_()
    for (a, b), (p, _) in want.items():
        P[a:b] = torch.from_numpy(p).cuda()


def test_shard_and_list_8(Z, data):
    n, P, G, C, S, want = data
    print(f"n={n}: shard", flush=True)
    Z.zero_shard_adam8_step(P, C, S, G, None, Z.AdamHyper(**HP), seed=5)
    torch.cuda.synchronize()
    check(n, P, C, S, model8(want, 0), "shard")
    reset(P, C, S, want)
    print(f"n={n}: list", flush=True)
    small = [torch.zeros(4, device="cuda"), torch.zeros(8, dtype=torch.uint8, device="cuda"),
             torch.zeros(2, dtype=torch.uint8, device="cuda"), torch.zeros(4, dtype=torch.bfloat16, device="cuda")]
    table = Z.TensorTable([small[0], P], [small[1], C], [small[2], S], [small[3], G], state_bits=8)
    Z.zero_multi_adam_step(table, [Z.AdamHyper(**HP)], seed=5)
    torch.cuda.synchronize()
    check(n, P, C, S, model8(want, 1), "list")
    reset(P, C, S, want)


def test_norm(Z, data):
    n, _, G, _, _, want = data
    table = Z.TensorTable.of_grads([G[:777], G])
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(table), dtype=torch.uint8, device="cuda")
    sq, ov = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    per = torch.zeros(2, dtype=torch.float64, device="cuda")
    Z.zero_multi_unscale_norm_overflow(table, 0.5, sq, ov, ws, per)
    exact = 0.25 * math.fsum(float(x) ** 2 for _, g in want.values() for x in g.float())
    # positive terms in float64: about 2^17 additions deep (2^34 elements over 512 blocks of 256 threads)
    assert abs(per[1].item() - exact) <= (2 ** 17 + 402) * 2.0 ** -53 * exact and ov.item() == 0
    first = 0.25 * math.fsum(float(x) ** 2 for x in want[0, 160][1].float())
    assert abs(per[0].item() - first) <= 402 * 2.0 ** -53 * first
    last = max(want)[1] - 1
    keep = G[last].clone()
    G[last] = float("inf")
    Z.zero_multi_unscale_norm_overflow(table, 0.5, sq, ov, ws, per)
    assert ov.item() == 1 and math.isinf(per[1].item()) and math.isfinite(per[0].item())
    G[last] = keep


def test_conversions(Z, data):
    n, P, _, C, S, want = data
    if n > 1 << 33:
        pytest.skip("both fp32 moments beside the fixture's buffers would not fit")
    M, V = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for (a, b), (p, _) in want.items():
        M[a:b], V[a:b] = torch.from_numpy(p).cuda(), torch.from_numpy(p * p).cuda()
    Z.zero_moments8_pack(C, S, M, V)
    for (a, b), (p, _) in want.items():
        root = np.sqrt(p * p)
        c, s = O8.pack(p, root.astype(np.float64) ** 2)
        assert np.array_equal(C[2 * a:2 * a + c.size].cpu().numpy(), c)
        assert np.array_equal(S[a // 16:a // 16 + s.size].cpu().numpy(), s)
    Z.zero_moments8_unpack(M, V, C, S)
    for (a, b), (p, _) in want.items():
        m, r = O8.decode(*O8.pack(p, np.sqrt(p * p).astype(np.float64) ** 2), b - a)
        assert np.array_equal(M[a:b].cpu().numpy(), m.astype(np.float32))
        assert np.array_equal(V[a:b].cpu().numpy(), (r * r).astype(np.float32))
    C.zero_(), S.zero_()


def test_list_32(Z, data):
    n, P, G, C, S, want = data
    if n > 1 << 33:
        pytest.skip("both fp32 moments beside the fixture's buffers would not fit")
    M, V = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    Z.zero_multi_adam_step(Z.TensorTable([P], [M], [V], [G]), [Z.AdamHyper(**HP)])
    for (a, b), (p, g) in want.items():
        got = [t[a:b].cpu().numpy() for t in (P, M, V)]
        for x, y in zip(got, adam_update(p, np.zeros_like(p), np.zeros_like(p), g.float().numpy(), 0.0, **HP)):
            assert np.array_equal(x, y), a
    reset(P, C, S, want)
