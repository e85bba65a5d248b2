"""GPU: a launch of the 32-bit list update and of the conversions whose tasks
pass one grid (2^34 elements), so that workgroups take a second task.  All is
zero but a few places on both sides of that border, whose results are the
float32 model's and the oracle's; the rest has to stay zero."""
import numpy as np
import pytest

import oracle.moments8 as O8
from f32model import adam_update

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=3, inv_loss_scale=1.0, max_grad_norm=0.0)
N = (1 << 34) + 100_003
# 2^26 - 1 workgroups of 256 elements fill one grid
PLACES = [(a, min(a + 160, N)) for a in (0, (1 << 32) + 4096, (1 << 34) - 512, (1 << 34) - 256, 1 << 34,
                                         (1 << 34) + 65_536, N // 32 * 32 - 64)]


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < 250e9:
        pytest.skip("needs 241 GB of device memory")
    yield Z
    torch.cuda.empty_cache()


def planted(seed, scale):
    rng = np.random.default_rng(seed)
    return {at: rng.normal(0, scale, at[1] - at[0]).astype(np.float32) for at in PLACES}


def put(t, values):
    for (a, b), x in values.items():
        t[a:b] = torch.from_numpy(x).to(t.dtype).cuda()


def taken(values, at):
    """The planted values as they stand in the buffer: a later place overwrites what an earlier one shares with it."""
    out = values[at].copy()
    for (a, b), x in list(values.items())[list(values).index(at) + 1:]:
        lo, hi = max(a, at[0]), min(b, at[1])
        if lo < hi:
            out[lo - at[0]:hi - at[0]] = x[lo - a:hi - a]
    return out


def nonzero(t):
    return sum(int(torch.count_nonzero(x)) for x in t.split(1 << 30))


def test_list_of_32_bit_moments(Z):
    P, M, V = (torch.zeros(N, device="cuda") for _ in range(3))
    G = torch.zeros(N, dtype=torch.bfloat16, device="cuda")
    p, g = planted(1, 0.02), planted(2, 1e-3)
    put(P, p), put(G, g)
    print("step", flush=True)
    Z.zero_multi_adam_step(Z.TensorTable([P], [M], [V], [G]), [Z.AdamHyper(**HP)])
    torch.cuda.synchronize()
    for at in PLACES:
        want_p, want_g = taken(p, at), torch.from_numpy(taken(g, at)).bfloat16().float().numpy()
        zero = np.zeros_like(want_p)
        for name, t, y in zip("pmv", (P, M, V), adam_update(want_p, zero, zero, want_g, 0.0, **HP)):
            assert np.array_equal(t[at[0]:at[1]].cpu().numpy(), y), (name, at)
    for (a, b) in PLACES:
        P[a:b], M[a:b], V[a:b] = 0, 0, 0
    assert nonzero(P) == nonzero(M) == nonzero(V) == 0
    del P, M, V, G
    torch.cuda.empty_cache()


def test_conversions(Z):
    M, V = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    C = torch.full((Z.zero_moments8_bytes(N),), 9, dtype=torch.uint8, device="cuda")
    S = torch.full((Z.zero_scales8_bytes(N),), 9, dtype=torch.uint8, device="cuda")
    m = planted(3, 0.02)
    v = {at: x * x for at, x in m.items()}
    put(M, m), put(V, v)
    print("pack", flush=True)
    Z.zero_moments8_pack(C, S, M, V)
    torch.cuda.synchronize()
    blocks = {}
    for a, b in PLACES:                                    # whole blocks of 32, as they stand in the buffers
        lo, hi = a // 32 * 32, min(-(-b // 32) * 32, N)
        x, y = M[lo:hi].cpu().numpy(), V[lo:hi].cpu().numpy()
        c, s = O8.pack(x, np.sqrt(y).astype(np.float64) ** 2)
        assert np.array_equal(C[2 * lo:2 * lo + c.size].cpu().numpy(), c), a
        assert np.array_equal(S[lo // 16:lo // 16 + s.size].cpu().numpy(), s), a
        blocks[lo, hi] = c, s
    M.zero_(), V.zero_()
    print("unpack", flush=True)
    Z.zero_moments8_unpack(M, V, C, S)
    torch.cuda.synchronize()
    for (lo, hi), (c, s) in blocks.items():
        dm, ds = O8.decode(c, s, hi - lo)
        assert np.array_equal(M[lo:hi].cpu().numpy(), dm.astype(np.float32)), lo
        assert np.array_equal(V[lo:hi].cpu().numpy(), (ds * ds).astype(np.float32)), lo
        M[lo:hi], V[lo:hi], C[2 * lo:2 * lo + c.size] = 0, 0, 0
    assert nonzero(M) == nonzero(V) == nonzero(C) == 0
    # a block of zeros has the smallest scale
    for lo, hi in blocks:
        S[lo // 16:lo // 16 + 2 * -(-(hi - lo) // 32)] = 1
    assert all(bool((x == 1).all()) for x in S.split(1 << 30))
    del M, V, C, S
    torch.cuda.empty_cache()
