"""Host-side tests of the list and 8-bit calls (no GPU): the table's contents,
and every refusal of the library and of the binding before anything is
enqueued."""
import ctypes
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import zero_sharded_mixed_partition_amd as Z  # noqa: E402
from zero_sharded_mixed_partition_amd import _lib as L  # noqa: E402

from test_binding_checks import FakeDev, FakeState  # noqa: E402

AL = 1 << 40                        # a plausible, 16-byte aligned device address
HDR = "<Iiiiiiqqqqqqqqqqqqq"


def tensor(base, n, gdt=L.ZERO_BF16, pdt=L.ZERO_BF16, group=0, bits=32, **over):
    """A zero_tensor with its buffers 1 MiB apart, starting at base."""
    t = L.zero_tensor(base, base + (1 << 20), base + (2 << 20), base + (3 << 20), base + (4 << 20), n, gdt, pdt, group, 0)
    for k, v in over.items():
        setattr(t, k, v)
    return t


def build(tensors, bits=32, capacity=None):
    lib = L.lib()
    arr = (L.zero_tensor * max(1, len(tensors)))(*tensors)
    size, dev = ctypes.c_size_t(), ctypes.c_size_t()
    st = lib.zero_multi_table_build(arr, len(tensors), bits, None, 0, ctypes.byref(size), ctypes.byref(dev))
    if st != L.ZERO_ENOSPC:
        return st, None, 0
    buf = ctypes.create_string_buffer(size.value + 16)
    st = lib.zero_multi_table_build(arr, len(tensors), bits, buf, size.value if capacity is None else capacity,
                                    ctypes.byref(size), ctypes.byref(dev))
    return st, buf, dev.value


def table_of(*numels, bits=32, **kw):
    st, buf, _ = build([tensor(AL + (i << 28), n, **kw) for i, n in enumerate(numels)], bits)
    assert st == L.ZERO_OK
    return buf


def test_sizes_of_the_8_bit_buffers():
    for n in (0, 1, 3, 4, 5, 31, 32, 33, 1000, 2 ** 33 + 1):
        assert Z.zero_moments8_bytes(n) == 8 * -(-n // 4)
        assert Z.zero_scales8_bytes(n) == 2 * -(-n // 32)
    assert Z.zero_moments8_bytes(-1) == Z.zero_scales8_bytes(-1) == 0


def test_table_contents():
    sizes = [5, 0, 8192, 8193, 0, 40000]
    tensors = [tensor(AL + (i << 28), n, group=i % 3) for i, n in enumerate(sizes)]
    st, buf, dev = build(tensors)
    assert st == L.ZERO_OK
    raw = buf.raw
    (_, bits, n_groups, n_user, n_tensors, n_empty, n_chunks, n_units, unit_log2, desc_at, chunks_at, units_at, empty_at,
     device_bytes, ranges_at, n_ranges, grads_at, n_grads, size) = struct.unpack_from(HDR, raw)
    assert (bits, n_groups, n_user, n_tensors, n_empty) == (32, 3, 6, 4, 2)
    chunks = [-(-n // 8192) for n in sizes]
    assert n_chunks == sum(chunks) and device_bytes == dev <= size
    refs = [struct.unpack_from("<II", raw, chunks_at + 8 * c) for c in range(n_chunks)]
    live = [i for i, n in enumerate(sizes) if n]
    assert refs == [(k, c) for k, i in enumerate(live) for c in range(chunks[i])]
    # 1 + 32 + 33 + 157 tasks; 8 a unit take 8 + 32 + 40 + 160 workgroups, 16 take 272, over a tenth more
    assert (unit_log2, n_units) == (3, 30)
    refs = [struct.unpack_from("<II", raw, units_at + 8 * c) for c in range(n_units)]
    assert refs == [(k, u) for k, i in enumerate(live) for u in range(-(-sizes[i] // 2048))]
    first = 0
    for k, i in enumerate(live):
        f = struct.unpack_from("<QQQQQqiiiIIIii", raw, desc_at + k * 80)
        t = tensors[i]
        assert f == (t.master, t.exp_avg, t.exp_avg_sq, t.grad, t.param_out, sizes[i], t.grad_dtype, t.param_dtype,
                     t.group, i, first, chunks[i], 0, 0)
        first += chunks[i]
    assert [struct.unpack_from("<I", raw, empty_at + 4 * j)[0] for j in range(2)] == [1, 4]
    ranges = [struct.unpack_from("<QQ", raw, ranges_at + 16 * j) for j in range(n_ranges)]
    want = sorted((p, p + nb) for i in live for p, nb in
                  ((tensors[i].master, 4 * sizes[i]), (tensors[i].exp_avg, 4 * sizes[i]),
                   (tensors[i].exp_avg_sq, 4 * sizes[i]), (tensors[i].param_out, 2 * sizes[i])))
    assert ranges == want
    grads = [struct.unpack_from("<QQ", raw, grads_at + 16 * j) for j in range(n_grads)]
    assert grads == [(tensors[i].grad, tensors[i].grad + 2 * sizes[i]) for i in live]


def test_table_joins_written_ranges():
    """Tensors end to end in flat buffers leave one range per buffer."""
    n, k = 100, 10
    tensors = [tensor(AL, n, master=AL + 4 * n * i, exp_avg=AL + (1 << 20) + 4 * n * i,
                      exp_avg_sq=AL + (2 << 20) + 4 * n * i, grad=AL + (3 << 20) + 2 * n * i,
                      param_out=AL + (4 << 20) + 2 * n * i) for i in range(k)]
    st, buf, _ = build(tensors)
    assert st == L.ZERO_OK and struct.unpack_from(HDR, buf.raw)[15] == 4


def test_table_refusals():
    ok = tensor(AL, 100)
    assert build([ok])[0] == L.ZERO_OK
    assert build([])[0] == L.ZERO_OK
    for bad in (dict(numel=-1), dict(grad_dtype=4), dict(grad_dtype=0), dict(param_dtype=L.ZERO_F32), dict(group=-1),
                dict(group=16), dict(master=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(grad=None)):
        assert build([tensor(AL, 100, **bad)])[0] == L.ZERO_EINVAL, bad
    for bad in (dict(master=AL + 2), dict(exp_avg=AL + (1 << 20) + 1), dict(exp_avg_sq=AL + (2 << 20) + 2),
                dict(grad=AL + (3 << 20) + 1), dict(param_out=AL + (4 << 20) + 1)):
        assert build([tensor(AL, 100, **bad)])[0] == L.ZERO_EALIGN, bad
    assert build([tensor(AL, 100, gdt=L.ZERO_F32, grad=AL + (3 << 20) + 2)])[0] == L.ZERO_EALIGN
    assert build([tensor(AL, 100, exp_avg=AL + (1 << 20) + 4)], 8)[0] == L.ZERO_EALIGN      # codes: 8 bytes
    assert build([tensor(AL, 100, exp_avg_sq=AL + (2 << 20) + 1)], 8)[0] == L.ZERO_EALIGN
    assert build([tensor(AL, 100, numel=2 ** 62)])[0] == L.ZERO_ERANGE
    assert build([ok], 16)[0] == L.ZERO_EINVAL
    assert build([ok], capacity=10)[0] == L.ZERO_ENOSPC
    lib = L.lib()
    s = ctypes.c_size_t()
    assert lib.zero_multi_table_build(None, 1, 32, None, 0, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EINVAL
    assert lib.zero_multi_table_build(None, -1, 32, None, 0, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EINVAL
    assert lib.zero_multi_table_build(None, 0, 32, None, 0, None, ctypes.byref(s)) == L.ZERO_EINVAL
    odd = ctypes.addressof(ctypes.create_string_buffer(4096)) // 8 * 8 + 4
    assert lib.zero_multi_table_build(None, 0, 32, odd, 4096, ctypes.byref(s), ctypes.byref(s)) == L.ZERO_EALIGN
    assert lib.zero_multi_adam_step(odd, None, None, 1, 0, None, None, None) in (L.ZERO_EALIGN, L.ZERO_EINVAL)


def test_table_refuses_overlaps():
    a = tensor(AL, 100)
    assert build([a, a])[0] == L.ZERO_EINVAL                                        # the same tensor twice
    far = AL + (1 << 30)
    for over in (dict(master=AL + 396), dict(exp_avg=AL), dict(param_out=AL + (2 << 20) + 200),
                 dict(grad=AL + (4 << 20)), dict(grad=AL)):
        assert build([a, tensor(far, 100, **over)])[0] == L.ZERO_EINVAL, over
    assert build([a, tensor(far, 100, grad=a.grad)])[0] == L.ZERO_OK                # gradients may be shared
    assert build([a, tensor(far, 100, master=AL + 400)])[0] == L.ZERO_OK            # end to end
    assert build([tensor(AL, 100, exp_avg=AL + 396)])[0] == L.ZERO_EINVAL
    # 8 bits: the codes are 8 * ceil(n / 4) bytes, the scales 2 * ceil(n / 32)
    assert build([tensor(AL, 33, exp_avg_sq=AL + (1 << 20) + 70)], 8)[0] == L.ZERO_EINVAL
    assert build([tensor(AL, 33, exp_avg_sq=AL + (1 << 20) + 72)], 8)[0] == L.ZERO_OK
    # a table of gradients looks at nothing else
    st, buf, _ = build([L.zero_tensor(None, None, None, AL, None, 100, L.ZERO_F16, 0, 0, 0)] * 2, 0)
    assert st == L.ZERO_OK and struct.unpack_from(HDR, buf.raw)[17] == 1     # gradients that overlap are one range


def test_workspace():
    lib = L.lib()
    assert lib.zero_multi_norm_workspace_bytes(None) == 0
    assert lib.zero_multi_norm_workspace_bytes(ctypes.create_string_buffer(256)) == 0
    small, large = table_of(5), table_of(5, 8192 * 5000, bits=0)      # gradients only: nothing overlaps
    assert lib.zero_multi_norm_workspace_bytes(small) == 256
    # blocks and tensors: a partial each, the scale's factor, and a flag per block
    want = lambda blocks, tensors: -(-((blocks + tensors + 1) * 8 + blocks * 4) // 256) * 256  # noqa: E731
    assert lib.zero_multi_norm_workspace_bytes(large) == want(512, 2)
    short = table_of(5, 8192 * 4095, bits=0)
    assert lib.zero_multi_norm_workspace_bytes(short) == want(1024, 2)
    many = build([tensor(AL + (i << 28), 8192 * 3, group=0) for i in range(2000)], 0)[1]
    assert lib.zero_multi_norm_workspace_bytes(many) == want(1024, 2000)


D = AL + (1 << 39)                  # where the scalars and the table's device copy lie


def test_norm_refusals():
    lib = L.lib()
    tab = table_of(100, 50)
    n = lib.zero_multi_norm_workspace_bytes(tab)

    def norm(table=tab, d=D, inv=1.0, sq=D + 4096, ov=D + 4104, per=D + 4352, ws=D + 8192, nb=n):
        return lib.zero_multi_unscale_norm_overflow(table, d, inv, sq, ov, per, ws, nb, None)

    for bad in (dict(table=None), dict(table=ctypes.create_string_buffer(512)), dict(d=None), dict(inv=0.0),
                dict(inv=float("inf")), dict(inv=float("nan")), dict(sq=None), dict(ov=None), dict(ws=None),
                dict(sq=D + 8192), dict(ov=D + 4096), dict(per=D + 4096), dict(per=D + 8192 + n - 8), dict(ws=D),
                dict(sq=AL + (3 << 20)), dict(per=AL + (1 << 28) + (3 << 20)), dict(ws=AL + (3 << 20))):
        assert norm(**bad) == L.ZERO_EINVAL, bad
    for bad in (dict(d=D + 8), dict(sq=D + 4100), dict(ov=D + 4106), dict(per=D + 4356), dict(ws=D + 8200)):
        assert norm(**bad) == L.ZERO_EALIGN, bad
    assert norm(nb=n - 1) == L.ZERO_ENOSPC

    hp = (L.zero_adam_hyper * 2)(*[L.zero_adam_hyper(1e-3, 0.9, 0.999, 1e-8, 0.0, 0.0)] * 2)

    def decide(hp=hp, g=2, st=D + 12288, co=D + 16384):
        return lib.zero_multi_norm_decide_dev(tab, D, 0, hp, g, st, D + 4096, D + 4104, None, co, D + 8192, n, None)

    for bad in (dict(hp=None), dict(g=0), dict(g=17), dict(st=None), dict(co=None), dict(co=D + 12288), dict(co=D + 4096)):
        assert decide(**bad) == L.ZERO_EINVAL, bad
    assert decide(st=D + 12292) == L.ZERO_EALIGN
    bad_hp = (L.zero_adam_hyper * 1)(L.zero_adam_hyper(1e-3, 1.0, 0.999, 1e-8, 0.0, 0.0))
    assert decide(hp=bad_hp, g=1) == L.ZERO_EINVAL
    f = lib.zero_multi_decide_dev
    assert f(hp, 2, 0, D, None, D + 4096, None) == L.ZERO_EINVAL
    assert f(hp, 2, 0, D, D + 1024, D + 64, None) == L.ZERO_EINVAL
    assert f(hp, 0, 0, D, D + 1024, D + 4096, None) == L.ZERO_EINVAL
    g = lib.zero_multi_unscale_norm_overflow_dev
    assert g(tab, D, 0, None, D + 4096, D + 4104, None, D + 8192, n, None) == L.ZERO_EINVAL


@pytest.mark.parametrize("bits", [32, 8])
def test_update_refusals(bits):
    lib = L.lib()
    tab = table_of(100, 50, bits=bits)
    good = L.zero_adam_params(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 1.0, 0.0)
    clip = L.zero_adam_params(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 1.0, 1.0)
    bad_hp = L.zero_adam_params(1e-3, 0.9, 1.5, 1e-8, 0.0, 1, 1.0, 0.0)
    arr = lambda *h: (L.zero_adam_params * len(h))(*h)  # noqa: E731
    far = (1 << 28)

    def step(table=tab, d=D, hp=arr(clip, clip), g=2, sq=D + 4096, ov=D + 4104):
        return lib.zero_multi_adam_step(table, d, hp, g, 0, sq, ov, None)

    for bad in (dict(table=None), dict(d=None), dict(hp=None), dict(g=0), dict(g=17), dict(hp=arr(good, bad_hp)),
                dict(sq=None), dict(sq=AL), dict(ov=AL + far + 4), dict(d=AL + (1 << 20)), dict(sq=AL + (4 << 20)),
                dict(ov=AL + far + (2 << 20))):
        assert step(**bad) == L.ZERO_EINVAL, bad
    for bad in (dict(d=D + 4), dict(sq=D + 4100), dict(ov=D + 4106)):
        assert step(**bad) == L.ZERO_EALIGN, bad
    grouped = table_of(100, 50, bits=bits, group=3)
    assert step(table=grouped, hp=arr(*[clip] * 3), g=3) == L.ZERO_EINVAL            # the table names group 3
    assert step(table=table_of(100, bits=0)) == L.ZERO_EINVAL                        # gradients only

    def coef(co=D + 16384, g=2, t=D + 8192, sq=D + 4096, ov=None):
        return lib.zero_multi_adam_step_coef(tab, D, co, g, 0, t, sq, ov, None)

    for bad in (dict(co=None), dict(sq=None), dict(g=0), dict(co=AL), dict(t=AL + 8)):
        assert coef(**bad) == L.ZERO_EINVAL, bad
    if bits == 8:
        assert coef(t=None) == L.ZERO_EINVAL
    for bad in (dict(co=D + 16388), dict(t=D + 8196)):
        assert coef(**bad) == L.ZERO_EALIGN, bad


def test_shard8_refusals():
    lib = L.lib()
    hp = L.zero_adam_params(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 1.0, 1.0)
    M = 1 << 20

    def step(p=AL, c=AL + M, s=AL + 2 * M, g=AL + 3 * M, gd=L.ZERO_BF16, o=AL + 4 * M, pd=L.ZERO_BF16, n=100, h=hp,
             sq=D, ov=D + 8):
        return lib.zero_shard_adam8_step(p, c, s, g, gd, o, pd, n, ctypes.byref(h) if h else None, 0, sq, ov, None)

    for bad in (dict(p=None), dict(c=None), dict(s=None), dict(g=None), dict(gd=7), dict(pd=L.ZERO_F32), dict(n=-1),
                dict(h=None), dict(sq=None), dict(c=AL), dict(s=AL + M + 192), dict(g=AL + 2 * M), dict(o=AL + 3 * M),
                dict(o=AL + 384), dict(sq=AL + 8), dict(ov=AL + M), dict(sq=AL + 2 * M),
                dict(h=L.zero_adam_params(1e-3, 0.9, 0.999, 1e-8, 0.0, 0, 1.0, 1.0))):
        assert step(**bad) == L.ZERO_EINVAL, bad
    for bad in (dict(p=AL + 8), dict(c=AL + M + 8), dict(s=AL + 2 * M + 2), dict(g=AL + 3 * M + 2), dict(o=AL + 4 * M + 4),
                dict(sq=D + 4), dict(ov=D + 10)):
        assert step(**bad) == L.ZERO_EALIGN, bad
    assert step(n=2 ** 62) == L.ZERO_ERANGE
    assert step(n=0, p=None, c=None, s=None, g=None, o=None) == L.ZERO_OK

    def coef(co=D + 64, t=D + 128, sq=D, ov=D + 8):
        return lib.zero_shard_adam8_step_coef(AL, AL + M, AL + 2 * M, AL + 3 * M, L.ZERO_F16, None, 0, 100, co, 0, t, sq,
                                              ov, None)

    for bad in (dict(co=None), dict(t=None), dict(sq=None), dict(co=AL), dict(t=AL + M), dict(sq=AL + 2 * M)):
        assert coef(**bad) == L.ZERO_EINVAL, bad
    for bad in (dict(co=D + 68), dict(t=D + 132), dict(ov=D + 9)):
        assert coef(**bad) == L.ZERO_EALIGN, bad

    for f in (lambda m, v, c, s, n: lib.zero_moments8_unpack(m, v, c, s, n, None),
              lambda m, v, c, s, n: lib.zero_moments8_pack(c, s, m, v, n, None)):
        assert f(AL, AL + M, AL + 2 * M, AL + 3 * M, -1) == L.ZERO_EINVAL
        assert f(None, None, None, None, 0) == L.ZERO_OK
        for k in range(4):
            a = [AL, AL + M, AL + 2 * M, AL + 3 * M]
            a[k] = None
            assert f(*a, 100) == L.ZERO_EINVAL
            a[k] = AL + 5 * M + (2, 2, 4, 1)[k]
            assert f(*a, 100) == L.ZERO_EALIGN
            a[k] = a[k - 1]
            assert f(*a, 100) == L.ZERO_EINVAL
        assert f(AL, AL + M, AL + 2 * M, AL + 3 * M, 2 ** 62) == L.ZERO_ERANGE


# ---------------------------------------------------------------- the binding

U8, F32, F64, I32, I64, BF16 = torch.uint8, torch.float32, torch.float64, torch.int32, torch.int64, torch.bfloat16


def test_binding_checks_8_bit_buffers():
    n = 1000
    good = dict(master=FakeDev(n, F32), moments8=FakeDev(2000, U8), scales8=FakeDev(64, U8), grad=FakeDev(n, BF16),
                param_out=FakeDev(n, BF16))

    def step(**over):
        Z.zero_shard_adam8_step(hp=Z.AdamHyper(), stream=0, **dict(good, **over))

    for name, bad in (("master", FakeDev(n, F64)), ("moments8", FakeDev(1999, U8)), ("moments8", FakeDev(2000, BF16)),
                      ("scales8", FakeDev(63, U8)), ("grad", FakeDev(n - 1, BF16)), ("param_out", FakeDev(n - 1, BF16))):
        with pytest.raises(ValueError):
            step(**{name: bad})
    with pytest.raises(ValueError, match="global_sqnorm"):
        step(global_sqnorm=FakeDev(1, F32))
    with pytest.raises(ValueError, match="d_step"):
        Z.zero_shard_adam8_step_coef(*good.values(), FakeDev(64, U8), FakeDev(1, I32), FakeDev(1, F64), stream=0)
    for name, args in (("exp_avg", (FakeDev(2000, U8), FakeDev(64, U8), FakeDev(n, BF16), FakeDev(n, F32))),
                       ("moments8", (FakeDev(1999, U8), FakeDev(64, U8), FakeDev(n, F32), FakeDev(n, F32))),
                       ("scales8", (FakeDev(2000, U8), FakeDev(62, U8), FakeDev(n, F32), FakeDev(n, F32)))):
        with pytest.raises(ValueError, match=name):
            Z.zero_moments8_pack(*args, n=n, stream=0)
        with pytest.raises(ValueError, match=name):
            Z.zero_moments8_unpack(args[2], args[3], args[0], args[1], n=n, stream=0)


def fake_list(numels, bits=32):
    cols = [[], [], [], [], []]
    for i, n in enumerate(numels):
        base = AL + (i << 30)
        moments = [(n, F32), (n, F32)] if bits == 32 else [(Z.zero_moments8_bytes(n), U8), (Z.zero_scales8_bytes(n), U8)]
        for c, (k, dt) in enumerate([(n, F32), *moments, (n, BF16), (n, BF16)]):
            cols[c].append(FakeDev(k, dt, base + (c << 24)))
    return cols


def test_binding_builds_and_checks_tables():
    for bits in (32, 8):
        m, a, b, g, p = fake_list([100, 7, 3000], bits)
        t = Z.TensorTable(m, a, b, g, p, groups=[0, 2, 1], state_bits=bits)
        assert t.n_tensors == 3 and t.n_groups == 3 and t.device is None
        assert Z.zero_multi_norm_workspace_bytes(t) == 256
        key = t._grad_key
        t.set_grads(g)
        assert t._grad_key is key
        other = fake_list([100, 7, 3000])[3]
        other[1] = FakeDev(7, F32, AL + (7 << 30))
        t.set_grads(other)
        assert t._grad_key != key
        with pytest.raises(ValueError, match="gradients"):
            t.set_grads(other[:2])
        with pytest.raises(ValueError, match="masters"):
            Z.TensorTable(m[:2], a, b, g, state_bits=bits)
        with pytest.raises(ValueError, match="groups"):
            Z.TensorTable(m, a, b, g, groups=[0], state_bits=bits)
        with pytest.raises(ValueError, match="state_bits"):
            Z.TensorTable(m, a, b, g, state_bits=16)
        with pytest.raises(Z.ZeroShardError):
            Z.TensorTable(m, a, b, g, groups=[0, 16, 1], state_bits=bits)
        for col, bad in ((0, FakeDev(6, F32)), (0, FakeDev(7, BF16)), (1, FakeDev(3, F32)), (2, FakeDev(0, U8)),
                         (4, FakeDev(6, BF16)), (4, FakeDev(7, F64))):
            cols = [list(c) for c in (m, a, b, g, p)]
            cols[col][1] = bad
            with pytest.raises(ValueError):
                Z.TensorTable(*cols, state_bits=bits)
        with pytest.raises(Z.ZeroShardError):
            Z.TensorTable(m + m[:1], a + a[:1], b + b[:1], g + g[:1], p + p[:1], state_bits=bits)
    assert Z.TensorTable.of_grads([]).n_tensors == 0


def test_binding_checks_list_calls():
    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    sq, ov, ws, per = FakeDev(1, F64), FakeDev(1, I32), FakeDev(256, U8), FakeDev(2, F64)
    for kw in (dict(sqnorm=FakeDev(1, F32)), dict(overflow=FakeDev(1, I64)), dict(tensor_sqnorm=FakeDev(1, F64))):
        with pytest.raises(ValueError):
            Z.zero_multi_unscale_norm_overflow(t, 1.0, **dict(dict(sqnorm=sq, overflow=ov, workspace=ws,
                                                                   tensor_sqnorm=per), **kw), stream=0)
        with pytest.raises(ValueError):
            Z.zero_multi_unscale_norm_overflow_dev(t, FakeState(), **dict(dict(sqnorm=sq, overflow=ov, workspace=ws,
                                                                               tensor_sqnorm=per), **kw), stream=0)
    hps = [Z.AdamHyper()] * 2
    for bad in ([], [Z.AdamHyper()] * 17):
        with pytest.raises(ValueError, match="hyperparameter"):
            Z.zero_multi_adam_step(t, bad, sq, ov, stream=0)
        with pytest.raises(ValueError, match="hyperparameter"):
            Z.zero_multi_decide_dev(bad, FakeState(), ov, FakeDev(4096, U8), stream=0)
    short = FakeDev(2 * Z.zero_adam_coef_bytes() - 1, U8)
    with pytest.raises(ValueError, match="d_coefs"):
        Z.zero_multi_adam_step_coef(t, short, 2, sq, ov, stream=0)
    with pytest.raises(ValueError, match="d_coefs"):
        Z.zero_multi_norm_decide_dev(t, hps, FakeState(), sq, ov, short, ws, stream=0)
    with pytest.raises(ValueError, match="global_sqnorm"):
        Z.zero_multi_adam_step(t, hps, FakeDev(1, F32), ov, stream=0)


def test_gradients_of_another_length_or_order_in_the_same_place_are_refused():
    """A view that begins where the described gradient does is not that gradient."""
    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    with pytest.raises(ValueError, match="elements"):
        t.set_grads([FakeDev(50, g[0].dtype, g[0].data_ptr()), g[1]])
    turned = FakeDev(100, g[0].dtype, g[0].data_ptr())
    turned.is_contiguous = lambda: False
    with pytest.raises(ValueError, match="contiguous"):
        t.set_grads([turned, g[1]])
    t.set_grads(g)
    assert t.grads == g


class Placed(FakeDev):
    """A stand-in that knows its device."""

    def __init__(self, numel, dtype, addr=1 << 40, index=0):
        super().__init__(numel, dtype, addr)
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


def test_tensors_on_another_device_are_refused(monkeypatch):
    from zero_sharded_mixed_partition_amd import moments8 as M8
    from zero_sharded_mixed_partition_amd import multi as MU
    cols = [[Placed(t.numel(), t.dtype, t.data_ptr()) for t in col] for col in fake_list([100, 7])]
    for col in range(5):
        bad = [list(c) for c in cols]
        t = bad[col][1]
        bad[col][1] = Placed(t.numel(), t.dtype, t.data_ptr(), index=1)
        with pytest.raises(ValueError, match="cuda:1"):
            Z.TensorTable(*bad)
    for module in (M8, MU):
        monkeypatch.setattr(module, "_current_device", lambda: 1)
    n = 100
    for k in range(5):
        args = [FakeDev(n, F32), FakeDev(200, U8), FakeDev(8, U8), FakeDev(n, BF16), FakeDev(n, BF16)]
        for i, t in enumerate(args):                        # all on the current device but one
            args[i] = Placed(t.numel(), t.dtype, t.data_ptr(), index=0 if i == k else 1)
        with pytest.raises(ValueError, match="current device is cuda:1"):
            Z.zero_shard_adam8_step(*args, Z.AdamHyper(), stream=0)
    class OtherStream:
        device_index, cuda_stream = 0, 4096

    with pytest.raises(ValueError, match="stream of cuda:0"):
        Z.zero_shard_adam8_step(*(Placed(t.numel(), t.dtype, t.data_ptr(), index=1) for t in args), Z.AdamHyper(),
                                stream=OtherStream())
    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    t._index = 0
    with pytest.raises(ValueError, match="current device is cuda:1"):
        Z.zero_multi_adam_step(t, [Z.AdamHyper()], FakeDev(1, F64), stream=0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        Z.zero_multi_unscale_norm_overflow(t, 1.0, FakeDev(1, F64), FakeDev(1, I32), FakeDev(256, U8), stream=0)


def test_the_device_copy_waits_for_every_stream_that_read_it(monkeypatch):
    """A table used on a stream other than its own is given back to the
    allocator with that stream recorded, once; a raw handle cannot be."""
    class Stream:
        def __init__(self, handle):
            self.cuda_stream, self.device_index = handle, 0

    class Device:
        def __init__(self):
            self.seen = []

        def record_stream(self, s):
            self.seen.append(s.cuda_stream)

        def data_ptr(self):
            return 1 << 45

    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    t._index, t.device, t._streams, t._captured = 0, Device(), {64}, True
    for handle in (64, 128, 192, 128):
        t._ptrs(0, Stream(handle))
    t._ptrs(0, 256)
    assert t.device.seen == [128, 192]
    monkeypatch.setattr(Z, "_raw_stream", lambda device: 512)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(512))
    t._ptrs(0, None)
    t._ptrs(0, None)
    assert t.device.seen == [128, 192, 512]


def test_np_seed_range():
    """Any integer seeds the rounding: it is taken modulo 2^64."""
    from zero_sharded_mixed_partition_amd.moments8 import _seed
    assert _seed(-1) == 2 ** 64 - 1 and _seed(2 ** 64 + 5) == 5 and _seed(np.int64(3)) == 3


def test_multi_adam_refuses_bad_lists():
    g = [FakeDev(5, BF16)]
    for kw in (dict(state_bits=16), dict(hyper=[]), dict(hyper=[{}] * 17), dict(hyper=[dict(lr=1.0, momentum=0.9)]),
               dict(groups=[1]), dict(groups=[-1])):
        with pytest.raises(ValueError):
            Z.MultiAdam([FakeDev(5, F32)], g, **kw)
    with pytest.raises(ValueError, match="empty"):
        Z.MultiAdam([], [])
    with pytest.raises(ValueError, match="fp32"):
        Z.ShardAdam8(FakeDev(5, BF16))
    with pytest.raises(ValueError, match="together"):
        Z.ShardAdam8(FakeDev(5, F32), moments8=FakeDev(16, U8))
    with pytest.raises(ValueError, match="uint8"):
        Z.ShardAdam8(FakeDev(5, F32), moments8=FakeDev(15, U8), scales8=FakeDev(2, U8))


def test_table_phases_and_units():
    """32-bit tensors whose master starts off a 256-byte boundary: the update's
    tasks start before the tensor, and take one more where that spills.  Units
    are as large as idle workgroups (at most a tenth of the tasks) allow."""
    for off, n, bits, count, want in ((1, 8192, 32, 1, (1, 2, 9)), (0, 8192, 32, 1, (0, 5, 1)), (64, 8192, 32, 1, (0, 5, 1)),
                                      (63, 8130, 32, 1, (63, 2, 9)), (63, 8129, 32, 1, (63, 5, 1)),
                                      (1, 8192, 8, 1, (0, 5, 1)), (5, 1, 32, 1, (5, 0, 1)), (0, 500, 32, 30, (0, 1, 30)),
                                      (0, 64, 8, 30, (0, 0, 30)), (0, 256 * 60, 32, 2, (0, 5, 4))):
        st, buf, _ = build([tensor(AL + (i << 28), n, master=AL + (i << 28) + 4 * off) for i in range(count)], bits)
        assert st == L.ZERO_OK
        h = struct.unpack_from(HDR, buf.raw)
        f = struct.unpack_from("<QQQQQqiiiIIIii", buf.raw, h[9])
        assert (f[12], h[8], h[7]) == want, (off, n, bits, f[12], h[8], h[7])




def test_checkpoint_of_parameters_of_several_dimensions(monkeypatch, tmp_path):
    """Arrays load into tensors of the shape they were saved with or of its flat
    form, and nothing is written when one does not fit or the groups differ."""
    from types import SimpleNamespace
    from zero_sharded_mixed_partition_amd import checkpoint
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(synchronize=lambda: None))

    def opt(*shapes, groups=1):
        cols = [torch.full(s, 1.0 + i) for i, s in enumerate(shapes)]
        return SimpleNamespace(state=None, t=0, scaler=Z.LossScaler(), hyper=[dict(lr=0.1)] * groups, seed=3, cols=cols,
                               checkpoint_arrays=lambda: {f"master_{i}": x for i, x in enumerate(cols)})

    shapes = [(3, 5), (), (0, 4), (7,)]
    a, b, flat = opt(*shapes), opt(*shapes), opt((15,), (1,), (0,), (7,))
    for x in a.cols:
        x.mul_(10)
    checkpoint.save(a, str(tmp_path))
    checkpoint.load(b, str(tmp_path))
    assert all(torch.equal(x, y) for x, y in zip(a.cols, b.cols))
    c = opt(*shapes)
    checkpoint.load_state_dict(c, checkpoint.state_dict(flat))
    assert all(torch.equal(x.reshape(-1), y) for x, y in zip(c.cols, flat.cols))
    for other, what in ((opt((5, 3), (), (0, 4), (7,)), "master_0"), (opt(*shapes, groups=2), "groups")):
        before = [x.clone() for x in other.cols]
        with pytest.raises(ValueError, match=what):
            checkpoint.load(other, str(tmp_path))
        assert all(torch.equal(x, y) for x, y in zip(before, other.cols))
