"""GPU: what a list's table keeps alive, and what its device copy waits for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIZES = [700, 5, 8192, 20_001]
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def normal(seed, scale, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(dtype).cuda() for n in SIZES]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_replay_reads_the_gradients_it_was_recorded_with(Z, bits):
    """They are described no longer and the caller has dropped them: the memory
    is not handed out again, and a replay steps with their values."""
    opts = [Z.MultiAdam(normal(1, 0.02), normal(2, 1e-2, torch.bfloat16), hyper=[HYPER], state_bits=bits,
                        device_state=True) for _ in range(2)]
    rec, eager = opts
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec.step()
    taken = {g.data_ptr() for g in rec.table.grads}
    rec.table.set_grads([torch.zeros_like(g) for g in rec.table.grads])
    fill = [torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda") for n in SIZES * 8]
    assert not taken & {x.data_ptr() for x in fill}
    for k in range(3):
        if k:
            eager.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(rec.masters, eager.masters) and same(rec.exp_avgs, eager.exp_avgs)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_stream_waits_for_a_table_built_on_another(Z, bits):
    """The table is built on a stream that still has work to do, and used on
    others that nobody made wait."""
    state = {32: lambda: [torch.zeros(n, device="cuda") for n in SIZES],
             8: lambda: [torch.zeros(2 * n + 8, dtype=torch.uint8, device="cuda") for n in SIZES]}[bits]
    grads = normal(2, 1e-2, torch.bfloat16)
    hp = [Z.AdamHyper(**HYPER, step=1)]
    want = normal(1, 0.02)
    Z.zero_multi_adam_step(Z.TensorTable(want, state(), state(), grads, state_bits=bits), hp)
    got, other = [(normal(1, 0.02), state(), state()) for _ in range(2)]
    torch.cuda.synchronize()
    build, first, second = (torch.cuda.Stream() for _ in range(3))
    with torch.cuda.stream(build):
        torch.cuda._sleep(20_000_000)                      # some milliseconds
        tables = [Z.TensorTable(*x, grads, state_bits=bits) for x in (got, other)]
    with torch.cuda.stream(first):
        Z.zero_multi_adam_step(tables[0], hp)
    Z.zero_multi_adam_step(tables[1], hp, stream=second)
    torch.cuda.synchronize()
    assert same(got[0], want) and same(other[0], want)


@pytest.mark.parametrize("bits", [32, 8])
def test_released_gradients_free_their_memory(Z, bits):
    """New gradients every step, dropped after it: the memory is free between
    the steps, the results are those of fixed buffers."""
    # of a size that the allocator serves from blocks of their own
    sizes = [3_000_001, 5_000_000]
    make = lambda k: [torch.randn(n, generator=torch.Generator("cuda").manual_seed(10 * k + i), device="cuda")  # noqa: E731
                      .mul_(1e-2).bfloat16() for i, n in enumerate(sizes)]
    masters = lambda: [torch.zeros(n, device="cuda") for n in sizes]  # noqa: E731
    fixed = make(0)
    want = Z.MultiAdam(masters(), fixed, hyper=[HYPER], max_grad_norm=1.0, state_bits=bits, device_state=True)
    got = Z.MultiAdam(masters(), make(0), hyper=[HYPER], max_grad_norm=1.0, state_bits=bits, device_state=True)
    got.release_grads()
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="released"):
        got.step()
    for k in range(4):
        for x, y in zip(fixed, make(k)):
            x.copy_(y)
        want.step()
        grads = make(k)
        got.step(grads)
        got.release_grads()
        del grads, x, y
        # the copy of a rebuilt table is all that may have come (less than its list's 2 bytes an element)
        assert torch.cuda.memory_allocated() - base < sum(sizes) * 2 // 10
    assert same(got.masters, want.masters) and same(got.exp_avgs, want.exp_avgs) and same(got.exp_avg_sqs, want.exp_avg_sqs)
