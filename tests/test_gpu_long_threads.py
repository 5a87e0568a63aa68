"""Host threads that make calls of one kernel with different sizes at once, and one graph that holds a large call before a
small one: what a call asks of the GPU is its own, whatever another call asks in between."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def zg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import generative_recommendation_constrained_gb300 as zg
    return zg


@pytest.fixture(scope="module")
def dev(zg):
    from generative_recommendation_constrained_gb300 import device
    return device


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def recorded(Z, call):
    """The library call that `call` makes, with its arguments as they reach C: a thread that repeats it is inside the
    library most of the time, without the interpreter's lock."""
    real, seen = Z.lib, []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: seen.append((getattr(real, name), a)) or 0

    Z.lib = Recorder()
    try:
        call()
    finally:
        Z.lib = real
    (f, args), = seen
    return f, args


def at_once(zg, dev, *calls, times=10000):
    """Each call `times` times from two threads, each on a stream of its own."""
    errors, start = [], threading.Barrier(2 * len(calls))

    def work(f, args):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(times):
            if f(*args):
                errors.append(dev.Z.lib.zg_last_error())
                return

    streams, threads = [torch.cuda.Stream() for _ in range(2 * len(calls))], []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            threads.append(threading.Thread(target=work, args=recorded(dev.Z, calls[i // 2])))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    zg.zg_check_device_status(0)
    assert not errors, errors


@pytest.mark.parametrize("fmt, dim, few", [("e4m3", 128, 1), ("e2m1", 64, 60)])
def test_weights_of_few_rows_and_of_many(zg, dev, fmt, dim, few):
    """A token's weights beside a window's, which have more queries in shared memory.  Histories are empty: the launch alone."""
    cache = dev.KVCache(4, 16, 1, dim, fmt)
    calls = []
    for R in (few, 500):
        q = torch.zeros((1, R, 4, dim), dtype=torch.bfloat16, device="cuda")
        a = (torch.zeros((1, 1, 16), device="cuda"), q, torch.zeros((1, R, 4), device="cuda"), ints([[0]]), ints([0]))
        calls.append(lambda a=a: cache.add_weights(*a))
    at_once(zg, dev, *calls)


@pytest.mark.parametrize("fmt, dim", [("int8", 32), ("e2m1", 128)])
def test_evictions_through_narrow_and_wide_tables(zg, dev, fmt, dim):
    cache = dev.KVCache(4, 16, 1, dim, fmt)
    calls = []
    for width in (1, 1 << 14):
        e = dev.CacheEviction(cache, 1, width, 1)
        a = (torch.zeros((1, 1, 16 * width), device="cuda"), torch.zeros((1, width), dtype=torch.int32, device="cuda"), ints([0]))
        calls.append(lambda e=e, a=a: e(*a))
    at_once(zg, dev, *calls)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_writes_of_few_and_of_many_tokens(zg, dev, fmt):
    """float32 rows of 64 and of 128 tokens, which stage 64 and 128 KB; none of them is new."""
    cache = dev.KVCache(4, 128, 1, 128, fmt)
    calls = []
    for T in (64, 128):
        x = torch.zeros((1, T, 1, 128), device="cuda")
        a = (x, x, ints([[0, 1]]), ints([0]), ints([0]))
        calls.append(lambda a=a: cache.append(*a))
    at_once(zg, dev, *calls)


def test_a_large_call_and_a_small_one_in_one_graph(zg, dev):
    """Weights of 500 rows, then of one; an eviction through a wide table, then through a narrow one."""
    def state(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache = dev.KVCache(40, 16, 1, 128, "e4m3")
        cache.k_codes.view(torch.uint8).zero_(), cache.v_codes.view(torch.uint8).zero_()
        cache.k_scale.zero_(), cache.v_scale.zero_()
        x = torch.randn((2, 300, 2, 128), generator=g, device="cuda").bfloat16()
        wide = torch.zeros((1, 1 << 14), dtype=torch.int32, device="cuda")
        wide[0, :20] = torch.arange(20, device="cuda")
        narrow = torch.arange(20, 40, dtype=torch.int32, device="cuda")[None].contiguous()
        length = ints([300])
        cache.append(x[:1, :, :1], x[:1, :, 1:], wide, ints([0]))
        cache.append(x[1:, :, :1], x[1:, :, 1:], narrow, ints([0]))
        tables = (wide, narrow)
        w = [torch.zeros((1, 1, 16 * t.shape[1]), device="cuda") for t in tables]
        q = [torch.randn((1, R, 4, 128), generator=g, device="cuda").bfloat16() for R in (500, 1)]
        lse = [torch.full((1, R, 4), 3.0, device="cuda") for R in (500, 1)]
        evict = [dev.CacheEviction(cache, 1, t.shape[1], 100, 3) for t in tables]

        def run():
            for i in range(2):
                cache.add_weights(w[i], q[i], lse[i], tables[i], length)
            for i in range(2):
                evict[i](w[i], tables[i], length)

        return run, [cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, *w, *(e.kept for e in evict)]

    run, eager = state(1)
    run()
    torch.cuda.synchronize()
    run, captured = state(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    zg.zg_check_device_status(0)
    for x, y in zip(eager, captured):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
