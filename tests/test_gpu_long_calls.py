"""Calls of the long histories' operators that share a GPU: two streams at once, one graph after another, requests that
bring no rows, budgets above every history."""
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


def ok(zg):
    torch.cuda.synchronize()
    zg.zg_check_device_status(0)


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Work:
    """A set of buffers and the calls over them: prompt attention, a write, many rows' attention, weights, an eviction."""

    def __init__(self, dev, seed, fmt):
        self.B, self.Hq, self.Hk, self.D, self.T, self.R, self.width = 6, 4, 2, 64, 700, 40, 12
        B, D = self.B, self.D
        self.length = ints([700, 3, 0, 511, 64, 650])
        self.starts = torch.cat([ints([0]), self.length.cumsum(0, dtype=torch.int32)])
        n = int(self.starts[-1])
        self.q, self.k, self.v = (randn((n, h, D), torch.bfloat16, seed + i) for i, h in enumerate((4, 2, 2)))
        self.kk, self.vv = (randn((B, self.T, 2, D), torch.bfloat16, seed + 5 + i) for i in range(2))
        self.rows = randn((B, self.R, 4, D), torch.bfloat16, seed + 9)
        self.cache = dev.KVCache(B * self.width, 64, 2, D, fmt)
        self.table = torch.arange(B * self.width, dtype=torch.int32, device="cuda").view(B, self.width)
        self.zero = torch.zeros_like(self.length)
        self.prompt = dev.PromptAttention(4, 2, D, lse=True)
        self.attend = dev.CacheAttention(self.cache, B, self.R, 4, self.width, lse=True)
        self.evict = dev.CacheEviction(self.cache, B, self.width, 300, 20)
        self.w = torch.zeros((B, 2, self.width * 64), device="cuda")
        self.out, self.lse = torch.empty_like(self.q), torch.empty((n, 4), device="cuda")

    def run(self):
        self.w.zero_()
        self.prompt(self.q, self.k, self.v, self.starts, self.out, self.lse)
        self.cache.append(self.kk, self.vv, self.table, self.zero, self.length)
        out, lse = self.attend(self.rows, self.table, self.length)
        self.cache.add_weights(self.w, self.rows, lse, self.table, self.length)
        new, kept = self.evict(self.w, self.table, self.length)
        after, _ = self.attend(self.rows, self.table, new)
        self.results = out, lse, new, kept, after

    def taken(self):
        return [x.clone() for x in (self.out, self.lse, self.w, *self.results)]


def alike(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("fmts", [("e2m1", "int8"), ("e4m3", "e2m1")])
def test_two_streams_at_once(zg, dev, fmts):
    works = [Work(dev, 100 * i, f) for i, f in enumerate(fmts)]
    want = []
    for x in works:
        x.run()
        ok(zg)
        want.append(x.taken())
    streams = [torch.cuda.Stream() for _ in works]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for x, s in zip(works, streams):
            with torch.cuda.stream(s):
                x.run()
    ok(zg)
    for x, w in zip(works, want):
        assert alike(x.taken(), w)


def test_two_graphs_replayed_at_once(zg, dev):
    works = [Work(dev, 100 * i, "e2m1") for i in range(2)]
    want, graphs = [], []
    for x in works:
        x.run()
        ok(zg)
        want.append(x.taken())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in works]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    ok(zg)
    for x, w in zip(works, want):
        assert alike(x.taken(), w)


def test_requests_without_rows_are_decayed(zg, dev):
    x = Work(dev, 7, "int8")
    x.run()
    out, lse = x.attend(x.rows, x.table, x.length)
    w = torch.rand_like(x.w)
    before = w.clone()
    x.cache.add_weights(w, x.rows, lse, x.table, x.length, n_rows=ints([0] * 6), decay=0.5)
    ok(zg)
    held = torch.arange(w.shape[2], device="cuda")[None] < x.length[:, None]
    assert torch.equal(w, torch.where(held[:, None], before * 0.5, before))
    x.cache.add_weights(w, x.rows[:, :0], lse[:, :0].contiguous(), x.table, x.length, decay=0.5)
    ok(zg)
    assert torch.equal(w, torch.where(held[:, None], before * 0.5, before))


def test_budgets_above_every_history(zg, dev):
    x = Work(dev, 9, "e2m1")
    x.run()
    codes, w = x.cache.k_codes.clone(), x.w.clone()
    new, kept = dev.CacheEviction(x.cache, x.B, x.width, 5000, 5000)(x.w, x.table, x.length)
    ok(zg)
    assert torch.equal(new, x.length) and torch.equal(x.w, w) and torch.equal(x.cache.k_codes, codes)
    n = torch.arange(5000, device="cuda", dtype=torch.int32)
    assert torch.equal(kept, torch.where(n < x.length[:, None], n, -1)[:, None].expand(x.B, 2, 5000))
