"""What cached tokens collect of attention, and eviction by it, on the GPU against their definitions: ties, NaN and zeros
of both signs among the weights, budgets from one token to all but one, heads that keep different tokens, every format."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

QMAX = {"e4m3": 448.0, "int8": 127.0}
LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed), device="cuda")).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def build(dev, fmt, heads, dim, bt, lengths, width, seed):
    """A cache as writes leave it, blocks in no order; behind every history and in other blocks NaN."""
    B = len(lengths)
    c = dev.KVCache(B * width + 2, bt, heads, dim, fmt)
    for x in (c.k_codes, c.v_codes):
        x.view(torch.uint8).fill_(0x7F)
    for x in (c.k_scale, c.v_scale):
        x.fill_(255 if fmt == "e2m1" else math.nan)
    table = torch.randperm(B * width + 2, generator=torch.Generator().manual_seed(seed))[:B * width].to(torch.int32).cuda().view(B, width)
    x = randn((B, max(max(lengths), 1), 2 * heads, dim), torch.float32, seed)
    x *= torch.exp(randn((B, x.shape[1], 2 * heads, 1), torch.float32, seed + 1))
    c.append(x[:, :, :heads], x[:, :, heads:], table, ints([0] * B), ints(lengths))
    used = (ints(lengths) + bt - 1) // bt
    table = torch.where(torch.arange(width, device="cuda")[None] < used[:, None], table, ints([-5])[None])
    return c, table.contiguous(), ints(lengths)


def keys(c, table, b, n):
    """Keys 0 .. n - 1 of request b in 64 bits: [heads, n, dim]."""
    blk = table[b, :-(-n // c.block_tokens)].long()
    x = c.k_codes[blk].cpu()
    if x.dtype == torch.uint8:
        code = torch.stack([x & 15, x >> 4], -1).flatten(-2).long()
        s = (c.k_scale[blk].cpu().to(torch.int16) << 7).view(torch.float16).double()
        v = LEVELS[code & 7] * (1 - 2 * (code >> 3)) * s.repeat_interleave(16, -1)
    else:
        v = x.float().double() * c.k_scale[blk].cpu().double()[..., None, None]
    return v.permute(1, 0, 2, 3).reshape(c.heads, -1, c.dim)[:, :n].cuda()


# ---------------------------------------------------------------- weights

def want_weights(c, q, lse, table, length, rows, known, causal, scale, decay, w):
    """The definition in 64 bits and the bound of what 32-bit sums cost."""
    B, R, Hq, D = q.shape
    G = Hq // c.heads
    out, tol = w.double().clone(), torch.zeros_like(w, dtype=torch.float64)
    for b in range(B):
        n, nr = int(length[b]), R if rows is None else int(rows[b])
        if not n:
            continue
        old = out[b, :, :n] * decay
        old[:, n if known is None else max(int(known[b]), 0):] = 0
        if decay == 0:
            old = torch.zeros_like(old)
        k = keys(c, table, b, n)
        qq = q[b, :nr].double().view(nr, c.heads, G, D).permute(1, 2, 0, 3)
        z = qq @ k[:, None].transpose(2, 3) * scale
        size = qq.abs() @ k[:, None].abs().transpose(2, 3) * scale
        see = torch.full((nr,), n, device="cuda") - ((nr - 1 - torch.arange(nr, device="cuda")) if causal else 0)
        ls = lse[b, :nr].double().view(nr, c.heads, G).permute(1, 2, 0)[..., None]
        mask = (torch.arange(n, device="cuda")[None] < see[:, None]) & (ls > -math.inf)
        p = torch.where(mask, torch.exp(z - torch.where(ls > -math.inf, ls, torch.zeros_like(ls))), torch.zeros_like(z))
        # a term: its score's D products and sums, the factors of score and log-sum-exp, and the exponential in 32 bits
        e = p * (size * ((D + 8) * 2.0 ** -24) + (z.abs() + ls.abs().nan_to_num(posinf=0)) * 2.0 ** -21 + 2.0 ** -20)
        out[b, :, :n] = old + p.sum((1, 2))
        # a term below the smallest normal number counts as 0: off by less than 2^-126 each
        tol[b, :, :n] = nr * G * 2.0 ** -126 + e.sum((1, 2)) * 1.01 + (nr * G + 4) * 2.0 ** -24 * out[b, :, :n].abs()
    return out, tol


def check_weights(zg, dev, c, q, table, length, rows=None, known=None, causal=False, scale=None, decay=1.0, seed=1):
    B, R, Hq, _ = q.shape
    a = dev.CacheAttention(c, B, R, Hq, table.shape[1], causal=causal, scale=scale, dtype=q.dtype, lse=True)
    lse = a(q, table, length, rows)[1].clone()
    tokens = table.shape[1] * c.block_tokens + 3
    w = torch.rand((B, c.heads, tokens), generator=gen(seed), device="cuda")
    if known is not None or decay == 0:                  # what does not exist yet may be anything
        for b in range(B):
            w[b, :, 0 if decay == 0 else max(int(known[b]), 0):int(length[b])] = math.nan
    want, tol = want_weights(c, q, lse, table, length, rows, known, causal, a.scale, decay, w)
    before = w.clone()
    got = c.add_weights(w, q, lse, table, length, rows, known, causal, scale, decay)
    ok(zg)
    assert got is w and torch.isfinite(w).all()
    err = (w.double() - want).abs()
    assert (err <= tol).all(), (float((err / tol.clamp(min=1e-30)).max()), (err > tol).nonzero()[:4].tolist())
    behind = torch.arange(tokens, device="cuda")[None] >= length[:, None]
    assert torch.equal(w.transpose(0, 1)[:, behind], before.transpose(0, 1)[:, behind])
    return lse


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "e2m1"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("bt", [16, 128])
def test_weights_of_one_token(zg, dev, fmt, dim, bt):
    lengths = [0, 1, bt - 1, bt + 1, 700]
    for heads, G, dtype in ((2, 1, torch.bfloat16), (1, 3, torch.float16), (2, 8, torch.bfloat16), (1, 20, torch.float16)):
        c, table, length = build(dev, fmt, heads, dim, bt, lengths, -(-700 // bt) + 1, 3 + G)
        q = randn((5, 1, heads * G, dim), dtype, 5, scale=2.0)
        check_weights(zg, dev, c, q, table, length)
        check_weights(zg, dev, c, q, table, length, known=ints([0, 0, 5, 999, -1]), decay=0.5)


@pytest.mark.parametrize("fmt, dim", [("e4m3", 64), ("int8", 128), ("e2m1", 96), ("e2m1", 128), ("e4m3", 32)])
@pytest.mark.parametrize("R, G", [(5, 1), (33, 4), (130, 2), (300, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_weights_of_many_rows(zg, dev, fmt, dim, R, G, causal):
    """Windows of rows, ragged, some that see nothing; more rows than lie in shared memory at once."""
    lengths = [0, 1, 15, R - 1, 300, 641]
    c, table, length = build(dev, fmt, 2, dim, 32, lengths, 21, 7)
    q = randn((6, R, 2 * G + 1, dim), torch.float16 if G == 1 else torch.bfloat16, 9)[:, :, :2 * G]
    check_weights(zg, dev, c, q, table, length, ints([R, R, 3, R, 0, R - 2]), None, causal, decay=0.0 if R == 5 else 0.75)


def test_weights_of_long_histories(zg, dev):
    """Several steps a CTA; a sum over tokens that equals the number of rows."""
    c, table, length = build(dev, "e2m1", 4, 64, 64, [70000, 5, 0, 41234] * 3, 1094, 11)
    q = randn((12, 2, 8, 64), torch.bfloat16, 2)
    check_weights(zg, dev, c, q, table, length)
    a = dev.CacheAttention(c, 12, 2, 8, 1094, lse=True)
    lse = a(q, table, length)[1]
    w = torch.zeros((12, 4, 1094 * 64), device="cuda")
    c.add_weights(w, q, lse, table, length)
    ok(zg)
    total = w.double().sum(-1)
    assert ((total - 4 * (length > 0)[:, None]).abs() < 1e-4).all()          # each of 4 rows' weights sum to 1


def test_weights_of_bad_blocks_and_lengths(zg, dev):
    c, table, length = build(dev, "int8", 1, 64, 16, [100, 60], 7, 3)
    q = randn((2, 1, 1, 64), torch.bfloat16, 4)
    lse = dev.CacheAttention(c, 2, 1, 1, 7, lse=True)(q, table, length)[1]
    w = torch.ones((2, 1, 112), device="cuda")
    want = c.add_weights(w.clone(), q, lse, table, length)
    ok(zg)
    broken = table.clone()
    broken[0, 2], broken[1, 0] = -1, c.n_blocks
    got = c.add_weights(w.clone(), q, lse, broken, length)
    torch.cuda.synchronize()
    with pytest.raises(zg.ZgError, match="out of range"):
        zg.zg_check_device_status(0)
    want[0, 0, 32:48], want[1, 0, :16] = 1, 1
    assert torch.equal(got, want)
    for bad, rows in ((ints([113, 60]), None), (ints([100, -1]), None), (length, ints([2, 1]))):
        c.add_weights(w.clone(), q, lse, table, bad, rows)
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)


def test_weights_on_a_stream_and_in_a_graph(zg, dev):
    c, table, length = build(dev, "e2m1", 2, 128, 32, [100, 37], 5, 3)
    q = randn((2, 3, 4, 128), torch.bfloat16, 2)
    a = dev.CacheAttention(c, 2, 3, 4, 5, lse=True)
    w = torch.zeros((2, 2, 160), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lse = a(q, table, length)[1]
        c.add_weights(w, q, lse, table, length)
    s.synchronize()
    one = w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lse = a(q, table, length)[1]
        c.add_weights(w, q, lse, table, length)
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, one)
    graph.replay()
    ok(zg)
    assert ((w - 2 * one).abs() <= 1e-6 * one).all()


# ---------------------------------------------------------------- eviction

def want_kept(w, n, keep, recent):
    """Places that one head keeps of n tokens: by weight (NaN below all, both zeros alike), equal ones in order."""
    if n <= keep:
        return list(range(n))
    key = [-math.inf if math.isnan(x) else x for x in w[:n - recent].tolist()]
    nan = [math.isnan(x) for x in w[:n - recent].tolist()]
    by = sorted(range(n - recent), key=lambda j: (nan[j], -key[j], j))[:keep - recent]
    return sorted(by) + list(range(n - recent, n))


def recoded(codes, s0, s1, fmt):
    """Rows of codes [.., dim] of scale s0 in terms of s1, as elementary float32 operations."""
    x = codes.float() * s0[..., None]
    x = x * torch.where(s1 > 0, 1.0 / s1, torch.zeros_like(s1))[..., None]
    x = x.clamp(-QMAX[fmt], QMAX[fmt])
    return (x.round().to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)).view(torch.uint8)


def check_evict(zg, dev, c, fmt, table, length, w, keep, recent, e=None):
    B, width, bt = len(length), table.shape[1], c.block_tokens
    e = e or dev.CacheEviction(c, B, width, keep, recent)
    for x in (e.length, e.kept):
        x.view(torch.uint8).fill_(0xC3)
    want = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale, w)]
    kept = torch.full((B, c.heads, keep), -1, dtype=torch.int32, device="cuda")
    old = w.cpu()
    for b, n in enumerate(length.tolist()):
        for h in range(c.heads):
            at = torch.tensor(want_kept(old[b, h], n, keep, recent), device="cuda", dtype=torch.long)
            kept[b, h, :len(at)] = at.int()
            if n <= keep:
                continue
            i = torch.arange(keep, device="cuda")
            want[4][b, h, :keep] = w[b, h, at]
            src, dst = table[b].long()[at // bt], table[b].long()[i // bt]
            for codes, scales, wc, ws in ((c.k_codes, c.k_scale, want[0], want[2]), (c.v_codes, c.v_scale, want[1], want[3])):
                if fmt == "e2m1":
                    wc[dst, h, i % bt] = codes[src, h, at % bt]
                    ws[dst, h, i % bt] = scales[src, h, at % bt]
                    continue
                s0 = scales[src, h]
                for blk in dst.unique().tolist():
                    ws[blk, h] = s0[dst == blk].max()
                wc.view(torch.uint8)[dst, h, i % bt] = recoded(codes.view(torch.uint8)[src, h, at % bt].view(codes.dtype), s0, ws[dst, h], fmt)
    got_n, got = e(w, table, length)
    ok(zg)
    assert torch.equal(got_n, length.clamp(max=keep)) and torch.equal(got, kept)
    for x, y in zip((c.k_codes, c.v_codes, c.k_scale, c.v_scale, w), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    return e


def some_weights(B, heads, tokens, seed, levels=0):
    w = torch.exp(2 * randn((B, heads, tokens), torch.float32, seed))
    if levels:
        w = (w * levels).round() / levels
    return w


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "e2m1"])
@pytest.mark.parametrize("dim, heads, bt", [(32, 3, 16), (64, 1, 32), (96, 2, 64), (128, 2, 128), (128, 5, 16)])
@pytest.mark.parametrize("keep, recent", [(1, 0), (1, 1), (40, 7), (100, 0), (257, 257), (699, 1), (699, 350)])
def test_evict(zg, dev, fmt, dim, heads, bt, keep, recent):
    """Budgets from one token to all but one; weights with many ties."""
    lengths = [700, 0, 1, keep, keep + 1, 400]
    width = -(-max(lengths) // bt) + 1
    c, table, length = build(dev, fmt, heads, dim, bt, lengths, width, 3)
    check_evict(zg, dev, c, fmt, table, length, some_weights(6, heads, width * bt, 5, levels=2), keep, recent)


@pytest.mark.parametrize("fmt", ["int8", "e2m1"])
def test_evict_long_histories(zg, dev, fmt):
    """Clusters of several CTAs, and rows in many batches, in the first places and behind them."""
    c, table, length = build(dev, fmt, 2, 64, 64, [50000, 2900, 31111], 790, 3)
    w = some_weights(3, 2, 790 * 64 + 5, 5)
    check_evict(zg, dev, c, fmt, table, length, w, 2800, 77)
    # again, with what stands there now
    length = ints([2801, 2800, 790 * 64 - 1])
    used = (length + 63) // 64
    assert (table >= 0).sum() > 0
    table = torch.where(torch.arange(790, device="cuda")[None] < used[:, None], table, ints([-5])[None]).contiguous()
    length = torch.minimum(length, (table >= 0).sum(1).int() * 64)
    if fmt == "e2m1":
        check_evict(zg, dev, c, fmt, table, length, some_weights(3, 2, 790 * 64, 6), 2800, 2799, e=dev.CacheEviction(c, 3, 790, 2800, 2799))


def test_evict_by_special_weights(zg, dev):
    """NaN, infinities, zeros of both signs, negative weights; all weights equal."""
    c, table, length = build(dev, "e2m1", 3, 32, 16, [300, 290], 19, 3)
    w = randn((2, 3, 304), torch.float32, 5)
    w[0, 0, ::7] = math.nan
    w[0, 0, 3::11] = math.inf
    w[0, 0, 5::13] = -math.inf
    w[0, 1] = 0
    w[0, 1, ::2] = -0.0
    w[0, 2] = math.nan
    w[1, 0] = 1e-42
    w[1, 0, 100:150] = 2e-42
    w[1, 1, :200] = -math.inf
    w[1, 1, :100] = math.nan
    check_evict(zg, dev, c, "e2m1", table, length, w, 200, 20)


def test_evict_of_equal_weights_keeps_the_first(zg, dev):
    c, table, length = build(dev, "int8", 1, 64, 32, [9000], 282, 3)
    e = check_evict(zg, dev, c, "int8", table, length, torch.ones((1, 1, 9024), device="cuda"), 5000, 10)
    assert torch.equal(e.kept[0, 0, :4990], torch.arange(4990, device="cuda", dtype=torch.int32))


def test_evict_of_bad_blocks_and_lengths(zg, dev):
    """Rows from blocks outside the cache become zeros; nothing outside is touched; the next call is sound."""
    c, table, length = build(dev, "e2m1", 1, 64, 16, [100], 7, 3)
    w = some_weights(1, 1, 112, 2)
    e = dev.CacheEviction(c, 1, 7, 50, 50)
    broken = table.clone()
    broken[0, 5] = c.n_blocks + 3                       # tokens 80 .. 95: rows 30 .. 45
    before = c.k_codes.clone()
    e(w, broken, length)
    torch.cuda.synchronize()
    with pytest.raises(zg.ZgError, match="out of range"):
        zg.zg_check_device_status(0)
    out = torch.empty((1, 50, 1, 64), device="cuda")
    c.read(table, ints([0]), None, out)
    ok(zg)
    assert not out[0, 30:46].any() and out[0, :30].any() and torch.isfinite(out).all()
    assert torch.equal(c.k_codes[table[0, 4:].long()], before[table[0, 4:].long()])
    for bad in (ints([113]), ints([-1])):
        e(w.clone(), table, bad)
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)
    c, table, length = build(dev, "e2m1", 1, 64, 16, [100], 7, 3)
    check_evict(zg, dev, c, "e2m1", table, length, some_weights(1, 1, 112, 2), 50, 5)


def test_evict_on_a_stream_and_in_a_graph(zg, dev):
    """Captured and replayed over the same histories."""
    c, table, length = build(dev, "e4m3", 2, 64, 32, [300, 200], 10, 3)
    start = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    w = some_weights(2, 2, 320, 2)
    e = dev.CacheEviction(c, 2, 10, 120, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w0 = w.clone()
    with torch.cuda.stream(s):
        e(w, table, length)
    s.synchronize()
    after = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale, w, e.kept, e.length)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e(w, table, length)
    for x, y in zip((c.k_codes, c.v_codes, c.k_scale, c.v_scale, w), (*start, w0)):
        x.copy_(y)
    graph.replay()
    ok(zg)
    for x, y in zip((c.k_codes, c.v_codes, c.k_scale, c.v_scale, w, e.kept, e.length), after):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_thinned_histories_in_use(zg, dev):
    """Writes, attention, weights, eviction and further writes, as a serving loop has them: the thinned history attends
    as a history of the kept tokens alone does."""
    B, Hk, G, D, bt, width, keep, recent = 3, 2, 2, 64, 16, 10, 48, 8
    c = dev.KVCache(B * width, bt, Hk, D, "e2m1")
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda().view(B, width)
    turn = dev.NormRope(D)
    x = randn((B, 120, 2 * G + 4, D), torch.bfloat16, 4)
    pos = torch.arange(120, device="cuda", dtype=torch.int32).expand(B, 120).contiguous()
    q, k = turn(x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], pos)
    v = x[:, :, 2 * G + 2:]
    attn = dev.CacheAttention(c, B, 1, Hk * G, width, lse=True)
    evict = dev.CacheEviction(c, B, width, keep, recent)
    w = torch.full((B, Hk, width * bt), math.nan, device="cuda")
    length = ints([0, 0, 0])
    places = [[list(range(0)) for _ in range(Hk)] for _ in range(B)]          # events that each head holds
    for t in range(120):
        c.append(k[:, t:t + 1], v[:, t:t + 1], table, length)
        known, length = length, length + 1
        out, lse = attn(q[:, t:t + 1], table, length)
        c.add_weights(w, q[:, t:t + 1], lse, table, length, known=known)
        for b in range(B):
            for h in range(Hk):
                places[b][h].append(t)
        if t % 20 == 19:
            new, kept = evict(w, table, length)
            length = new.clone()
            kept = kept.cpu()
            places = [[[places[b][h][i] for i in kept[b, h].tolist() if i >= 0] for h in range(Hk)] for b in range(B)]
    ok(zg)
    assert length.tolist() == [keep] * B and torch.isfinite(w[:, :, :keep]).all()
    whole = dev.KVCache(B * width, bt, Hk, D, "e2m1")
    whole.append(k, v, table, ints([0] * B))
    kf, vf = (torch.empty((B, 120, Hk, D), device="cuda") for _ in range(2))
    whole.read(table, ints([0] * B), None, kf, vf)
    got_k, got_v = (torch.empty((B, keep, Hk, D), device="cuda") for _ in range(2))
    c.read(table, ints([0] * B), None, got_k, got_v)
    ok(zg)
    for b in range(B):
        for h in range(Hk):
            at = torch.tensor(places[b][h], device="cuda")
            assert torch.equal(got_k[b, :, h], kf[b, at, h]) and torch.equal(got_v[b, :, h], vf[b, at, h])
            assert at[-recent:].tolist() == list(range(120 - recent, 120))
    out, _ = attn(q[:, -1:], table, length)
    ok(zg)
    z = torch.einsum("bhgd,bnhd->bhgn", q[:, -1].double().view(B, Hk, G, D), got_k.double()) * D ** -0.5
    want = torch.einsum("bhgn,bnhd->bhgd", torch.softmax(z, -1), got_v.double()).reshape(B, Hk * G, D)
    # a probability as a half, 32-bit scores, one rounding to bf16
    assert ((out[:, 0].double() - want).abs() <= got_v.abs().max() * (2.0 ** -11 + 2.0 ** -16) + 2.0 ** -8 * 1.001 * want.abs() + 1e-6).all()
