"""Evictions whose kept rows do not fit a cluster's shared memory at once, and whose weights do not: rows moved in several
batches by one CTA a head and by eight, weights read from memory again, a second eviction over what the first has left."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_evict import build, check_evict, dev, ints, some_weights, zg  # noqa: E402, F401 (zg and dev are fixtures)


def plan(fmt, heads, dim, tokens, B, keep):
    """CTAs a head, batches of kept rows, and the tokens whose weights a head's CTAs hold."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ranks = 1
    while ranks < 8 and (tokens > ranks * 4096 or keep > ranks * 512) and B * heads * ranks * 2 <= sms:
        ranks *= 2
    row = dim // 2 if fmt == "e2m1" else dim
    rows = min(min(131072 // (2 * row) // 128 * 128, 1024), (-(-keep // ranks) + 127) // 128 * 128)
    return ranks, -(-keep // (ranks * rows)), ranks * 32768


# one CTA a head (more than half the SMs have one), two to five batches
@pytest.mark.parametrize("fmt, dim, bt, heads, keep, recent, batches", [
    ("e4m3", 128, 32, 2, 1601, 40, 4), ("int8", 96, 16, 2, 2900, 2899, 5), ("e2m1", 128, 128, 2, 2500, 0, 3),
    ("e4m3", 32, 64, 4, 1999, 1, 2), ("int8", 128, 128, 2, 1300, 700, 3), ("e2m1", 64, 16, 2, 1027, 5, 2)])
def test_one_cta_in_batches(zg, dev, fmt, dim, bt, heads, keep, recent, batches):  # noqa: F811
    B = 160 // heads // 2 + 1
    lengths = [(keep - 3, keep + 1, 3800, 0, keep + bt, keep)[b % 6] + (b if b % 6 == 2 else 0) for b in range(B)]
    width = -(-max(lengths) // bt) + 1
    assert plan(fmt, heads, dim, width * bt, B, keep)[:2] == (1, batches)
    c, table, length = build(dev, fmt, heads, dim, bt, lengths, width, 3)
    check_evict(zg, dev, c, fmt, table, length, some_weights(B, heads, width * bt, 5, levels=2), keep, recent)


@pytest.mark.parametrize("fmt, dim, bt, keep, batches", [("e4m3", 128, 64, 6000, 2), ("int8", 64, 16, 9001, 2), ("e2m1", 96, 32, 17000, 3)])
def test_eight_ctas_in_batches(zg, dev, fmt, dim, bt, keep, batches):  # noqa: F811
    """And again with other weights over what the first eviction has left."""
    lengths = [keep + 4000, keep + 1, 2 * keep]
    width = -(-max(lengths) // bt) + 1
    assert plan(fmt, 1, dim, width * bt, 3, keep)[:2] == (8, batches)
    c, table, length = build(dev, fmt, 1, dim, bt, lengths, width, 3)
    check_evict(zg, dev, c, fmt, table, length, some_weights(3, 1, width * bt, 5), keep, 77)
    less = keep - 1500
    check_evict(zg, dev, c, fmt, table, length.clamp(max=keep), some_weights(3, 1, width * bt, 6, levels=3), less, 3)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_weights_beyond_shared_memory(zg, dev, fmt):  # noqa: F811
    """One CTA a head holds 32,768 weights; those behind them are read again in every pass."""
    B, bt, keep = 80, 128, 2100
    lengths = [41000 if b == 3 else 33000 if b == 60 else 32768 if b == 7 else 40 * b for b in range(B)]
    width = -(-max(lengths) // bt)
    ranks, batches, held = plan(fmt, 1, 32, width * bt, B, keep)
    assert ranks == 1 and batches > 2 and held < max(lengths)
    c, table, length = build(dev, fmt, 1, 32, bt, lengths, width, 3)
    w = some_weights(B, 1, width * bt, 5, levels=1)
    w[3, 0, 30000:] *= 2                     # many of the kept ones, and of the equal ones, lie behind
    check_evict(zg, dev, c, fmt, table, length, w, keep, 5)


def test_lengths_handed_back(zg, dev):  # noqa: F811
    """A loop that adds to the returned lengths in place and hands them to the next eviction, as one that keeps copies."""
    def loop(own):
        B, width, bt = 3, 12, 16
        c = dev.KVCache(B * width, bt, 2, 64, "e2m1")
        c.k_codes.zero_(), c.v_codes.zero_(), c.k_scale.zero_(), c.v_scale.zero_()
        table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
        e = dev.CacheEviction(c, B, width, 40, 4)
        length, w = ints([0, 7, 33]), some_weights(B, 2, width * bt, 9)
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn((6, 2, B, 30, 2, 64), generator=g, device="cuda").bfloat16()
        seen = []
        for k, v in x:
            c.append(k, v, table, length)
            length += 30
            new, kept = e(w, table, length)
            length = new if own else new.clone()
            seen += [length.clone(), kept.clone()]
        return [c.k_codes, c.v_codes, c.k_scale, c.v_scale, w, *seen]

    got, want = loop(True), loop(False)
    torch.cuda.synchronize()
    zg.zg_check_device_status(0)
    assert got[-2].tolist() == [40] * 3
    for x, y in zip(got, want):
        assert torch.equal(x, y)
