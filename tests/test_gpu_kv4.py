"""The history cache in 4 bits on the GPU against its definition in 64 bits: the write, the read back, attention.  The
cases are the places where such kernels go wrong: ties of the rounding, scales at both ends of their range, blocks that
end inside a tile, rows that see nothing, NaN scales behind a history, every head size, offsets past 32 bits, other streams,
captured graphs."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}    # half a step, relative
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
SCALES = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)    # of every byte; NaN from 249 on


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


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def coded(x):
    """x [.., D] in 64 bits -> values [.., D] and scale bytes [.., D/16]: the nearest scale, then the nearest level, ties
    to the even byte and the even code."""
    y = np.abs(x).reshape(*x.shape[:-1], -1, 16)
    want = y.max(-1, keepdims=True) / 6
    grid = SCALES[:227]
    at = np.searchsorted(grid, want).clip(1, 226)
    lo, hi = want - grid[at - 1], grid[at] - want
    byte = np.where(hi < lo, at, np.where(lo < hi, at - 1, at - at % 2)).clip(0, 226)
    byte = np.where(want <= 0, 0, byte)
    s = grid[byte]
    # nearest level: x / s against the midpoints, a tie to the even code
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    code = np.zeros(y.shape, int)
    for i, m in enumerate(mid):
        code += (y > m * s) | ((y == m * s) & ((i + 1) % 2 == 0))
    code = np.where(s > 0, code, 0)
    return (LEVELS[code] * s).reshape(x.shape) * np.where(x < 0, -1, 1), byte[..., 0]


def values(codes, scales):
    """The cache's bytes as values in 64 bits: [blocks, heads, rows, dim]."""
    c, u = codes.cpu().numpy(), scales.cpu().numpy()
    n = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    return LEVELS[n & 7] * np.where(n & 8, -1, 1) * np.repeat(SCALES[u], 16, -1)


def new_cache(dev, n, bt, heads, dim, fill=0xFF):
    c = dev.KVCache(n, bt, heads, dim, "e2m1")
    for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale):
        x.fill_(fill)                    # NaN scales
    return c


def place(table, start, bt, T):
    p = start.cpu().numpy()[:, None] + np.arange(T)[None]
    return np.take_along_axis(table.cpu().numpy(), np.minimum(p // bt, table.shape[1] - 1), 1), p % bt


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim, heads, bt", [(32, 3, 16), (64, 1, 32), (96, 2, 64), (128, 2, 128), (128, 4, 64), (64, 70, 16)])
def test_append(zg, dev, dtype, dim, heads, bt):
    """Chunks of every kind of length, one behind the other, strided: scales and values are the definition's, exactly;
    nothing else changes."""
    B, width = 3, 8
    n_blocks = B * width + 1
    table = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(5))[:B * width].to(torch.int32).cuda().view(B, width)
    c = new_cache(dev, n_blocks, bt, heads, dim)
    start = ints([0, 0, 0])
    for step, (T, news) in enumerate([(1, [1, 1, 0]), (bt + 3, [bt + 3, 2, 1]), (5, [5, 0, 5]), (2 * bt + 1, [1, 2 * bt + 1, 17])]):
        x = randn((B, T, 2 * heads + 1, dim), dtype, 20 + step, scale=0.01 * 10.0 ** step)
        k, v = x[:, :, :heads], x[:, :, heads:2 * heads]
        sides = ((k, c.k_codes, c.k_scale), (v, c.v_codes, c.v_scale))
        want = [(codes.cpu().numpy().copy(), scales.cpu().numpy().copy()) for _, codes, scales in sides]
        c.append(k, v, table, start, ints(news))
        ok(zg)
        blk, row = place(table, start, bt, T)
        for (src, codes, scales), (old_codes, old_scales) in zip(sides, want):
            y, u = coded(src.double().cpu().numpy())
            got, gu = values(codes, scales), scales.cpu().numpy()
            for b in range(B):
                i, r = blk[b, :news[b]], row[b, :news[b]]
                assert np.array_equal(gu[i, :, r], u[b, :news[b]])
                assert np.array_equal(got[i, :, r], y[b, :news[b]])
                old_codes[i, :, r] = codes.cpu().numpy()[i, :, r]
                old_scales[i, :, r] = gu[i, :, r]
            assert np.array_equal(codes.cpu().numpy(), old_codes) and np.array_equal(gu, old_scales)
        start = start + ints(news)


def test_append_ties_and_ends(zg, dev):
    """Every scale with its ties: elements on the midpoints between levels and the numbers next to them, largest values on
    the midpoints between scales and next to them, the ends of the range."""
    rows = []
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    for byte in range(1, 227):
        s = np.float32(SCALES[byte])
        near = np.concatenate([[np.nextafter(np.float32(m * s), np.float32(d)) for d in (0, 1e9)] + [np.float32(m * s)] for m in mid[:5]])
        rows.append(np.concatenate([near, [np.float32(6 * s)]]))
        near = np.array([np.nextafter(np.float32(m * s), np.float32(d)) for m in mid[5:] for d in (0, 1e9)] + [m * s for m in mid[5:]], np.float32)
        rows.append(np.concatenate([-near, near[:6], [0, -0.0, 6 * s, 0.1 * s]]).astype(np.float32)[:16])
        if byte < 226:
            top = np.float32(6 * (SCALES[byte] + SCALES[byte + 1]) / 2)
            for t in (top, np.nextafter(top, np.float32(0)), np.nextafter(top, np.float32(1e9))):
                rows.append(np.float32(t) * np.float32([1, -1, 0.5, 0.25, 0, 1 / 12, 5 / 6, -5 / 12] * 2))
    rows += [np.full(16, x, np.float32) for x in (0, 1e-42, 2.0 ** -18, 6 * 2.0 ** -18, np.nextafter(np.float32(6 * 2.0 ** -18), np.float32(1)),
                                                  61440, 70000, 3e38, -3e38)]
    x = np.stack(rows).astype(np.float32)
    x = np.concatenate([x, np.zeros((-len(x) % 8, 16), np.float32)]).reshape(1, -1, 1, 128)
    t = torch.from_numpy(x).cuda()
    n = -(-t.shape[1] // 16)
    c = new_cache(dev, n, 16, 1, 128)
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    c.append(t, -t, table, ints([0]))
    out, out2 = torch.empty_like(t), torch.empty_like(t)
    c.read(table, ints([0]), None, out, out2)
    ok(zg)
    want, _ = coded(x.astype(np.float64))
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert np.array_equal(out2.double().cpu().numpy(), -want)


def test_append_special_values(zg, dev):
    """NaN is stored as 0, an infinity as 6 scales of the finite values; both recorded, only where they are written."""
    c = new_cache(dev, 2, 16, 1, 64)
    table = ints([[1]])
    x = randn((1, 3, 1, 64), torch.float32, 1)
    x[0, 1, 0, :5] = torch.tensor([math.nan, math.inf, -math.inf, 2.0, -3.0])
    x[0, 1, 0, 5:16] = 0.25
    x[0, 1, 0, 16:32] = math.inf           # nothing finite: 0
    x[0, 1, 0, 32:48] = -math.nan
    c.append(x, x, table, ints([0]))
    torch.cuda.synchronize()
    with pytest.raises(zg.ZgError, match="NaN or infinity"):
        zg.zg_check_device_status(0)
    out = torch.empty_like(x)
    c.read(table, ints([0]), None, out)
    ok(zg)
    assert out[0, 1, 0, :5].tolist() == [0, 3, -3, 2, -3] and not out[0, 1, 0, 16:48].any()
    y = x.clone()
    y[0, 1, 0, :48] = 0
    want, _ = coded(y.double().cpu().numpy())
    keep = torch.ones(64, dtype=torch.bool)
    keep[:16] = False
    assert np.array_equal(out.double().cpu().numpy()[0, 1, 0, keep.numpy()], want[0, 1, 0, keep.numpy()])
    assert np.array_equal(out.double().cpu().numpy()[0, [0, 2]], want[0, [0, 2]])
    # behind n_new: not read; with eps 0 a row of zeros has no norm only where it is a row
    z = torch.zeros((1, 2, 1, 64), device="cuda")
    z[0, 1] = math.nan
    c.append(z, z, table, ints([3]), ints([1]))
    c.append(z[:, :, :, :], z, table, ints([4]), ints([0]), norm_rope=dev.NormRope(64, eps=0.0))
    ok(zg)


@pytest.mark.parametrize("inter, rot", [(False, 96), (False, 48), (False, 8), (True, 96), (True, 40), (False, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_turns_keys_and_queries(zg, dev, inter, rot, dtype):
    """The fused write: queries as the stand-alone call turns them; keys as the write of keys turned alone in 32 bits,
    but for codes where the two turns' last bits fall on two sides of a midpoint."""
    B, T, Hq, Hk, D, bt = 2, 41, 6, 2, 96, 32
    x = randn((B, T, Hq + 2 * Hk, D), dtype, 31)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    g = 1 + 0.1 * randn((D,), torch.float32, 1)
    nr = dev.NormRope(D, g, g, rot_dim=rot, interleaved=inter)
    c, c2 = new_cache(dev, 9, bt, Hk, D), new_cache(dev, 9, bt, Hk, D)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    start = ints([19, 0])
    q_out = c.append(k, v, table, start, q=q, norm_rope=nr)
    pos = (start[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
    alone, _ = nr(q, None, pos)
    kf = nr(None, k.float(), pos)[1]
    c2.append(kf, v.float(), table, start)
    ok(zg)
    assert torch.equal(q_out, alone)
    assert torch.equal(c.v_codes[:8], c2.v_codes[:8]) and torch.equal(c.v_scale[:8], c2.v_scale[:8])
    a, b = (torch.empty_like(kf) for _ in range(2))
    c.read(table, start, None, a)
    c2.read(table, start, None, b)
    ok(zg)
    # a code is its neighbour only where x / s lies within 2^-20 of a midpoint: of 2.2 * 2^-20 expected
    # places an element, fewer than 1 in 1,000 elements here
    assert (a != b).float().mean() < 1e-3
    assert ((a - kf).abs() <= (kf.abs() / 3 + kf.abs().unflatten(-1, (-1, 16)).amax(-1, keepdim=True).expand(*kf.shape[:-1], D // 16, 16).flatten(-2) * 0.25)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_read(zg, dev, dtype, dim):
    """Windows of every kind back, exactly, into strided rows; rows behind them zero, others untouched."""
    c = new_cache(dev, 6, 16, 5, dim)
    x = randn((2, 40, 5, dim), torch.float32, 4)
    table = ints([[5, 0, 3], [1, 4, 2]])
    c.append(x, x * 2, table, ints([0, 0]))
    buf = torch.full((2, 50, 11, dim), 9.0, dtype=dtype, device="cuda")
    start, n = ints([3, 39]), ints([37, 1])
    c.read(table, start, n, k_out=buf[:, :, :5], v_out=buf[:, :, 6:])
    ok(zg)
    blk, row = place(table, start, 16, 50)
    for out, codes, scales in ((buf[:, :, :5], c.k_codes, c.k_scale), (buf[:, :, 6:], c.v_codes, c.v_scale)):
        want = values(codes, scales)
        for b in range(2):
            m = int(n[b])
            assert np.array_equal(out[b, :m].double().cpu().numpy(), want[blk[b, :m], :, row[b, :m]])
            assert not out[b, m:].any()
    assert (buf[:, :, 5] == 9).all()


def test_bad_tables_are_reported(zg, dev):
    c = new_cache(dev, 4, 16, 2, 64)
    x, q = randn((1, 20, 2, 64), torch.bfloat16, 1), randn((1, 1, 2, 64), torch.bfloat16, 2)
    good = ints([[2, 1]])
    attn = dev.CacheAttention(c, 1, 1, 2, 2)
    c.append(x, x, good, ints([0]))
    ok(zg)
    kept = [t.clone() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    buf = torch.empty_like(x)
    for f in (lambda: c.append(x, x, ints([[4, -1]]), ints([0])), lambda: c.append(x, x, good, ints([-1])),
              lambda: c.append(x, x, good, ints([13])), lambda: c.append(x, x, good, ints([0]), ints([21])),
              lambda: c.append(x, x, good, ints([0]), ints([-1])), lambda: c.append(x, x, good, ints([2 ** 31 - 1])),
              lambda: c.read(good, ints([14]), None, k_out=buf), lambda: c.read(ints([[0, 77]]), ints([0]), None, k_out=buf),
              lambda: c.read(good, ints([-2]), None, v_out=buf), lambda: attn(q, ints([[2, 4]]), ints([20])),
              lambda: attn(q, good, ints([33])), lambda: attn(q, good, ints([-1]))):
        f()
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)
        assert all(torch.equal(a, b) for a, b in zip(kept, (c.k_codes, c.v_codes, c.k_scale, c.v_scale)))
    check(zg, dev, c, q, good, ints([20]))


# -------------------------------------------------------------------- attention

def build(dev, heads, dim, bt, lengths, width, seed, spread=1.0):
    """A cache as writes leave it, blocks in no order, NaN scales behind every history and in every other block."""
    B = len(lengths)
    c = new_cache(dev, B * width + 2, bt, heads, dim)
    order = torch.randperm(B * width + 2, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    table = order[:B * width].view(B, width).contiguous()
    x = randn((B, max(max(lengths), 1), 2 * heads, dim), torch.float32, seed)
    x *= torch.exp(spread * randn((B, x.shape[1], 2 * heads, 1), torch.float32, seed + 1))
    c.append(x[:, :, :heads], x[:, :, heads:], table, ints([0] * B), ints(lengths))
    used = (ints(lengths) + bt - 1) // bt
    table = torch.where(torch.arange(width, device="cuda")[None] < used[:, None], table, ints([-5])[None])
    return c, table.contiguous(), ints(lengths)


def want_attention(c, q, table, length, rows, causal, scale):
    """The definition in 64 bits: outputs, log-sum-exps, and the bounds of what 32-bit sums and half operands cost."""
    B, R, Hq, D = q.shape
    G, bt = Hq // c.heads, c.block_tokens
    out = torch.zeros((B, R, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n, nr = int(length[b]), R if rows is None else int(rows[b])
        if not n or not nr:
            continue
        blk = table[b, :-(-n // bt)].long()
        k, v = (torch.from_numpy(values(x[blk], s[blk])).cuda().permute(1, 0, 2, 3).reshape(c.heads, -1, D)[:, :n]
                for x, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)))
        qq = q[b, :nr].double().view(nr, c.heads, G, D).permute(1, 2, 0, 3)          # [heads][G][nr][D]
        z = qq @ k[:, None].transpose(2, 3) * scale
        size = qq.abs() @ k[:, None].abs().transpose(2, 3) * scale
        see = torch.full((nr,), n, device="cuda") - ((nr - 1 - torch.arange(nr, device="cuda")) if causal else 0)
        mask = torch.arange(n, device="cuda")[None] < see[:, None]
        z = torch.where(mask, z, torch.full_like(z, -math.inf))
        some = see > 0
        # scores: D products and sums in 32 bits (bf16 and f16 queries are halves exactly, but for the smallest bf16)
        dz = torch.where(mask, size, torch.zeros_like(size)).amax(-1) * ((D + 8) * 2.0 ** -24)
        p = torch.nan_to_num(torch.softmax(z, -1))
        o, mass, ls = p @ v[:, None], p @ v[:, None].abs(), torch.logsumexp(z, -1)
        # probabilities: a half (2^-11), the scores' error twice (p and the sum), the exponential and the running sums in
        # 32 bits; a probability below 2^-14 of its row's reference is a subnormal half: absolute error 2^-25 each
        t = mass * (2.0 ** -11 + 2 * dz[..., None] + 2.0 ** -18)
        t = t + v.abs().amax((1, 2))[:, None, None, None] * 2.0 ** -25 * (see.clamp(min=0) / torch.exp(ls - z.amax(-1)))[..., None]
        put = lambda x: torch.where(some.view(1, 1, nr, *[1] * (x.dim() - 3)), x, torch.zeros_like(x)).permute(2, 0, 1, *range(3, x.dim())).flatten(1, 2)  # noqa: E731
        out[b, :nr], tol[b, :nr], ltol[b, :nr] = put(o), put(t), put(dz + 2.0 ** -18 + ls.abs() * 2.0 ** -22)
        lse[b, :nr] = ls.permute(2, 0, 1).flatten(1, 2)
    return out, lse, tol, ltol


def check(zg, dev, c, q, table, length, rows=None, causal=False, scale=None, a=None):
    B, R, Hq, D = q.shape
    a = a or dev.CacheAttention(c, B, R, Hq, table.shape[1], causal=causal, scale=scale, dtype=q.dtype, lse=True)
    a.out.fill_(math.nan)
    a.lse.fill_(math.nan)
    a.ws.fill_(0xFF)                                   # contents of a workspace are not defined
    got, lse = a(q, table, length, rows)
    ok(zg)
    want, wlse, tol, ltol = want_attention(c, q, table, length, rows, causal, a.scale)
    got, lse = got.double(), lse.double()
    err = (got - want).abs()
    bound = tol + U[q.dtype] * 1.001 * (want.abs() + tol) + (2.0 ** -25 if q.dtype == torch.float16 else 0)
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), (float((err / bound.clamp(min=1e-30)).max()), (err > bound).nonzero()[:4].tolist())
    assert torch.equal(lse == -math.inf, wlse == -math.inf)
    seen = wlse > -math.inf
    assert ((lse - wlse).abs()[seen] <= ltol[seen]).all(), float((lse - wlse).abs()[seen].max())
    return a


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("bt", [16, 32, 64, 128])
def test_attention_one_token(zg, dev, dim, bt):
    """Every kind of length for one token a request, shared heads or not, both types, one and two tiles of rows."""
    lengths = [0, 1, bt - 1, bt, bt + 1, 5 * bt + 7, 700]
    width = -(-700 // bt) + 1
    for heads, G, dtype in ((2, 1, torch.bfloat16), (1, 3, torch.float16), (2, 8, torch.bfloat16), (1, 20, torch.float16)):
        c, table, length = build(dev, heads, dim, bt, lengths, width, 3 + G)
        check(zg, dev, c, randn((len(lengths), 1, heads * G, dim), dtype, 5, scale=2.0), table, length)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("R, G, bt", [(33, 1, 16), (40, 3, 32), (130, 2, 64), (257, 1, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_many_rows(zg, dev, dim, R, G, bt, causal):
    """Beams and causal chunks: ragged rows, some that see nothing, histories shorter than the chunk."""
    lengths = [0, 1, 15, R - 1, 300, 641]
    c, table, length = build(dev, 2, dim, bt, lengths, -(-641 // bt), 7)
    q = randn((6, R, 2 * G, dim), torch.float16 if G == 1 else torch.bfloat16, 9, scale=2.0)
    check(zg, dev, c, q, table, length, ints([R, R, 3, R, 0, R - 2]), causal)


@pytest.mark.parametrize("R", [1, 2, 100])
def test_attention_long_histories_in_parts(zg, dev, R):
    """Histories over many CTAs, whose parts are joined; a small scale and a large one; strided queries."""
    lengths = [20000, 3, 0, 7777]
    c, table, length = build(dev, 2, 64, 64, lengths, 313, 11)
    q = randn((4, R, 9, 64), torch.bfloat16, 2)[:, :, 1:9:2]
    check(zg, dev, c, q, table, length)
    check(zg, dev, c, q.contiguous(), table, length, scale=3.0)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("R, bt, width", [(1, 64, 5), (7, 16, 40), (64, 64, 5), (64, 16, 300), (300, 32, 21)])
def test_keys_of_bad_blocks_are_left_out(zg, dev, dim, R, bt, width):
    n = [width * bt, (width - 1) * bt - 3, 2 * bt]
    c, table, length = build(dev, 2, dim, bt, n, width, 7)
    q = randn((3, R, 4, dim), torch.bfloat16, 2)
    bad = [[0, width // 2], [width - 2], [0, 1]]
    broken, kept, left = table.clone(), torch.full_like(table, -5), []
    for b, out in enumerate(bad):
        for i in out:
            broken[b, i] = c.n_blocks + 7 * i if i % 2 else -1 - i
        stay = [i for i in range(-(-n[b] // bt)) if i not in out]
        kept[b, :len(stay)] = table[b, stay]
        left.append(n[b] - sum(min(bt, n[b] - i * bt) for i in out))
    a = dev.CacheAttention(c, 3, R, 4, width, lse=True)
    got, lse = (t.clone() for t in a(q, broken, length))
    torch.cuda.synchronize()
    with pytest.raises(zg.ZgError, match="out of range"):
        zg.zg_check_device_status(0)
    want, wlse, tol, ltol = want_attention(c, q, kept, ints(left), None, False, a.scale)
    assert ((got.double() - want).abs() <= tol + U[q.dtype] * 1.001 * (want.abs() + tol)).all()
    assert torch.equal(lse == -math.inf, wlse == -math.inf) and not got[2].any()
    seen = wlse > -math.inf
    assert ((lse.double() - wlse).abs()[seen] <= ltol[seen]).all()


@pytest.mark.parametrize("R", [1, 60])
def test_scales_at_the_ends_and_special_queries(zg, dev, R):
    """Keys and values of the smallest and the largest scales; a NaN in a query shows in its own rows alone."""
    for size in (2.0 ** -15, 9000.0):
        c, table, length = build(dev, 1, 64, 32, [200, 1], 7, 13, spread=0.2)
        x = randn((2, 200, 2, 64), torch.float32, 3, scale=size)
        c.append(x[:, :, :1], x[:, :, 1:], table, ints([0, 0]), length)
        q = randn((2, R, 2, 64), torch.bfloat16, 4)
        a = check(zg, dev, c, q, table, length, scale=0.1 / size)
        q2 = q.clone()
        q2[0, 0, 1, 5] = math.nan
        before = a.out.clone()
        o, lse = a(q2, table, length)
        ok(zg)
        assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
        o[0, 0, 1], before[0, 0, 1] = 0, 0
        assert torch.equal(o, before)


def test_cache_past_32_bits(zg, dev):
    """A pool whose codes pass 4 GiB a side: blocks at its end."""
    heads, bt, dim, n = 8, 128, 128, 66000
    assert n * heads * bt * dim // 2 > 2 ** 32
    c = dev.KVCache(n, bt, heads, dim, "e2m1")
    table = ints([[n - 1, 0, n - 2], [n - 3, n - 4, 1]])
    x = randn((2, 300, heads, dim), torch.bfloat16, 2)
    c.append(x, x, table, ints([0, 0]))
    out = torch.empty_like(x)
    c.read(table, ints([0, 0]), None, k_out=out)
    ok(zg)
    want, _ = coded(x.double().cpu().numpy())
    assert np.array_equal(out.double().cpu().numpy(), want)
    check(zg, dev, c, randn((2, 1, 8, dim), torch.bfloat16, 5), table, ints([300, 257]))
    check(zg, dev, c, randn((2, 40, 8, dim), torch.bfloat16, 5), table, ints([300, 257]))


def test_other_stream_and_captured_graph(zg, dev):
    """Write, read and attention on a stream of their own, then captured and replayed over new inputs."""
    c, table, length = build(dev, 2, 128, 32, [100, 37], 5, 3)
    x, q = randn((2, 4, 4, 128), torch.bfloat16, 1), randn((2, 1, 4, 128), torch.bfloat16, 2)
    a = dev.CacheAttention(c, 2, 1, 4, 5, lse=True)
    out = torch.empty((2, 4, 2, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()

    def step():
        c.append(x[:, :, :2], x[:, :, 2:], table, length - 4, stream=None)
        c.read(table, length - 4, None, out)
        a(q, table, length)

    table = torch.where(table < 0, 0, table).contiguous()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6):
        x.copy_(randn(x.shape, torch.bfloat16, seed))
        q.copy_(randn(q.shape, torch.bfloat16, seed + 1))
        graph.replay()
        ok(zg)
        want, _ = coded(x[:, :, :2].double().cpu().numpy())
        assert np.array_equal(out.double().cpu().numpy(), want)
        replayed = a.out.clone(), a.lse.clone()
        check(zg, dev, c, q, table, length, a=a)
        assert torch.equal(replayed[0], a.out) and torch.equal(replayed[1], a.lse)


def test_empty_calls_and_refusals(zg, dev):
    c = new_cache(dev, 4, 16, 2, 64)
    x = torch.empty((1, 0, 2, 64), device="cuda", dtype=torch.bfloat16)
    t = ints([[0, 1]])
    c.append(x, x, t, ints([0]), q=x, norm_rope=dev.NormRope(64))
    c.read(t, ints([0]), None, x, x)
    ok(zg)
    assert (c.k_codes == 0xFF).all()
    for f in (lambda: dev.KVCache.over(c.k_codes, c.v_codes, c.k_scale, c.v_scale[:2]),
              lambda: dev.KVCache.over(c.k_codes, c.v_codes, c.k_scale.float(), c.v_scale.float()),
              lambda: dev.KVCache.over(c.k_codes, c.v_codes, c.k_scale[..., :2], c.v_scale[..., :2]),
              lambda: dev.KVCache.over(c.k_codes, c.k_codes.to(torch.int8), c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            f()


def test_expired_wait_is_reported(zg, dev):
    c, table, length = build(dev, 1, 64, 64, [700, 300], 11, 3)
    q = randn((2, 200, 1, 64), torch.bfloat16, 3)
    attn = dev.CacheAttention(c, 2, 200, 1, 11)
    zg.zg_debug_set_wait_limit(1)
    try:
        attn(q, table, length)
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="wait expired"):
            zg.zg_check_device_status(0)
    finally:
        zg.zg_debug_set_wait_limit(0)
    check(zg, dev, c, q, table, length)
