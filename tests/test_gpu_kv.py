"""The history cache on the GPU against its definition in 64 bits: norm and
rotation, the quantised write, the read back, attention.  The cases are the
places where such kernels go wrong: lengths of zero and one, blocks that end
inside a tile, rows that see nothing, NaN behind a history, strides, heads of
every supported size, offsets past 32 bits, other streams, captured graphs."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

QMAX = {"e4m3": 448.0, "int8": 127.0}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}    # half a step, relative


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


# ---------------------------------------------------------------- norm, rotation

def turned(x, gain, pos, rot, theta, inter, norm, eps=1e-6, freq=None):
    """The definition in 64 bits, and the size of the pair each element comes from (its error's scale)."""
    y = x.double().cpu().numpy()
    if norm:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps)
        if gain is not None:
            y = y * gain.double().cpu().numpy()
    size = np.abs(y)
    if rot:
        f = np.array(freq) if freq is not None else theta ** (-2.0 * np.arange(rot // 2) / rot)
        a = (pos.cpu().numpy().astype(np.float64)[..., None] * f)[:, :, None]
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        u, v = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a)
        size[..., ia] = size[..., ib] = np.hypot(u, v)
    return y, size


def near_turned(got, want, size, far=0):
    # 32-bit arithmetic: at most 32 roundings of the pair's size on the way (sum of squares, root, gain, sine and
    # cosine with their argument's rounding, two products), positions cost p * 2^-52 turns; then one rounding
    err = np.abs(got.double().cpu().numpy() - want)
    bound = U[got.dtype] * np.abs(want) * 1.001 + (32 * 2.0 ** -24 + far * 2.0 ** -49) * size
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim, rot, inter", [(32, 32, False), (64, 64, True), (64, 24, False), (96, 96, False),
                                             (96, 40, True), (128, 128, False), (128, 64, True), (128, 8, False),
                                             (64, 0, False)])
def test_norm_rope(zg, dev, dtype, dim, rot, inter):
    for B, T, Hq, Hk, far in ((1, 1, 1, 1, 3), (3, 1, 8, 2, 9_000_000), (2, 37, 5, 3, 200_000), (1, 2100, 4, 4, 10)):
        x = randn((B, T, Hq + Hk, dim), dtype, 7 * B + T)
        q, k = x[:, :, :Hq], x[:, :, Hq:]
        gq, gk = randn((dim,), torch.float32, 1), randn((dim,), torch.float32, 2)
        pos = (ints([[far * (b + 1)] for b in range(B)]) + torch.arange(T, device="cuda", dtype=torch.int32)[None]).contiguous()
        nr = dev.NormRope(dim, gq, gk, rot_dim=rot, theta=500000.0, interleaved=inter)
        qo, ko = nr(q, k, pos)
        ok(zg)
        for got, src, g in ((qo, q, gq), (ko, k, gk)):
            near_turned(got, *turned(src, g, pos, rot, 500000.0, inter, True), far=far * B + T)


def test_norm_rope_forms(zg, dev):
    """In place, one side only, without gains, without the norm, given frequencies, negative positions."""
    q = randn((2, 5, 3, 64), torch.float32, 3)
    pos = ints([[-7, -1, 0, 1, 2 ** 31 - 1], [5, 5, 5, 5, -2 ** 31]])
    freq = [1.0 / (i + 1) for i in range(16)]
    want = turned(q, None, pos, 32, 0, True, False, freq=freq)
    nr = dev.NormRope(64, rot_dim=32, interleaved=True, norm=False, freq=freq)
    out, none = nr(q, None, pos, q_out=q)
    ok(zg)
    assert out is q and none is None
    near_turned(q, *want, far=2 ** 31)
    k = randn((2, 5, 3, 64), torch.bfloat16, 4)
    none, ko = dev.NormRope(64, rot_dim=0)(None, k, pos)
    ok(zg)
    near_turned(ko, *turned(k, None, pos, 0, 0, False, True))
    g = randn((64,), torch.float32, 5)                   # the gains belong to the norm: without it they do nothing
    ko = dev.NormRope(64, g, g, norm=False)(None, k, pos)[1]
    ok(zg)
    near_turned(ko, *turned(k, g, pos, 64, 10000.0, False, False), far=2 ** 31)
    z = torch.zeros((1, 1, 2, 96), device="cuda")
    assert not dev.NormRope(96)(z, z, ints([[4]]))[0].any()
    ok(zg)


def test_norm_rope_refuses_shapes(dev):
    nr = dev.NormRope(64)
    q = torch.zeros((1, 2, 2, 64), device="cuda")
    for bad in (ints([[1]]), ints([[1, 2]]).long(), ints([[1, 0, 2, 0]])[:, ::2]):
        with pytest.raises(ValueError):
            nr(q, None, bad)
    with pytest.raises(ValueError):
        nr(q.transpose(2, 3).contiguous().transpose(2, 3), None, ints([[1, 2]]))
    with pytest.raises(ValueError):
        nr(q, q[:, :1], ints([[1, 2]]))
    with pytest.raises(ValueError):
        dev.NormRope(64, q_gain=torch.ones(32, device="cuda"))


# ------------------------------------------------------------------ write, read

def half_step(code, fmt):
    """Half the distance between neighbouring codes around |code| (64-bit array)."""
    if fmt == "int8":
        return np.full_like(code, 0.5)
    e = np.floor(np.log2(np.maximum(np.abs(code), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def place(table, start, bt, T):
    p = start.cpu().numpy()[:, None] + np.arange(T)[None]
    return np.take_along_axis(table.cpu().numpy(), np.minimum(p // bt, table.shape[1] - 1), 1), p % bt


def new_cache(dev, fmt, n, bt, heads, dim):
    c = dev.KVCache(n, bt, heads, dim, fmt)
    for x in (c.k_codes, c.v_codes):
        x.view(torch.uint8).fill_(0x7F)      # e4m3: NaN
    c.k_scale.fill_(math.nan)
    c.v_scale.fill_(math.nan)
    return c


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim, heads, bt", [(32, 3, 16), (64, 1, 32), (96, 2, 64), (128, 2, 128), (128, 4, 64), (64, 2, 16)])
def test_append_codes(zg, dev, fmt, dtype, dim, heads, bt):
    """Chunks of every kind of length, one behind the other: scales and codes against their definition."""
    B, width = 3, 8
    n_blocks = B * width + 1
    order = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    table = order[:B * width].view(B, width).contiguous()
    c = new_cache(dev, fmt, n_blocks, bt, heads, dim)
    start = ints([0, 0, 0])
    top = {}                                            # (side, block) -> largest |x| so far, by head
    for step, (T, news) in enumerate([(1, [1, 1, 0]), (bt + 3, [bt + 3, 2, 1]), (5, [5, 0, 5]), (bt, [bt, bt - 1, bt]),
                                      (2 * bt + 1, [1, 2 * bt + 1, 17 % (2 * bt)])]):
        x = randn((B, T, 2 * heads + 1, dim), dtype, 20 + step, scale=0.1 * 3.0 ** step)
        k, v = x[:, :, :heads], x[:, :, heads:2 * heads]
        new = ints(news)
        before = [t.view(torch.uint8).clone() for t in (c.k_codes, c.v_codes)]
        c.append(k, v, table, start, new)
        ok(zg)
        blk, row = place(table, start, bt, T)
        for side, (src, codes, scales, old) in enumerate(((k, c.k_codes, c.k_scale, before[0]), (v, c.v_codes, c.v_scale, before[1]))):
            xs = src.double().cpu().numpy()
            code, s = codes.float().double().cpu().numpy(), scales.double().cpu().numpy()
            touched = set()
            for b in range(B):
                for t in range(news[b]):
                    kb = (side, int(blk[b, t]))
                    if row[b, t] == 0:
                        top[kb] = 0
                    top[kb] = np.maximum(top.get(kb, 0), np.abs(xs[b, t]).max(-1))
                    touched.add(kb[1])
                for t in range(news[b]):
                    i = int(blk[b, t])
                    # the scale: the quotient of the largest value and Q, rounded once
                    assert np.array_equal(s[i], (top[(side, i)].astype(np.float32) / np.float32(QMAX[fmt])).astype(np.float64))
                    # the code: the nearest to x / s; the product with 1 / s costs two roundings in 32 bits
                    got = code[i, :, row[b, t]]
                    y = xs[b, t] / s[i][:, None]
                    assert (np.abs(got - y) <= half_step(got, fmt) * 1.0001 + np.abs(y) * 2.0 ** -22).all()
            for i in range(n_blocks):      # nothing else has changed
                if i not in touched:
                    assert torch.equal(codes.view(torch.uint8)[i], old[i])
        start = start + new
    # what was coded again on the way is within the roundings it went through: half a step of each code it had,
    # which no later scale makes finer
    n = int(start.max())
    ko = torch.empty((B, n, heads, dim), device="cuda")
    c.read(table, ints([0] * B), start, k_out=ko)
    ok(zg)
    assert torch.isfinite(ko).all()
    for b in range(B):
        assert not ko[b, int(start[b]):].any()


def test_append_recodes_held_rows(zg, dev):
    """A growing scale: earlier rows keep their values to half a step of the new scale (int8)."""
    c = new_cache(dev, "int8", 2, 32, 2, 64)
    table = ints([[1]])
    x = randn((1, 30, 2, 64), torch.float32, 9)
    x[:, 20:] *= 50
    for a, n in ((0, 7), (7, 1), (8, 12), (20, 1), (21, 9)):
        c.append(x[:, a:a + n], x[:, a:a + n], table, ints([a]))
    ok(zg)
    got = torch.empty_like(x)
    c.read(table, ints([0]), None, k_out=got)
    ok(zg)
    s = c.k_scale[1].double()[None, None, :, None]
    # at most five roundings of at most half the final step each
    assert ((got.double() - x.double()).abs() <= 5 * 0.5 * s * 1.001).all()
    last = (got[:, 21:].double() - x[:, 21:].double()).abs()
    assert (last <= 0.5 * s * 1.001).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim, heads, bt", [(96, 4, 16), (64, 4, 32), (128, 2, 128), (32, 1, 64)])
def test_append_codes_of_elementary_operations(zg, dev, fmt, dtype, dim, heads, bt):
    """Codes are bit for bit those of the same steps in torch's float32, where a division by a number is a product
    with its reciprocal; the stored scale is the quotient rounded once, at most two units in the last place off."""
    Q, B, T, more = QMAX[fmt], 3, 1001, 2 * bt + 5
    nb = -(-(T + more) // bt)

    def coded(y):
        y = y.clamp(-Q, Q)
        return (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)).view(torch.uint8)

    def blocks(x, first):        # [B, T, heads, dim] from row `first` of a block on -> [B, blocks, bt, heads, dim], zeros around
        n = -(-(first + x.shape[1]) // bt)
        y = torch.zeros((B, n * bt, heads, dim), device="cuda")
        y[:, first:first + x.shape[1]] = x.float()
        return y.view(B, n, bt, heads, dim)

    c = new_cache(dev, fmt, B * nb, bt, heads, dim)
    table = torch.randperm(B * nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda().view(B, nb).contiguous()
    for start, x in ((0, randn((B, T, 2 * heads, dim), dtype, 3)), (T, randn((B, more, 2 * heads, dim), dtype, 4, scale=3.0))):
        n, j, first = x.shape[1], start // bt, start % bt
        at = table[:, j:-(-(start + n) // bt)].long()
        sides = ((x[:, :, :heads], c.k_codes, c.k_scale), (x[:, :, heads:], c.v_codes, c.v_scale))
        before = [(codes.view(torch.uint8)[at[:, 0]].clone(), scales[at[:, 0]].clone()) for _, codes, scales in sides]
        c.append(x[:, :, :heads], x[:, :, heads:], table, ints([start] * B))
        ok(zg)
        for (src, codes, scales), (old, s0) in zip(sides, before):
            f = blocks(src, first)
            s = f.abs().amax((2, 4)) / Q
            if first:
                s[:, 0] = torch.maximum(s[:, 0], s0)
            inverse = 1.0 / s
            want = coded(f * inverse[:, :, None, :, None]).permute(0, 1, 3, 2, 4)
            got = codes.view(torch.uint8)[at]
            row = torch.arange(at.shape[1] * bt, device="cuda").view(1, -1, 1, bt, 1)
            assert not ((got != want) & (row >= first) & (row < first + n)).any()
            if first:                # rows held before: coded again where the scale has grown
                held = old.view(codes.dtype).float() * s0[:, :, None, None]
                again = torch.where((s[:, 0] > s0)[:, :, None, None], coded(held * inverse[:, 0, :, None, None]), old)
                assert torch.equal(got[:, 0, :, :first], again[:, :, :first])
            assert ((scales[at].double() - s.double()).abs() <= s.double() * 2.0 ** -22).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_special_values(zg, dev, fmt):
    c = new_cache(dev, fmt, 2, 16, 1, 64)
    x = torch.zeros((1, 2, 1, 64), device="cuda")
    table = ints([[0]])
    c.append(x, x, table, ints([0]))                     # all zero: scale 0, codes 0
    ok(zg)
    assert float(c.k_scale[0]) == 0 and not c.k_codes.view(torch.uint8)[0, :, :2].any()
    x[0, 0, 0, :4] = torch.tensor([1e-42, -1e-39, 0, 1e-40])      # below the smallest scale: held as zero
    c.append(x, x, table, ints([0]))
    ok(zg)
    assert float(c.v_scale[0]) == 0 and not c.v_codes[0, :, :2].float().any()     # a zero may have a sign
    x[0, 1, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 2.0])
    c.append(x, x, table, ints([0]))
    torch.cuda.synchronize()
    with pytest.raises(zg.ZgError, match="NaN or infinity"):
        zg.zg_check_device_status(0)
    got = torch.empty_like(x)
    c.read(table, ints([0]), None, k_out=got)
    ok(zg)
    assert got[0, 1, 0, :4].tolist() == [0.0, 2.0, -2.0, 2.0]
    big = torch.full((1, 1, 1, 64), 3.0e38, device="cuda")
    c.append(big, big, table, ints([0]))
    ok(zg)
    c.read(table, ints([0]), None, v_out=big)
    ok(zg)
    assert (big / 3.0e38 - 1).abs().max() < 1e-6


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_turns_keys_and_queries(zg, dev, fmt):
    """The fused write equals the turn in 64 bits to half a code's step, and turns q as the stand-alone call does."""
    B, T, Hq, Hk, D, bt = 2, 41, 6, 2, 96, 32
    x = randn((B, T, Hq + 2 * Hk, D), torch.bfloat16, 31)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    g = randn((D,), torch.float32, 1)
    nr = dev.NormRope(D, g, g, rot_dim=48)
    c = new_cache(dev, fmt, 9, bt, Hk, D)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4).contiguous()
    start = ints([19, 0])
    c.append(k[:, :19].contiguous(), v[:, :19].contiguous(), table, ints([0, 0]), ints([19, 0]))   # rows held before
    q_out = c.append(k, v, table, start, q=q, norm_rope=nr)
    pos = (start[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
    alone, _ = nr(q, None, pos)
    ok(zg)
    assert torch.equal(q_out, alone)
    plain = c.append(k, v, table, start, q=q, norm_rope=dev.NormRope(D, g, g, norm=False, rot_dim=96, interleaved=True))
    ok(zg)
    near_turned(plain, *turned(q, g, pos, 96, 10000.0, True, False), far=100)
    c.append(k[:, :19].contiguous(), v[:, :19].contiguous(), table, ints([0, 0]), ints([19, 0]))
    c.append(k, v, table, start, q=q, norm_rope=nr)
    ok(zg)
    want, size = turned(k, g, pos, 48, 10000.0, False, True)
    blk, row = place(table, start, bt, T)
    code, s = c.k_codes.float().double().cpu().numpy(), c.k_scale.double().cpu().numpy()
    for b in range(B):
        for t in range(T):
            got, sc = code[blk[b, t], :, row[b, t]], s[blk[b, t]][:, None]
            err = np.abs(got * sc - want[b, t])
            assert (err <= half_step(got, fmt) * sc * 1.0001 + 40 * 2.0 ** -24 * size[b, t]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_read(zg, dev, dtype):
    for fmt, dim in (("e4m3", 96), ("int8", 32)):
        c = new_cache(dev, fmt, 6, 16, 3, dim)
        x = randn((2, 40, 3, dim), torch.float32, 4)
        table = ints([[5, 0, 3], [1, 4, 2]])
        c.append(x, x * 2, table, ints([0, 0]))
        buf = torch.full((2, 50, 8, dim), 9.0, dtype=dtype, device="cuda")
        start, n = ints([3, 39]), ints([37, 1])
        c.read(table, start, n, k_out=buf[:, :, 1:4], v_out=buf[:, :, 5:])
        ok(zg)
        blk, row = place(table, start, 16, 50)
        for out, codes, scales in ((buf[:, :, 1:4], c.k_codes, c.k_scale), (buf[:, :, 5:], c.v_codes, c.v_scale)):
            cd, sc = codes.float().double().cpu().numpy(), scales.double().cpu().numpy()
            for b in range(2):
                m = int(n[b])
                want = cd[blk[b, :m], :, row[b, :m]] * sc[blk[b, :m]][..., None]
                err = np.abs(out[b, :m].double().cpu().numpy() - want)
                # the product is rounded to 32 bits, then to the output's type
                assert (err <= (U[dtype] + 2.0 ** -24) * 1.001 * np.abs(want) + 2.0 ** -25).all()
                assert not out[b, m:].any()
        assert (buf[:, :, 0] == 9).all() and (buf[:, :, 4] == 9).all()


def test_bad_tables_are_reported(zg, dev):
    """Blocks and lengths outside the cache: left out, recorded, and the next call is sound."""
    c = new_cache(dev, "e4m3", 4, 16, 2, 64)
    x = randn((1, 20, 2, 64), torch.bfloat16, 1)
    q = randn((1, 1, 2, 64), torch.bfloat16, 2)
    good = ints([[2, 1]])
    attn = dev.CacheAttention(c, 1, 1, 2, 2)
    c.append(x, x, good, ints([0]))
    ok(zg)
    kept = c.k_codes.view(torch.uint8).clone()
    buf = torch.empty_like(x)
    for f in (lambda: c.append(x, x, ints([[4, -1]]), ints([0])), lambda: c.append(x, x, good, ints([-1])),
              lambda: c.append(x, x, good, ints([13])), lambda: c.append(x, x, good, ints([0]), ints([21])),
              lambda: c.append(x, x, good, ints([0]), ints([-1])), lambda: c.read(good, ints([14]), None, k_out=buf),
              lambda: c.read(ints([[0, 77]]), ints([0]), None, k_out=buf), lambda: c.read(good, ints([-2]), None, v_out=buf),
              lambda: attn(q, ints([[2, 4]]), ints([20])), lambda: attn(q, good, ints([33])),
              lambda: attn(q, good, ints([-1])), lambda: attn(q, good, ints([20]), ints([2]))):
        f()
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)
        assert torch.equal(c.k_codes.view(torch.uint8), kept)
    check_attention(zg, dev, c, q, good, ints([20]), None, False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("R, bt, width", [(1, 64, 5), (7, 16, 40), (64, 64, 5), (64, 16, 300), (300, 32, 21)])
def test_keys_of_bad_blocks_are_left_out(zg, dev, fmt, dim, R, bt, width):
    """Blocks outside the cache, first, in the middle, at a history's end: recorded, and the rest of the history is
    attended to as if their keys were not there, for few rows and many; a history of such blocks alone gives nothing."""
    n = [width * bt, (width - 1) * bt - 3, 2 * bt]
    c, table, length = build(dev, fmt, 3, 2, dim, bt, n, width, 7)
    q = randn((3, R, 4, dim), torch.bfloat16, 2)
    bad = [[0, width // 2], [width - 2], [0, 1]]
    broken = table.clone()
    kept, left = torch.full_like(table, -5), []
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
    err = (got.double().cpu() - want).abs()
    assert (err <= tol + U[q.dtype] * 1.001 * (want.abs() + tol)).all()
    assert torch.equal(lse.cpu() == -math.inf, wlse == -math.inf) and not got[2].any()
    seen = wlse > -math.inf
    assert ((lse.double().cpu() - wlse).abs()[seen] <= ltol[seen]).all()


# -------------------------------------------------------------------- attention

def fill(c, seed):
    """Codes and scales of any size within the format, NaN codes never among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for codes, scales in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        m = 127 if codes.dtype == torch.int8 else 448
        x = (torch.randn(codes.shape, generator=g, device="cuda") * (m / 4)).clamp(-m, m)
        codes.copy_(x.round().to(codes.dtype) if codes.dtype == torch.int8 else x.to(codes.dtype))
        scales.copy_(4.0 / m * torch.exp(1.5 * torch.randn(scales.shape, generator=g, device="cuda")))


def behind(c, table, length):
    """NaN codes behind every request's last token."""
    if c.k_codes.dtype == torch.int8:
        return
    bt = c.block_tokens
    for b, n in enumerate(length.tolist()):
        if n % bt:
            for x in (c.k_codes, c.v_codes):
                x.view(torch.uint8)[int(table[b, n // bt]), :, n % bt:] = 0x7F


def want_attention(c, q, table, length, rows, causal, scale):
    """The definition in 64 bits: outputs, log-sum-exps, and the bounds of what 32-bit sums and half operands cost."""
    B, R, Hq, D = q.shape
    G, bt = Hq // c.heads, c.block_tokens
    out = torch.zeros((B, R, Hq, D), dtype=torch.float64)
    lse = torch.full((B, R, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n, nr = int(length[b]), R if rows is None else int(rows[b])
        if not n:
            continue
        blk = table[b, :-(-n // bt)].long()
        k, v = ((x[blk].float().double() * s[blk].double()[..., None, None]).permute(1, 0, 2, 3).reshape(c.heads, -1, D)[:, :n].cpu()
                for x, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)))
        for r in range(nr):
            see = n - (nr - 1 - r) if causal else n
            if see <= 0:
                continue
            qq = q[b, r].double().cpu().view(c.heads, G, 1, D)
            z = (qq * k[:, None, :see]).sum(-1) * scale
            # scores: D products and sums in 32 bits, q rounded to a half (relative 2^-11) unless it is one already
            dz = ((qq.abs() * k[:, None, :see].abs()).sum(-1) * scale).amax(-1) * ((D + 8) * 2.0 ** -24)
            p = torch.softmax(z, -1)
            out[b, r] = (p @ v[:, :see]).reshape(Hq, D)
            lse[b, r] = torch.logsumexp(z, -1).reshape(Hq)
            mass = (p @ v[:, :see].abs()).reshape(Hq, D)
            # probabilities: a half (2^-11), the scores' error twice (p and the sum), the exponential and the
            # running sums in 32 bits
            tol[b, r] = mass * (2.0 ** -11 + 2 * dz.reshape(Hq)[:, None] + 2.0 ** -18)
            # a probability below 2^-14 of its row's reference is a subnormal half: absolute error 2^-25 each
            big = v[:, :see].abs().amax((1, 2)).repeat_interleave(G)[:, None]
            tol[b, r] += big * 2.0 ** -25 * (see / torch.exp(torch.logsumexp(z, -1) - z.amax(-1))).reshape(Hq)[:, None]
            ltol[b, r] = dz.reshape(Hq) + 2.0 ** -18 + lse[b, r].abs() * 2.0 ** -22
    return out, lse, tol, ltol


def check_attention(zg, dev, c, q, table, length, rows, causal, scale=None, out=None):
    B, R, Hq, D = q.shape
    a = dev.CacheAttention(c, B, R, Hq, table.shape[1], causal=causal, scale=scale, dtype=q.dtype, lse=True)
    a.out.fill_(math.nan)
    a.lse.fill_(math.nan)
    a.ws.fill_(0xFF)                                   # contents of a workspace are not defined
    got, lse = a(q, table, length, rows)
    ok(zg)
    want, wlse, tol, ltol = want_attention(c, q, table, length, rows, causal, a.scale)
    got, lse = got.double().cpu(), lse.double().cpu()
    err = (got - want).abs()
    bound = tol + U[q.dtype] * 1.001 * (want.abs() + tol) + (2.0 ** -25 if q.dtype == torch.float16 else 0)
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), (float((err / bound.clamp(min=1e-30)).max()), (err > bound).nonzero()[:4].tolist())
    assert torch.equal(lse == -math.inf, wlse == -math.inf)
    seen = wlse > -math.inf
    assert ((lse - wlse).abs()[seen] <= ltol[seen]).all(), float((lse - wlse).abs()[seen].max())
    return a


def build(dev, fmt, B, heads, dim, bt, lengths, width, seed):
    c = dev.KVCache(B * width + 2, bt, heads, dim, fmt)
    fill(c, seed)
    order = torch.randperm(B * width + 2, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    table = order[:B * width].view(B, width).contiguous()
    length = ints(lengths)
    behind(c, table, length)
    used = (length + bt - 1) // bt
    table = torch.where(torch.arange(width, device="cuda")[None] < used[:, None], table, ints([-5])[None])
    return c, table.contiguous(), length


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("bt", [16, 32, 64, 128])
def test_attention_one_token(zg, dev, fmt, dim, bt):
    """Every kind of length for one token a request, shared heads or not, both types."""
    lengths = [0, 1, bt - 1, bt, bt + 1, 5 * bt + 7, 700]
    width = -(-700 // bt) + 1
    for heads, G, dtype in ((2, 1, torch.bfloat16), (1, 3, torch.float16), (2, 8, torch.bfloat16), (1, 20, torch.float16)):
        c, table, length = build(dev, fmt, len(lengths), heads, dim, bt, lengths, width, 3 + G)
        q = randn((len(lengths), 1, heads * G, dim), dtype, 5, scale=2.0)
        check_attention(zg, dev, c, q, table, length, None, False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim, heads, G, bt", [(64, 2, 1, 16), (128, 1, 1, 64), (96, 2, 2, 32), (32, 1, 4, 128), (128, 2, 4, 16), (64, 1, 3, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_many_rows(zg, dev, fmt, dim, heads, G, bt, causal):
    """Beams and causal chunks: rows that see nothing, fewer rows than R, lengths around tiles."""
    for R, lengths, rows in ((9, [0, 5, 64, 200], [9, 9, 1, 0]), (65, [1, 64, 129, 300], [65, 64, 65, 7]),
                             (150, [40, 128, 257, 500], None)):
        c, table, length = build(dev, fmt, 4, heads, dim, bt, lengths, -(-500 // bt), R)
        q = randn((4, R, heads * G, dim), torch.bfloat16 if R != 65 else torch.float16, R, scale=2.0)
        check_attention(zg, dev, c, q, table, length, ints(rows) if rows else None, causal)


def test_attention_long(zg, dev):
    """Long histories: the keys split over many parts, lengths that leave most parts empty."""
    c, table, length = build(dev, "e4m3", 3, 1, 64, 64, [20011, 3, 9000], 320, 8)
    q = randn((3, 1, 2, 64), torch.bfloat16, 1, scale=3.0)
    check_attention(zg, dev, c, q, table, length, None, False)
    q = randn((3, 33, 2, 64), torch.float16, 1)
    check_attention(zg, dev, c, q, table, length, ints([33, 5, 1]), True)


def test_attention_extremes(zg, dev):
    """Scores and scales over many orders: the running maximum and reference scale move on every tile."""
    for fmt in ("e4m3", "int8"):
        c, table, length = build(dev, fmt, 2, 1, 64, 16, [333, 200], 24, 4)
        ramp = torch.exp2(torch.arange(24, device="cuda").float() * 1.7 - 20)
        for b in range(2):
            used = table[b][table[b] >= 0].long()
            c.v_scale[used, 0] = ramp[:len(used)] if b == 0 else ramp[:len(used)].flip(0)
        c.v_scale[table[1, 2].long()] = 0
        q = randn((2, 3, 4, 64), torch.bfloat16, 6, scale=30.0)
        q[0, 1] = 0                                              # uniform weights
        q[1, 2] *= 1e4
        check_attention(zg, dev, c, q, table, length, None, False, scale=0.02)
        check_attention(zg, dev, c, (q * 1e30).to(torch.bfloat16), table, length, None, True, scale=1e-32)
        q = randn((2, 140, 4, 64), torch.bfloat16, 6, scale=30.0)
        check_attention(zg, dev, c, q, table, length, None, False, scale=0.02)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_scale_of_unseen_blocks(zg, dev, fmt):
    """A value scale of a block that a causal row does not see leaves the row's precision alone; nor does a large
    scale that a row sees with no weight."""
    for R in (10, 90):
        c, table, length = build(dev, fmt, 1, 1, 64, 16, [96], 6, 9)
        for j, x in enumerate((1.0, 2.0 ** 30, 2.0 ** -30, 1.0, 2.0 ** 60, 2.0 ** 90)):
            c.v_scale[table[0, j].long()] = x
        q = randn((1, R, 2, 64), torch.bfloat16, 6, scale=2.0)
        check_attention(zg, dev, c, q, table, length, None, True)
        # keys of the large blocks far below the others: their weight times their values is nothing
        blk = table[0].long()
        c.v_scale[blk] = torch.tensor([[1.0], [4.0], [1.0], [2.0 ** 18], [1.0], [2.0 ** 20]], device="cuda")
        for j in (3, 5):
            c.k_codes.view(torch.uint8)[blk[j]] = c.k_codes.view(torch.uint8)[blk[j], :, :1].clone()
        q = (-40 * torch.sign(c.k_codes[blk[3], 0, 0].float() + c.k_codes[blk[5], 0, 0].float())).expand(1, R, 2, 64).to(torch.bfloat16).contiguous()
        check_attention(zg, dev, c, q, table, length, None, False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("factor", [2.0 ** -96, 2.0 ** -105, 2.0 ** -112, 2.0 ** 60, 2.0 ** 115])
@pytest.mark.parametrize("R, n", [(1, 320), (12, 5000), (64, 700), (150, 3000)])
def test_attention_value_scales_of_any_size(zg, dev, fmt, factor, R, n):
    """Value scales from the smallest that a write holds (2^-126) up to where values leave 32 bits."""
    c, table, length = build(dev, fmt, 2, 1, 64, 64, [n, 77], -(-n // 64), 3)
    c.v_scale.copy_((c.v_scale * factor).clamp(2.0 ** -126, 2.0 ** 118))
    c.v_scale[table[1, 0].long()] = 0                # a block of nothing first
    c.v_codes.view(torch.uint8)[table[1, 0].long()] = 0
    check_attention(zg, dev, c, randn((2, R, 2, 64), torch.bfloat16, 2), table, length, None, False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("bt", [16, 64])
@pytest.mark.parametrize("R, n", [(1, 700), (10, 4000), (64, 700), (150, 3000)])
def test_attention_blocks_of_nothing(zg, dev, fmt, bt, R, n):
    """Blocks whose values are all zero (scale 0) weigh in the softmax, whatever the scales around them: at the
    beginning, between and at the end, beside scales of 2^40 and of 2^-40, and alone."""
    c, table, length = build(dev, fmt, 4, 1, 64, bt, [n, n - 1, n // 2, 100], -(-n // bt), 3)
    g = torch.Generator().manual_seed(5)
    for b, factor in ((0, 2.0 ** 40), (1, 2.0 ** -40), (2, None), (3, 0)):
        blk = table[b][table[b] >= 0].long()
        f = torch.full((len(blk), 1), 1.0 if factor is None else factor, device="cuda")
        if factor is None:
            f = torch.exp2(torch.randint(-50, 50, (len(blk), 1), generator=g).float()).cuda()
        none = (torch.rand(len(blk), generator=g) < 0.5).cuda()
        none[0] = True
        f[none] = 0
        c.v_scale[blk] *= f
        c.v_codes.view(torch.uint8)[blk[none]] = 0
    check_attention(zg, dev, c, randn((4, R, 2, 64), torch.bfloat16, 2), table, length, None, False)
    check_attention(zg, dev, c, randn((4, R, 2, 64), torch.bfloat16, 4), table, length, None, True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale", [1e2, 1e6, 1e8, 1e12, 1e30])
@pytest.mark.parametrize("R, n", [(1, 320), (64, 320), (200, 2000)])
def test_attention_scores_of_any_size(zg, dev, dim, R, n, scale):
    """Scores far past the size at which 32 bits hold single units: finite, one value or a mean of values as near as
    the scores' own rounding leaves them."""
    c, table, length = build(dev, "int8", 1, 1, dim, 64, [n], -(-n // 64), 3)
    check_attention(zg, dev, c, randn((1, R, 2, dim), torch.bfloat16, 3), table, length, None, False, scale=scale)
    same = c.k_codes[table[0, 0].long(), :, :1].clone()              # all keys of the second block alike
    c.k_codes[table[0, 1].long()] = same
    check_attention(zg, dev, c, randn((1, R, 2, dim), torch.float16, 4), table, length, None, True, scale=scale)


@pytest.mark.parametrize("top", [1e-38, 1e-30, 1.6e38, 2e38, 3.2e38])
@pytest.mark.parametrize("R", [1, 10, 64, 200])
def test_attention_queries_of_any_size(zg, dev, R, top):
    """Query rows up to the largest bf16 and down to the smallest normal ones, beside one of ordinary size."""
    c, table, length = build(dev, "int8", 1, 1, 64, 64, [320], 5, 3)
    q = randn((1, R, 2, 64), torch.float32, 2)
    q = q / q.abs().amax(-1, keepdim=True) * top
    q[0, R // 2, 1] = randn((64,), torch.float32, 3)
    q = q.to(torch.bfloat16)
    assert torch.isfinite(q).all()
    check_attention(zg, dev, c, q, table, length, None, False, scale=min(2.0 / top, 1e30))


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("R, n", [(1, 320), (1, 5000), (3, 320), (11, 9000), (64, 320), (64, 20000), (120, 90), (300, 5000)])
def test_attention_of_a_nan(zg, dev, R, n, causal, value):
    """A query row with a NaN (or an infinity: codes of both signs and none) has NaN for its output and its
    log-sum-exp, in one part and in many; the rows beside it are none the wiser, and a row that sees nothing stays
    empty whatever its query holds."""
    c, table, length = build(dev, "int8", 2, 1, 64, 64, [n, 70], -(-n // 64), 3)
    c.k_codes[table[:, 0].long(), :, :, 5] = torch.tensor([0, 1, -1, 2], dtype=torch.int8, device="cuda").repeat(16)
    q = randn((2, R, 2, 64), torch.bfloat16, 2)
    bad = R // 2
    want = q.clone()
    q[:, bad, 1, 5] = value
    rows = ints([R, max(1, R - 2)])
    q[1, R - 1, :, 7] = value              # a row behind the last but for R of 1
    a = dev.CacheAttention(c, 2, R, 2, table.shape[1], causal=causal, lse=True)
    o1, l1 = (t.clone() for t in a(want, table, length, rows))
    o2, l2 = a(q, table, length, rows)
    ok(zg)
    sees = torch.tensor([[(m - (nr - 1 - r) if causal else m) if r < nr else 0 for r in range(R)]
                         for m, nr in zip((n, 70), rows.tolist())], device="cuda") > 0
    hit = torch.zeros((2, R, 2), dtype=torch.bool, device="cuda")
    hit[:, bad, 1] = True
    hit[1, R - 1] = True
    hit &= sees[..., None]
    assert hit.any() and torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], o1[~hit]) and torch.equal(l2[~hit], l1[~hit])
    assert not o2[~sees].any() and (l2[~sees] == -math.inf).all()


def test_attention_strides_and_streams(zg, dev):
    """q inside a packed buffer, outputs into a wider one, on a stream that is not the current one."""
    c, table, length = build(dev, "int8", 2, 2, 64, 32, [100, 77], 5, 2)
    for R in (1, 70):
        x = randn((2, R, 8, 64), torch.bfloat16, 11)
        want = dev.CacheAttention(c, 2, R, 4, 5)(x[:, :, 2:6].contiguous(), table, length)[0].clone()
        wide = torch.zeros((2, R, 9, 68), dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(zg.zg_kv_attention_workspace_size(c.struct, 5, 2, R, 4), dtype=torch.uint8, device="cuda")
        q = x[:, :, 2:6]
        o = wide[:, :, 5:]
        zg.zg_kv_attention(c.struct, table, 5, length, None, zg.make_rows(q, zg.ZG_BF16, *q.stride()[:3]),
                           zg.make_rows(o, zg.ZG_BF16, *o.stride()[:3]), None, 2, R, 4, 0.125, False, ws, ws.numel(),
                           s.cuda_stream)
        s.synchronize()
        ok(zg)
        assert torch.equal(o[..., :64], want) and not wide[:, :, :5].any() and not wide[..., 64:].any()


def test_new_outputs_on_another_stream(zg, dev):
    """Outputs made by a call on a stream that is not the current one are none of the current stream's memory: blocks
    given back there may still be read by queued work."""
    q = randn((4, 300, 4, 64), torch.bfloat16, 1)
    pos = torch.arange(300, dtype=torch.int32, device="cuda").repeat(4, 1).contiguous()
    nr = dev.NormRope(64)
    c = new_cache(dev, "int8", 80, 16, 4, 64)
    table = torch.arange(80, dtype=torch.int32, device="cuda").view(4, 20).contiguous()
    start = ints([0] * 4)
    want = nr(q, None, pos)[0].clone()
    ok(zg)
    free = [torch.empty_like(q) for _ in range(4)]
    mine = {x.data_ptr() for x in free}
    del free                                     # four blocks of the outputs' size in the current stream's memory
    for handle in (torch.cuda.Stream().cuda_stream, 0):
        with torch.cuda.stream(torch.cuda.Stream()) if handle == 0 else torch.cuda.stream(None):
            here = [torch.empty_like(q) for _ in range(4)]
            taken = mine | {x.data_ptr() for x in here}
            del here
            outs = [*nr(q, q, pos, stream=handle), c.append(q, q, table, start, q=q, norm_rope=nr, stream=handle)]
        ok(zg)
        assert all(torch.equal(o, want) for o in outs)
        if handle:
            assert not taken & {o.data_ptr() for o in outs}


def test_attention_in_a_graph(zg, dev):
    """Write, then attend, captured once and replayed on new data."""
    c = new_cache(dev, "e4m3", 8, 16, 2, 64)
    table = ints([[3, 1], [0, 6]])
    x = randn((2, 3, 8, 64), torch.bfloat16, 2)
    start, length = ints([0, 0]), ints([3, 3])
    nr = dev.NormRope(64)
    attn = dev.CacheAttention(c, 2, 3, 4, 2, causal=True)
    q = torch.empty((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")

    def step():
        c.append(x[:, :, 4:6], x[:, :, 6:], table, start, q=x[:, :, :4], q_out=q, norm_rope=nr)
        attn(q, table, length)

    step()
    ok(zg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(randn((2, 3, 8, 64), torch.bfloat16, 3))
    start.copy_(ints([3, 3]))
    length.copy_(ints([6, 6]))
    g.replay()
    ok(zg)
    got = attn.out.clone()
    step()
    ok(zg)
    assert torch.equal(got, attn.out)
    check_attention(zg, dev, c, q, table, ints([3, 3]), None, True)


@pytest.mark.parametrize("R", [1, 10, 160])
def test_split_attention_in_a_graph(zg, dev, R):
    """A history in many parts, captured: replays follow the lengths that the device holds then."""
    c, table, length = build(dev, "int8", 2, 1, 64, 64, [5000, 3000], 80, 5)
    q = randn((2, R, 2, 64), torch.bfloat16, 5)
    attn = dev.CacheAttention(c, 2, R, 2, 80, lse=True)
    assert attn.ws_bytes > 0
    attn(q, table, length)
    ok(zg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn(q, table, length)
    for lengths in ([100, 2999], [4999, 0], [5000, 3000]):
        length.copy_(ints(lengths))
        g.replay()
        ok(zg)
        got, lse = attn.out.clone(), attn.lse.clone()
        attn(q, table, length)
        ok(zg)
        assert torch.equal(got, attn.out) and torch.equal(lse, attn.lse)
    check_attention(zg, dev, c, q, table, length, None, False)


def test_attention_repeats(zg, dev):
    """The same call gives the same bits."""
    c, table, length = build(dev, "e4m3", 5, 2, 128, 64, [5000, 0, 1, 4097, 300], 90, 12)
    for R in (1, 200):
        q = randn((5, R, 4, 128), torch.bfloat16, 3)
        a = dev.CacheAttention(c, 5, R, 4, 90, lse=True)
        o, l = (t.clone() for t in a(q, table, length))
        for _ in range(3):
            o2, l2 = a(q, table, length)
            assert torch.equal(o, o2) and torch.equal(l, l2)


def test_parts_merge_by_lse(zg, dev):
    """Two halves of a history, each with its own table, merged by their log-sum-exps."""
    c, table, length = build(dev, "int8", 1, 1, 64, 16, [160], 10, 3)
    q = randn((1, 40, 2, 64), torch.float16, 3)
    whole = check_attention(zg, dev, c, q, table, length, None, False)
    o1, l1 = (t.clone() for t in dev.CacheAttention(c, 1, 40, 2, 4, dtype=q.dtype, lse=True)(q, table[:, :4].contiguous(), ints([64])))
    o2, l2 = dev.CacheAttention(c, 1, 40, 2, 6, dtype=q.dtype, lse=True)(q, table[:, 4:].contiguous(), ints([96]))
    w = torch.softmax(torch.stack([l1, l2]), 0)[..., None]
    merged = w[0] * o1.float() + w[1] * o2.float()
    # three results, each within half a step of its type and 2^-10 of the values' size
    assert (merged - whole.out.float()).abs().max() <= 3 * 2.0 ** -10 * float((o1.abs().max() + o2.abs().max()))


def test_attention_of_tables_near_2_31_tokens(zg, dev):
    """A length of 2^31 - 2^20 beside a short one: a table of one block again and again, so that outputs are the block's own and the
    log-sum-exp grows by the logarithm of its count."""
    B, blocks, bt, D = 2, 2 ** 24 - 2 ** 13, 128, 32
    c = dev.KVCache(2, bt, 1, D, "int8")
    fill(c, 1)
    table = torch.zeros((B, blocks), dtype=torch.int32, device="cuda")
    lengths = [blocks * bt] + [bt] * (B - 1)
    q = randn((B, 64, 1, D), torch.bfloat16, 2)
    o, lse = dev.CacheAttention(c, B, 64, 1, blocks, lse=True)(q, table, ints(lengths))
    o1, l1 = dev.CacheAttention(c, B, 64, 1, 1, lse=True)(q, table[:, :1].contiguous(), ints([bt] * B))
    ok(zg)
    gain = torch.tensor([math.log(n / bt) for n in lengths], device="cuda")[:, None, None]
    # each part's sums are of 2^25 / 16 terms in 32 bits, each rounded to 2^-24: a drift of 1 / 8 at most
    assert ((lse - l1 - gain).abs() < 0.25).all(), float((lse - l1 - gain).abs().max())
    assert torch.equal(o[1:], o1[1:])
    # weights and their sum drift apart by as much at most
    assert ((o - o1).abs().float() < 0.25 * float(o1.abs().max())).all()


def test_cache_past_32_bits(zg, dev):
    """A pool whose codes pass 4 GiB a side: blocks at its end."""
    heads, bt, dim, n = 8, 128, 128, 33000
    assert n * heads * bt * dim > 2 ** 32
    c = dev.KVCache(n, bt, heads, dim, "int8")
    table = ints([[n - 1, 0, n - 2], [n - 3, n - 4, 1]])
    for b in table.flatten().tolist():
        for x in (c.k_codes, c.v_codes):
            x[b].fill_(0)
    x = randn((2, 300, heads, dim), torch.bfloat16, 2)
    c.append(x, x, table, ints([0, 0]))
    out = torch.empty_like(x)
    c.read(table, ints([0, 0]), None, k_out=out)
    ok(zg)
    assert ((out.float() - x.float()).abs() <= x.float().abs() * 2.0 ** -8 + 6.0 / 254 * 1.01).all()
    check_attention(zg, dev, c, randn((2, 1, 8, dim), torch.bfloat16, 5), table, ints([300, 257]), None, False)
    check_attention(zg, dev, c, randn((2, 20, 8, dim), torch.bfloat16, 5), table, ints([300, 257]), None, False)


def test_empty_tensors(zg, dev):
    """Calls of no tokens or no requests: nothing runs, nothing changes."""
    c = new_cache(dev, "int8", 4, 16, 2, 64)
    x = torch.empty((1, 0, 2, 64), device="cuda", dtype=torch.bfloat16)
    t = ints([[0, 1]])
    c.append(x, x, t, ints([0]), q=x, norm_rope=dev.NormRope(64))
    c.read(t, ints([0]), None, x, x)
    assert dev.NormRope(64)(x, x, torch.empty((1, 0), dtype=torch.int32, device="cuda"))[0].shape == x.shape
    assert dev.CacheAttention(c, 1, 0, 2, 2)(x, t, ints([5]))[0].numel() == 0
    ok(zg)
    assert (c.k_codes.view(torch.uint8) == 0x7F).all()


def test_wrappers_refuse_shapes(dev):
    c = dev.KVCache(4, 16, 2, 64)
    x = torch.zeros((1, 2, 2, 64), device="cuda", dtype=torch.bfloat16)
    t, s = ints([[0, 1]]), ints([0])
    for f in (lambda: c.append(x, x[:, :1], t, s), lambda: c.append(x, x, t.long(), s), lambda: c.append(x, x, t, ints([0, 0])),
              lambda: c.append(x.double(), x, t, s), lambda: c.read(t, s, None, x[:, :, :1]),
              lambda: dev.CacheAttention(c, 1, 1, 2, 2)(x, t, s), lambda: dev.CacheAttention(c, 1, 2, 2, 3)(x, t, s),
              lambda: dev.KVCache.over(c.k_codes, c.v_codes, c.k_scale, c.v_scale[:2]),
              lambda: dev.KVCache.over(c.k_codes.cpu(), c.v_codes.cpu(), c.k_scale.cpu(), c.v_scale.cpu()),
              lambda: c.append(x.cpu(), x, t, s), lambda: c.append(x, x, t.cpu(), s), lambda: c.append(x, x, t, s.cpu()),
              lambda: dev.NormRope(64, torch.ones(64))):
        with pytest.raises(ValueError):
            f()


def test_expired_wait_is_reported(zg, dev):
    """A pipeline wait that runs out ends the many-rows kernel early with a status; the next call is sound."""
    c, table, length = build(dev, "e4m3", 2, 1, 64, 64, [700, 300], 11, 3)
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
    check_attention(zg, dev, c, q, table, length, None, False)


@pytest.mark.parametrize("R, G", [(1, 2), (9, 1)])
def test_expired_wait_of_few_rows_is_reported(zg, dev, R, G):
    """The same for few rows, where a CTA's share holds several items and items lie in several CTAs: the items that a
    CTA leaves out are passed by, whatever the workspace held before."""
    lengths = [1 + 31 * b % 200 for b in range(120)] + [20000, 0, 3000, 9000]
    c, table, length = build(dev, "int8", len(lengths), 2, 64, 64, lengths, 313, 3)
    q = randn((len(lengths), R, 2 * G, 64), torch.bfloat16, 3)
    attn = dev.CacheAttention(c, len(lengths), R, 2 * G, 313)
    assert attn.ws_bytes > 0
    attn.ws.fill_(0x41)
    zg.zg_debug_set_wait_limit(1)
    try:
        attn(q, table, length)
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="wait expired"):
            zg.zg_check_device_status(0)
    finally:
        zg.zg_debug_set_wait_limit(0)
    want = torch.full_like(attn.out, math.nan)
    want.copy_(attn(q, table, length)[0])
    ok(zg)
    some = [3, 117, 120, 121, 122]
    check_attention(zg, dev, c, q[some].contiguous(), table[some].contiguous(), length[some].contiguous(), None, False)
    attn.ws.fill_(0x41)
    assert torch.equal(attn(q, table, length)[0], want)
    ok(zg)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_example_history_decode(zg, fmt):
    """The example's path end to end: the request vectors against attention in 64 bits over what the cache holds, and
    items of the catalogue only."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "history_decode.py")
    spec = importlib.util.spec_from_file_location("history_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(["--users", "9", "--events", "70", "--fmt", fmt])
    items = {tuple(s) for s in r["items"].tolist()}
    assert all(tuple(s) in items for s in r["sids"].reshape(-1, r["sids"].shape[-1]).tolist())
    assert torch.isfinite(r["rescored"]).all() and torch.isfinite(r["lse"]).all()
    # the new event's query again, attending in 64 bits
    q, _, _ = r["layer"].project(r["x"])
    q, _ = r["layer"].turn(q, None, (r["length"] - 1)[:, None].contiguous())
    want, _, tol, _ = want_attention(r["cache"], q, r["table"], r["length"], None, False, m.DIM ** -0.5)
    err = (r["a1"].double().cpu() - want).abs()
    assert (err <= tol + 2.0 ** -8 * 1.001 * (want.abs() + tol)).all()
