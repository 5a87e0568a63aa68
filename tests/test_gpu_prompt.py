"""Attention over whole prompts on the GPU against its definition in 64 bits: packed sequences of every kind of length,
grouped heads of every count, strides, rows in no sequence, what is not finite in masked places, streams and graphs."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}    # half a step, relative


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


def starts_of(lengths, first=0):
    at = [first]
    for n in lengths:
        at.append(at[-1] + n)
    return ints(at)


def want_prompt(q, k, v, starts, causal, scale):
    """The definition in 64 bits over what each row sees alone: outputs, log-sum-exps, and the bounds of what 32-bit sums
    and rounded probabilities cost."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    edge = starts.tolist()
    u = U[q.dtype]
    for a, b in zip(edge[:-1], edge[1:]):
        n = b - a
        if not n:
            continue
        i = torch.arange(n, device="cuda")
        mask = i[None] <= i[:, None] if causal else torch.ones((n, n), dtype=torch.bool, device="cuda")
        for h in range(Hq):
            qq, kk, vv = q[a:b, h].double(), k[a:b, h // G].double(), v[a:b, h // G].double()
            z = torch.where(mask, qq @ kk.T * scale, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            dz = torch.where(mask, qq.abs() @ kk.abs().T * scale, torch.zeros_like(z)).amax(-1) * ((D + 8) * 2.0 ** -24)
            p = torch.softmax(z, -1)
            seen = mask & (p > 0)
            # products of what is seen alone
            x = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv))
            o, mass = p @ x, p @ x.abs()
            if not torch.isfinite(vv).all():
                odd = (seen.double() @ (~torch.isfinite(vv)).double()) > 0
                o = torch.where(odd, torch.full_like(o, math.nan), o)
            out[a:b, h], lse[a:b, h] = o, torch.logsumexp(z, -1)
            # probabilities: a rounding each, the scores' error twice (p and the sum), the exponential and the running
            # sums in 32 bits; of halves, those below 2^-14 of a reference that the largest passes by 2^8 at most: 2^-25 each
            tol[a:b, h] = mass * (u + 2 * dz[:, None] + n * 2.0 ** -24 + 2.0 ** -18)
            if q.dtype == torch.float16:
                tol[a:b, h] += x.abs().amax() * 2.0 ** -25 * (mask.sum(-1) / torch.exp(lse[a:b, h] - z.amax(-1)))[:, None]
            ltol[a:b, h] = dz + 2.0 ** -18 + n * 2.0 ** -24 + lse[a:b, h].abs() * 2.0 ** -21
    return out, lse, tol, ltol


def check(zg, dev, q, k, v, starts, causal, scale=None, out=None):
    T, Hq, D = q.shape
    a = dev.PromptAttention(Hq, k.shape[1], D, causal=causal, scale=scale)
    fresh = out is None
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda") if fresh else out
    lse = torch.full((T, Hq), 7.0, device="cuda")
    want, wlse, tol, ltol = want_prompt(q, k, v, starts, causal, a.scale)
    got, l2 = a(q, k, v, starts, out, lse)
    ok(zg)
    assert got is out and l2 is lse
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    for x, y in zip(starts.tolist()[:-1], starts.tolist()[1:]):
        inside[x:y] = True
    if fresh:
        assert (out[~inside] == 7).all()
    assert (lse[~inside] == 7).all()
    got, want, tol = got[inside].double(), want[inside], tol[inside]
    bound = tol + U[q.dtype] * 1.001 * (want.abs() + tol) + (2.0 ** -25 if q.dtype == torch.float16 else 0)
    assert torch.equal(torch.isnan(want), torch.isnan(got) | (torch.isinf(got) & torch.isnan(want)))
    fine = torch.isfinite(want)
    err = (got - want).abs()[fine]
    assert (err <= bound[fine]).all(), float((err / bound[fine]).max())
    l, w = lse[inside].double(), wlse[inside]
    assert torch.equal(torch.isnan(l), torch.isnan(w))
    fine = torch.isfinite(w)
    assert ((l - w).abs()[fine] <= ltol[inside][fine]).all(), float((l - w).abs()[fine].max())
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("Hq, Hk", [(1, 1), (2, 2), (6, 2), (8, 2), (5, 1), (40, 1), (300, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(zg, dev, dtype, dim, Hq, Hk, causal):
    """Sequences of no row, one, around a tile and a step, several steps; one buffer for q, k and v."""
    lengths = [1, 0, 127, 128, 129, 2, 255, 257, 0, 31] if Hq < 40 else [1, 0, 40, 129]
    T = sum(lengths)
    x = randn((T, Hq + 2 * Hk, dim), dtype, 3 + Hq)
    check(zg, dev, 2 * x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], starts_of(lengths), causal)


@pytest.mark.parametrize("dtype, dim, Hq, Hk", [(torch.bfloat16, 128, 4, 1), (torch.float16, 64, 3, 3), (torch.bfloat16, 96, 2, 1),
                                                (torch.float16, 32, 2, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_sequences(zg, dev, dtype, dim, Hq, Hk, causal):
    """The ring goes round many times; rows before, between the last and the end in no sequence."""
    lengths = [3000, 5, 1777]
    T = sum(lengths) + 30
    q, k, v = randn((T, Hq, dim), dtype, 1, 2.0), randn((T, Hk, dim), dtype, 2), randn((T, Hk, dim), dtype, 3)
    starts = starts_of(lengths, 17)
    for x in (q, k, v):                       # what lies in no sequence is not used
        x[:17], x[17 + sum(lengths):] = math.nan, math.inf
    check(zg, dev, q, k, v, starts, causal)
    check(zg, dev, q, k, v, starts, causal, scale=1.5)


def test_many_sequences(zg, dev):
    """More sequences than threads, most of them short, some empty."""
    g = torch.Generator().manual_seed(3)
    lengths = [int(torch.randint(0, 9, (), generator=g)) for _ in range(1500)] + [600] + [0] * 50
    T = sum(lengths)
    q, k, v = (randn((T, h, 64), torch.bfloat16, h) for h in (4, 2, 2))
    v = randn((T, 2, 64), torch.bfloat16, 9)
    check(zg, dev, q, k, v, starts_of(lengths), True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("Hq, Hk", [(2, 2), (6, 2)])
def test_what_is_not_finite_stays_behind_the_mask(zg, dev, dtype, dim, Hq, Hk):
    """A NaN or an infinity in a key, a value or a query reaches the rows that see it, and no other."""
    lengths = [200, 300, 70]
    T = sum(lengths)
    q, k, v = randn((T, Hq, dim), dtype, 1), randn((T, Hk, dim), dtype, 2), randn((T, Hk, dim), dtype, 3)
    starts = starts_of(lengths)
    v[150, 0, 3], v[199, 1, :] = math.inf, math.nan          # the last row of a sequence among them
    v[200 + 128, 0, 9], v[200 + 130, 0, 9], v[200 + 299, 1, 40] = math.nan, -math.inf, math.inf
    k[200 + 250, 1, 5] = math.nan
    q[520, 0, 7] = math.nan
    a = dev.PromptAttention(Hq, Hk, dim, lse=True)
    out, lse = a(q, k, v, starts)
    ok(zg)
    clean_v, clean_k, clean_q = (torch.nan_to_num(x, 0.0, 0.0, 0.0) for x in (v, k, q))
    o2, l2 = a(clean_q, clean_k, clean_v, starts)
    ok(zg)
    G = Hq // Hk
    touched = torch.zeros((T, Hq, dim), dtype=torch.bool, device="cuda")
    for t, h, d, end in ((150, 0, 3, 200), (328, 0, 9, 500), (330, 0, 9, 500), (499, 1, 40, 500)):
        touched[t:end, h * G:(h + 1) * G, d] = True
    touched[199, G:2 * G] = True
    touched[450:500, G:2 * G] = True
    touched[520, 0] = True
    assert not torch.isfinite(out[touched]).any()
    assert torch.isnan(out[520, 0]).all() and torch.isnan(lse[520, 0]) and torch.isnan(lse[450:500, G:2 * G]).all()
    assert (out[150:200, :G, 3] == math.inf).all() and torch.isnan(out[330:500, :G, 9]).all()
    # the others as if it were not there, but for up to three values' rows that are added apart, without the rounding of
    # their probabilities (at most 1 together); and one rounding of each output
    err = (out.double() - o2.double()).abs()[~touched]
    assert (err <= 2.01 * U[dtype] * o2.double().abs()[~touched] + 2.0 ** -24 + 1.01 * U[dtype] * float(clean_v.abs().max())).all()
    before = torch.ones(T, dtype=torch.bool, device="cuda")
    before[150:200], before[328:500], before[520:] = False, False, False
    assert torch.equal(out[before], o2[before]) and torch.equal(lse[before], l2[before])
    # not causal: all rows of the sequence see it, the others nothing
    b = dev.PromptAttention(Hq, Hk, dim, causal=False)
    o3, o4 = b(q, k, v, starts)[0], b(clean_q, clean_k, clean_v, starts)[0]
    ok(zg)
    assert not torch.isfinite(o3[:200, :G, 3]).any() and not torch.isfinite(o3[200:500, :G, 9]).any()
    assert torch.equal(o3[500:520], o4[500:520]) and torch.equal(o3[521:], o4[521:])


def test_scores_of_any_size(zg, dev):
    """Scores far apart, large and equal; a row's reference moves often."""
    T, D = 700, 64
    k = randn((T, 1, D), torch.float16, 2)
    q = randn((T, 2, D), torch.float16, 1)
    v = randn((T, 1, D), torch.float16, 3)
    grow = k * torch.linspace(0.01, 30, T, device="cuda")[:, None, None].half()
    for kk, scale in ((grow, 1.0), (grow.flip(0), 1.0), (torch.zeros_like(k), 1.0), (k, 1e-6)):
        check(zg, dev, q, kk, v, starts_of([T]), True, scale=scale)
        check(zg, dev, q, kk, v, starts_of([300, 400]), False, scale=scale)
    # scores of 2^27 and more: one key has it all; out is its value to the rounding of two types
    big = dev.PromptAttention(2, 1, D, causal=False, scale=3e4)
    big_k = (8 * k).clamp(-60, 60)
    o, _ = big((100 * q), big_k, v, starts_of([T]))
    ok(zg)
    best = torch.einsum("thd,jd->thj", (100 * q).double(), big_k[:, 0].double()).argmax(-1)
    assert ((o.double() - v[:, 0].double()[best]).abs() <= 2.0 ** -9 * v.abs().max()).float().mean() > 0.999


def test_strides_in_place_and_wrapper_outputs(zg, dev):
    """Heads before tokens, gaps between rows, the output over the queries; new outputs."""
    lengths = [130, 77]
    T, Hq, Hk, D = 207, 4, 2, 96
    q = randn((Hq, T, D), torch.bfloat16, 1).transpose(0, 1)
    k = randn((Hk, T + 3, D + 8), torch.bfloat16, 2)[:, 3:, :D].transpose(0, 1)
    v = randn((T, 3, Hk, D), torch.bfloat16, 3)[:, 1]
    starts = starts_of(lengths)
    out, lse = check(zg, dev, q, k, v, starts, True)
    a = dev.PromptAttention(Hq, Hk, D, lse=True)
    o, l2 = a(q, k, v, starts)
    q2 = q.clone()
    o2, none = dev.PromptAttention(Hq, Hk, D)(q2, k, v, starts, out=q2)
    ok(zg)
    assert torch.equal(o, out) and torch.equal(l2, lse) and torch.equal(q2, out) and none is None
    buf = torch.full((T, Hq + 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    a(q, k, v, starts, out=buf[:, 1:])
    ok(zg)
    assert torch.equal(buf[:, 1:], out) and (buf[:, 0] == 5).all()


def test_bad_starts_are_reported(zg, dev):
    T = 100
    q, k, v = randn((T, 2, 64), torch.bfloat16, 1), randn((T, 1, 64), torch.bfloat16, 2), randn((T, 1, 64), torch.bfloat16, 3)
    a = dev.PromptAttention(2, 1, 64)
    for bad in ([0, 101], [-1, 50], [50, 40, 100], [2 ** 31 - 1, 5], [0, 2 ** 31 - 1, -2 ** 31]):
        a(q, k, v, ints(bad))
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)
    check(zg, dev, q, k, v, ints([0, 100]), True)


def test_stream_and_captured_graph(zg, dev):
    """On another stream, captured, replayed over new rows and new starts."""
    T = 900
    q, k, v = randn((T, 4, 128), torch.bfloat16, 1), randn((T, 2, 128), torch.bfloat16, 2), randn((T, 2, 128), torch.bfloat16, 3)
    starts = starts_of([300, 600])
    a = dev.PromptAttention(4, 2, 128)
    out, lse = torch.empty_like(q), torch.empty((T, 4), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o1, _ = a(q, k, v, starts, stream=s.cuda_stream)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a(q, k, v, starts, out, lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o1)
    for seed, lengths in ((5, [900, 0]), (6, [1, 700])):
        q.copy_(randn(q.shape, torch.bfloat16, seed))
        starts.copy_(starts_of(lengths))
        graph.replay()
        ok(zg)
        got = out.clone(), lse.clone()
        o2, l2 = check(zg, dev, q, k, v, starts, True)
        n = sum(lengths)
        assert torch.equal(got[0][:n], o2[:n]) and torch.equal(got[1][:n], l2[:n])


def test_rows_past_32_bits(zg, dev):
    """Rows whose offsets pass 2^31 elements."""
    T, Hq, Hk, D = 1 << 19, 32, 1, 128
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((T, 64, D), dtype=torch.bfloat16, device="cuda")[:, :1] for _ in range(2))
    n = 200
    for x, s in ((q, 1), (k, 2), (v, 3)):
        x[T - n:] = randn(x[T - n:].shape, torch.bfloat16, s)
    starts = ints([T - n, T])
    o, _ = dev.PromptAttention(Hq, Hk, D)(q, k, v, starts, out=q.clone())
    ok(zg)
    part, _ = dev.PromptAttention(Hq, Hk, D)(q[T - n:].contiguous(), k[T - n:].contiguous(), v[T - n:].contiguous(), ints([0, n]))
    ok(zg)
    assert torch.equal(o[T - n:], part) and not o[:T - n].any()


def test_empty_and_refused(zg, dev):
    x = torch.zeros((8, 2, 64), device="cuda", dtype=torch.bfloat16)
    a = dev.PromptAttention(2, 2, 64)
    e = x[:0]
    assert a(e, e, e, ints([0, 0]))[0].shape == (0, 2, 64)
    y = torch.full_like(x, 3.0)
    a(x, x, x, ints([0]), out=y)                       # no sequence
    ok(zg)
    assert (y == 3).all()
    for f in (lambda: a(x, x[:, :1], x[:, :1], ints([0, 8])), lambda: a(x, x[:4], x[:4], ints([0, 8])), lambda: a(x, x, x, ints([0, 8]).long()),
              lambda: a(x, x, x, ints([[0, 8]])), lambda: a(x, x, x, ints([0, 8]), out=x[:4]), lambda: a(x, x, x.cpu(), ints([0, 8])),
              lambda: a(x, x, x, ints([0, 8]), lse=torch.zeros((8, 3), device="cuda")), lambda: dev.PromptAttention(3, 2, 64),
              lambda: a(x.transpose(1, 2).contiguous().transpose(1, 2), x, x, ints([0, 8]))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: a(x.float(), x.float(), x.float(), ints([0, 8])), lambda: a(x, x.half(), x, ints([0, 8])),
              lambda: dev.PromptAttention(2, 1, 64)(x, x[:, :1].expand(8, 1, 64).as_strided((8, 1, 64), (4, 4, 1)), x[:, :1], ints([0, 8]))):
        with pytest.raises(zg.ZgError):
            f()


def test_expired_wait_is_reported(zg, dev):
    T = 2000
    q, k, v = randn((T, 2, 128), torch.bfloat16, 1), randn((T, 1, 128), torch.bfloat16, 2), randn((T, 1, 128), torch.bfloat16, 3)
    a = dev.PromptAttention(2, 1, 128)
    zg.zg_debug_set_wait_limit(1)
    try:
        a(q, k, v, ints([0, T]))
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="wait expired"):
            zg.zg_check_device_status(0)
    finally:
        zg.zg_debug_set_wait_limit(0)
    check(zg, dev, q, k, v, ints([0, T]), True)
