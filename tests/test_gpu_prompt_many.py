"""Prompt attention over hundreds and thousands of packed sequences: which CTA takes which rows, by any mixture of lengths,
and a time in proportion to the rows."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_prompt import check, dev, ints, ok, randn, starts_of, zg  # noqa: E402, F401 (zg and dev are fixtures)

FEW = 128      # sequences of the calls that the others are compared with


def rows(T, Hq, Hk, dim, dtype):
    return tuple(randn((T, h, dim), dtype, 3 + i) for i, h in enumerate((Hq, Hk, Hk)))


def in_parts(a, q, k, v, starts, out, lse):
    """The same sequences, FEW a call."""
    for i in range(0, starts.shape[0] - 1, FEW):
        a(q, k, v, starts[i:i + FEW + 1].contiguous(), out, lse)


def mixture(kind, B):
    r = random.Random(B)
    if kind == "some empty":
        return [r.choice([0, 1, 2, r.randrange(300)]) for _ in range(B)]
    if kind == "mostly empty":
        return [r.randrange(1, 300) if r.random() < 0.05 else 0 for _ in range(B - 1)] + [0]
    n = [r.randrange(40) for _ in range(B)]
    n[B // 3], n[-1] = 2500, 700           # "long ones among short ones"
    return n


@pytest.mark.parametrize("kind", ["some empty", "mostly empty", "long ones among short ones"])
@pytest.mark.parametrize("B", [129, 160, 1025, 5000])
@pytest.mark.parametrize("Hq, Hk", [(4, 1), (3, 3), (10, 2)])
@pytest.mark.parametrize("first, last", [(0, 0), (17, 200)])
def test_as_the_same_sequences_in_several_calls(zg, dev, kind, B, Hq, Hk, first, last):  # noqa: F811
    """Bit for bit; rows in no sequence stay as they are."""
    lengths = mixture(kind, B)
    starts = starts_of(lengths, first)
    T, dim = int(starts[-1]) + last, 64
    q, k, v = rows(T, Hq, Hk, dim, torch.bfloat16)
    a = dev.PromptAttention(Hq, Hk, dim, lse=True)
    got, want = ((torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")) for _ in range(2))
    a(q, k, v, starts, *got)
    in_parts(a, q, k, v, starts, *want)
    ok(zg)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    edge = torch.arange(T, device="cuda")
    outside = (edge < first) | (edge >= T - last)
    assert (got[0][outside] == 7).all() and (got[1][~outside] != 7).all()


@pytest.mark.parametrize("causal", [True, False])
def test_against_the_definition(zg, dev, causal):  # noqa: F811
    r = random.Random(5)
    lengths = [r.choice([0, 1, 5, 130, r.randrange(200)]) for _ in range(300)]
    q, k, v = rows(sum(lengths), 3, 1, 96, torch.float16)
    check(zg, dev, q, k, v, starts_of(lengths), causal)


def test_more_sequences_than_rows(zg, dev):  # noqa: F811
    """100,000 sequences, fifty of one row among empty ones: each row's output is its value."""
    T, B = 50, 100_000
    q, k, v = rows(T, 4, 2, 64, torch.bfloat16)
    starts = (torch.arange(B + 1, device="cuda") * T // B).int()
    out, _ = dev.PromptAttention(4, 2, 64)(q, k, v, starts)
    ok(zg)
    assert torch.equal(out, v.repeat_interleave(2, 1))


def test_bad_starts_of_many_sequences_are_reported(zg, dev):  # noqa: F811
    """Falling, negative, behind the rows: held inside them."""
    T = 900
    q, k, v = rows(T, 4, 2, 64, torch.bfloat16)
    a = dev.PromptAttention(4, 2, 64)
    r = random.Random(3)
    for bad in ([r.randrange(-100, T + 100) for _ in range(401)], [0] * 200 + [T + 1], [-1] + [T] * 150, [2 ** 31 - 1, -2 ** 31] * 100,
                list(range(T, T - 300, -1))):
        a(q, k, v, ints(bad))
        torch.cuda.synchronize()
        with pytest.raises(zg.ZgError, match="out of range"):
            zg.zg_check_device_status(0)
    check(zg, dev, q, k, v, ints([0] * 150 + [T] * 10), True)


def test_time_in_proportion_to_the_rows(zg, dev):  # noqa: F811
    """4,096 sequences take a few times as long as the same rows in 32 calls at most (they took sixteen times as long when
    each CTA counted all sequences anew)."""
    lengths = [20 + b * 7919 % 281 for b in range(32 * FEW)]
    starts = starts_of(lengths)
    q, k, v = rows(sum(lengths), 8, 2, 64, torch.float16)
    a = dev.PromptAttention(8, 2, 64)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    parts = [starts[i:i + FEW + 1].contiguous() for i in range(0, 32 * FEW, FEW)]

    def time(f):
        e, best = [torch.cuda.Event(enable_timing=True) for _ in range(2)], []
        for _ in range(4):
            e[0].record()
            f()
            e[1].record()
            torch.cuda.synchronize()
            best.append(e[0].elapsed_time(e[1]))
        return min(best[1:])

    whole = time(lambda: a(q, k, v, starts, out, lse))
    apart = time(lambda: [a(q, k, v, s, out, lse) for s in parts])
    ok(zg)
    assert whole < 4 * apart, (whole, apart)
