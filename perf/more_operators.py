"""Operators for long histories as measurable cases: attention over whole prompts, a cache held in 4 bits (written,
read back, attended to), the attention weights that its tokens collect, and eviction by them.

A recommendation model takes a user's events in at once (prompt attention), holds their keys and values in 4 bits,
lets single events and the beams of a decode attend to them, and drops the events that nothing attends to once a
history has grown past its budget.  The cases are those moves at small, ordinary and large sizes.

`own` False: elementary torch operations in 32 bits (64 for the angles).  `own` True: the calls a user makes.

Definitions.
  prompt     packed rows, sequence b = rows starts[b] .. starts[b + 1] - 1: softmax(scale * q k^T) v over its own
             sequence (causal: row i of it sees rows 0 .. i), and the log-sum-exp of each row and head
  4 bits     16 neighbouring elements of a token's head share a scale: max |x| / 6 rounded to the nearest half whose
             bits are u << 7 (u the byte that is stored; ties to even), at most 10240; an element is x / scale rounded to the
             nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), within 6, and its sign; two codes a byte, the
             earlier element in the low half.  value = code * scale
  8 bits     e4m3 or int8 codes, one float32 scale a (block, head)
  weights    w[b][h][j] = decay * w[b][h][j] + sum of exp(scale * q k_j - lse) over the rows that see token j and the
             query heads of key head h; tokens behind a history keep what they have
  eviction   a request of n > keep tokens keeps, for each key head, its last `recent` ones and of the others the keep -
             recent with the largest weights (equal ones: the earlier); they move to the front in their order, and so do their
             weights.  8 bits: a block's new scale is the largest of its rows' old ones, rows are coded again by it
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the histories of a serving batch (64 users, up to 500 events), short and uneven: latency and packing
        dict(name="prompt short", op="prompt", dtype="f16", B=64, Hq=8, Hk=2, D=64, length=500, causal=True, ragged=True),
        # four lifelong histories at once, bound by the tensor cores
        dict(name="prompt long", op="prompt", dtype="bf16", B=4, Hq=16, Hk=4, D=128, length=11000, causal=True,
             ragged=True),
        # the newest event of 64 users: norm, rotation and the write in one call, then read back
        dict(name="write one token", op="write", dtype="bf16", B=64, T=1, Hq=8, Hk=2, D=128, block=64, start=1500,
             norm=True),
        # new users' whole histories (their keys already turned: prompt attention took them), written and read back
        dict(name="write histories", op="write", dtype="bf16", B=32, T=2048, Hq=0, Hk=4, D=128, block=64, start=0,
             norm=False),
        # few users, odd lengths that begin inside a block, a head of 96, fp32 activations
        dict(name="write odd f32", op="write", dtype="f32", B=3, T=1001, Hq=0, Hk=4, D=96, block=16, start=5,
             norm=False),
        # one token for each of 64 users with a few thousand events
        dict(name="attend one token", op="attend", dtype="bf16", fmt="e2m1", B=64, R=1, Hq=8, Hk=2, D=128, block=64,
             length=4096, causal=False, ragged=True),
        # lifelong histories: few requests, a long cache
        dict(name="attend lifelong", op="attend", dtype="f16", fmt="e2m1", B=8, R=1, Hq=16, Hk=4, D=128, block=64,
             length=131072, causal=False, ragged=True),
        # the beams of the large catalogue (64 requests, 256 beams, width 512 over four heads)
        dict(name="attend 256 beams", op="attend", dtype="bf16", fmt="e2m1", B=64, R=256, Hq=4, Hk=4, D=128, block=64,
             length=2048, causal=False, ragged=True),
        # the weights of one decoded token over lifelong histories
        dict(name="weights lifelong", op="weights", dtype="bf16", fmt="e2m1", B=8, R=1, Hq=16, Hk=4, D=128, block=64,
             length=131072, causal=False, ragged=True, decay=1.0),
        # the last 33 events of 16 long histories look back: which tokens the eviction after them keeps
        dict(name="weights window", op="weights", dtype="f16", fmt="e4m3", B=16, R=33, Hq=16, Hk=4, D=64, block=32,
             length=8190, causal=True, ragged=True, decay=0.5),
        # a serving batch of ordinary histories cut to a quarter
        dict(name="evict 64 users", op="evict", fmt="int8", B=64, Hk=2, D=64, block=32, length=2047, keep=500, recent=33,
             ragged=True),
        # lifelong histories cut to 8,192 tokens a head
        dict(name="evict lifelong", op="evict", fmt="e2m1", B=8, Hk=4, D=128, block=64, length=131072, keep=8192,
             recent=1024, ragged=True),
    ]


def _log(rng, a, b):
    """A whole number between a and b, spread over the logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "write", "attend", "attend", "weights", "evict"])
    D = rng.choice([32, 64, 64, 96, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    fmt = rng.choice(["e2m1", "e2m1", "e4m3", "int8"])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    ragged = rng.random() < 0.8
    if op == "prompt":
        B = _log(rng, 1, 96)
        most = min(11000, int(math.sqrt(5e9 / (B * Hq))), 300_000_000 // (B * Hq * D))
        return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, D=D, length=_log(rng, 2, most), causal=rng.random() < 0.7,
                    ragged=ragged)
    if op == "write":
        B = _log(rng, 1, 96)
        T = 1 if rng.random() < 0.3 else _log(rng, 2, min(5000, 30_000_000 // (B * Hk * D)))
        start = rng.choice([0, rng.randrange(1, 3000)])
        if T == 1:   # single tokens are turned on the way, histories come turned
            return dict(op=op, dtype=dtype, B=B, T=1, Hq=Hq, Hk=Hk, D=D, block=block, start=start, norm=True)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=B, T=T, Hq=0, Hk=Hk, D=D, block=block,
                    start=start, norm=False)
    if op == "evict":
        B = _log(rng, 1, 96)
        length = _log(rng, 2, min(100_000, 300_000_000 // (B * Hk * D)))
        keep = _log(rng, 1, length)
        return dict(op=op, fmt=fmt, B=B, Hk=Hk, D=D, block=block, length=length, keep=keep,
                    recent=rng.choice([0, keep, rng.randrange(0, keep + 1)]), ragged=ragged)
    kind = rng.choice(["token", "token", "beams", "chunk"])
    B = _log(rng, 1, 96)
    R = 1 if kind == "token" else _log(rng, 2, 400 if op == "attend" else 80)
    while B * R * Hq * D > 100_000_000:
        B, R = max(1, B // 2), max(1, R // 2) if B == 1 else R
    # the codes of one side, and the scores of all rows, bound the length
    most = int(min(300_000_000 / (B * Hk * D), 400_000_000 / (B * Hq * R), 100_000))
    c = dict(op=op, dtype=dtype, fmt="e2m1" if op == "attend" else fmt, B=B, R=R, Hq=Hq, Hk=Hk, D=D, block=block,
             length=_log(rng, 1 if kind == "token" else 17, most), causal=kind == "chunk", ragged=ragged)
    return c | {"decay": rng.choice([1.0, 0.9])} if op == "weights" else c


def _spread(B, low, high, ragged):
    """B whole numbers from low to high: an even spread in an order of its own, the same for every seed."""
    if not ragged:
        return [high] * B
    got = [low + int((high - low) * math.modf((b + 1) * 0.6180339887498949)[0]) for b in range(B)]
    got[-1] = high
    if B > 3:
        got[1] = 0           # a user without a history
    return got


def _lengths(c):
    return _spread(c["B"], c["length"] // 4, c["length"], c["ragged"])


def _rows(c):
    """Rows of each request: ragged in causal chunks."""
    return _spread(c["B"], max(1, c["R"] // 2), c["R"], c["ragged"] and c["causal"])


def _starts(c):
    return _spread(c["B"], c["start"] // 2, c["start"], c["start"] > 0)


def _news(c):
    """Tokens written for each request."""
    return _spread(c["B"], max(1, c["T"] // 3), c["T"], c["T"] > 1)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, counts, T, more):
    """Blocks in a shuffled order: [B][max_blocks] with -1 where a request has none, and the pool's size."""
    need = [max(0, -(-n // T)) for n in counts]
    width, total = max(1, max(need)), max(1, sum(need)) + more
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(width, device="cuda")[None, :]
    n = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(n, 0) - n
    flat = (first + at).clamp(max=total - 1)
    return torch.where(at < n, order[flat], torch.full_like(order[flat], -1)), total


def _pool(g, total, c, behind):
    """Codes and scales as normal keys and values leave them; what lies behind a request's last token (`behind`: block and
    row numbers) is not defined: here NaN, or the largest codes."""
    shape = (total, c["Hk"], c["block"], c["D"])
    out = []
    for _ in range(2):
        if c["fmt"] == "e2m1":
            x = _randn(g, shape, torch.float16) * torch.exp(0.4 * _randn(g, shape[:2])).half()[:, :, None, None]
            codes, scales = _to_4_bits(x)
            scales[behind[0], :, behind[1]] = 0xFF      # NaN
        else:
            q = QMAX[c["fmt"]]
            x = _randn(g, shape, torch.float16).mul_(q / 4.2).clamp_(-q, q)
            codes = x.round_().to(torch.int8) if c["fmt"] == "int8" else x.to(torch.float8_e4m3fn)
            scales = torch.exp(0.4 * _randn(g, shape[:2])) * (4.2 / q)
        codes.view(torch.uint8)[behind[0], :, behind[1]] = 0x7F     # e4m3: NaN
        out.append((codes, scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _behind(table, lengths, block):
    """Rows of each request's last block that lie behind its last token."""
    last = torch.tensor([n - 1 for n in lengths], device="cuda")
    blk = table.long().gather(1, last.clamp(min=0).div(block, rounding_mode="floor")[:, None])[:, 0]
    dead = torch.arange(block, device="cuda")[None, :] > (last % block)[:, None]
    b, t = (dead & (last >= 0)[:, None]).nonzero(as_tuple=True)
    return blk[b], t


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if own:
        from generative_recommendation_constrained_gb300 import device as dev
    if c["op"] == "prompt":
        dt, lengths = DT[c["dtype"]], _lengths(c)
        s["starts"] = _ints([0] + torch.tensor(lengths).cumsum(0).tolist())
        s["scale"] = 1.0 / math.sqrt(c["D"])
        # projections of the events, side by side in one buffer as one matrix product leaves them
        x = _randn(g, (sum(lengths), c["Hq"] + 2 * c["Hk"], c["D"]), torch.float16 if c["dtype"] == "f16" else torch.float32)
        x[:, :c["Hq"]] *= 2.0
        x = x.to(dt)
        s["q"], s["k"], s["v"] = x[:, :c["Hq"]], x[:, c["Hq"]:c["Hq"] + c["Hk"]], x[:, c["Hq"] + c["Hk"]:]
        if own:
            s["attn"] = dev.PromptAttention(c["Hq"], c["Hk"], c["D"], causal=c["causal"], scale=s["scale"], lse=True)
        return s
    if c["op"] == "write":
        dt, starts, news = DT[c["dtype"]], _starts(c), _news(c)
        heads = c["Hq"] + 2 * c["Hk"]
        x = _randn(g, (c["B"], c["T"], heads, c["D"]), torch.float16 if c["dtype"] == "f16" else torch.float32)
        x = (x * (0.5 + torch.rand((1, 1, heads, 1), generator=g, device="cuda"))).to(dt)
        s["q"], s["k"], s["v"] = x[:, :, :c["Hq"]], x[:, :, c["Hq"]:c["Hq"] + c["Hk"]], x[:, :, c["Hq"] + c["Hk"]:]
        s["gq"], s["gk"] = (1.0 + 0.2 * _randn(g, (c["D"],)) for _ in range(2))
        s["table"], total = _table(g, [a + n for a, n in zip(starts, news)], c["block"], 2)
        s["kc"], s["vc"] = (torch.zeros((total, c["Hk"], c["block"], c["D"] // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros((total, c["Hk"], c["block"], c["D"] // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
        s["start"], s["new"] = _ints(starts), _ints(news)
        s["q_out"] = torch.empty(s["q"].shape, dtype=dt, device="cuda") if c["Hq"] else None
        s["k_out"], s["v_out"] = (torch.empty(s["k"].shape, dtype=dt, device="cuda") for _ in range(2))
        if own:
            s["cache"] = dev.KVCache.over(s["kc"], s["vc"], s["ks"], s["vs"])
            s["nr"] = dev.NormRope(c["D"], s["gq"], s["gk"], eps=EPS) if c["norm"] else None
        return s
    lengths = _lengths(c)
    s["table"], total = _table(g, lengths, c["block"], 3)
    s["kc"], s["vc"], s["ks"], s["vs"] = _pool(g, total, c, _behind(s["table"], lengths, c["block"]))
    s["length"] = _ints(lengths)
    if own:
        s["cache"] = dev.KVCache.over(s["kc"], s["vc"], s["ks"], s["vs"])
    most = s["table"].shape[1] * c["block"]
    if c["op"] == "evict":
        # what tokens collect over many rows: a few much, most little, some nothing at all
        w = torch.exp(2.0 * _randn(g, (c["B"], c["Hk"], most)) - 4.0)
        s["w"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
        if own:
            s["evict"] = dev.CacheEviction(s["cache"], c["B"], s["table"].shape[1], c["keep"], c["recent"])
        return s
    dt = DT[c["dtype"]]
    s["rows"] = _ints(_rows(c))
    s["q"] = (2.0 * _randn(g, (c["B"], c["R"], c["Hq"], c["D"]))).to(dt)
    s["scale"] = 1.0 / math.sqrt(c["D"])
    if c["op"] == "weights":
        z, m = _scores(s)
        s["lse"] = (m + torch.log(z.sub_(m).exp_().sum(-1, keepdim=True)))[..., 0].permute(0, 3, 1, 2).reshape(c["B"], c["R"], c["Hq"]).contiguous()
        s["w"] = torch.rand((c["B"], c["Hk"], most), generator=g, device="cuda")
    elif own:
        s["attn"] = dev.CacheAttention(s["cache"], c["B"], c["R"], c["Hq"], s["table"].shape[1], causal=c["causal"],
                                       scale=s["scale"], dtype=dt, lse=True)
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _to_4_bits(x):
    """x [..][D] -> packed codes [..][D/2] and scale bytes [..][D/16], by exact quotients."""
    x = x.float().unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=x.device)
    top = torch.div(x.abs().amax(-1), six)
    # 4 bits of mantissa, down to steps of 2^-17
    _, e = torch.frexp(top)
    step = torch.ldexp(torch.ones_like(top), torch.clamp(e - 4, min=-17))
    scale = (torch.round(top / step) * step).clamp_(max=10240.0)
    u = scale.half().view(torch.int16).bitwise_right_shift(7).to(torch.uint8)
    y = torch.where(scale[..., None] > 0, x.abs() / scale[..., None], torch.zeros_like(x))
    i = (y > 0.25).to(torch.uint8)
    for edge, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (y >= edge) if tie_up else (y > edge)
    i = (i | ((x < 0).to(torch.uint8) << 3)).flatten(-2)
    return i[..., 0::2] | (i[..., 1::2] << 4), u


def _levels(dtype=torch.float32):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device="cuda")
    return torch.cat([v, -v])


def _from_4_bits(codes, u, dtype=torch.float32):
    """Packed codes [..][D/2] and scale bytes [..][D/16] -> values [..][D]."""
    at = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = (u.to(torch.int16) << 7).view(torch.float16).to(dtype)
    return (_levels(dtype)[at.int()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _values(fmt, codes, scales, blk, dtype=torch.float32):
    """Values of the blocks `blk` [..] -> [..][heads][block][D]."""
    if fmt == "e2m1":
        return _from_4_bits(codes[blk], scales[blk], dtype)
    return codes.view(torch.uint8)[blk].view(CODE[fmt]).to(dtype) * scales[blk][..., None, None].to(dtype)


def _side(s, codes, scales):
    """One side of every request's history, [B][Hk][L][D]; zero behind it."""
    c = s["case"]
    L = s["table"].shape[1] * c["block"]
    held = torch.arange(L, device="cuda")[None, :] < s["length"][:, None]
    x = _values(c["fmt"], codes, scales, s["table"].long().clamp(min=0))
    x = x.permute(0, 2, 1, 3, 4).reshape(c["B"], c["Hk"], L, c["D"])
    return torch.where(held[:, None, :, None], x, torch.zeros((), device="cuda"))


def _scores(s):
    """Scores [B][Hk][G][R][L] of a cache's keys, -inf where a row does not see, and each row's largest (0 if it sees nothing)."""
    c = s["case"]
    B, R, Hk, G, D = c["B"], c["R"], c["Hk"], c["Hq"] // c["Hk"], c["D"]
    k = _side(s, s["kc"], s["ks"])
    L = k.shape[2]
    q = s["q"].float().reshape(B, R, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * R, D)
    z = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    row = torch.arange(R, device="cuda")[None, :]
    sees = s["length"][:, None].expand(B, R)
    if c["causal"]:
        sees = sees - (s["rows"][:, None] - 1 - row)
    sees = torch.where(row < s["rows"][:, None], sees, torch.zeros_like(sees))
    mask = torch.arange(L, device="cuda")[None, None, :] < sees[:, :, None]
    z = z.view(B, Hk, G, R, L).masked_fill_(~mask[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    return z, torch.where(m == -math.inf, torch.zeros_like(m), m)


def _attend(s):
    c = s["case"]
    B, R, Hk, G, D = c["B"], c["R"], c["Hk"], c["Hq"] // c["Hk"], c["D"]
    z, m = _scores(s)
    L = z.shape[-1]
    z = z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hk, G * R, L), _side(s, s["vc"], s["vs"])).view(B, Hk, G, R, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, R, Hk * G, D).to(DT[c["dtype"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, R, Hk * G)}


def _weights(s):
    c = s["case"]
    B, R, Hk, G = c["B"], c["R"], c["Hk"], c["Hq"] // c["Hk"]
    z, _ = _scores(s)
    lse = s["lse"].view(B, R, Hk, G).permute(0, 2, 3, 1)[..., None]
    p = z.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_().sum((2, 3))
    held = torch.arange(p.shape[-1], device="cuda")[None, None, :] < s["length"][:, None, None]
    s["w"].copy_(torch.where(held, s["w"] * c["decay"] + p, s["w"]))
    return {"w": s["w"]}


def _prompt(s):
    """All sequences at once, padded to the longest."""
    c = s["case"]
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    G, n = Hq // Hk, (s["starts"][1:] - s["starts"][:-1]).long()
    L = max(1, int(c["length"]))
    at = torch.arange(L, device="cuda")
    held = at[None, :] < n[:, None]                                                    # [B][L]
    b, t = held.nonzero(as_tuple=True)
    row = s["starts"].long()[b] + t

    def padded(x):
        y = torch.zeros((B, L, x.shape[1], D), device="cuda")
        y[b, t] = x.float()[row]
        return y.permute(0, 2, 1, 3)

    q, k, v = padded(s["q"]).reshape(B, Hk, G * L, D), padded(s["k"]), padded(s["v"])
    z = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hk, G, L, L)
    mask = held[:, None, :].expand(B, L, L)
    if c["causal"]:
        mask = mask & (at[None, None, :] <= at[None, :, None])
    z.masked_fill_(~mask[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    z = z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hk, G * L, L), v).view(B, Hk, G, L, D) / l
    lse = (m + torch.log(l))[..., 0]
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, L, Hq, D)[b, t].to(DT[c["dtype"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, L, Hq)[b, t]}


def _turned(c, x, gain, pos):
    """Norm, gain, and the rotation of pairs (i, i + D/2) by position * 10000^(-2i/D), angles in 64 bits first."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain
    i = torch.arange(0, c["D"], 2, device="cuda", dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -i / c["D"])
    cos, sin, h = a.cos().float()[:, :, None], a.sin().float()[:, :, None], c["D"] // 2
    return torch.cat([y[..., :h] * cos - y[..., h:] * sin, y[..., :h] * sin + y[..., h:] * cos], -1)


def _write(s):
    c = s["case"]
    p = s["start"].long()[:, None] + torch.arange(c["T"], device="cuda")[None, :]
    ok = torch.arange(c["T"], device="cuda")[None, :] < s["new"][:, None]
    blk = s["table"].long().gather(1, (p // c["block"]).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k = s["k"]
    if c["norm"]:
        s["q_out"].copy_(_turned(c, s["q"], s["gq"], p))
        k = _turned(c, k, s["gk"], p)
    b, t = ok.nonzero(as_tuple=True)
    got = {}
    for name, x, codes, scales in (("k", k, s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        at = (blk[b, t], slice(None), p[b, t] % c["block"])
        codes[at], scales[at] = _to_4_bits(x[b, t])
        y = _from_4_bits(codes[blk, :, p % c["block"]], scales[blk, :, p % c["block"]])
        out = s[name + "_out"]
        out.copy_(torch.where(ok[:, :, None, None], y, torch.zeros_like(y)))
        got[name] = out
    return got | ({"q": s["q_out"]} if c["Hq"] else {})


def _evict(s):
    c = s["case"]
    B, Hk, T, keep, recent = c["B"], c["Hk"], c["block"], c["keep"], c["recent"]
    n, most = s["length"].long(), s["table"].shape[1] * T
    at = torch.arange(most, device="cuda")[None, :].expand(B, most)
    # rank of every token: the last ones before all others, then by weight, equal ones in order, then what is not there
    late = at >= (n - recent)[:, None]
    key = torch.where(late[:, None], torch.full_like(s["w"], math.inf), s["w"])
    key = torch.where((at < n[:, None])[:, None], key, torch.full_like(key, -1.0))
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :min(keep, most)]
    new = n.clamp(max=keep)
    slot = torch.arange(first.shape[-1], device="cuda")[None, None, :]
    # histories inside the budget stay as they are
    first = torch.where((n > keep)[:, None, None], first, slot.expand_as(first))
    first = torch.where(slot < new[:, None, None], first, torch.full_like(first, most)).sort(-1).values
    kept = torch.full((B, Hk, keep), -1, dtype=torch.int32, device="cuda")
    ok = slot < new[:, None, None]
    kept[..., :first.shape[-1]] = torch.where(ok, first, torch.full_like(first, -1)).to(torch.int32)
    b, h, i = (ok & (n > keep)[:, None, None]).expand_as(first).nonzero(as_tuple=True)
    j = first[b, h, i]
    s["w"][b, h, i] = s["w"][b, h, j]
    src, dst = s["table"].long()[b, j // T], s["table"].long()[b, i // T]
    for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        raw = codes.view(torch.uint8)
        if c["fmt"] == "e2m1":
            raw[dst, h, i % T] = raw[src, h, j % T]
            scales[dst, h, i % T] = scales[src, h, j % T]
            continue
        s0 = scales[src, h]
        s1 = torch.zeros_like(scales).view(-1).scatter_reduce_(0, dst * Hk + h, s0, "amax").view_as(scales)
        inv = torch.where(s1 > 0, 1.0 / s1, torch.zeros_like(s1))
        x = raw[src, h, j % T].view(CODE[c["fmt"]]).float() * s0[:, None]
        x = (x * inv[dst, h][:, None]).clamp(-QMAX[c["fmt"]], QMAX[c["fmt"]])
        raw[dst, h, i % T] = (x.round().to(torch.int8) if c["fmt"] == "int8" else x.to(torch.float8_e4m3fn)).view(torch.uint8)
        scales[dst, h] = s1[dst, h]
    return {"length": new.to(torch.int32), "kept": kept, "w": s["w"], "k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"prompt": _prompt, "write": _write, "attend": _attend, "weights": _weights, "evict": _evict}[c["op"]](s)
    if c["op"] == "prompt":
        out, lse = s["attn"](s["q"], s["k"], s["v"], s["starts"])
        return {"out": out, "lse": lse}
    if c["op"] == "write":
        s["cache"].append(s["k"], s["v"], s["table"], s["start"], s["new"], q=s["q"] if c["Hq"] else None,
                          q_out=s["q_out"], norm_rope=s["nr"])
        s["cache"].read(s["table"], s["start"], s["new"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]} | ({"q": s["q_out"]} if c["Hq"] else {})
    if c["op"] == "attend":
        out, lse = s["attn"](s["q"], s["table"], s["length"], s["rows"])
        return {"out": out, "lse": lse}
    if c["op"] == "weights":
        s["cache"].add_weights(s["w"], s["q"], s["lse"], s["table"], s["length"], n_rows=s["rows"], causal=c["causal"],
                               scale=s["scale"], decay=c["decay"])
        return {"w": s["w"]}
    length, kept = s["evict"](s["w"], s["table"], s["length"])
    return {"length": length, "kept": kept, "w": s["w"], "k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"]}


def _side_bytes(c, tokens, blocks):
    """Codes and scales of one side of a cache."""
    if c.get("fmt", "e2m1") == "e2m1":
        return tokens * c["Hk"] * (c["D"] // 2 + c["D"] // 16)
    return tokens * c["Hk"] * c["D"] + blocks * c["Hk"] * 4


def work(case):
    c = case
    if c["op"] == "prompt":
        e, n = SIZE[c["dtype"]], _lengths(c)
        seen = sum(x * (x + 1) // 2 if c["causal"] else x * x for x in n)
        return {"bytes": sum(n) * ((2 * c["Hq"] + 2 * c["Hk"]) * c["D"] * e + 4 * c["Hq"]) + 4 * (c["B"] + 1),
                "flops": 4 * seen * c["Hq"] * c["D"]}
    if c["op"] == "write":
        e, tokens, rows = SIZE[c["dtype"]], sum(_news(c)), c["B"] * c["T"]
        q, kv = rows * c["Hq"] * c["D"], tokens * 2 * c["Hk"] * c["D"]
        # activations in, codes and scales out and in again, values out (zeros behind a request's rows among them)
        return {"bytes": 2 * q * e + kv * e + 4 * _side_bytes(c, tokens, 0) + rows * 2 * c["Hk"] * c["D"] * e + 8 * c["B"],
                "flops": 7 * q + 6 * kv}
    lengths = _lengths(c)
    blocks = sum(-(-n // c["block"]) for n in lengths)
    if c["op"] == "evict":
        moved = sum(c["keep"] for n in lengths if n > c["keep"])
        moved_blocks = sum(-(-c["keep"] // c["block"]) for n in lengths if n > c["keep"])
        weighed = sum(n for n in lengths if n > c["keep"]) * c["Hk"]
        return {"bytes": 4 * _side_bytes(c, moved, moved_blocks) + 4 * weighed + 4 * moved * c["Hk"] + 4 * c["B"] * c["Hk"] * c["keep"] + 4 * blocks,
                "flops": weighed}
    rows = _rows(c)
    seen = 0
    for n, r in zip(lengths, rows):
        if c["causal"]:   # the last min(n, r) rows see n, n - 1, ... tokens
            m = min(n, r)
            seen += m * n - m * (m - 1) // 2
        else:
            seen += n * r
    q = c["B"] * c["R"] * c["Hq"]
    if c["op"] == "weights":
        return {"bytes": _side_bytes(c, sum(lengths), blocks) + 4 * blocks + q * (c["D"] * SIZE[c["dtype"]] + 4) + 8 * sum(lengths) * c["Hk"],
                "flops": 2 * seen * c["Hq"] * c["D"]}
    return {"bytes": 2 * _side_bytes(c, sum(lengths), blocks) + 4 * blocks + q * (2 * c["D"] * SIZE[c["dtype"]] + 4),
            "flops": 4 * seen * c["Hq"] * c["D"]}


# ------------------------------------------------------------------------------------ from the definition

def exact(case, seed):
    global own
    c = case
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] != "write" and c["op"] != "evict" and work(c)["flops"] > 2e12:
        return None
    return {"prompt": _exact_prompt, "write": _exact_write, "attend": _exact_attend, "weights": _exact_weights,
            "evict": _exact_evict}[c["op"]](s)


def _softmax_of(z, mask, v):
    """Rows of scores [R][n] in 64 bits: outputs and log-sum-exps; rows whose mask leaves nothing give 0 and -inf."""
    z = torch.where(mask, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return p @ v, lse


def _exact_prompt(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    edge = s["starts"].tolist()
    for a, b in zip(edge[:-1], edge[1:]):
        i = torch.arange(b - a, device="cuda")
        mask = i[None, :] <= i[:, None] if c["causal"] else torch.ones((b - a, b - a), dtype=torch.bool, device="cuda")
        for h in range(c["Hq"] if b > a else 0):
            g = h // (c["Hq"] // c["Hk"])
            z = s["q"][a:b, h].double() @ s["k"][a:b, g].double().T * s["scale"]
            out[a:b, h], lse[a:b, h] = _softmax_of(z, mask, s["v"][a:b, g].double())
    return {"out": out, "lse": lse}


def _history(s, b, h, codes, scales, n):
    """Tokens 0 .. n - 1 of request b and key head h in 64 bits, element by element of the stored bytes."""
    c, T = s["case"], s["case"]["block"]
    p = torch.arange(n, device="cuda")
    blk, row = s["table"][b].long()[p // T], p % T
    if c.get("fmt", "e2m1") != "e2m1":
        return codes.view(torch.uint8)[blk, h, row].view(CODE[c["fmt"]]).double() * scales[blk, h].double()[:, None]
    byte = codes[blk, h, row].long()
    nibble = torch.empty((n, c["D"]), dtype=torch.long, device="cuda")
    nibble[:, 0::2], nibble[:, 1::2] = byte % 16, byte // 16
    sign, e, m = 1.0 - 2.0 * (nibble // 8), (nibble // 2) % 4, nibble % 2
    value = sign * torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + 0.5 * m), 0.5 * m)
    u = scales[blk, h, row].double()
    e, m = torch.floor(u / 8), u % 8
    scale = torch.where(e > 0, torch.exp2(e - 15) * (1 + m / 8), torch.exp2(e - 14) * m / 8)
    return value * scale.repeat_interleave(16, -1)


def _exact_attend(s):
    c = s["case"]
    out = torch.zeros((c["B"], c["R"], c["Hq"], c["D"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["R"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hk"]
    for b, (n, rows) in enumerate(zip(_lengths(c), _rows(c))):
        for h in range(c["Hk"] if n else 0):
            k, v = _history(s, b, h, s["kc"], s["ks"], n), _history(s, b, h, s["vc"], s["vs"], n)
            i = torch.arange(rows, device="cuda")
            mask = torch.arange(n, device="cuda")[None, :] < (n - (rows - 1 - i) if c["causal"] else torch.full_like(i, n))[:, None]
            for j in range(h * G, (h + 1) * G):
                out[b, :rows, j], lse[b, :rows, j] = _softmax_of(s["q"][b, :rows, j].double() @ k.T * s["scale"], mask, v)
    return {"out": out, "lse": lse}


def _exact_weights(s):
    c = s["case"]
    w, G = s["w"].double(), c["Hq"] // c["Hk"]
    for b, (n, rows) in enumerate(zip(_lengths(c), _rows(c))):
        for h in range(c["Hk"] if n else 0):
            k = _history(s, b, h, s["kc"], s["ks"], n)
            w[b, h, :n] *= c["decay"]
            i = torch.arange(rows, device="cuda")
            mask = torch.arange(n, device="cuda")[None, :] < (n - (rows - 1 - i) if c["causal"] else torch.full_like(i, n))[:, None]
            for j in range(h * G, (h + 1) * G):
                z = s["q"][b, :rows, j].double() @ k.T * s["scale"] - s["lse"][b, :rows, j].double()[:, None]
                w[b, h, :n] += torch.where(mask, torch.exp(z), torch.zeros_like(z)).sum(0)
    return {"w": w}


def _exact_write(s):
    c = s["case"]
    got = {"k": torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")}
    got["v"] = torch.zeros_like(got["k"])
    level = _levels(torch.float64)[:8]
    if c["norm"]:   # pairs as complex numbers times e^(i angle)
        def turned(x, gain):
            y = x.double()
            y = y * gain.double() / (y.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()
            f = torch.exp(-math.log(10000.0) * 2.0 * torch.arange(c["D"] // 2, device="cuda", dtype=torch.float64) / c["D"])
            pos = s["start"].double()[:, None] + torch.arange(c["T"], device="cuda")[None, :]
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, :, None, None] * f)
            z = torch.complex(y[..., :c["D"] // 2], y[..., c["D"] // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)
        got["q"] = turned(s["q"], s["gq"])
        got["k"] = None     # the codes of turned keys hang on single roundings: they have no value in 64 bits
    for name in ("k", "v"):
        if got[name] is None:
            continue
        for b, n in enumerate(_news(c)):
            x = s[name][b, :n].double().reshape(n, c["Hk"], c["D"] // 16, 16)
            top = x.abs().amax(-1) / 6.0
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -60)))
            e = torch.where(torch.exp2(e) > top, e - 1, e)
            e = torch.where(torch.exp2(e + 1) <= top, e + 1, e).clamp(min=-14)
            scale = (torch.round(top / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(max=10240.0)[..., None]
            # the nearest level of every element; where two are as near, that of the even code
            near = (x.abs()[..., None] - level * scale[..., None]).abs()
            near[..., 1::2] *= 1 + 1e-13
            y = level[near.argmin(-1)] * scale * torch.sign(x)
            got[name][b, :n] = y.reshape(n, c["Hk"], c["D"])
    return got


def _exact_evict(s):
    """The kept tokens' weights alone: the rest of the outputs are whole numbers and codes."""
    c = s["case"]
    w = s["w"].double()
    for b, n in enumerate(_lengths(c)):
        if n <= c["keep"]:
            continue
        for h in range(c["Hk"]):
            old = s["w"][b, h, :n].tolist()
            by = sorted(range(n - c["recent"]), key=lambda j: (-old[j], j))
            at = sorted(by[:c["keep"] - c["recent"]] + list(range(n - c["recent"], n)))
            w[b, h, :c["keep"]] = s["w"][b, h, torch.tensor(at, device="cuda")].double()
    none = None
    return {"length": none, "kept": none, "w": w, "k": none, "v": none, "ks": none, "vs": none}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(1)) for _ in range(3)]:
        print(case.get("name", "drawn"), work(case))
