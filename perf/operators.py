"""The history-cache operators as measurable cases: a per-head norm with the position rotation, the write of
keys and values into an 8-bit block cache, the read back, and attention over that cache.

A recommendation model serves a request in three moves: the user's history (item tokens) is written into the
cache, later events are appended one at a time, and the beams of a decode attend to the history.  The cases are
those moves at small, ordinary and large sizes.

`own` False: elementary torch operations in 32 bits (64 for the angles).  `own` True: the calls a user makes.

Definitions.
  norm       y = x / sqrt(mean(x^2) + eps) * gain, over one head's `dim` elements
  rotation   pairs (a, b) of the first `rot` elements -> (a cos - b sin, a sin + b cos), angle = position *
             theta^(-2 i / rot) for pair i; pairs are (i, i + rot/2), or (2i, 2i + 1) interleaved
  cache      codes [block][head][token][dim] in e4m3 or int8, one float32 scale a (block, head); value = code *
             scale; a request's token p is row p % T of block table[b][p / T]
  write      scale = max(scale of the rows that the block already holds, largest |x| written / Q) with Q = 448 or
             127; code = round(x * (1 / scale)) to nearest even, clamped to +-Q; rows already there are coded
             again where the scale has grown
  attention  softmax(scale * q k^T) v over the first `length` tokens; causal: row r of n rows sees the first
             length - (n - 1 - r); a row that sees nothing gives zeros and a log-sum-exp of -inf
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
TINY = 2.0 ** -126        # a scale below the smallest normal number is held as zero


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # norm + rotation of one new token a request: a serving batch of the large catalogue (64 requests)
        dict(name="rotate one token", op="rotate", dtype="bf16", B=64, T=1, Hq=8, Hk=2, D=128, rot=128,
             inter=False, far=100000, theta=10000.0),
        # full histories of a training-size batch at once, bound by memory
        dict(name="rotate histories", op="rotate", dtype="bf16", B=32, T=4096, Hq=16, Hk=4, D=128, rot=128,
             inter=False, far=1, theta=1000000.0),
        # the newest event of 64 users: norm, rotation and the quantised write in one call
        dict(name="write one token", op="write", dtype="bf16", fmt="e4m3", B=64, T=1, Hq=8, Hk=2, D=128, rot=128,
             inter=False, block=64, start=1500, theta=10000.0, norm=True),
        # a batch of new users: whole histories written at once
        dict(name="write histories", op="write", dtype="bf16", fmt="e4m3", B=32, T=2048, Hq=16, Hk=4, D=128,
             rot=128, inter=False, block=64, start=0, theta=10000.0, norm=True),
        # ragged chunks that begin inside a block, int8, written and read back
        dict(name="write and read int8", op="roundtrip", dtype="f16", fmt="int8", B=16, T=1000, Hq=0, Hk=4, D=64,
             rot=0, inter=False, block=32, start=77, theta=10000.0, norm=False),
        # few users, odd lengths, a head of 96 (the dense-early width 384 over four heads), fp32 activations
        dict(name="write and read odd f32", op="roundtrip", dtype="f32", fmt="e4m3", B=3, T=1001, Hq=0, Hk=4, D=96,
             rot=0, inter=False, block=16, start=5, theta=10000.0, norm=False),
        # one user, one event: latency
        dict(name="attend one user", op="attend", dtype="bf16", fmt="e4m3", B=1, R=1, Hq=4, Hk=4, D=64, block=16,
             length=509, causal=False, ragged=False),
        # one token for each of 64 users with a few thousand events
        dict(name="attend one token", op="attend", dtype="bf16", fmt="e4m3", B=64, R=1, Hq=8, Hk=2, D=128,
             block=64, length=4096, causal=False, ragged=True),
        # lifelong histories: few requests, a long cache
        dict(name="attend lifelong", op="attend", dtype="bf16", fmt="int8", B=8, R=1, Hq=16, Hk=4, D=128, block=64,
             length=131072, causal=False, ragged=True),
        # the beams of a mid-size decode (32 requests, 64 beams, width 256 over four heads) over short histories
        dict(name="attend 64 beams", op="attend", dtype="f16", fmt="int8", B=32, R=64, Hq=4, Hk=4, D=64, block=32,
             length=1000, causal=False, ragged=True),
        # the beams of the large catalogue (64 requests, 256 beams, width 512 over four heads)
        dict(name="attend 256 beams", op="attend", dtype="bf16", fmt="e4m3", B=64, R=256, Hq=4, Hk=4, D=128,
             block=64, length=2048, causal=False, ragged=True),
        # a long history taken in by chunks: each row sees the tokens before it
        dict(name="attend chunk causal", op="attend", dtype="bf16", fmt="e4m3", B=2, R=2048, Hq=16, Hk=4, D=128,
             block=64, length=16384, causal=True, ragged=True),
    ]


def _log(rng, a, b):
    """A whole number between a and b, spread over the logarithm."""
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["rotate", "write", "roundtrip", "attend", "attend", "attend"])
    D = rng.choice([32, 64, 64, 96, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    fmt = rng.choice(["e4m3", "int8"])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    inter = rng.random() < 0.5
    if op == "attend":
        kind = rng.choice(["token", "token", "beams", "chunk"])
        B = _log(rng, 1, 96)
        if kind == "token":
            R, causal, most = 1, False, 300_000_000
        elif kind == "beams":
            R, causal, most = _log(rng, 2, 512), False, 300_000_000
        else:
            R, causal, most = _log(rng, 2, 2500), True, 300_000_000
        while B * R * Hq * D > 150_000_000:
            B, R = max(1, B // 2), max(1, R // 2) if B == 1 else R
        # the codes of one side, and the scores of all rows, bound the length
        most_len = min(most / (B * Hk * D), 500_000_000 / (B * Hq * R), 100_000)
        while most_len < 40:
            B, most_len = max(1, B // 2), most_len * 2
            if B == 1 and most_len < 40:
                R = max(1, R // 2)
                most_len = 500_000_000 / (Hq * R)
        length = _log(rng, 1 if kind == "token" else 17, int(most_len))
        return dict(op=op, dtype=dtype, fmt=fmt, B=B, R=R, Hq=Hq, Hk=Hk, D=D, block=block, length=length,
                    causal=causal, ragged=rng.random() < 0.8)
    B = _log(rng, 1, 96)
    T = 1 if rng.random() < 0.3 else _log(rng, 2, min(5000, 80_000_000 // (B * (Hq + 2 * Hk) * D)))
    rot = rng.choice([D, D, D // 2])
    theta = rng.choice([10000.0, 500000.0, 1000000.0])
    if op == "rotate":
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot,
                    inter=inter, far=_log(rng, 1, 10_000_000), theta=theta)
    if op == "write":
        return dict(op=op, dtype=dtype, fmt="e4m3", B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, inter=inter, block=block,
                    start=rng.choice([0, rng.randrange(1, 3000)]), theta=theta, norm=rng.random() < 0.8)
    return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), fmt=fmt, B=B, T=T, Hq=0, Hk=Hk, D=D, rot=0, inter=False, block=block,
                start=rng.choice([0, rng.randrange(1, 3000)]), theta=theta, norm=False)


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
    return _spread(c["B"], max(1, c["T"] // 3), c["T"], c["op"] == "roundtrip" and c["T"] > 1)


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


def _pool(g, total, c):
    """Codes and scales as normal keys and values leave them: a block's largest |x| is near 4.2 sigma."""
    shape = (total, c["Hk"], c["block"], c["D"])
    q, out = QMAX[c["fmt"]], []
    for _ in range(2):
        x = _randn(g, shape, torch.float16).mul_(q / 4.2).clamp_(-q, q)
        out.append(x.round_().to(torch.int8) if c["fmt"] == "int8" else x.to(torch.float8_e4m3fn))
    scales = [torch.exp(0.4 * _randn(g, shape[:2])) * (4.2 / q) for _ in range(2)]
    return out[0], out[1], scales[0], scales[1]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    dt = DT[c["dtype"]]
    if c["op"] == "attend":
        lengths, rows = _lengths(c), _rows(c)
        s["table"], total = _table(g, lengths, c["block"], 3)
        s["kc"], s["vc"], s["ks"], s["vs"] = _pool(g, total, c)
        if c["fmt"] == "e4m3":   # what lies behind a request's last token is not defined: NaN codes here
            last = torch.tensor([n - 1 for n in lengths], device="cuda")
            blk = s["table"].long().gather(1, last.clamp(min=0).div(c["block"], rounding_mode="floor")[:, None])[:, 0]
            dead = torch.arange(c["block"], device="cuda")[None, :] > (last % c["block"])[:, None]
            dead &= (last >= 0)[:, None]
            b, t = dead.nonzero(as_tuple=True)
            s["kc"].view(torch.uint8)[blk[b], :, t] = 0x7F
            s["vc"].view(torch.uint8)[blk[b], :, t] = 0x7F
        s["length"], s["rows"] = _ints(lengths), _ints(rows)
        s["q"] = (2.0 * _randn(g, (c["B"], c["R"], c["Hq"], c["D"]))).to(dt)
        s["scale"] = 1.0 / math.sqrt(c["D"])
        if own:
            from generative_recommendation_constrained_gb300.device import CacheAttention, KVCache
            cache = KVCache.over(s["kc"], s["vc"], s["ks"], s["vs"])
            s["attn"] = CacheAttention(cache, c["B"], c["R"], c["Hq"], s["table"].shape[1], causal=c["causal"],
                                       scale=s["scale"], dtype=dt, lse=True)
        return s
    # projections of a history: q, k and v side by side in one buffer, as one matrix product leaves them
    heads = c["Hq"] + c["Hk"] * (1 if c["op"] == "rotate" else 2)
    x = _randn(g, (c["B"], c["T"], heads, c["D"]), torch.float16 if c["dtype"] == "f16" else torch.float32)
    x = (x * (0.5 + torch.rand((1, 1, heads, 1), generator=g, device="cuda"))).to(dt)
    s["q"], s["k"] = x[:, :, :c["Hq"]], x[:, :, c["Hq"]:c["Hq"] + c["Hk"]]
    s["gq"], s["gk"] = (1.0 + 0.2 * _randn(g, (c["D"],)) for _ in range(2))
    if c["op"] == "rotate":
        first = torch.randint(0, c["far"], (c["B"], 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(c["T"], device="cuda")[None, :]).to(torch.int32)
        s["q_out"], s["k_out"] = torch.empty(s["q"].shape, dtype=dt, device="cuda"), torch.empty(s["k"].shape, dtype=dt, device="cuda")
        if own:
            from generative_recommendation_constrained_gb300.device import NormRope
            s["nr"] = NormRope(c["D"], s["gq"], s["gk"], eps=EPS, rot_dim=c["rot"], theta=c["theta"],
                               interleaved=c["inter"])
        return s
    s["v"] = x[:, :, c["Hq"] + c["Hk"]:]
    starts, news = _starts(c), _news(c)
    s["table"], total = _table(g, [a + n for a, n in zip(starts, news)], c["block"], 2)
    s["kc"], s["vc"], s["ks"], s["vs"] = _pool(g, total, c)
    s["start"], s["new"] = _ints(starts), _ints(news)
    s["q_out"] = torch.empty(s["q"].shape, dtype=dt, device="cuda") if c["Hq"] else None
    if c["op"] == "roundtrip":
        s["k_out"], s["v_out"] = (torch.empty(s["k"].shape, dtype=dt, device="cuda") for _ in range(2))
    if own:
        from generative_recommendation_constrained_gb300.device import KVCache, NormRope
        s["cache"] = KVCache.over(s["kc"], s["vc"], s["ks"], s["vs"])
        s["nr"] = NormRope(c["D"], s["gq"], s["gk"], eps=EPS, rot_dim=c["rot"], theta=c["theta"],
                           interleaved=c["inter"], norm=c["norm"]) if c["norm"] or c["rot"] else None
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _angles(c, pos):
    """cos and sin [.., rot/2] of every position's angles, in 64 bits first."""
    i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"), -i / c["rot"])
    return a.cos().float(), a.sin().float()


def _norm_rotate(c, x, gain, cos, sin, norm):
    y = x.float()
    if norm:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain
    if not c["rot"]:
        return y
    y = y.clone()
    cos, sin, h = cos[:, :, None], sin[:, :, None], c["rot"] // 2
    a, b = (y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]) if c["inter"] else (y[..., :h], y[..., h:c["rot"]])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    if c["inter"]:
        y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = ra, rb
    else:
        y[..., :h], y[..., h:c["rot"]] = ra, rb
    return y


def _code(x, inverse, fmt):
    x = (x * inverse).clamp(-QMAX[fmt], QMAX[fmt])
    return x.round().to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)


def _write(c, x, codes, scales, table, start, new):
    """x [B][T][Hk][D] float32 into one side of the cache, in place."""
    B, T, bt, fmt = c["B"], c["T"], c["block"], c["fmt"]
    p = start.long()[:, None] + torch.arange(T, device="cuda")[None, :]
    ok = torch.arange(T, device="cuda")[None, :] < new[:, None]
    width = table.shape[1]
    blk = table.long().gather(1, (p // bt).clamp(max=width - 1))
    b, t = ok.nonzero(as_tuple=True)
    blk, row, x = blk[b, t], p[b, t] % bt, x[b, t]
    # largest |x| of every touched block and head, and the scale of the rows that it holds already
    top = torch.zeros_like(scales)
    top.scatter_reduce_(0, blk[:, None].expand(-1, c["Hk"]), x.abs().amax(-1), "amax")
    s1 = top / QMAX[fmt]
    held = start.long() % bt                                    # rows held in each request's first block
    part = ((held > 0) & (new > 0)).nonzero()[:, 0]
    fb = table.long().gather(1, (start.long() // bt).clamp(max=width - 1)[:, None])[part, 0]
    s0 = scales[fb]
    s1[fb] = torch.maximum(s1[fb], s0)
    s1 = torch.where(s1 < TINY, torch.zeros_like(s1), s1)
    inverse = torch.where(s1 > 0, 1.0 / s1, torch.zeros_like(s1))
    raw = codes.view(torch.uint8)                               # indexed writes of 8-bit values
    old = raw[fb].view(CODE[fmt])
    again = _code(old.float() * s0[:, :, None, None], inverse[fb][:, :, None, None], fmt)
    grown = (s1[fb] > s0)[:, :, None, None] & (torch.arange(bt, device="cuda")[None, :] < held[part][:, None])[:, None, :, None]
    raw[fb] = torch.where(grown, again.view(torch.uint8), old.view(torch.uint8))
    raw[blk, :, row] = _code(x, inverse[blk][:, :, None], fmt).view(torch.uint8)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda")
    touched[blk] = True
    scales.copy_(torch.where(touched[:, None], s1, scales))


def _read(c, codes, scales, table, start, new, out):
    p = start.long()[:, None] + torch.arange(c["T"], device="cuda")[None, :]
    ok = torch.arange(c["T"], device="cuda")[None, :] < new[:, None]
    blk = table.long().gather(1, (p // c["block"]).clamp(max=table.shape[1] - 1)).clamp(min=0)
    x = codes.view(torch.uint8)[blk, :, p % c["block"]].view(CODE[c["fmt"]]).float() * scales[blk][..., None]
    out.copy_(torch.where(ok[:, :, None, None], x, torch.zeros_like(x)))
    return out


def _attend(s):
    c = s["case"]
    B, R, Hq, Hk, D, bt = (c[k] for k in ("B", "R", "Hq", "Hk", "D", "block"))
    G, width = Hq // Hk, s["table"].shape[1]
    L = width * bt
    blk = s["table"].long().clamp(min=0)
    key = torch.arange(L, device="cuda")
    held = key[None, :] < s["length"][:, None]                                          # [B][L]

    def side(codes, scales):
        x = codes.view(torch.uint8)[blk].view(CODE[c["fmt"]]).float() * scales[blk][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D)
        return torch.where(held[:, None, :, None], x, torch.zeros((), device="cuda"))

    q = s["q"].float().reshape(B, R, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * R, D)
    z = torch.matmul(q, side(s["kc"], s["ks"]).transpose(2, 3)) * s["scale"]            # [B][Hk][G R][L]
    sees = s["length"][:, None].expand(B, R)
    row = torch.arange(R, device="cuda")[None, :]
    if c["causal"]:
        sees = sees - (s["rows"][:, None] - 1 - row)
    sees = torch.where(row < s["rows"][:, None], sees, torch.zeros_like(sees))
    mask = key[None, None, :] < sees[:, :, None]                                        # [B][R][L]
    z = z.view(B, Hk, G, R, L).masked_fill_(~mask[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    z = z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hk, G * R, L), side(s["vc"], s["vs"])).view(B, Hk, G, R, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, R, Hq, D).to(DT[c["dtype"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, R, Hq)}


def run(state):
    s, c = state, state["case"]
    if c["op"] == "attend":
        if own:
            out, lse = s["attn"](s["q"], s["table"], s["length"], s["rows"])
            return {"out": out, "lse": lse}
        return _attend(s)
    if c["op"] == "rotate":
        if own:
            s["nr"](s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
        else:
            cos, sin = _angles(c, s["pos"])
            s["q_out"].copy_(_norm_rotate(c, s["q"], s["gq"], cos, sin, True))
            s["k_out"].copy_(_norm_rotate(c, s["k"], s["gk"], cos, sin, True))
        return {"q": s["q_out"], "k": s["k_out"]}
    if own:
        s["cache"].append(s["k"], s["v"], s["table"], s["start"], s["new"], q=s["q"] if c["Hq"] else None,
                          q_out=s["q_out"], norm_rope=s["nr"])
        if c["op"] == "roundtrip":
            s["cache"].read(s["table"], s["start"], s["new"], s["k_out"], s["v_out"])
    else:
        k, cos, sin = s["k"].float(), None, None
        if c["rot"]:
            pos = s["start"].long()[:, None] + torch.arange(c["T"], device="cuda")[None, :]
            cos, sin = _angles(c, pos)
        if c["norm"] or c["rot"]:
            k = _norm_rotate(c, s["k"], s["gk"], cos, sin, c["norm"])
            if c["Hq"]:
                s["q_out"].copy_(_norm_rotate(c, s["q"], s["gq"], cos, sin, c["norm"]))
        elif c["Hq"]:
            s["q_out"].copy_(s["q"])
        _write(c, k, s["kc"], s["ks"], s["table"], s["start"], s["new"])
        _write(c, s["v"].float(), s["vc"], s["vs"], s["table"], s["start"], s["new"])
        if c["op"] == "roundtrip":
            _read(c, s["kc"], s["ks"], s["table"], s["start"], s["new"], s["k_out"])
            _read(c, s["vc"], s["vs"], s["table"], s["start"], s["new"], s["v_out"])
    if c["op"] == "roundtrip":
        return {"k": s["k_out"], "v": s["v_out"], "ks": s["ks"], "vs": s["vs"]}
    got = {"k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"]}
    return got | {"q": s["q_out"]} if c["Hq"] else got


def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "attend":
        lengths, rows = _lengths(c), _rows(c)
        seen = 0
        for n, r in zip(lengths, rows):
            if c["causal"]:   # the last min(n, r) rows see n, n - 1, ... tokens
                m = min(n, r)
                seen += m * n - m * (m - 1) // 2
            else:
                seen += n * r
        blocks = sum(-(-n // c["block"]) for n in lengths)
        held = sum(lengths) * c["Hk"] * c["D"] * 2 + blocks * (8 * c["Hk"] + 4)
        q = c["B"] * c["R"] * c["Hq"] * (2 * c["D"] * e + 4)
        return {"bytes": held + q, "flops": 4 * seen * c["Hq"] * c["D"]}
    rows = c["B"] * c["T"]
    if c["op"] == "rotate":
        n = rows * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * e + 4 * rows, "flops": 7 * n}
    tokens = sum(_news(c))
    q = rows * c["Hq"] * c["D"]
    kv = tokens * 2 * c["Hk"] * c["D"]
    blocks = sum(-(-(a + n) // c["block"]) - a // c["block"] for a, n in zip(_starts(c), _news(c)))
    b = 2 * q * e + kv * (e + 1) + blocks * (8 * c["Hk"] + 4)
    if c["op"] == "roundtrip":
        b += kv * 1 + rows * 2 * c["Hk"] * c["D"] * e
    return {"bytes": b, "flops": 7 * q + 6 * kv}


# ------------------------------------------------------------------------------------ from the definition

def _exact_rotated(c, x, gain, pos, norm):
    """Rows x [T][H][D] of one request in 64 bits: pairs as complex numbers times e^(i angle)."""
    y = x.double()
    if norm:
        y = y * gain.double() / (y.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()
    r = c["rot"]
    if not r:
        return y
    freq = torch.exp(-math.log(c["theta"]) * 2.0 * torch.arange(r // 2, device="cuda", dtype=torch.float64) / r)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None, None] * freq)
    pairs = y[..., :r].reshape(*y.shape[:-1], r // 2, 2) if c["inter"] else y[..., :r].reshape(*y.shape[:-1], 2, r // 2).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.reshape(*y.shape[:-1], r) if c["inter"] else z.transpose(-1, -2).reshape(*y.shape[:-1], r)
    return torch.cat([z, y[..., r:]], -1)


def exact(case, seed):
    global own
    c = case
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "rotate":
        f = lambda x, g: torch.stack([_exact_rotated(c, x[b], g, s["pos"][b], True) for b in range(c["B"])])  # noqa: E731
        return {"q": f(s["q"], s["gq"]), "k": f(s["k"], s["gk"])}
    if c["op"] == "attend":
        return _exact_attend(s)
    q_max, bt = QMAX[c["fmt"]], c["block"]
    scales = {"ks": s["ks"].double(), "vs": s["vs"].double()}
    q = []
    for b, (a, n) in enumerate(zip(_starts(c), _news(c))):
        pos = torch.arange(a, a + c["T"], device="cuda")
        if c["Hq"]:
            q.append(_exact_rotated(c, s["q"][b], s["gq"], pos, c["norm"]))
        k = _exact_rotated(c, s["k"][b, :n], s["gk"], pos[:n], c["norm"])
        for side, x in (("ks", k), ("vs", s["v"][b, :n].double())):
            at = a
            while at < a + n:                       # block by block of this request
                end = min(a + n, (at // bt + 1) * bt)
                blk = int(s["table"][b, at // bt])
                top = x[at - a:end - a].abs().amax(-1).amax(0) / q_max
                scales[side][blk] = torch.maximum(top, scales[side][blk]) if at % bt else top
                at = end
    if c["op"] == "roundtrip":   # the values read back hang on single roundings: codes have no value in 64 bits
        return {"k": None, "v": None, **scales}
    got = {"k": None, "v": None, **scales}
    return got | {"q": torch.stack(q)} if c["Hq"] else got


def _exact_attend(s):
    c = s["case"]
    bt, G = c["block"], c["Hq"] // c["Hk"]
    out = torch.zeros((c["B"], c["R"], c["Hq"], c["D"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["R"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    if work(c)["flops"] > 1e12:
        return None
    for b, (n, rows) in enumerate(zip(_lengths(c), _rows(c))):
        if not n:
            continue
        blk = s["table"][b, :-(-n // bt)].long()
        for h in range(c["Hk"]):
            k, v = ((x.view(torch.uint8)[blk, h].view(CODE[c["fmt"]]).double() * y[blk, h][:, None, None].double()).reshape(-1, c["D"])[:n]
                    for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            sees = torch.arange(rows, device="cuda") + (n - rows + 1) if c["causal"] else torch.full((rows,), n, device="cuda")
            for j in range(h * G, (h + 1) * G):
                z = s["q"][b, :rows, j].double() @ k.T * s["scale"]
                z = torch.where(torch.arange(n, device="cuda")[None, :] < sees[:, None], z, torch.full_like(z, -math.inf))
                some = sees > 0
                lse[b, :rows, j] = torch.logsumexp(z, -1)
                out[b, :rows, j] = torch.where(some[:, None], torch.nan_to_num(torch.softmax(z, -1)) @ v, torch.zeros((), dtype=torch.float64, device="cuda"))
    return {"out": out, "lse": lse}
