"""From users' histories to constrained recommendations, on one GPU.

Every user has a history of item events.  One attention layer with random
weights stands for the model that makes the decoder's request vectors:

  1. the histories are written into an 8-bit block cache in one call (keys
     normalised per head and rotated by position on the way);
  2. a new event of every user is appended, and its query attends to the whole
     history: the result is the request vector u;
  3. zg_decode searches the catalogue with beams, constrained to real items;
  4. the returned items attend to the history they were made from, all beams of
     a user at once over the one cache, and are re-scored by it.

    python examples/history_decode.py [--users 64] [--events 500] [--fmt int8]

The weights are random: the numbers show the path, not quality.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import generative_recommendation_constrained_gb300 as zg
import synth
from generative_recommendation_constrained_gb300.device import CacheAttention, Decoder, DeviceModel, KVCache, NormRope

HEADS, KV_HEADS, DIM, BLOCK = 8, 2, 64, 32


class HistoryLayer:
    """Query, key, value and output projections of one attention layer over a user's events."""

    def __init__(self, d: int, seed: int):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.wqkv = torch.randn((d, (HEADS + 2 * KV_HEADS) * DIM), generator=g, device="cuda").mul_(d ** -0.5).bfloat16()
        self.wo = torch.randn((HEADS * DIM, d), generator=g, device="cuda").mul_((HEADS * DIM) ** -0.5).bfloat16()
        gain = [1 + 0.1 * torch.randn((DIM,), generator=g, device="cuda") for _ in range(2)]
        self.turn = NormRope(DIM, *gain)

    def project(self, x: torch.Tensor):
        """q, k, v [B, T, heads, DIM] of events x [B, T, d]: views of one product's output."""
        y = (x.bfloat16() @ self.wqkv).view(*x.shape[:2], HEADS + 2 * KV_HEADS, DIM)
        return y[:, :, :HEADS], y[:, :, HEADS:HEADS + KV_HEADS], y[:, :, HEADS + KV_HEADS:]

    def output(self, a: torch.Tensor) -> torch.Tensor:
        return (a.flatten(2) @ self.wo).float()


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--events", type=int, default=500, help="events of the longest history")
    ap.add_argument("--fmt", choices=("e4m3", "int8"), default="e4m3")
    ap.add_argument("--seed", type=int, default=1)
    a = ap.parse_args(argv)

    cfg = synth.CONFIGS["tiny"]
    sids = synth.make_catalogue(cfg)
    model = synth.make_model(cfg.L, cfg.V, cfg.d, cfg.w_dtype)
    dm = DeviceModel(model)
    index = zg.zg_index_build(sids, cfg.V, stream=torch.cuda.current_stream().cuda_stream)
    layer = HistoryLayer(cfg.d, a.seed)
    tokens = torch.from_numpy(np.ascontiguousarray(sids)).long().cuda()

    def embed(items):                                   # an item: the sum of its tokens' vectors
        t = tokens[items]
        return sum(dm.C[s][t[..., s]] for s in range(cfg.L - 1))

    # histories of uneven length, padded on the right, and one new event each
    g = torch.Generator(device="cuda").manual_seed(a.seed)
    B, T = a.users, a.events
    held = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    events = torch.randint(0, len(sids), (B, T), generator=g, device="cuda")
    latest = torch.randint(0, len(sids), (B, 1), generator=g, device="cuda")

    # the cache: blocks of every user, in no order
    width = -(-(T + 1) // BLOCK)
    cache = KVCache(B * width, BLOCK, KV_HEADS, DIM, a.fmt)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    zero = torch.zeros((B,), dtype=torch.int32, device="cuda")
    one = CacheAttention(cache, B, 1, HEADS, width)
    beams = CacheAttention(cache, B, cfg.topk, HEADS, width, lse=True)
    decoder = Decoder(index, None, dm, B, cfg.beam, cfg.topk)

    # 1. the histories
    _, k, v = layer.project(embed(events))
    cache.append(k, v, table, zero, held, norm_rope=layer.turn)

    # 2. the new event: written, and its query over everything
    x = embed(latest)
    q, k, v = layer.project(x)
    q = cache.append(k, v, table, held, q=q, norm_rope=layer.turn)
    length = held + 1
    a1, _ = one(q, table, length)
    u = (x + layer.output(a1))[:, 0].contiguous()

    # 3. the constrained search
    out_sids, scores = decoder(u)

    # 4. the found items (as events one position on) over the same history
    found = embed_sids(out_sids, dm, cfg.L)
    q, _, _ = layer.project(found)
    pos = length[:, None].expand(B, cfg.topk).contiguous()
    q, _ = layer.turn(q, None, pos)
    a2, lse = beams(q, table, length)
    again = scores + (found * layer.output(a2)).sum(-1) * cfg.d ** -0.5

    torch.cuda.synchronize()
    zg.zg_check_device_status(0)
    best = again.argmax(1)
    print(f"{B} users, {int(length.sum())} events in {cache.n_blocks} blocks of {BLOCK} ({a.fmt}); "
          f"{cfg.topk} items each, re-scoring moves the first place of {int((best != 0).sum())}")
    return {"u": u, "sids": out_sids, "scores": scores, "rescored": again, "lse": lse, "length": length,
            "table": table, "cache": cache, "layer": layer, "x": x, "items": sids, "a1": a1}


def embed_sids(sids: torch.Tensor, dm: DeviceModel, L: int) -> torch.Tensor:
    t = sids.long().clamp(min=0)
    return sum(dm.C[s][t[..., s]] for s in range(L - 1))


if __name__ == "__main__":
    main()
