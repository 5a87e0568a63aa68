"""The operators of long histories together, as the example uses them: prompt attention, a cache in 4 or 8 bits, weights,
eviction, cached attention and the decode."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("history_decode", os.path.join(ROOT, "examples", "history_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("keep", [0, 30, 5])
def test_example(example, fmt, keep):
    r = example.main(["--users", "9", "--events", "70", "--fmt", fmt, "--keep", str(keep)])
    items = {tuple(s) for s in r["items"].tolist()}
    assert all(tuple(s) in items for s in r["sids"].reshape(-1, r["sids"].shape[-1]).tolist())
    assert torch.isfinite(r["rescored"]).all() and torch.isfinite(r["lse"]).all()
    held = r["held"]
    assert torch.equal(r["length"], (held.clamp(max=keep) if keep else held) + 1)
    # the states of the histories against attention in 64 bits
    q, k, v = (x.double() for x in r["packed"])
    G = example.HEADS // example.KV_HEADS
    edge = r["starts"].tolist()
    for a, b in zip(edge[:-1], edge[1:]):
        if a == b:
            continue
        z = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(G, 1)) * example.DIM ** -0.5
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1), -float("inf"))
        p, vv = torch.softmax(z, -1), v[a:b].repeat_interleave(G, 1)
        want, mass = torch.einsum("hij,jhd->ihd", p, vv), torch.einsum("hij,jhd->ihd", p, vv.abs())
        # probabilities rounded to bf16, 32-bit scores (norm 1 keys and queries: below 64 in size), one rounding
        tol = mass * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -8 * 1.001 * want.abs()
        assert ((r["states"][a:b].double() - want).abs() <= tol + 1e-6).all()
    # the new event's query over what the cache holds
    cache, table, length, layer = r["cache"], r["table"], r["length"], r["layer"]
    n = int(length.max())
    kf, vf = (torch.zeros((9, n, example.KV_HEADS, example.DIM), device="cuda") for _ in range(2))
    cache.read(table, torch.zeros_like(length), length, kf, vf)
    q, _, _ = layer.project(r["x"])
    q, _ = layer.turn(q, None, held[:, None].contiguous())
    z = torch.einsum("bhd,bjhd->bhj", q[:, 0].double(), kf.double().repeat_interleave(G, 2)) * example.DIM ** -0.5
    z = z.masked_fill(torch.arange(n, device="cuda")[None, None] >= length[:, None, None], -float("inf"))
    p, vv = torch.softmax(z, -1), vf.double().repeat_interleave(G, 2)
    want, mass = torch.einsum("bhj,bjhd->bhd", p, vv), torch.einsum("bhj,bjhd->bhd", p, vv.abs())
    # probabilities as halves, values read back within a rounding to 32 bits, one rounding to bf16
    tol = mass * (2.0 ** -11 + 2.0 ** -14) + 2.0 ** -8 * 1.001 * want.abs()
    assert ((r["a1"][:, 0].double() - want).abs() <= tol + 1e-6).all()
    if keep:
        # every event's weights: each of the window's rows gives 1 a query head
        rows = held.clamp(max=example.WINDOW)
        assert r["weights"].shape[:2] == (9, example.KV_HEADS) and torch.isfinite(r["weights"]).all()
        short = held <= keep
        total = r["weights"].sum(-1)[short]
        assert ((total - (G * rows)[short][:, None]).abs() < 1e-3).all()
