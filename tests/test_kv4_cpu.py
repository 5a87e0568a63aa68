"""Refusals of the 4-bit history cache, without a GPU: every argument check comes before any CUDA call, so the pointers
here are never followed."""
import pytest
from test_kv_cpu import Rows, fake_cuda  # noqa: F401 (a fixture)

P = 1 << 20      # an aligned address that nothing follows


@pytest.fixture(scope="module")
def zg():
    import __graft_entry__
    __graft_entry__.build()
    import generative_recommendation_constrained_gb300 as zg
    return zg


def cache(zg, **kw):
    a = dict(fmt=zg.ZG_KV_E2M1, n_blocks=8, heads=2, block_tokens=16, dim=64, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    a.update(kw)
    return zg.make_kv_cache(**a)


def refused(zg, status, words, f, *a, **kw):
    with pytest.raises(zg.ZgError) as e:
        f(*a, **kw)
    assert e.value.status == status and words in str(e.value), str(e.value)


@pytest.mark.parametrize("kw, status, words", [(dict(fmt=3), 1, "format"), (dict(dim=80), 4, "dim"), (dict(k_scale=P + 4), 1, "16-byte"),
                                               (dict(v_scale=P + 8), 1, "16-byte"), (dict(v_codes=P + 8), 1, "16-byte"),
                                               (dict(k_scale=None), 1, "NULL"), (dict(block_tokens=8), 1, "block_tokens")])
def test_bad_caches(zg, kw, status, words):
    c, r = cache(zg, **kw), zg.make_rows(P, zg.ZG_BF16, 256, 128, 64)
    refused(zg, status, words, zg.zg_kv_append, c, None, r, r, None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, status, words, zg.zg_kv_read, c, P, 4, P, None, 1, 1, r, r)
    refused(zg, status, words, zg.zg_kv_attention, c, P, 4, P, None, r, r, None, 1, 1, 2, 1.0, False, P, 1 << 30)
    refused(zg, status, words, zg.zg_kv_attention_workspace_size, c, 4, 1, 1, 2)


def test_append_refusals(zg):
    c, r, n = cache(zg), zg.make_rows(P, zg.ZG_BF16, 256, 128, 64), zg.make_norm_rope(True, 1e-6, None, None, 64, False, 1e4)
    f = zg.zg_kv_append
    refused(zg, 1, "start", f, c, n, r, r, None, None, 0, P, 4, None, None, 1, 1)
    refused(zg, 1, "v must", f, c, n, r, zg.make_rows(P, zg.ZG_F16, 256, 128, 64), None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, "without a norm_rope", f, c, None, r, r, r, r, 2, P, 4, P, None, 1, 1)
    refused(zg, 4, "tokens", f, c, n, r, r, None, None, 0, P, 4, P, None, 2 ** 31 - 1, 2 ** 31 - 1)
    refused(zg, 4, "CTAs", f, c, n, r, r, None, None, 0, P, 4, P, None, 2 ** 20, 2 ** 18)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 0, 1)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 1, 0)


def test_weights_refusals(zg):
    c, r = cache(zg), zg.make_rows(P, zg.ZG_BF16, 256, 128, 64)
    ok = dict(cache=c, table=P, max_blocks=4, length=P, n_rows=None, known=None, q=r, lse=P, weights=P, w_tokens=64,
              decay=1.0, B=1, R=1, Hq=2, scale=1.0, causal=False)

    def no(status, words, **kw):
        refused(zg, status, words, zg.zg_kv_weights, **{**ok, **kw})

    no(1, "Hq", Hq=3)
    no(1, "B and R", B=-1)
    no(1, "2^31", B=1 << 15, R=1 << 16)
    no(4, "65,535", B=65536)
    no(1, "w_tokens", w_tokens=63)
    no(1, "decay", decay=-1.0)
    no(1, "decay", decay=float("nan"))
    no(1, "scale", scale=float("inf"))
    no(1, "lse", lse=None)
    no(1, "lse", weights=P + 2)
    no(1, "length", length=None)
    no(4, "ZG_BF16 or ZG_F16", q=zg.make_rows(P, zg.ZG_F32, 256, 128, 64))
    no(4, "tokens in a table", max_blocks=2 ** 27 - 1, w_tokens=2 ** 31 - 1)
    zg.zg_kv_weights(**{**ok, "B": 0, "lse": None})
    zg.zg_kv_weights(**{**ok, "R": 0, "lse": None})


def test_evict_refusals(zg):
    c = cache(zg)
    ok = dict(cache=c, table=P, max_blocks=4, length=P, weights=P, w_tokens=64, keep=8, recent=2, new_length=2 * P, kept=P, B=1)

    def no(status, words, **kw):
        refused(zg, status, words, zg.zg_kv_evict, **{**ok, **kw})

    no(1, "keep", keep=0)
    no(4, "keep", keep=2 ** 30 + 1)
    no(1, "recent", recent=9)
    no(1, "recent", recent=-1)
    no(1, "B must", B=-1)
    no(4, "65,535", B=32768)
    no(1, "w_tokens", w_tokens=63)
    no(1, "NULL", weights=None)
    no(1, "NULL", kept=None)
    no(1, "4-byte", kept=P + 2)
    no(1, "new_length", new_length=P)
    no(1, "table", table=None)
    no(4, "tokens in a table", max_blocks=2 ** 27 - 1, w_tokens=2 ** 31 - 1)
    zg.zg_kv_evict(**{**ok, "B": 0, "length": None})


@pytest.fixture
def recorded(fake_cuda, monkeypatch):  # noqa: F811
    """The new calls recorded too."""
    dev, seen = fake_cuda
    for name in ("zg_prompt_attention", "zg_kv_weights", "zg_kv_evict"):
        monkeypatch.setattr(dev.Z, name, lambda *a, name=name: seen["calls"].append((name, a[-1])))
    return dev, seen


def some(dev, index=0):
    """A 4-bit cache, its weights and what the calls take, on device `index`."""
    import torch
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    codes, scales = Rows((8, 4, 16, 32), u8, index), Rows((8, 4, 16, 4), u8, index)
    return dict(c=dev.KVCache.over(codes, codes, scales, scales), w=Rows((2, 4, 80), f32, index), q=Rows((2, 3, 8, 64), index=index),
                lse=Rows((2, 3, 8), f32, index), table=Rows((2, 5), i32, index), length=Rows((2,), i32, index),
                pq=Rows((9, 8, 64), index=index), pk=Rows((9, 4, 64), index=index), starts=Rows((3,), i32, index))


@pytest.mark.parametrize("stream, of", [(None, 7), (7, 7), (42, 42), (0, 0)])
def test_streams_and_outputs(recorded, stream, of):
    """Calls go to the stream given or the current one; a new output comes from that stream's memory."""
    dev, seen = recorded
    s = some(dev)
    assert (s["c"].dim, s["c"].block_tokens, s["c"].heads) == (64, 16, 4)
    s["c"].add_weights(s["w"], s["q"], s["lse"], s["table"], s["length"], stream=stream)
    dev.CacheEviction(s["c"], 2, 5, 30, 3)(s["w"], s["table"], s["length"], stream=stream)
    seen["made"].clear()
    out, lse = dev.PromptAttention(8, 4, 64, lse=True)(s["pq"], s["pk"], s["pk"], s["starts"], stream=stream)
    assert seen["made"] == [of, of] and tuple(out.shape) == (9, 8, 64) and tuple(lse.shape) == (9, 8)
    assert seen["calls"] == [("zg_kv_weights", of), ("zg_kv_evict", of), ("zg_prompt_attention", of)]


def test_tensors_of_another_device_are_refused(recorded):
    dev, seen = recorded
    s, o = some(dev), some(dev, 1)
    prompt, evict = dev.PromptAttention(8, 4, 64), dev.CacheEviction(s["c"], 2, 5, 30, 3)
    for f in (lambda: s["c"].add_weights(o["w"], s["q"], s["lse"], s["table"], s["length"]),
              lambda: s["c"].add_weights(s["w"], o["q"], s["lse"], s["table"], s["length"]),
              lambda: s["c"].add_weights(s["w"], s["q"], o["lse"], s["table"], s["length"]),
              lambda: s["c"].add_weights(s["w"], s["q"], s["lse"], o["table"], s["length"]),
              lambda: s["c"].add_weights(s["w"], s["q"], s["lse"], s["table"], o["length"]),
              lambda: s["c"].add_weights(s["w"], s["q"], s["lse"], s["table"], s["length"], n_rows=o["length"]),
              lambda: s["c"].add_weights(s["w"], s["q"], s["lse"], s["table"], s["length"], known=o["length"]),
              lambda: o["c"].add_weights(o["w"], o["q"], o["lse"], o["table"], o["length"]),
              lambda: evict(o["w"], s["table"], s["length"]), lambda: evict(s["w"], o["table"], s["length"]),
              lambda: evict(s["w"], s["table"], o["length"]), lambda: dev.CacheEviction(o["c"], 2, 5, 30),
              lambda: prompt(o["pq"], s["pk"], s["pk"], s["starts"]), lambda: prompt(s["pq"], o["pk"], s["pk"], s["starts"]),
              lambda: prompt(s["pq"], s["pk"], o["pk"], s["starts"]), lambda: prompt(s["pq"], s["pk"], s["pk"], o["starts"]),
              lambda: prompt(s["pq"], s["pk"], s["pk"], s["starts"], out=o["pq"])):
        with pytest.raises(ValueError, match="device"):
            f()
    assert seen["calls"] == []


def test_shapes_and_types_are_refused(recorded):
    import torch
    dev, seen = recorded
    s = some(dev)
    prompt, evict = dev.PromptAttention(8, 4, 64), dev.CacheEviction(s["c"], 2, 5, 30, 3)
    add = lambda **kw: s["c"].add_weights(**{**dict(weights=s["w"], q=s["q"], lse=s["lse"], table=s["table"], length=s["length"]), **kw})  # noqa: E731
    for f in (lambda: add(weights=Rows((2, 4, 79), torch.float32)), lambda: add(weights=Rows((2, 3, 80), torch.float32)),
              lambda: add(weights=Rows((2, 4, 80))), lambda: add(q=Rows((2, 3, 6, 64))), lambda: add(q=Rows((2, 3, 8, 32))),
              lambda: add(lse=Rows((2, 8, 3), torch.float32)), lambda: add(table=Rows((3, 5), torch.int32)),
              lambda: add(length=Rows((2,), torch.int64)), lambda: add(known=Rows((3,), torch.int32)),
              lambda: evict(Rows((2, 4, 64), torch.float32), s["table"], s["length"]), lambda: evict(s["w"], Rows((2, 6), torch.int32), s["length"]),
              lambda: dev.CacheEviction(s["c"], 2, 5, 30, 31), lambda: dev.CacheEviction(s["c"], 2, 5, 0),
              lambda: prompt(Rows((9, 6, 64)), s["pk"], s["pk"], s["starts"]), lambda: prompt(s["pq"], s["pk"], Rows((8, 4, 64)), s["starts"]),
              lambda: prompt(s["pq"], Rows((8, 4, 64)), Rows((8, 4, 64)), s["starts"]), lambda: prompt(s["pq"], s["pk"], s["pk"], Rows((3,), torch.int64)),
              lambda: prompt(s["pq"], s["pk"], s["pk"], Rows((3, 1), torch.int32)), lambda: prompt(s["pq"], s["pk"], s["pk"], s["starts"], out=Rows((9, 8, 32))),
              lambda: prompt(s["pq"], s["pk"], s["pk"], s["starts"], lse=Rows((9, 4), torch.float32)),
              lambda: dev.KVCache.over(Rows((8, 4, 16, 32), torch.uint8), Rows((8, 4, 16, 32), torch.uint8), Rows((8, 4), torch.float32), Rows((8, 4), torch.float32))):
        with pytest.raises(ValueError):
            f()
    assert seen["calls"] == []
