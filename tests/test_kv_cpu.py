"""Refusals and sizes of the history-cache calls, without a GPU: every argument
check comes before any CUDA call, so the pointers here are never followed."""
import ctypes as C
import math

import pytest


@pytest.fixture(scope="module")
def zg():
    import __graft_entry__
    __graft_entry__.build()
    import generative_recommendation_constrained_gb300 as zg
    return zg


P = 1 << 20      # an aligned address that nothing follows


def cache(zg, **kw):
    a = dict(fmt=zg.ZG_KV_E4M3, n_blocks=8, heads=2, block_tokens=16, dim=64, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    a.update(kw)
    return zg.make_kv_cache(**a)


def rows(zg, data=P, dtype=None, sb=256, st=128, sh=64):
    return zg.make_rows(data, zg.ZG_BF16 if dtype is None else dtype, sb, st, sh)


def nrope(zg, **kw):
    a = dict(norm=True, eps=1e-6, q_gain=None, k_gain=None, rot_dim=64, interleaved=False, theta=1e4)
    a.update(kw)
    return zg.make_norm_rope(**a)


def refused(zg, status, words, f, *a, **kw):
    with pytest.raises(zg.ZgError) as e:
        f(*a, **kw)
    assert e.value.status == status and words in str(e.value), str(e.value)


BAD_CACHE = [(dict(fmt=2), 1, "format"), (dict(n_blocks=0), 1, "n_blocks"), (dict(heads=0), 1, "heads"),
             (dict(heads=1025), 1, "heads"), (dict(block_tokens=24), 1, "block_tokens"), (dict(dim=80), 4, "dim"),
             (dict(dim=256), 4, "dim"), (dict(k_codes=None), 1, "NULL"), (dict(v_scale=None), 1, "NULL"),
             (dict(v_codes=P + 8), 1, "16-byte"), (dict(k_scale=P + 2), 1, "4-byte")]


@pytest.mark.parametrize("kw, status, words", BAD_CACHE)
def test_bad_caches(zg, kw, status, words):
    c, r = cache(zg, **kw), rows(zg)
    refused(zg, status, words, zg.zg_kv_append, c, None, r, r, None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, status, words, zg.zg_kv_read, c, P, 4, P, None, 1, 1, r, r)
    refused(zg, status, words, zg.zg_kv_attention, c, P, 4, P, None, r, r, None, 1, 1, 2, 1.0, False, P, 1 << 30)
    refused(zg, status, words, zg.zg_kv_attention_workspace_size, c, 4, 1, 1, 2)


@pytest.mark.parametrize("kw, words", [(dict(data=None), "NULL"), (dict(dtype=3), "dtype"), (dict(sb=-4), "strides"),
                                       (dict(st=130), "strides"), (dict(sh=2), "strides"), (dict(data=P + 4), "aligned"),
                                       (dict(data=P + 8, dtype=0), "aligned")])
def test_bad_rows(zg, kw, words):
    r, good, c, n = rows(zg, **kw), rows(zg), cache(zg), nrope(zg)
    refused(zg, 1, words, zg.zg_qk_norm_rope, n, r, None, good, None, P, 1, 1, 2, 0, 64)
    refused(zg, 1, words, zg.zg_kv_append, c, None, r, good, None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, words, zg.zg_kv_read, c, P, 4, P, None, 1, 1, r, None)
    refused(zg, 1, words, zg.zg_kv_attention, c, P, 4, P, None, r, good, None, 1, 1, 2, 1.0, False, P, 1 << 30)


@pytest.mark.parametrize("kw, words", [(dict(rot_dim=-8), "rot_dim"), (dict(rot_dim=72), "rot_dim"),
                                       (dict(rot_dim=12), "rot_dim"), (dict(eps=-1.0), "eps"),
                                       (dict(eps=float("nan")), "eps"), (dict(theta=0.5), "theta"),
                                       (dict(theta=float("inf")), "theta"), (dict(q_gain=P + 2), "gains"),
                                       (dict(rot_dim=8, freq=[1.0, 0.1, -0.1, 0.0]), "freq"),
                                       (dict(rot_dim=8, freq=[1.0, 4.1, 0.1, 0.0]), "freq"),
                                       (dict(rot_dim=8, freq=[1.0, float("nan"), 0.1, 0.0]), "freq")])
def test_bad_norm_ropes(zg, kw, words):
    n, r, c = nrope(zg, **kw), rows(zg), cache(zg)
    refused(zg, 1, words, zg.zg_qk_norm_rope, n, r, r, r, r, P, 1, 1, 2, 2, 64)
    refused(zg, 1, words, zg.zg_kv_append, c, n, r, r, None, None, 0, P, 4, P, None, 1, 1)


def test_norm_rope_refusals(zg):
    n, r = nrope(zg), rows(zg)
    f = zg.zg_qk_norm_rope
    refused(zg, 1, "norm_rope", f, None, r, r, r, r, P, 1, 1, 2, 2, 64)
    refused(zg, 4, "dim", f, n, r, r, r, r, P, 1, 1, 2, 2, 48)
    refused(zg, 1, "B and T", f, n, r, r, r, r, P, -1, 1, 2, 2, 64)
    refused(zg, 1, "Hq and Hk", f, n, r, r, r, r, P, 1, 1, 2000, 2, 64)
    refused(zg, 1, "exactly when", f, n, r, None, r, None, P, 1, 1, 2, 2, 64)
    refused(zg, 1, "neither", f, n, None, None, None, None, P, 1, 1, 0, 0, 64)
    refused(zg, 1, "type of the other", f, n, r, rows(zg, dtype=zg.ZG_F16), r, r, P, 1, 1, 2, 2, 64)
    refused(zg, 1, "q_out", f, n, r, r, None, r, P, 1, 1, 2, 2, 64)
    refused(zg, 1, "positions", f, n, r, r, r, r, None, 1, 1, 2, 2, 64)
    f(n, r, r, r, r, P, 0, 5, 2, 2, 64)          # nothing to do: no launch
    f(n, r, r, r, r, P, 5, 0, 2, 2, 64)


def test_append_refusals(zg):
    c, n, r = cache(zg), nrope(zg), rows(zg)
    f = zg.zg_kv_append
    refused(zg, 1, "cache is NULL", f, None, n, r, r, None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, "table", f, c, n, r, r, None, None, 0, None, 4, P, None, 1, 1)
    refused(zg, 1, "max_blocks", f, c, n, r, r, None, None, 0, P, 0, P, None, 1, 1)
    refused(zg, 1, "max_blocks", f, c, n, r, r, None, None, 0, P, 1 << 27, P, None, 1, 1)
    refused(zg, 1, "start", f, c, n, r, r, None, None, 0, P, 4, None, None, 1, 1)
    refused(zg, 1, "B and T", f, c, n, r, r, None, None, 0, P, 4, P, None, 1, -1)
    refused(zg, 1, "v must", f, c, n, r, rows(zg, dtype=zg.ZG_F16), None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, "Hq", f, c, n, r, r, r, r, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, "Hq", f, c, n, r, r, None, None, 2, P, 4, P, None, 1, 1)
    refused(zg, 1, "without a norm_rope", f, c, None, r, r, r, r, 2, P, 4, P, None, 1, 1)
    refused(zg, 1, "q_out", f, c, n, r, r, r, None, 2, P, 4, P, None, 1, 1)
    refused(zg, 4, "CTAs", f, c, n, r, r, None, None, 0, P, 4, P, None, 1 << 30, 16)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 0, 1)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 1, 0)


def test_read_refusals(zg):
    c, r = cache(zg), rows(zg)
    refused(zg, 1, "neither", zg.zg_kv_read, c, P, 4, P, None, 1, 1, None, None)
    refused(zg, 1, "start", zg.zg_kv_read, c, P, 4, None, None, 1, 1, r, r)
    refused(zg, 1, "table", zg.zg_kv_read, c, None, 4, P, None, 1, 1, r, r)
    zg.zg_kv_read(c, P, 4, P, None, 0, 1, r, None)


def test_attention_refusals(zg):
    c, r = cache(zg), rows(zg)
    f = zg.zg_kv_attention
    ok = dict(cache=c, table=P, max_blocks=4, length=P, n_rows=None, q=r, out=r, lse=None, B=1, R=1, Hq=2, scale=1.0,
              causal=False, workspace=P, ws_bytes=1 << 30)

    def no(status, words, **kw):
        refused(zg, status, words, f, **{**ok, **kw})

    no(1, "Hq", Hq=3)
    no(1, "Hq", Hq=0)
    no(1, "Hq", Hq=1026)
    no(1, "2^31", B=1 << 20, R=1 << 11)
    no(1, "B and R", R=-1)
    no(4, "ZG_BF16 or ZG_F16", q=rows(zg, dtype=zg.ZG_F32), out=rows(zg, dtype=zg.ZG_F32))
    no(1, "out must", out=rows(zg, dtype=zg.ZG_F16))
    no(1, "length", length=None)
    no(1, "table", table=None)
    no(1, "scale", scale=0.0)
    no(1, "scale", scale=float("nan"))
    no(1, "lse", lse=P + 2)
    long = dict(max_blocks=4096)
    assert zg.zg_kv_attention_workspace_size(c, 4096, 1, 1, 2) > 0
    no(1, "workspace", workspace=None, **long)
    no(1, "workspace", workspace=P + 64, **long)
    no(1, "workspace", ws_bytes=16, **long)
    f(**{**ok, "B": 0})
    f(**{**ok, "R": 0})
    from generative_recommendation_constrained_gb300._lib import lib
    assert lib.zg_kv_attention_workspace_size(C.byref(c), 4, 1, 1, 2, None) == 1


def test_attention_leaves_room_below_2_31(zg):
    """Tables and units of work so near 2^31 that a look ahead would pass it are refused."""
    c, r = cache(zg), rows(zg)
    most = (2 ** 31 - 2 ** 20) // 16
    a = dict(n_rows=None, q=r, out=r, lse=None, R=1, Hq=2, scale=1.0, causal=False, workspace=P, ws_bytes=1 << 60)
    refused(zg, 4, "tokens in a table", zg.zg_kv_attention, c, P, most + 1, P, B=1, **a)
    refused(zg, 4, "tokens in a table", zg.zg_kv_attention_workspace_size, c, most + 1, 1, 1, 2)
    assert zg.zg_kv_attention_workspace_size(c, most, 1, 1, 2) > 0
    # 2 heads, tables of 2^20 - 1 units of 128 tokens: 1,024 requests make 2^31 - 2^11, 1,025 more than 2^31
    for B in (1024, 1025):
        refused(zg, 4, "units of work", zg.zg_kv_attention, c, P, (2 ** 20 - 1) * 8, P, B=B, **a)


def test_sizes_past_64_bits_are_refused(zg):
    """B and T whose products with heads and lanes leave 64 bits, and writes of so many pieces that a step past the
    last leaves 32: refused before any launch."""
    c, n, r, far = cache(zg, heads=1024, dim=128), nrope(zg, rot_dim=128), rows(zg), 2 ** 31 - 1
    for B, T in ((far, far), (2 ** 30, 2 ** 11), (2 ** 21, 2 ** 20)):
        refused(zg, 4, "tokens", zg.zg_qk_norm_rope, n, r, r, r, r, P, B, T, 1024, 1024, 128)
        refused(zg, 4, "tokens", zg.zg_kv_append, c, n, r, r, r, r, 1024, P, 4, P, None, B, T)
        refused(zg, 4, "tokens", zg.zg_kv_read, c, P, 4, P, None, B, T, r, r)
    one = cache(zg, heads=1)
    for B in (2 ** 30 - 1, 2 ** 30 - 2 ** 18, 2 ** 30 + 1):        # two pieces each
        refused(zg, 4, "pieces", zg.zg_kv_append, one, None, r, r, None, None, 0, P, 4, P, None, B, 1)


def test_empty_calls_need_no_rows(zg):
    """Sizes of 0 do nothing, and an empty tensor has no address."""
    c, n, e, r = cache(zg), nrope(zg), rows(zg, data=None), rows(zg)
    for B, T in ((0, 3), (3, 0)):
        zg.zg_qk_norm_rope(n, e, e, e, e, None, B, T, 2, 2, 64)
        zg.zg_kv_append(c, n, e, e, None, None, 0, P, 4, None, None, B, T)
        zg.zg_kv_read(c, P, 4, None, None, B, T, e, e)
        zg.zg_kv_attention(c, P, 4, None, None, e, e, None, B, T, 2, 1.0, False, None, 0)
    refused(zg, 1, "B and T", zg.zg_kv_read, c, P, 4, P, None, -1, 0, r, r)


def test_workspace_covers_smaller_calls(zg):
    """A workspace sized for a batch serves no less than the same batch needs: equal sizes, equal answers."""
    c = cache(zg)
    assert zg.zg_kv_attention_workspace_size(c, 64, 0, 4, 2) == 0
    a = zg.zg_kv_attention_workspace_size(c, 4096, 2, 3, 4)
    assert a == zg.zg_kv_attention_workspace_size(c, 4096, 2, 3, 4) and isinstance(a, int)


@pytest.mark.parametrize("R", [1, 9, 64, 256, 700])
@pytest.mark.parametrize("blocks", [3, 500, 65536])
def test_workspace_serves_every_smaller_batch(zg, R, blocks):
    """A workspace sized for the largest batch is enough for each smaller one: sizes never fall with the batch."""
    c = cache(zg, heads=4)
    sizes = [zg.zg_kv_attention_workspace_size(c, blocks, B, R, 4) for B in range(0, 200)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert zg.zg_kv_attention_workspace_size(c, blocks, 5000, R, 4) >= sizes[-1]


def test_binding_structs_match_the_header(zg):
    """Sizes of the argument structs as the C compiler lays them out."""
    from generative_recommendation_constrained_gb300 import _lib
    assert C.sizeof(_lib.zg_rows) == 40 and C.sizeof(_lib.zg_kv_cache) == 56 and C.sizeof(_lib.zg_norm_rope) == 48


class Rows:
    """A stand-in for a tensor on the GPU: what the wrappers ask of one."""
    is_cuda = True

    def __init__(self, shape, dtype=None, index=0):
        import torch
        self.shape = torch.Size(shape if isinstance(shape, tuple) else (shape,))
        self.dtype, self.device = dtype or torch.bfloat16, torch.device("cuda", index)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return P

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index


@pytest.fixture
def fake_cuda(zg, monkeypatch):
    """The wrappers with a current device and stream (handle 7) of no GPU; calls into the library are recorded."""
    import contextlib

    import torch
    from generative_recommendation_constrained_gb300 import device
    seen = {"stream": 7, "made": [], "calls": [], "device": 0}

    @contextlib.contextmanager
    def current(s):
        before, seen["stream"] = seen["stream"], s
        yield
        seen["stream"] = before

    def empty(shape, dtype=None, device=None):
        seen["made"].append(seen["stream"])
        return Rows(shape, dtype, torch.device(device).index or 0)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: seen["device"])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: seen["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: seen["stream"], raising=False)
    for name in ("zg_qk_norm_rope", "zg_kv_append", "zg_kv_read", "zg_kv_attention"):
        monkeypatch.setattr(device.Z, name, lambda *a, name=name: seen["calls"].append((name, a[-1])))
    monkeypatch.setattr(device.Z, "zg_kv_attention_workspace_size", lambda *a: 256)
    return device, seen


@pytest.mark.parametrize("stream, of", [(None, 7), (7, 7), (42, 42), (0, 0)])
def test_outputs_belong_to_the_stream_that_writes_them(fake_cuda, stream, of):
    """A new output comes from the memory of the stream that the kernel runs on, not from the current one's."""
    import torch
    dev, seen = fake_cuda
    x, pos = Rows((2, 3, 4, 64)), Rows((2, 3), torch.int32)
    nr = dev.NormRope(64)
    nr(x, x, pos, stream=stream)
    assert seen["made"] == [of, of] and seen["calls"] == [("zg_qk_norm_rope", of)]
    codes, scales = Rows((8, 4, 16, 64), torch.int8), Rows((8, 4), torch.float32)
    dev.KVCache.over(codes, codes, scales, scales).append(x, x, Rows((2, 5), torch.int32), Rows((2,), torch.int32), q=x,
                                                          norm_rope=nr, stream=stream)
    assert seen["made"] == [of] * 3 and seen["calls"][1:] == [("zg_kv_append", of)]


def test_tensors_of_another_device_are_refused(fake_cuda):
    """The library launches on the current device, so every tensor of a call has to be there; nothing is called
    otherwise."""
    import torch
    dev, seen = fake_cuda
    i32, f32, i8 = torch.int32, torch.float32, torch.int8

    def cache(index, odd=None):
        return dev.KVCache.over(*(Rows(s, t, odd if j == 3 and odd is not None else index)
                                  for j, (s, t) in enumerate((((8, 4, 16, 64), i8), ((8, 4, 16, 64), i8), ((8, 4), f32), ((8, 4), f32)))))

    x, y = Rows((2, 3, 4, 64)), Rows((2, 3, 4, 64), index=1)
    table, start = Rows((2, 5), i32), Rows((2,), i32)
    pos, gain = Rows((2, 3), i32), Rows((64,), f32, 1)
    c, nr = cache(0), dev.NormRope(64)
    attn = dev.CacheAttention(c, 2, 3, 4, 5)
    for f in (lambda: nr(y, None, pos), lambda: nr(x, y, pos), lambda: nr(x, None, Rows((2, 3), i32, 1)), lambda: nr(x, None, pos, y),
              lambda: dev.NormRope(64, gain)(x, None, pos), lambda: dev.NormRope(64, gain, Rows((64,), f32)),
              lambda: c.append(y, y, table, start), lambda: c.append(x, y, table, start),
              lambda: c.append(x, x, Rows((2, 5), i32, 1), start), lambda: c.append(x, x, table, Rows((2,), i32, 1)),
              lambda: c.append(x, x, table, start, Rows((2,), i32, 1)), lambda: c.append(x, x, table, start, q=y, norm_rope=nr),
              lambda: c.append(x, x, table, start, q=x, norm_rope=dev.NormRope(64, gain)), lambda: cache(1).append(x, x, table, start),
              lambda: cache(0, 1), lambda: c.read(table, start, None, y), lambda: c.read(Rows((2, 5), i32, 1), start, None, x),
              lambda: cache(1).read(table, start, None, x), lambda: attn(y, table, start), lambda: attn(x, Rows((2, 5), i32, 1), start),
              lambda: attn(x, table, start, Rows((2,), i32, 1)), lambda: dev.CacheAttention(cache(1), 2, 3, 4, 5)):
        with pytest.raises(ValueError, match="device"):
            f()
    seen["device"] = 1
    for f in (lambda: c.append(x, x, table, start), lambda: c.read(table, start, None, x), lambda: attn(x, table, start),
              lambda: nr(x, None, pos)):
        with pytest.raises(ValueError, match="device"):
            f()
    assert seen["calls"] == []
    seen["device"] = 0
    nr(x, x, pos)
    c.append(x, x, table, start)
    c.read(table, start, None, x)
    attn(x, table, start)
    assert [name for name, _ in seen["calls"]] == ["zg_qk_norm_rope", "zg_kv_append", "zg_kv_read", "zg_kv_attention"]


def test_wrappers_want_something_to_do(fake_cuda):
    import torch
    dev, seen = fake_cuda
    codes, scales = Rows((8, 4, 16, 64), torch.int8), Rows((8, 4), torch.float32)
    c = dev.KVCache.over(codes, codes, scales, scales)
    start = Rows((2,), torch.int32)
    for f, words in ((lambda: dev.NormRope(64)(None, None, None), "neither"),
                     (lambda: c.read(Rows((2, 5), torch.int32), start), "neither"),
                     (lambda: c.read(Rows((10,), torch.int32), start, None, Rows((2, 3, 4, 64))), "max_blocks")):
        with pytest.raises(ValueError, match=words):
            f()
    assert seen["calls"] == []
