"""Device-memory plumbing around the C ABI: torch tensors hold the model,
workspace and outputs; the library's kernels do all the work."""
from __future__ import annotations

import struct

import numpy as np
import torch

from . import _lib as Z


def _to_device_weights(w: np.ndarray, w_dtype: str, device) -> torch.Tensor:
    if w_dtype == "f32":
        return torch.from_numpy(np.ascontiguousarray(w, np.float32)).to(device)
    if w_dtype == "bf16":      # uint16 bfloat16 bit patterns
        bits = np.ascontiguousarray(w, np.uint16).view(np.int16)
        return torch.from_numpy(bits).to(device).view(torch.bfloat16)
    if w_dtype == "f16":
        return torch.from_numpy(np.ascontiguousarray(w, np.float16)).to(device)
    raise ValueError(w_dtype)


def _f32(x, device):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(device)


class DeviceModel:
    """Uploads a synthetic model (C_s float32, W_s in its storage dtype) and,
    optionally, a light decoder's weights (deco: the hidden vectors then come
    from the decoder and the decode's input is the concept vectors), and
    builds the zg_model struct pointing at the device copies."""

    def __init__(self, model, device="cuda", deco=None):
        self.L, self.V, self.d, self.w_dtype = model.L, model.V, model.d, model.w_dtype
        self.C = [_f32(c, device) for c in model.C]
        self.W = [_to_device_weights(w, model.w_dtype, device) for w in model.W]
        dstruct = None
        if deco is not None:
            self.deco = {"E": [_f32(e, device) for e in deco.E], "P": _f32(deco.P, device)}
            for n in ("Wq", "Wk", "Wv", "Wo", "W1", "W2"):
                self.deco[n] = [_f32(w, device) for w in getattr(deco, n)]
            t = self.deco
            dstruct = Z.make_deco(deco.M, deco.heads, deco.ffn, [e.data_ptr() for e in t["E"]],
                                  t["P"].data_ptr(), *[[w.data_ptr() for w in t[n]]
                                                       for n in ("Wq", "Wk", "Wv", "Wo", "W1", "W2")])
        self.struct = Z.make_model(self.L, self.V, self.d, Z.DTYPES[self.w_dtype],
                                   [c.data_ptr() for c in self.C], [w.data_ptr() for w in self.W], dstruct)


class Decoder:
    """Workspace and outputs for repeated zg_decode calls with fixed shapes."""

    def __init__(self, idx, plan, dmodel: DeviceModel, B: int, beam: int, K: int, device="cuda"):
        self.idx, self.plan, self.dm = idx, plan, dmodel
        self.B, self.beam, self.K = B, beam, K
        self.ws_bytes = Z.zg_decode_workspace_size(idx, plan, dmodel.struct, B, beam, K)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.out_sids = torch.empty((B, K, dmodel.L), dtype=torch.int32, device=device)
        self.out_scores = torch.empty((B, K), dtype=torch.float32, device=device)

    def __call__(self, u: torch.Tensor, stream: int | None = None):
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        Z.zg_decode(self.idx, self.plan, self.dm.struct, u, self.B, self.beam, self.K, self.out_sids,
                    self.out_scores, self.ws, self.ws_bytes, stream)
        return self.out_sids, self.out_scores

    def trace(self, u: torch.Tensor, stream: int | None = None) -> list[dict]:
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        return Z.zg_decode_trace(self.idx, self.plan, self.dm.struct, u, self.B, self.beam, self.K,
                                 self.out_sids, self.out_scores, self.ws, self.ws_bytes, stream)


_ROW_TYPES = {torch.float32: Z.ZG_F32, torch.bfloat16: Z.ZG_BF16, torch.float16: Z.ZG_F16}
_CODE_TYPES = {torch.float8_e4m3fn: Z.ZG_KV_E4M3, torch.int8: Z.ZG_KV_INT8}


# The library launches on the current device; the classes below refuse tensors of another one.

_pack_rows = struct.Struct("Piiqqq").pack      # zg_rows as bytes: a fraction of a ctypes struct's cost


def _rows(x: torch.Tensor | None, gpu: int):
    """zg_rows of a [B, T, heads, dim] tensor on device `gpu` whose last dimension is contiguous."""
    if x is None:
        return None
    dt = _ROW_TYPES.get(x.dtype)
    if dt is None:
        raise ValueError(f"rows must be float32, bfloat16 or float16, not {x.dtype}")
    sb, st, sh, se = x.stride()
    if se != 1:
        raise ValueError("the last dimension of the rows must be contiguous")
    if x.get_device() != gpu:
        raise ValueError(f"the rows must be on the GPU, on the current device (cuda:{gpu})")
    if sb < 0 or st < 0 or sh < 0:
        raise ValueError("strides of the rows must not be negative")
    return _pack_rows(x.data_ptr(), dt, 0, sb, st, sh)


def _stream(stream, gpu: int):
    """The stream given, or the current one of device `gpu` (its number alone: a Stream object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream


def _out_like(x: torch.Tensor, stream, gpu: int):
    """A new output like x for work on `stream`.  It comes from that stream's memory: a block that the current stream
    has given back may still be read by work queued there."""
    if stream is None or stream == torch._C._cuda_getCurrentRawStream(gpu):
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    on = torch.cuda.ExternalStream(stream, device=gpu) if stream else torch.cuda.default_stream(gpu)
    with torch.cuda.stream(on):
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _int32(x: torch.Tensor | None, shape, name: str, gpu: int):
    if x is not None and (x.dtype != torch.int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != gpu):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on the GPU, on the current device "
                         f"(cuda:{gpu})")


def _current(held: int, what: str) -> int:
    """The current device, on which the library launches: what a call is given, and what it `held` before (-1: nothing),
    has to be there."""
    gpu = torch._C._cuda_getDevice()     # current_device() without its check of the start-up: there are tensors already
    if held != gpu and held >= 0:
        raise ValueError(f"{what} on cuda:{held}, but the current device is cuda:{gpu}")
    return gpu


class NormRope:
    """Norm and rotation of query and key heads (zg_norm_rope).  gains: float32 [dim] device tensors or None;
    norm False leaves the norm out, rot_dim 0 the rotation; freq: radians a position of each pair instead of
    theta^(-2i / rot_dim)."""

    def __init__(self, dim: int, q_gain=None, k_gain=None, eps: float = 1e-6, rot_dim: int | None = None,
                 theta: float = 10000.0, interleaved: bool = False, norm: bool = True, freq=None):
        for g in (q_gain, k_gain):
            if g is not None and (g.dtype != torch.float32 or tuple(g.shape) != (dim,) or not g.is_contiguous() or
                                  not g.is_cuda):
                raise ValueError("gains must be contiguous float32 tensors of shape [dim] on the GPU")
        self.gpu = max([g.get_device() for g in (q_gain, k_gain) if g is not None], default=-1)
        if any(g is not None and g.get_device() != self.gpu for g in (q_gain, k_gain)):
            raise ValueError("gains must be on one device")
        self.dim, self.q_gain, self.k_gain = dim, q_gain, k_gain
        self.struct = Z.make_norm_rope(norm, eps, q_gain, k_gain, dim if rot_dim is None else rot_dim, interleaved,
                                       theta, freq)

    def __call__(self, q, k, positions, q_out=None, k_out=None, stream: int | None = None):
        """Rows q [B, T, Hq, dim] and k [B, T, Hk, dim] (either may be None) at int32 positions [B, T]; outputs
        default to new tensors and may be the inputs themselves.  New tensors belong to `stream` (the raw handle; the
        current stream when None) as if made while it was current."""
        x = q if q is not None else k
        if x is None:
            raise ValueError("neither q nor k given")
        gpu = _current(self.gpu, "the gains are")
        B, T = x.shape[:2]
        _int32(positions, (B, T), "positions", gpu)
        heads = [0, 0]
        for n, i in enumerate((q, k)):
            if i is not None:
                shape = i.shape                          # each look at a tensor's shape costs 0.1 us
                if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != self.dim:
                    raise ValueError("q and k must be [B, T, heads, dim]")
                heads[n] = shape[2]
                o = (q_out, k_out)[n]
                if o is not None and o.shape != shape:
                    raise ValueError("an output must have its input's shape")
        if q is not None and q_out is None:
            q_out = _out_like(q, stream, gpu)
        if k is not None and k_out is None:
            k_out = _out_like(k, stream, gpu)
        Z.zg_qk_norm_rope(self.struct, _rows(q, gpu), _rows(k, gpu), _rows(q_out, gpu) if q is not None else None,
                          _rows(k_out, gpu) if k is not None else None, positions, B, T, heads[0], heads[1], self.dim,
                          _stream(stream, gpu))
        return q_out, k_out


class KVCache:
    """A cache of keys and values in 8 bits (zg_kv_cache): codes [n_blocks, heads, block_tokens, dim] and a scale a
    (block, head) and side.  Block tables [B, max_blocks], lengths and counts [B] are int32 device tensors that the
    caller keeps; entries past a request's tokens are not read."""

    def __init__(self, n_blocks: int, block_tokens: int, heads: int, dim: int, fmt: str = "e4m3", device="cuda"):
        dt = torch.float8_e4m3fn if Z.KV_FORMATS[fmt] == Z.ZG_KV_E4M3 else torch.int8
        codes = [torch.empty((n_blocks, heads, block_tokens, dim), dtype=dt, device=device) for _ in range(2)]
        scales = [torch.empty((n_blocks, heads), dtype=torch.float32, device=device) for _ in range(2)]
        self._set(*codes, *scales)

    @classmethod
    def over(cls, k_codes, v_codes, k_scale, v_scale) -> "KVCache":
        """A cache in tensors that the caller holds."""
        self = cls.__new__(cls)
        self._set(k_codes, v_codes, k_scale, v_scale)
        return self

    def _set(self, k_codes, v_codes, k_scale, v_scale):
        if k_codes.dtype not in _CODE_TYPES or k_codes.dim() != 4:
            raise ValueError("codes must be float8_e4m3fn or int8 [n_blocks, heads, block_tokens, dim]")
        for x, like in ((v_codes, k_codes), (k_scale, None), (v_scale, None)):
            if like is not None and (x.dtype != like.dtype or x.shape != like.shape):
                raise ValueError("k_codes and v_codes must be alike")
            if like is None and (x.dtype != torch.float32 or x.shape != k_codes.shape[:2]):
                raise ValueError("scales must be float32 [n_blocks, heads]")
        if not all(x.is_contiguous() and x.is_cuda for x in (k_codes, v_codes, k_scale, v_scale)):
            raise ValueError("codes and scales must be contiguous and on the GPU")
        self.gpu = k_codes.get_device()
        if any(x.get_device() != self.gpu for x in (v_codes, k_scale, v_scale)):
            raise ValueError("codes and scales must be on one device")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.n_blocks, self.heads, self.block_tokens, self.dim = k_codes.shape
        self.struct = Z.make_kv_cache(_CODE_TYPES[k_codes.dtype], self.n_blocks, self.heads, self.block_tokens,
                                      self.dim, k_codes, v_codes, k_scale, v_scale)

    def append(self, k, v, table, start, n_new=None, q=None, q_out=None, norm_rope: NormRope | None = None,
               stream: int | None = None):
        """Writes k, v [B, T, heads, dim] behind the start[b] tokens that each request holds (n_new[b] of the T
        rows, all when None); norm_rope turns the keys on the way, and q [B, T, Hq, dim] into q_out, which is
        returned (a new tensor when None; it belongs to `stream`, as in NormRope)."""
        gpu = _current(self.gpu, "the cache is")
        shape = k.shape                                  # each look at a tensor's shape costs 0.1 us
        if len(shape) != 4 or v.shape != shape or shape[2] != self.heads or shape[3] != self.dim:
            raise ValueError("k and v must be [B, T, heads, dim] of the cache")
        B, T, _, _ = shape
        if table.dim() != 2:
            raise ValueError("table must be [B, max_blocks]")
        width, Hq = table.shape[1], 0
        if norm_rope is not None and norm_rope.dim != self.dim:
            raise ValueError("norm_rope and the cache differ in dim")
        if norm_rope is not None and norm_rope.gpu != gpu and norm_rope.gpu >= 0:
            _current(norm_rope.gpu, "the gains are")
        _int32(table, (B, width), "table", gpu)
        _int32(start, (B,), "start", gpu)
        _int32(n_new, (B,), "n_new", gpu)
        if q is not None:
            q_shape = q.shape
            if len(q_shape) != 4 or q_shape[0] != B or q_shape[1] != T or q_shape[3] != self.dim:
                raise ValueError("q must be [B, T, Hq, dim]")
            Hq = q_shape[2]
            if q_out is None:
                q_out = _out_like(q, stream, gpu)
            elif q_out.shape != q_shape:
                raise ValueError("q_out must have q's shape")
        Z.zg_kv_append(self.struct, norm_rope.struct if norm_rope is not None else None, _rows(k, gpu), _rows(v, gpu),
                       _rows(q, gpu), _rows(q_out, gpu) if q is not None else None, Hq, table, width, start, n_new, B, T,
                       _stream(stream, gpu))
        return q_out

    def read(self, table, start, n=None, k_out=None, v_out=None, stream: int | None = None):
        """Tokens start[b] .. start[b] + n[b] - 1 back into k_out, v_out [B, T, heads, dim] (either may be None);
        rows from n[b] on become zero."""
        x = k_out if k_out is not None else v_out
        if x is None:
            raise ValueError("neither k_out nor v_out given")
        if table.dim() != 2:
            raise ValueError("table must be [B, max_blocks]")
        gpu = _current(self.gpu, "the cache is")
        shape, width = x.shape, table.shape[1]
        if len(shape) != 4 or shape[2] != self.heads or shape[3] != self.dim or (x is k_out and v_out is not None and
                                                                                 v_out.shape != shape):
            raise ValueError("outputs must be [B, T, heads, dim] of the cache")
        B, T, _, _ = shape
        _int32(table, (B, width), "table", gpu)
        _int32(start, (B,), "start", gpu)
        _int32(n, (B,), "n", gpu)
        Z.zg_kv_read(self.struct, table, width, start, n, B, T, _rows(k_out, gpu), _rows(v_out, gpu),
                     _stream(stream, gpu))
        return k_out, v_out


class CacheAttention:
    """Workspace and outputs for repeated zg_kv_attention calls with fixed shapes: B requests of R query rows and Hq
    heads over `cache` through tables of max_blocks blocks."""

    def __init__(self, cache: KVCache, B: int, R: int, Hq: int, max_blocks: int, causal: bool = False,
                 scale: float | None = None, dtype=torch.bfloat16, lse: bool = False):
        device, gpu = cache.k_codes.device, _current(cache.gpu, "the cache is")   # the workspace's size is the device's
        self.cache, self.B, self.R, self.Hq, self.max_blocks = cache, B, R, Hq, max_blocks
        self.causal, self.scale = causal, cache.dim ** -0.5 if scale is None else scale
        self.ws_bytes = Z.zg_kv_attention_workspace_size(cache.struct, max_blocks, B, R, Hq)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.out = torch.empty((B, R, Hq, cache.dim), dtype=dtype, device=device)
        self.lse = torch.empty((B, R, Hq), dtype=torch.float32, device=device) if lse else None
        self._shape, self._out_rows = self.out.shape, _rows(self.out, gpu)

    def __call__(self, q, table, length, n_rows=None, stream: int | None = None):
        """q [B, R, Hq, dim] over the first length[b] tokens of each request; returns (out, lse or None), this
        object's own buffers."""
        if q.shape != self._shape:
            raise ValueError("q must be [B, R, Hq, dim]")
        gpu = _current(self.cache.gpu, "the cache is")
        _int32(table, (self.B, self.max_blocks), "table", gpu)
        _int32(length, (self.B,), "length", gpu)
        _int32(n_rows, (self.B,), "n_rows", gpu)
        Z.zg_kv_attention(self.cache.struct, table, self.max_blocks, length, n_rows, _rows(q, gpu), self._out_rows,
                          self.lse, self.B, self.R, self.Hq, self.scale, self.causal, self.ws, self.ws_bytes,
                          _stream(stream, gpu))
        return self.out, self.lse
