// The history cache in 4 bits: writes and reads.  16 neighbouring elements of a
// token's head share a scale,
//
//   scale  the nearest to max |x| / 6 of the halves whose bits are u << 7 (five
//          bits of exponent, three of mantissa; u is what is stored), at most 10240
//   code   x / scale to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, and its sign
//
// both to nearest even of the exact quotient.  A scale depends on its 16
// elements alone, so a write never touches rows that are there already, and
// code * scale is a half exactly (2 + 4 significant bits, 2^-18 to 61440),
// which is what the attention's products take.  The byte has an exponent bit
// more than e4m3 in place of its sign: scales are normal numbers from 2^-14 on,
// not from 2^-6, so that values need no scale of their own a head.
#include <cfloat>

#include "kv.cuh"

namespace zg {
namespace {

// a / b rounded once, from r = 1/b rounded once: the quotient's error is found
// exactly and added (Markstein).  Not for quotients near the ends of the range.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

__device__ __forceinline__ float scale_value(uint32_t u) {
  return __half2float(__ushort_as_half((unsigned short)(u << 7)));
}

// The scale byte of 16 elements whose largest is `top`.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const float y = quotient(top, 6.f, 1.f / 6.f);
  if (y < 0x1p-14f) return (uint32_t)__float2int_rn(y * 0x1p17f);  // steps of 2^-17; 8 of them are the first normal one
  uint32_t b = __float_as_uint(y);
  b += 0x7FFFFu + ((b >> 20) & 1);  // to nearest even at the third bit of the mantissa
  return min((b >> 20) - (112u << 3), 226u);  // 10240
}

// 1 / s rounded once, s the value of a scale byte: one step of Newton's from
// the approximation, which for each of those 226 numbers gives the nearest
// from any start within a unit in the last place.
__device__ __forceinline__ float scale_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.f), r, r);
}

// Largest |.| of three, NaN if one is.
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Eight elements of a lane to codes; two neighbouring lanes share a scale.
// Every lane of the warp takes part.  NaN -> 0, an infinity -> +-6 of what the
// finite elements give; `bad` is set.
__device__ __forceinline__ uint32_t codes8(float* x, uint32_t& u, bool& bad) {
  float top = abs_max3(abs_max3(x[0], x[1], x[2]), abs_max3(x[3], x[4], x[5]), abs_max3(x[6], x[7], x[7]));
  const bool odd = !(top <= FLT_MAX);  // a NaN or an infinity
  if (odd) {
    bad = true;
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) <= FLT_MAX) top = fmaxf(top, fabsf(x[i]));
      else if (isnan(x[i])) x[i] = 0.f;
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  u = scale_byte(top);
  const float s = scale_value(u), r = u ? scale_reciprocal(s) : 0.f;
  if (odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (isinf(x[i])) x[i] = copysignf(8.f * s, x[i]);
  }
  const uint64_t r2 = pair(r, r), s2 = pair(-s, -s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // quotient() of two
    const uint64_t a = pair(x[i], x[i + 1]), y = mul2(a, r2);
    unpair(fma2(fma2(y, s2, a), r2, y), q[i], q[i + 1]);
  }
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

template <typename T>
struct Append4Args {
  CacheView c;
  Rows<T> k, v, q, qo;
  const int32_t *start, *n_new;
  int32_t B, T_, Hq, chunk, nchunk;
  int32_t turn_ctas, side0, sides, nplain, wide;  // CTAs of what is turned; sides that are not, chunks of kAtOnce heads
  NormRopeArgs nr;
};

// x / d and x % d, in 32 bits where they fit (a 64-bit division is some hundred instructions).
struct Quot {
  int64_t q, r;
};
__device__ __forceinline__ Quot divide(int64_t x, int64_t d) {
  if (((x | d) >> 32) == 0) return {(uint32_t)x / (uint32_t)d, (uint32_t)x % (uint32_t)d};
  return {x / d, x % d};
}

constexpr int kAtOnce = 4;  // heads that a lane group codes at once

// Eight neighbouring elements of a lane as they lie in memory; `wide`: those of
// 16 bits are aligned to 16 bytes.
template <typename T>
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p, bool wide) {
    if (wide) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + 4);
      w = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ void get(float* x) const {
    load4(reinterpret_cast<const T*>(&w.x), x);
    load4(reinterpret_cast<const T*>(&w.z), x + 4);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// Where token t of request b goes: its block (-1: nowhere, recorded) and row.
struct Place {
  int blk, row;
};
__device__ __forceinline__ Place place_of(const CacheView& c, int b, int t, int T, int start, int n, bool live, bool report) {
  Place p = {-1, 0};
  if (start < 0 || n < 0 || n > T || (int64_t)start + n > (int64_t)c.max_blocks * c.bt) {
    if (report && live) atomicOr(c.status, kStatusCache);
  } else if (live && t < n) {
    const uint32_t at = (uint32_t)start + t;
    p.row = at % c.bt;
    p.blk = c.table[(int64_t)b * c.max_blocks + at / c.bt];
    if (p.blk < 0 || p.blk >= c.n_blocks) {
      if (report) atomicOr(c.status, kStatusCache);
      p.blk = -1;
    }
  }
  return p;
}

// What is only coded: a group of lanes a (token, side, four heads), neighbouring
// tokens side by side.  The rows are asked for before the place they go to is
// known.
template <typename T, int D>
__device__ __forceinline__ void code_plain(const Append4Args<T>& a, int64_t g, int l) {
  const int64_t tokens = (int64_t)a.B * a.T_;
  const Quot of = divide(g, tokens);
  const bool live = of.q < a.sides * a.nplain;
  const Quot bt = divide(live ? of.r : 0, a.T_);
  const int b = (int)bt.q, t = (int)bt.r, part = live ? (int)of.q : 0, Hk = a.c.heads;
  const int side = a.side0 + part / a.nplain, h0 = part % a.nplain * kAtOnce;
  const int start = a.start[b], n = a.n_new ? a.n_new[b] : a.T_;
  const bool mine = live && t < n && l < HeadLanes<D>::kUsed;
  const Rows<T>& src = side ? a.v : a.k;
  const T* from = src.at(b, t, h0) + 8 * l;
  Raw8<T> raw[kAtOnce];
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i)
    if (mine && h0 + i < Hk) raw[i].load(from + i * src.sh, a.wide);
  const Place to = place_of(a.c, b, t, a.T_, start, n, live, l == 0);
  const int64_t at = ((int64_t)max(to.blk, 0) * Hk + h0) * a.c.bt + to.row;
  uint32_t* w = reinterpret_cast<uint32_t*>((side ? a.c.vc : a.c.kc) + at * Row4<D>::kCodes) + l;
  uint8_t* s = reinterpret_cast<uint8_t*>(side ? a.c.vs : a.c.ks) + at * Row4<D>::kScales + l / 2;
  if (!__any_sync(0xFFFFFFFFu, mine && to.blk >= 0)) return;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) {
    const bool writes = mine && to.blk >= 0 && h0 + i < Hk;
    float x[8] = {};
    if (writes) raw[i].get(x);
    uint32_t u;
    const uint32_t c = codes8(x, u, bad);
    if (writes) {
      *w = c;
      if (!(l & 1)) *s = (uint8_t)u;
    }
    w += a.c.bt * (Row4<D>::kCodes / 4);
    s += a.c.bt * Row4<D>::kScales;
  }
  if (bad) atomicOr(a.c.status, kStatusNonFinite);
}

// A write of rows that are turned already, or not to be.  Bound by issue and the
// chain token -> request -> block -> row: 32 x up to 2,048 tokens of 4 heads of
// 128 (bf16, 110 MB) written and read back take 61 us, some 33 of them here (3.3
// TB/s, 75 % of issue slots busy); 70 with CUDA's division, 77 with rows asked for
// behind their place.  Of float32 both take 104 us (496 MB in all).
template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 4 : 5) k_kv_code4(const __grid_constant__ Append4Args<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  after_predecessor();
  code_plain<T, D>(a, ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS, threadIdx.x % GS);
}

// A write that turns the keys.  CTAs before turn_ctas: one group of lanes a
// (token, chunk of heads), as in the norm and rotation alone, heads 0 .. Hq - 1
// the queries, then the keys; a lane holds parts of two places of a head, so
// the turned keys go through shared memory to lanes that hold eight
// neighbours.  The others code the values.  The histories above with 16 query
// heads, normalised and rotated on the way, take 146 us with the read back (810
// MB in all, 82 % of the copy rate); 64 of up to 500 tokens (8 + 2 heads of 64) 29.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256) k_kv_append4(const __grid_constant__ Append4Args<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  __shared__ __align__(16) T ring[kAhead * 2 * 256 * 4];
  __shared__ __align__(16) float turned[256 * 8];
  after_predecessor();
  const int l = threadIdx.x % GS, Hk = a.c.heads;
  if ((int)blockIdx.x >= a.turn_ctas) {
    code_plain<T, D>(a, ((int64_t)(blockIdx.x - a.turn_ctas) * blockDim.x + threadIdx.x) / GS, l);
    return;
  }
  const Quot of = divide(((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS, a.nchunk);
  const bool live = of.q < (int64_t)a.B * a.T_;
  const Quot bt = divide(live ? of.q : 0, a.T_);
  const int b = (int)bt.q, t = (int)bt.r, part = (int)of.r;
  const int start = a.start[b], n = a.n_new ? a.n_new[b] : a.T_;
  const Place to = place_of(a.c, b, t, a.T_, start, n, live, l == 0);
  const bool writes = live && to.blk >= 0 && l < HeadLanes<D>::kUsed;
  bool bad = false;
  T* mine = ring + threadIdx.x * 4;
  const int h0 = part * a.chunk, h1 = min(h0 + a.chunk, a.Hq + Hk);
  const LaneMap m = lane_map<D, INTER>(a.nr, l);
  float sn[4], cs[4];
  lane_angles(a.nr, m, l, (int)((uint32_t)start + (uint32_t)t), sn, cs);
  if (a.Hq) {
    const Turn tq = turn_of(sn, cs, lane_gain<INTER>(a.nr.q_gain, m));
    turn_heads<T, D, INTER>(a.nr, m, tq, a.q.at(b, t, h0), a.q.sh, a.qo.at(b, t, h0), a.qo.sh,
                            live && m.used ? min(h1, a.Hq) - h0 : 0, min(a.chunk, a.Hq), mine, 256 * 4);
  }
  // the keys, kAhead of them in flight as in turn_heads
  const Turn tk = turn_of(sn, cs, lane_gain<INTER>(a.nr.k_gain, m));
  const int k0 = max(h0 - a.Hq, 0), count = writes ? h1 - a.Hq - k0 : 0;
  float* place = turned + threadIdx.x / GS * (GS * 8);
  const T* from = a.k.at(b, t, k0) + m.e0;
  const int d = m.e1 - m.e0;
  const int64_t at = ((int64_t)max(to.blk, 0) * Hk + k0) * a.c.bt + to.row;
  uint32_t* w = reinterpret_cast<uint32_t*>(a.c.kc + at * Row4<D>::kCodes) + l;
  uint8_t* s = reinterpret_cast<uint8_t*>(a.c.ks) + at * Row4<D>::kScales + l / 2;
  auto fetch = [&](int i) {
    if (i < count) {
      T* held = mine + (i % kAhead) * 2 * 256 * 4;
      copy4_async(held, from);
      copy4_async(held + 256 * 4, from + d);
    }
    from += a.k.sh;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch(i);
  for (int i = 0; i < min(a.chunk, Hk); ++i) {
    fetch(i + kAhead - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    float x[8] = {};
    if (i < count) {
      const T* held = mine + (i % kAhead) * 2 * 256 * 4;
      load4(held, x);
      load4(held + 256 * 4, x + 4);
    }
    norm_rotate<D, INTER>(a.nr, tk, x);
    if (!INTER && a.nr.rot) {
      if (m.used) {
        store4(place + m.e0, x);
        store4(place + m.e1, x + 4);
      }
      __syncwarp();
      if (m.used) {
        load4(place + 8 * l, x);
        load4(place + 8 * l + 4, x + 4);
      }
      __syncwarp();
    }
    uint32_t u;
    bool odd = false;
    const uint32_t c = codes8(x, u, odd);
    if (i < count) {
      bad |= odd;
      *w = c;
      if (!(l & 1)) *s = (uint8_t)u;
    }
    w += a.c.bt * (Row4<D>::kCodes / 4);
    s += a.c.bt * Row4<D>::kScales;
  }
  if (bad) atomicOr(a.c.status, kStatusNonFinite);
}

template <typename T>
struct Read4Args {
  CacheView c;
  Rows<T> ko, vo;
  const int32_t *start, *n;
  int32_t B, T_, sides, side0, chunk, nchunk;  // heads a group walks; such chunks a (token, side)
};

// One group of lanes a (token, side, chunk of heads), eight codes a lane and
// head, four heads in flight.  Values are exact in every type of rows.  Bound by
// memory: the same histories (163 MB) in 28 us, 5.8 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv_read4(const __grid_constant__ Read4Args<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  after_predecessor();
  const int l = threadIdx.x % GS;
  const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS;
  if (g >= (int64_t)a.B * a.T_ * a.sides * a.nchunk || l >= HeadLanes<D>::kUsed) return;
  uint32_t x = (uint32_t)g;  // below 2^31
  const int h0 = (int)(x % a.nchunk) * a.chunk, h1 = min(h0 + a.chunk, a.c.heads);
  x /= a.nchunk;
  const int side = a.side0 + (int)(x % a.sides);
  x /= a.sides;
  const int t = (int)(x % a.T_), b = (int)(x / a.T_);
  const int n = a.n ? a.n[b] : a.T_, start = a.start[b];
  int blk = -1, row = 0;
  if (t < n) {
    const int64_t p = (int64_t)start + t;
    if (start >= 0 && p < (int64_t)a.c.max_blocks * a.c.bt) {
      blk = a.c.table[(int64_t)b * a.c.max_blocks + (uint32_t)p / a.c.bt];
      row = (uint32_t)p % a.c.bt;
    }
    if (blk < 0 || blk >= a.c.n_blocks) {
      if (l == 0) atomicOr(a.c.status, kStatusCache);
      blk = -1;
    }
  }
  const Rows<T>& out = side ? a.vo : a.ko;
  T* o = out.at(b, t, h0) + 8 * l;
  const int64_t at = ((int64_t)max(blk, 0) * a.c.heads + h0) * a.c.bt + row;
  const uint8_t* codes = (side ? a.c.vc : a.c.kc) + at * Row4<D>::kCodes + 4 * l;
  const uint8_t* scales = reinterpret_cast<const uint8_t*>(side ? a.c.vs : a.c.ks) + at * Row4<D>::kScales + l / 2;
  const int64_t codes_step = (int64_t)a.c.bt * Row4<D>::kCodes, scales_step = (int64_t)a.c.bt * Row4<D>::kScales;
  for (int h = h0; h < h1; h += 4, codes += 4 * codes_step, scales += 4 * scales_step) {
    uint32_t w[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = u[i] = 0;
      if (blk >= 0 && h + i < h1) {
        w[i] = *reinterpret_cast<const uint32_t*>(codes + i * codes_step);
        u[i] = scales[i * scales_step];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + i >= h1) break;
      uint32_t y2[4];
      e2m1_half8(w[i], scale_twice(u[i]), y2);
      float y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y2[k]));
        y[2 * k] = f.x;
        y[2 * k + 1] = f.y;
      }
      store4(o, y);
      store4(o + 4, y + 4);
      o += out.sh;
    }
  }
}

}  // namespace

cudaError_t launch_append4(const CacheView& c, int dim, const NormRopeArgs* nr, const zg_rows* k, const zg_rows* v,
                           const zg_rows* q, const zg_rows* q_out, int32_t Hq, const int32_t* start, const int32_t* n_new,
                           int32_t B, int32_t T, int64_t turn_ctas, int64_t plain_ctas, int chunk, int nchunk,
                           cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  auto wide = [&](const zg_rows* r) {
    return reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && (r->stride_b | r->stride_t | r->stride_h) % 8 == 0;
  };
  for_type(k->dtype, [&](auto e) {
    using E = typename decltype(e)::type;
    const Append4Args<E> a = {c, rows_of<E>(k), rows_of<E>(v), rows_of<E>(q), rows_of<E>(q_out), start, n_new, B, T, Hq,
                              chunk, nchunk, (int32_t)turn_ctas, nr ? 1 : 0, nr ? 1 : 2,
                              (c.heads + kAtOnce - 1) / kAtOnce, wide(k) && wide(v), nr ? *nr : NormRopeArgs{}};
    for_dim(dim, [&](auto dv) {
      constexpr int D = decltype(dv)::value;
      auto kern = !nr ? k_kv_code4<E, D> : a.nr.inter ? k_kv_append4<E, D, true> : k_kv_append4<E, D, false>;
      err = launch_early(kern, turn_ctas + plain_ctas, 256, 0, st, a);
    });
  });
  return err;
}

int append4_plain(int heads, bool turned) { return (heads + kAtOnce - 1) / kAtOnce * (turned ? 1 : 2); }

cudaError_t launch_read4(const CacheView& c, int dim, const zg_rows* k_out, const zg_rows* v_out, const int32_t* start,
                         const int32_t* n, int32_t B, int32_t T, int chunk, int nchunk, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  const int sides = (k_out ? 1 : 0) + (v_out ? 1 : 0);
  const int64_t ctas = ((int64_t)B * T * sides * nchunk * group_lanes(dim) + 255) / 256;
  for_type(k_out ? k_out->dtype : v_out->dtype, [&](auto e) {
    using E = typename decltype(e)::type;
    const Read4Args<E> a = {c, rows_of<E>(k_out), rows_of<E>(v_out), start, n, B, T, sides, k_out ? 0 : 1, chunk, nchunk};
    for_dim(dim, [&](auto dv) { err = launch_early(k_kv_read4<E, decltype(dv)::value>, ctas, 256, 0, st, a); });
  });
  return err;
}

}  // namespace zg
