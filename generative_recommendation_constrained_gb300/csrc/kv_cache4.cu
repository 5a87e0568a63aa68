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

// Eight elements of a lane to codes; two neighbouring lanes share a scale.
// Every lane of the warp takes part.  NaN -> 0, an infinity -> +-6 of what the
// finite elements give; `bad` is set.
__device__ __forceinline__ uint32_t codes8(float* x, uint32_t& u, bool& bad) {
  float top = 0.f, all = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(x[i]));
    all += x[i];
  }
  const bool odd = !(fabsf(all) <= FLT_MAX);  // a NaN or an infinity (or a sum past the range)
  if (odd) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) <= FLT_MAX) {
        top = fmaxf(top, fabsf(x[i]));
      } else {
        bad = true;
        if (isnan(x[i])) x[i] = 0.f;
      }
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  u = scale_byte(top);
  const float s = scale_value(u), r = u ? __frcp_rn(s) : 0.f;
  if (odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (isinf(x[i])) x[i] = copysignf(8.f * s, x[i]);
  }
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(x[i], s, r);
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
  int32_t B, T_, Hq, chunk, nchunk, has_nr;
  NormRopeArgs nr;
};

// Where a lane group's codes and scale bytes go: its lane's word and byte of a
// row, `step` to the next head.
struct To4 {
  uint8_t *codes, *scales;
  int64_t codes_step, scales_step;
};

// `n` heads of one token to codes, kAhead of them in flight as in turn_heads.
// With TURN each is normalised and rotated first; a lane then holds parts of
// two places (m), and the elements go through `row`, the group's place in
// shared memory, to lanes that hold eight neighbours.
template <typename T, int D, bool INTER, bool TURN>
__device__ __forceinline__ void code_heads(const NormRopeArgs& a, const LaneMap& m, const Turn& t, int l, const T* from,
                                           int64_t from_step, To4 to, int n, int most, T* ring, int step, float* row,
                                           bool& bad) {
  from += m.e0;
  const int d = m.e1 - m.e0;
  auto fetch = [&](int i) {
    if (i < n) {
      T* s = ring + (i % kAhead) * 2 * step;
      copy4_async(s, from);
      copy4_async(s + step, from + d);
    }
    from += from_step;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch(i);
  for (int i = 0; i < most; ++i) {
    fetch(i + kAhead - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    float x[8] = {};
    if (i < n) {
      const T* s = ring + (i % kAhead) * 2 * step;
      load4(s, x);
      load4(s + step, x + 4);
    }
    if constexpr (TURN) {
      norm_rotate<D, INTER>(a, t, x);
      if (!INTER && a.rot) {
        if (m.used) {
          store4(row + m.e0, x);
          store4(row + m.e1, x + 4);
        }
        __syncwarp();
        if (m.used) {
          load4(row + 8 * l, x);
          load4(row + 8 * l + 4, x + 4);
        }
        __syncwarp();
      }
    }
    uint32_t u;
    bool odd = false;
    const uint32_t w = codes8(x, u, odd);
    if (i < n) {
      bad |= odd;
      *reinterpret_cast<uint32_t*>(to.codes) = w;
      if (!(l & 1)) *to.scales = (uint8_t)u;
    }
    to.codes += to.codes_step;
    to.scales += to.scales_step;
  }
}

// One group of lanes a (token, chunk of heads), as in the norm and rotation
// alone; heads 0 .. Hq - 1 are the queries, then the keys, then the values.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256) k_kv_append4(const __grid_constant__ Append4Args<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  __shared__ __align__(16) T ring[kAhead * 2 * 256 * 4];
  __shared__ __align__(16) float turned[256 * 8];
  after_predecessor();
  const int l = threadIdx.x % GS;
  const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS;
  const int64_t token = g / a.nchunk;
  const bool live = token < (int64_t)a.B * a.T_;
  const int b = live ? (int)(token / a.T_) : 0, t = live ? (int)(token % a.T_) : 0;
  const int Hk = a.c.heads, h0 = (int)(g % a.nchunk) * a.chunk, h1 = min(h0 + a.chunk, a.Hq + 2 * Hk);
  const int start = a.start[b], n = a.n_new ? a.n_new[b] : a.T_;
  T* mine = ring + threadIdx.x * 4;

  int blk = -1, row = 0;
  if (start < 0 || n < 0 || n > a.T_ || (int64_t)start + n > (int64_t)a.c.max_blocks * a.c.bt) {
    if (l == 0 && live) atomicOr(a.c.status, kStatusCache);
  } else if (live && t < n) {
    const uint32_t p = (uint32_t)start + t;
    row = p % a.c.bt;
    blk = a.c.table[(int64_t)b * a.c.max_blocks + p / a.c.bt];
    if (blk < 0 || blk >= a.c.n_blocks) {
      if (l == 0) atomicOr(a.c.status, kStatusCache);
      blk = -1;
    }
  }
  const LaneMap m = lane_map<D, INTER>(a.nr, l);
  const bool on = live && m.used, writes = on && blk >= 0;
  float sn[4], cs[4];
  lane_angles(a.nr, m, l, (int)((uint32_t)start + (uint32_t)t), sn, cs);
  if (a.Hq) {
    const Turn tq = turn_of(sn, cs, lane_gain<INTER>(a.nr.q_gain, m));
    turn_heads<T, D, INTER>(a.nr, m, tq, a.q.at(b, t, h0), a.q.sh, a.qo.at(b, t, h0), a.qo.sh,
                            on ? min(h1, a.Hq) - h0 : 0, min(a.chunk, a.Hq), mine, 256 * 4);
  }
  // the first of this chunk's keys (values), and where a row's codes go
  auto to = [&](uint8_t* codes, float* scales, int h) -> To4 {
    const int64_t at = ((int64_t)max(blk, 0) * Hk + h) * a.c.bt + row;
    return {codes + at * Row4<D>::kCodes + 4 * l, reinterpret_cast<uint8_t*>(scales) + at * Row4<D>::kScales + l / 2,
            (int64_t)a.c.bt * Row4<D>::kCodes, (int64_t)a.c.bt * Row4<D>::kScales};
  };
  bool bad = false;
  float* place = turned + threadIdx.x / GS * (GS * 8);
  const int most = min(a.chunk, Hk), k0 = max(h0 - a.Hq, 0), k1 = min(h1 - a.Hq, Hk);
  const int v0 = max(h0 - a.Hq - Hk, 0), v1 = h1 - a.Hq - Hk;
  const LaneMap plain = {8 * l, 8 * l + 4, m.used, false};
  const int nk = writes ? k1 - k0 : 0, nv = writes ? v1 - v0 : 0;
  if (a.has_nr) {
    const Turn tk = turn_of(sn, cs, lane_gain<INTER>(a.nr.k_gain, m));
    code_heads<T, D, INTER, true>(a.nr, m, tk, l, a.k.at(b, t, k0), a.k.sh, to(a.c.kc, a.c.ks, k0), nk, most, mine, 256 * 4,
                                  place, bad);
  } else {
    code_heads<T, D, INTER, false>(a.nr, plain, Turn{}, l, a.k.at(b, t, k0), a.k.sh, to(a.c.kc, a.c.ks, k0), nk, most, mine,
                                   256 * 4, place, bad);
  }
  code_heads<T, D, INTER, false>(a.nr, plain, Turn{}, l, a.v.at(b, t, v0), a.v.sh, to(a.c.vc, a.c.vs, v0), nv, most, mine,
                                 256 * 4, place, bad);
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
// head, four heads in flight.  Values are exact in every type of rows.
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
                           int32_t B, int32_t T, int chunk, int nchunk, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  const int64_t ctas = ((int64_t)B * T * nchunk * group_lanes(dim) + 255) / 256;
  for_type(k->dtype, [&](auto e) {
    using E = typename decltype(e)::type;
    const Append4Args<E> a = {c, rows_of<E>(k), rows_of<E>(v), rows_of<E>(q), rows_of<E>(q_out), start, n_new, B, T, Hq,
                              chunk, nchunk, nr != nullptr, nr ? *nr : NormRopeArgs{}};
    for_dim(dim, [&](auto dv) {
      auto kern = a.nr.inter ? k_kv_append4<E, decltype(dv)::value, true> : k_kv_append4<E, decltype(dv)::value, false>;
      err = launch_early(kern, ctas, 256, 0, st, a);
    });
  });
  return err;
}

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
