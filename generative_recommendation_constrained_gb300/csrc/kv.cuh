// Device helpers of the history cache: rows of activations in three types,
// the 8-bit codes, and the norm and rotation of one head.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "zg_internal.h"

namespace zg {

// zg_rows as a kernel argument.
template <typename T>
struct Rows {
  T* data;
  int64_t sb, st, sh;
  __device__ __forceinline__ T* at(int b, int t, int h) const { return data + b * sb + t * st + h * sh; }
};

template <typename T>
inline Rows<T> rows_of(const zg_rows* r) {
  Rows<T> o = {};
  if (r) o = {static_cast<T*>(r->data), r->stride_b, r->stride_t, r->stride_h};
  return o;
}

// Four neighbouring elements, widened to or rounded from float.
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const __half* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__half* p, const float* v) {
  const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Two e4m3 codes (low byte first) as halves; every e4m3 value is one exactly.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}

// Four codes to four halves, exactly: (code 0, code 1), (code 2, code 3).
// int8: the code with its sign bit flipped is code + 128 = the low mantissa
// bits of the half 1024 + that; subtracting 1152 leaves the code.
template <bool INT8>
__device__ __forceinline__ void codes_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (INT8) {
    w ^= 0x80808080u;
    lo = __byte_perm(w, 0x64646464u, 0x4140);
    hi = __byte_perm(w, 0x64646464u, 0x4342);
    const uint32_t off = 0x64806480u;
    *reinterpret_cast<__half2*>(&lo) =
        __hsub2(*reinterpret_cast<__half2*>(&lo), *reinterpret_cast<const __half2*>(&off));
    *reinterpret_cast<__half2*>(&hi) =
        __hsub2(*reinterpret_cast<__half2*>(&hi), *reinterpret_cast<const __half2*>(&off));
  } else {
    lo = e4m3x2_half2(w & 0xFFFFu);
    hi = e4m3x2_half2(w >> 16);
  }
}

template <bool INT8>
__device__ __forceinline__ void codes_float4(uint32_t w, float* v) {
  uint32_t lo, hi;
  codes_half4<INT8>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// Four values times `inv` to codes: to nearest even, within +-Q.
template <bool INT8>
__device__ __forceinline__ uint32_t float4_codes(const float* v, float inv) {
  if constexpr (INT8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = __float2int_rn(fminf(fmaxf(v[i] * inv, -127.f), 127.f));
      w |= ((uint32_t)q & 0xFFu) << (8 * i);
    }
    return w;
  } else {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(v[1] * inv), "f"(v[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(v[3] * inv), "f"(v[2] * inv));
    return (uint32_t)a | ((uint32_t)b << 16);
  }
}

// Lanes of a head's row: eight elements a lane, groups of a power of two
// (a head of 96 leaves four of its sixteen lanes idle).
template <int D>
struct HeadLanes {
  static constexpr int kUsed = D / 8;
  static constexpr int kGroup = D == 96 ? 16 : D / 8;
};

// zg_norm_rope as a kernel argument: pair i turns by turns[i] * 2^-64 of a
// full turn a position.  Products with the position wrap modulo 2^64, which
// takes the turns modulo 1 exactly, whatever the position.
struct NormRopeArgs {
  int32_t norm, rot, inter;
  float eps;
  const float *q_gain, *k_gain;
  uint64_t turns[64];
};

// What one lane holds of a head: elements e0..e0+3 and e1..e1+3, four pairs:
// (e0 + i, e1 + i), or INTER neighbours.  Pairs past rot_dim are not turned.
struct LaneMap {
  int e0, e1;
  bool used, rotated;
};

template <int D, bool INTER>
__device__ __forceinline__ LaneMap lane_map(const NormRopeArgs& a, int l) {
  LaneMap m;
  m.used = l < HeadLanes<D>::kUsed;
  m.rotated = m.used && 8 * l < a.rot;
  if (INTER || !m.rotated) {
    m.e0 = 8 * l;
    m.e1 = 8 * l + 4;
  } else {
    m.e0 = 4 * l;
    m.e1 = 4 * l + a.rot / 2;
  }
  return m;
}

// Pairs of floats in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Sine and cosine of turn * 2^-32 of a full turn: the nearest quarter off,
// then Taylor's series to t^9 and t^10 on [-pi/4, pi/4] (remainders below
// 2e-9).  Some 20 instructions against 40 of sincospif, in kernels that come
// near their issue limit.
__device__ __forceinline__ void turn_sincos(int32_t turn, float& sn, float& cs) {
  const int32_t quarter = (int32_t)((uint32_t)turn + 0x20000000u) >> 30;  // wraps
  const float t = (float)(int32_t)((uint32_t)turn - ((uint32_t)quarter << 30)) * (6.283185307f / 4294967296.f);
  const float u = t * t;
  float s = fmaf(u, 2.7557319e-6f, -1.9841270e-4f), c = fmaf(u, -2.7557319e-7f, 2.4801587e-5f);
  s = fmaf(u, s, 8.3333333e-3f);
  c = fmaf(u, c, -1.3888889e-3f);
  s = fmaf(u, s, -0.16666667f);
  c = fmaf(u, c, 4.1666667e-2f);
  s = fmaf(u * t, s, t);
  c = fmaf(u, c, -0.5f);
  c = fmaf(u, c, 1.f);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  sn = quarter & 2 ? -a : a;
  cs = (quarter + 1) & 2 ? -b : b;
}

// The turn of a lane's four pairs at one position, gains included: the pair
// (u, v) becomes (u uu + v uv, u vu + v vv) times the norm's factor.
struct Turn {
  float uu[4], uv[4], vu[4], vv[4];
};

// Gains of a lane's pairs (nullptr: 1).
struct LaneGain {
  float u[4], v[4];
};
template <bool INTER>
__device__ __forceinline__ LaneGain lane_gain(const float* gain, const LaneMap& m) {
  LaneGain g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g.u[i] = g.v[i] = 1.f;
    if (gain && m.used) {
      g.u[i] = gain[INTER ? m.e0 + 2 * i : m.e0 + i];
      g.v[i] = gain[INTER ? m.e0 + 2 * i + 1 : m.e1 + i];
    }
  }
  return g;
}

__device__ __forceinline__ void lane_angles(const NormRopeArgs& a, const LaneMap& m, int l, int pos, float* sn,
                                            float* cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sn[i] = 0.f;
    cs[i] = 1.f;
    if (m.rotated) turn_sincos((int32_t)(((uint64_t)(int64_t)pos * a.turns[4 * l + i]) >> 32), sn[i], cs[i]);
  }
}

__device__ __forceinline__ Turn turn_of(const float* sn, const float* cs, const LaneGain& g) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.uu[i] = g.u[i] * cs[i];
    t.uv[i] = -g.v[i] * sn[i];
    t.vu[i] = g.u[i] * sn[i];
    t.vv[i] = g.v[i] * cs[i];
  }
  return t;
}

// x[0..3] = elements e0.., x[4..7] = elements e1.. of one head, in place.
// Every lane of the warp takes part (group sums by shuffles).
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(const NormRopeArgs& a, const Turn& t, float* x) {
  float inv = 1.f;
  if (a.norm) {
    uint64_t s2 = mul2(pair(x[0], x[1]), pair(x[0], x[1]));
#pragma unroll
    for (int i = 2; i < 8; i += 2) s2 = fma2(pair(x[i], x[i + 1]), pair(x[i], x[i + 1]), s2);
    float ss, s1;
    unpair(s2, ss, s1);
    ss += s1;
#pragma unroll
    for (int o = HeadLanes<D>::kGroup / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    inv = rsqrtf(ss * (1.f / D) + a.eps);
  }
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], v = x[2 * i + 1];
      x[2 * i] = (u * t.uu[i] + v * t.uv[i]) * inv;
      x[2 * i + 1] = (u * t.vu[i] + v * t.vv[i]) * inv;
    }
  } else {
    const uint64_t i2 = pair(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t u = pair(x[i], x[i + 1]), v = pair(x[4 + i], x[5 + i]);
      const uint64_t y = fma2(u, pair(t.uu[i], t.uu[i + 1]), mul2(v, pair(t.uv[i], t.uv[i + 1])));
      const uint64_t z = fma2(u, pair(t.vu[i], t.vu[i + 1]), mul2(v, pair(t.vv[i], t.vv[i + 1])));
      unpair(mul2(y, i2), x[i], x[i + 1]);
      unpair(mul2(z, i2), x[4 + i], x[5 + i]);
    }
  }
}

// Four elements from global to shared memory, asynchronously.
template <typename T>
__device__ __forceinline__ void copy4_async(T* to, const T* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
               "n"(4 * sizeof(T))
               : "memory");
}

// Kernels of the history cache are launched so that they may start while their
// predecessor in the stream ends (some 2 us a call: 64 beams 20.7 -> 18.8, 64
// single tokens 27.1 -> 25.2): each waits here, before it touches memory, until
// everything before it is complete, and lets its successor be put in place.
__device__ __forceinline__ void after_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kern)(P...), int64_t ctas, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Run-time head size and type as template arguments: f(Dim<D>{}), f(Elem<T>{}).
template <int D>
using Dim = std::integral_constant<int, D>;
template <typename T>
struct Elem {
  using type = T;
};

template <typename F>
void for_dim(int dim, F&& f) {
  switch (dim) {
    case 32: f(Dim<32>{}); break;
    case 64: f(Dim<64>{}); break;
    case 96: f(Dim<96>{}); break;
    default: f(Dim<128>{}); break;
  }
}

// host checks shared by the entry points (kv_cache.cu)
zg_status bad_arg(const char* call, const std::string& what);
zg_status check_rows(const zg_rows* r, const char* name, int dtype, const char* call);
zg_status check_cache(const zg_kv_cache* c, const int32_t* table, int32_t max_blocks, const char* call);

}  // namespace zg
