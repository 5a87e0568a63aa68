// What the attention kernels over a history cache share.
#pragma once

#include "kv.cuh"

namespace zg {

struct AttnArgs {
  const uint8_t *kc, *vc;
  const float *ks, *vs;      // 8 bits: a scale a (block, head)
  const uint8_t *kg, *vg;    // 4 bits: a scale byte for 16 elements
  const int32_t *table, *length, *n_rows;
  uint32_t* status;
  float* lse;
  float* part;      // [slot][tile][D] outputs, then [slot][tile][2] (max, sum)
  int64_t slots;    // many rows: item * splits + part; few rows: two a CTA
  int2* info;       // few rows: each item's first slot and number of parts
  int32_t n_blocks, heads, bt, bt_log2, max_blocks;
  int32_t B, R, Hq, G, splits, causal;
  int32_t tile, mt;  // query rows an item (power of two), such items a (request, key head)
  int32_t chunk;     // keys of a part, a multiple of 512, up to 2^30
  float scale;  // scale * log2(e)
};

// The requests' lengths and rows, held inside what the tables can hold.
struct Seen {
  int len, rows;
};
__device__ __forceinline__ Seen seen_of(const AttnArgs& a, int b, bool report) {
  Seen s = {a.length[b], a.n_rows ? a.n_rows[b] : a.R};
  const int most = a.max_blocks * a.bt;
  if (s.len < 0 || s.len > most || s.rows < 0 || s.rows > a.R) {
    if (report) atomicOr(a.status, kStatusCache);
    s.len = min(max(s.len, 0), most);
    s.rows = min(max(s.rows, 0), a.R);
  }
  return s;
}

// Tokens that query row r sees.
__device__ __forceinline__ int visible(const AttnArgs& a, const Seen& s, int r) {
  if (r >= s.rows) return 0;
  return a.causal ? max(0, s.len - (s.rows - 1 - r)) : s.len;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a value block's scale.  With a scale of 0 (so count those below
// 2^-126) the values are 0 and their codes are left out, but the keys count in
// the row's sum: the scale stands where the last one before it does, or else
// the first of the same step, or else at kNoScale, so that its weights neither
// vanish beside the others' nor make theirs vanish.  (Where a part begins with
// blocks of scale 0 and goes on with scales below 2^-114, those values lose
// bits: half a step is 2^-125 then.)
constexpr float kNoScale = -100.f;
__device__ __forceinline__ bool has_scale(float vs) { return vs >= 0x1p-126f; }
__device__ __forceinline__ float scale_log2(float vs, float last) { return has_scale(vs) ? log2_fast(vs) : last; }

// What a key's weight counts for in the row's sum is 1 / scale.  Scales range
// from 2^-126 to 2^121, more than a sum of many such terms has room for in 32
// bits: where a part's keys begin with a scale this small, its sums are kept
// times 2^-40.
__device__ __forceinline__ bool small_scale(float vs) { return has_scale(vs) && vs < 0x1p-64f; }
__device__ __forceinline__ float sum_weight(float lv, bool small) { return exp2_fast(-lv) * (small ? 0x1p-40f : 1.f); }

// A row's sum when its reference moves from m to n: by halves, since a sum over
// small scales outlives a factor below 2^-126.
__device__ __forceinline__ float moved_sum(float l, float m, float n) {
  const float h = m == -INFINITY ? 0.f : exp2_fast(0.5f * (m - n));
  return l * h * h;
}

// A row at its part's end in the terms in which parts are joined: the sum
// brought near 1, the reference moved by as much, so that it is that of the
// scores alone and the scales of different parts do not meet; `down` is the
// factor of the row's output.  A NaN among the row's scores leaves its sum NaN;
// an infinite reference carries that through every join.
struct PartEnd {
  float m, l, down;
};
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ PartEnd part_end(float m, float l, bool small) {
  if (isnan(l)) return {INFINITY, l, 1.f};
  if (!(l > 0.f)) return {-INFINITY, 0.f, 1.f};
  const int kept = small ? 40 : 0, e = min((int)(__float_as_uint(l) >> 23) - 127 + kept, 126);  // a subnormal sum: -127
  return {m + (float)e, l * power_of_2(kept - e), power_of_2(-e)};
}

// Tokens of a table at most, and units of work of a call: room below 2^31 for
// the steps that kernels look ahead and for a share more than there are.
constexpr int64_t kMostTokens = 0x7FF00000, kMostUnits = 0x7FF00000;

// Parts that the keys of an item are in.
__device__ __forceinline__ int parts_of(const AttnArgs& a, int keys) { return 1 + max(keys - 1, 0) / a.chunk; }

// The power of two that brings a row's largest |q| to [1, 2), as an exponent;
// from 2^127 on to [2, 4), since its reciprocal has to be a normal number.
__device__ __forceinline__ int row_exponent(float top) {
  if (!(top > 0.f) || !(top < INFINITY)) return 0;
  const int e = (int)((__float_as_uint(top) >> 23) & 0xFF) - 127;
  return min(max(e, -120), 126);
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// Bounded wait for the phase of the given parity; false on expiry.  A poll
// suspends the thread for up to a microsecond or so; under a limit of a few
// polls (the debug hook's) it does not, so that the wait does run out.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
  const uint32_t a = smem_u32(bar);
  for (uint32_t it = 0; it < limit; ++it) {
    uint32_t done;
    if (limit > 64)
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
          : "=r"(done)
          : "r"(a), "r"(parity)
          : "memory");
    else
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
          : "=r"(done)
          : "r"(a), "r"(parity)
          : "memory");
    if (done) return true;
  }
  return false;
}
// The same for a whole warp: one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, limit));
}

__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_16816_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// What one lane takes of 16 keys and values (rows of D codes in shared
// memory): of keys g and g + 8 (lane = 4 g + c) the dims of `dim_of`, of values
// 2c, 2c + 1, 2c + 8, 2c + 9 the dims g * D/8 and on.  The order of the dims
// inside a product is free, so that a lane reads neighbouring bytes.
template <int D>
struct Tile16 {
  static constexpr int KW = D / 16, VW = D / 32;  // words of a key, of a value
  static constexpr int kBytes = 16 * D;           // of the keys, of the values
  static __device__ __forceinline__ int dim_of(int w, int c) {
    return w < D / 64 * 4 ? w / 4 * 64 + 16 * c + 4 * (w % 4) : D / 64 * 64 + 8 * c + 4 * (w - D / 64 * 4);
  }
  static __device__ __forceinline__ void keys(const uint8_t* at, int g, int c, uint32_t (&k)[2][KW]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* p = at + (n * 8 + g) * D;
      if constexpr (D == 128) {
        // rows of 128 bytes: odd rows read their halves the other way round, so that eight lanes meet all banks
        const int o = (g & 1) * 64;
        const uint4 x = *reinterpret_cast<const uint4*>(p + o + 16 * c);
        const uint4 y = *reinterpret_cast<const uint4*>(p + (64 - o) + 16 * c);
        *reinterpret_cast<uint4*>(&k[n][0]) = o ? y : x;
        *reinterpret_cast<uint4*>(&k[n][4]) = o ? x : y;
      } else {
        if constexpr (D >= 64) *reinterpret_cast<uint4*>(&k[n][0]) = *reinterpret_cast<const uint4*>(p + 16 * c);
        if constexpr (D % 64 != 0)
          *reinterpret_cast<uint2*>(&k[n][D / 64 * 4]) = *reinterpret_cast<const uint2*>(p + D / 64 * 64 + 8 * c);
      }
    }
  }
  static __device__ __forceinline__ void values(const uint8_t* at, int g, int c, uint32_t (&v)[4][VW]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* p = at + (2 * c + (j & 1) + (j >> 1) * 8) * D + g * (D / 8);
      if constexpr (D == 128) *reinterpret_cast<uint4*>(v[j]) = *reinterpret_cast<const uint4*>(p);
      else if constexpr (D == 64) *reinterpret_cast<uint2*>(v[j]) = *reinterpret_cast<const uint2*>(p);
      else
#pragma unroll
        for (int w = 0; w < VW; ++w) v[j][w] = *reinterpret_cast<const uint32_t*>(p + 4 * w);
    }
  }
};

// The same of 4-bit codes: 16 rows of D/2 bytes, then their scale bytes.  A
// word is eight codes; of keys a lane takes the dims c * D/4 and on (rows side
// by side: every bank once), of values whole words (and a half one where 64 does not divide D),
// so that a word never lies in two scales.
template <int D>
struct Tile16x4 {
  static constexpr int KW = D / 32;                           // words of a key
  static constexpr int FW = D / 64, HW = D % 64 / 32;         // whole words of a value, half ones
  static constexpr int kCodes = 16 * Row4<D>::kCodes, kBytes = kCodes + 16 * Row4<D>::kScales;
  // the first of the four dims of product w of the keys
  static __device__ __forceinline__ int dim_of(int w, int c) { return c * (D / 4) + 4 * w; }
  // the first of the two dims of product j of the values
  static __device__ __forceinline__ int value_dim(int j, int g) {
    return j < 4 * FW ? g * 8 * FW + 2 * j : 64 * FW + 4 * g + 2 * (j - 4 * FW);
  }
  // Codes at `at`, scale bytes at `scales`.
  static __device__ __forceinline__ void keys(const uint8_t* at, const uint8_t* scales, int g, int c,
                                              uint32_t (&k)[2][KW], uint32_t (&s)[2][KW]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* p = at + (n * 8 + g) * Row4<D>::kCodes + c * (D / 8);
      const uint8_t* u = scales + (n * 8 + g) * Row4<D>::kScales;
      if constexpr (KW == 4) *reinterpret_cast<uint4*>(k[n]) = *reinterpret_cast<const uint4*>(p);
      else if constexpr (KW == 2) *reinterpret_cast<uint2*>(k[n]) = *reinterpret_cast<const uint2*>(p);
      else
#pragma unroll
        for (int w = 0; w < KW; ++w) k[n][w] = *reinterpret_cast<const uint32_t*>(p + 4 * w);
      if constexpr (KW == 4) {
        const uint32_t two = *reinterpret_cast<const uint16_t*>(u + 2 * c);
        s[n][0] = s[n][1] = scale_twice(two & 0xFF);
        s[n][2] = s[n][3] = scale_twice(two >> 8);
      } else {
#pragma unroll
        for (int w = 0; w < KW; ++w) s[n][w] = scale_twice(u[(c * (D / 4) + 8 * w) / 16]);
      }
    }
  }
  // Words of keys 2c, 2c + 1, 2c + 8, 2c + 9 and their scales; keys from `seen` on (not defined, may be NaN) as zeros.
  static __device__ __forceinline__ void values(const uint8_t* at, int g, int c, int seen, uint32_t (&v)[4][FW + HW],
                                                uint32_t (&s)[4][FW + HW]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 2 * c + (j & 1) + (j >> 1) * 8;
      const uint8_t* p = at + row * Row4<D>::kCodes;
      const uint8_t* u = at + kCodes + row * Row4<D>::kScales;
      if constexpr (FW == 2) {
        *reinterpret_cast<uint2*>(v[j]) = *reinterpret_cast<const uint2*>(p + 8 * g);
        s[j][0] = s[j][1] = row < seen ? u[g] : 0;
      } else {
        if constexpr (FW) {
          v[j][0] = *reinterpret_cast<const uint32_t*>(p + 4 * g);
          s[j][0] = row < seen ? u[g / 2] : 0;
        }
        if constexpr (HW) {
          v[j][FW] = *reinterpret_cast<const uint16_t*>(p + 32 * FW + 2 * g);
          s[j][FW] = row < seen ? u[4 * FW + g / 4] : 0;
        }
      }
    }
  }
};

// Many query rows: the products on the tensor cores' tcgen05 path
// (kv_attention_tc.cu).  Query rows of an item, and its launch.
int attn_tc_tile(int64_t rows);
cudaError_t launch_attn_tc(const AttnArgs& a, const zg_rows* q, const zg_rows* out, int dim, int format,
                           int64_t items, cudaStream_t st);

}  // namespace zg
