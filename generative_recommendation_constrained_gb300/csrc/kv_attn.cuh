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

// Many query rows: the products on the tensor cores' tcgen05 path
// (kv_attention_tc.cu).  Query rows of an item, and its launch.
int attn_tc_tile(int64_t rows);
cudaError_t launch_attn_tc(const AttnArgs& a, const zg_rows* q, const zg_rows* out, int dim, int format,
                           int64_t items, cudaStream_t st);

}  // namespace zg
