// What cached tokens collect of attention:
//
//   w_j = decay * w_j + sum over rows and heads of exp(scale * q . k_j - lse)
//
// with the rows' log-sum-exps from the attention itself, so one pass over the
// keys does.  A warp has 32 keys as halves in registers (the long side of the
// products) and meets all query rows, eight an instruction, which lie in
// shared memory in the order of the fragments: a key's sum stays in its lanes,
// nothing is added atomically, and what is not defined behind a history stays
// with keys that are not written.
// Measured: one token over 8 histories of up to 131,072 tokens (16 heads over 4
// of 128, 4 bits, 201 MB with the weights) 53 us, 3.8 TB/s, bound by chains of
// dependent instructions (decoding, products, softmax) in 16 warps an SM: 60 %
// of issue slots are busy, in the others no warp is ready; with keys read into
// registers one step ahead 119 us.  33 rows back over 16 histories of up to
// 8,190 tokens (16 heads over 4 of 64, e4m3) 34 us: every CTA brings all queries
// in for its few steps (38 us with a row in flight at a time), CTAs unevenly on
// the SMs.  A CTA's share of keys follows the table's width, not the lengths:
// behind tables 16 times as wide the two take 73 and 66 us.
#include <cmath>

#include "kv_attn.cuh"

namespace zg {
namespace {

constexpr int kWarps = 4, kKeys = 32 * kWarps;  // keys of a CTA's step
constexpr int kStages = 4;                      // steps of a warp in shared memory, one of them in use
constexpr int kMostSteps = 16;                  // of a CTA

struct WeightArgs {
  const uint8_t* kc;
  const float* ks;
  const uint8_t* kg;
  const int32_t *table, *length, *n_rows, *known;
  uint32_t* status;
  const float* lse;
  float* w;
  int32_t n_blocks, heads, bt, bt_log2, max_blocks, w_tokens;
  int32_t B, R, Hq, G, causal, steps, rows_at_once;
  float scale, decay;  // scale * log2(e)
};

template <int D, int FMT>
struct WeightShape {
  static constexpr bool k4 = FMT == ZG_KV_E2M1;
  static constexpr int kRow = k4 ? Row4<D>::kCodes : D;
  // a stage: two tiles of 16 keys, then (4 bits) their scale bytes or the two blocks' scales, then the 32 weights
  static constexpr int kCodes = 32 * kRow, kScales = k4 ? 32 * Row4<D>::kScales : 16, kStage = kCodes + kScales + 128;
  static constexpr int kRing = kWarps * kStages * kStage;
};

__device__ __forceinline__ void copy16_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4b_async(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A warp's keys come into its own ring of shared memory three steps ahead, and
// the weights that they have so far with them; the CTA's block numbers are
// read before, at once.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps) k_kv_weights(const __grid_constant__ WeightArgs a, const Rows<T> q) {
  using Sh = WeightShape<D, FMT>;
  constexpr bool k4 = Sh::k4;
  constexpr int KS = D / 16;  // products of 16 dims
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* frag = reinterpret_cast<uint4*>(smem + Sh::kRing);  // [row / 8][KS / 2][lane]
  const int most = a.rows_at_once;
  float4* par = reinterpret_cast<float4*>(frag + most / 8 * (KS / 2) * 32);  // [row / 2]: factors of both rows, minus their log-sum-exps
  int2* sees = reinterpret_cast<int2*>(par + most / 2);                      // [row / 2]: tokens that they see
  __shared__ int s_blk[kMostSteps * kKeys / 16];  // of every 16 keys, -1: not there
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  after_predecessor();

  const int h = blockIdx.y, b = blockIdx.z;
  Seen s = {a.length[b], a.n_rows ? a.n_rows[b] : a.R};
  const int room = a.max_blocks * a.bt;
  if (s.len < 0 || s.len > room || s.rows < 0 || s.rows > a.R) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.status, kStatusCache);
    s.len = min(max(s.len, 0), room);
    s.rows = min(max(s.rows, 0), a.R);
  }
  const int64_t begin = (int64_t)blockIdx.x * a.steps * kKeys;
  if (begin >= s.len) return;
  const int key0 = (int)begin;
  const int steps = min(a.steps, (s.len - key0 + kKeys - 1) / kKeys);
  const int M = s.rows * a.G;
  const int known = a.known ? a.known[b] : s.len;
  for (int i = threadIdx.x; i < steps * kKeys / 16; i += 32 * kWarps) {
    const int key = key0 + 16 * i;
    int blk = -1;
    if (key < s.len) {
      blk = a.table[(int64_t)b * a.max_blocks + (key >> a.bt_log2)];
      if (blk < 0 || blk >= a.n_blocks) {
        atomicOr(a.status, kStatusCache);
        blk = -1;
      }
    }
    s_blk[i] = blk;
  }

  float* w = a.w + ((int64_t)b * a.heads + h) * a.w_tokens;
  uint8_t* ring = smem + warp * (kStages * Sh::kStage);
  auto fetch = [&](int step) {
    if (step < steps) {
      uint8_t* to = ring + step % kStages * Sh::kStage;
      const int key = key0 + step * kKeys + warp * 32;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int blk = s_blk[step * (kKeys / 16) + warp * 2 + n];
        if (blk < 0) continue;
        const int64_t bh = (int64_t)blk * a.heads + h, row = bh * a.bt + ((key + 16 * n) & (a.bt - 1));
        const uint8_t* from = a.kc + row * Sh::kRow;
#pragma unroll
        for (int i = lane; i < Sh::kRow; i += 32) copy16_async(to + (n * Sh::kRow + i) * 16, from + i * 16);
        if constexpr (k4) {
          if (lane < Row4<D>::kScales)
            copy16_async(to + Sh::kCodes + (n * Row4<D>::kScales + lane) * 16,
                         a.kg + row * Row4<D>::kScales + lane * 16);
        } else {
          if (lane == 0) copy4b_async(to + Sh::kCodes + 4 * n, a.ks + bh);
        }
      }
      // of the token that this lane writes (below)
      const int mine = key + 16 * (c >> 1) + 8 * (c & 1) + g;
      if (mine < s.len && mine < known) copy4b_async(to + Sh::kCodes + Sh::kScales + 4 * lane, w + mine);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // rows m0 .. m0 + most - 1 into shared memory: a lane has four dims of a row (a head of 96: 24 lanes), which are
  // one half of a fragment
  auto stage = [&](int m0) {
    constexpr int kLanes = D / 4, kSlot = D == 96 ? 32 : kLanes, kAt = 32 / kSlot;
    const int l = lane % kSlot, d = 4 * l;
    int dw, cc;  // of the lane's dims: Tile16(x4)::dim_of(dw, cc) = d
    if constexpr (k4) {
      cc = d / (D / 4), dw = d % (D / 4) / 4;
    } else if (d < D / 64 * 64) {
      cc = d % 64 / 16, dw = d / 64 * 4 + d % 16 / 4;
    } else {
      cc = d % 64 % 32 / 8, dw = D / 64 * 4 + d % 8 / 4;
    }
    const int upto = min(most, (M - m0 + 7) / 8 * 8);
    constexpr int kMany = 8;  // rows of a lane in flight at once
    for (int r0 = warp * kAt + lane / kSlot; r0 - lane / kSlot < upto; r0 += kMany * kWarps * kAt) {
      uint4 raw[kMany];  // four elements in the first half
      float ls[kMany];
      int vis[kMany];
#pragma unroll
      for (int k = 0; k < kMany; ++k) {
        const int r = r0 + k * kWarps * kAt, m = m0 + r;
        const bool live = r < upto && m < M;
        const int row = live ? m / a.G : 0, qh = h * a.G + (live ? m - row * a.G : 0);
        raw[k] = make_uint4(0, 0, 0, 0);
        ls[k] = -INFINITY;
        if (live && l < kLanes) *reinterpret_cast<uint2*>(&raw[k]) = *reinterpret_cast<const uint2*>(q.at(b, row, qh) + d);
        if (live) ls[k] = a.lse[((int64_t)b * a.R + row) * a.Hq + qh];
        vis[k] = !live ? 0 : a.causal ? max(0, s.len - (s.rows - 1 - row)) : s.len;
      }
#pragma unroll
      for (int k = 0; k < kMany; ++k) {
        const int r = r0 + k * kWarps * kAt;
        if (r - lane / kSlot >= upto) break;  // the same for all lanes
        if (ls[k] == -INFINITY) vis[k] = 0;
        float x[4] = {};
        if (vis[k] > 0) load4(reinterpret_cast<const T*>(&raw[k]), x);  // a row that sees nothing, whatever it holds: 0
        float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
        for (int o = kSlot / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int ex = row_exponent(top);
        const float dn = power_of_2(-ex);
        if (r < upto && l < kLanes)
          reinterpret_cast<uint2*>(frag)[(((r >> 3) * (KS / 2) + (dw >> 1)) * 32 + (r & 7) * 4 + cc) * 2 + (dw & 1)] =
              make_uint2(pack_half2(x[0] * dn, x[1] * dn), pack_half2(x[2] * dn, x[3] * dn));
        if (r < upto && l == 0) {
          float* of = reinterpret_cast<float*>(par + (r >> 1)) + (r & 1);
          of[0] = a.scale * power_of_2(ex);
          of[2] = vis[k] == 0 ? -INFINITY : ls[k] * -1.4426950408889634f;
          reinterpret_cast<int*>(sees)[r] = vis[k];
        }
      }
    }
  };

  // all steps for the rows that are in shared memory, then for the next ones
  for (int m0 = 0; m0 == 0 || m0 < M; m0 += most) {
    __syncthreads();  // the block numbers are there; the last rows are not read any more
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    stage(m0);
    __syncthreads();
    const int groups = (min(M - m0, most) + 7) / 8;
    for (int step = 0; step < steps; ++step) {
      fetch(step + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* at = ring + step % kStages * Sh::kStage;
      // the keys as fragments
      uint32_t ka[2][KS][4];
      float ks[2];
      bool here[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        here[n] = s_blk[step * (kKeys / 16) + warp * 2 + n] >= 0;
        if constexpr (k4) {
          constexpr int W = Tile16x4<D>::KW;
          uint32_t k[2][W], u[2][W];
          Tile16x4<D>::keys(at + n * 16 * Sh::kRow, at + Sh::kCodes + n * 16 * Row4<D>::kScales, g, c, k, u);
          ks[n] = 1.f;
#pragma unroll
          for (int i = 0; i < W; ++i) {
            uint32_t x[4], y[4];
            e2m1_half8(k[0][i], u[0][i], x);
            e2m1_half8(k[1][i], u[1][i], y);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              ka[n][2 * i + v][0] = x[2 * v];
              ka[n][2 * i + v][1] = y[2 * v];
              ka[n][2 * i + v][2] = x[2 * v + 1];
              ka[n][2 * i + v][3] = y[2 * v + 1];
            }
          }
        } else {
          constexpr int W = Tile16<D>::KW;
          uint32_t k[2][W];
          Tile16<D>::keys(at + n * 16 * Sh::kRow, g, c, k);
          ks[n] = reinterpret_cast<const float*>(at + Sh::kCodes)[n];
#pragma unroll
          for (int i = 0; i < W; ++i) {
            codes_half4<FMT == ZG_KV_INT8>(k[0][i], ka[n][i][0], ka[n][i][2]);
            codes_half4<FMT == ZG_KV_INT8>(k[1][i], ka[n][i][1], ka[n][i][3]);
          }
        }
      }
      const float had = reinterpret_cast<const float*>(at + Sh::kCodes + Sh::kScales)[lane];
      const int first = key0 + step * kKeys + warp * 32;
      // rows that see nothing count for nothing anyhow, so only causal ones need a mask, and only of the last keys
      const bool masked = a.causal && first + 32 > s.len - (s.rows - 1);
      const uint64_t ks2[2] = {pair(ks[0], ks[0]), pair(ks[1], ks[1])};
      uint64_t sum2[2][2] = {};  // keys g and g + 8 of both tiles, even and odd rows
#pragma unroll 2
      for (int n8 = 0; n8 < groups; ++n8) {
        float z[2][4];
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 f = frag[(n8 * (KS / 2) + i) * 32 + lane];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (i == 0) mma_16816_first(z[n], ka[n][0], f.x, f.y);
            else mma_16816(z[n], ka[n][2 * i], f.x, f.y);
            mma_16816(z[n], ka[n][2 * i + 1], f.z, f.w);
          }
        }
        const ulonglong2 p = reinterpret_cast<const ulonglong2*>(par)[n8 * 4 + c];
        int2 v;
        if (masked) v = sees[n8 * 4 + c];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint64_t f = k4 ? p.x : mul2(p.x, ks2[n]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float e0, e1;
            unpair(fma2(pair(z[n][2 * i], z[n][2 * i + 1]), f, p.y), e0, e1);
            e0 = exp2_fast(e0);
            e1 = exp2_fast(e1);
            if (masked) {
              const int key = first + 16 * n + 8 * i + g;
              if (key >= v.x) e0 = 0.f;
              if (key >= v.y) e1 = 0.f;
            }
            sum2[n][i] = add2(sum2[n][i], pair(e0, e1));
          }
        }
      }
      float sum[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float odd;
          unpair(sum2[n][i], sum[n][i], odd);
          sum[n][i] += odd;
        }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum[n][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][i], 1);
          sum[n][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][i], 2);
        }
      // lane (g, c) writes key g + 8 (c & 1) of tile c / 2
      const int key = first + 16 * (c >> 1) + 8 * (c & 1) + g;
      const float mine = c == 0 ? sum[0][0] : c == 1 ? sum[0][1] : c == 2 ? sum[1][0] : sum[1][1];
      if (key < s.len) {
        const float old = m0 > 0 ? w[key] : key < known && a.decay != 0.f ? had * a.decay : 0.f;
        w[key] = old + ((c >> 1 ? here[1] : here[0]) ? mine : 0.f);
      }
      __syncwarp();  // the stage is free again
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" zg_status zg_kv_weights(const zg_kv_cache* cache, const int32_t* table, int32_t max_blocks,
                                   const int32_t* length, const int32_t* n_rows, const int32_t* known, const zg_rows* q,
                                   const float* lse, float* weights, int32_t w_tokens, float decay, int32_t B, int32_t R,
                                   int32_t Hq, float scale, int32_t causal, void* stream) try {
  const char* call = "zg_kv_weights";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if (B < 0 || R < 0) return bad_arg(call, "B and R must be >= 0");
  if (Hq < 1 || Hq > 1024 || Hq % cache->heads) return bad_arg(call, "Hq must be a multiple of cache.heads, at most 1024");
  if ((int64_t)B * R >= 0x80000000LL / Hq) return bad_arg(call, "B * R * Hq must be below 2^31");
  const int64_t tokens = (int64_t)max_blocks * cache->block_tokens;
  if (tokens > kMostTokens) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_weights: more than 2^31 - 2^20 tokens in a table");
  if (B > 65535) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_weights: more than 65,535 requests");
  if (w_tokens < tokens) return bad_arg(call, "w_tokens must be at least max_blocks * block_tokens");
  if (!(decay >= 0.f && std::isfinite(decay))) return bad_arg(call, "decay must be finite and >= 0");
  if (!(scale > 0.f && std::isfinite(scale))) return bad_arg(call, "scale must be finite and > 0");
  if (B == 0 || R == 0) return ZG_OK;
  if ((st = check_rows(q, "q", -1, call)) != ZG_OK) return st;
  if (q->dtype == ZG_F32) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_weights: q must be ZG_BF16 or ZG_F16");
  if (!length) return bad_arg(call, "length is NULL");
  if (!lse || !weights || (reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(weights)) % 4)
    return bad_arg(call, "lse and weights must be given, 4-byte aligned");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  WeightArgs a = {};
  a.kc = static_cast<const uint8_t*>(cache->k_codes);
  a.ks = cache->k_scale;
  a.kg = reinterpret_cast<const uint8_t*>(cache->k_scale);
  a.table = table;
  a.length = length;
  a.n_rows = n_rows;
  a.known = known;
  a.status = status;
  a.lse = lse;
  a.w = weights;
  a.n_blocks = cache->n_blocks;
  a.heads = cache->heads;
  a.bt = cache->block_tokens;
  while ((1 << a.bt_log2) < a.bt) ++a.bt_log2;
  a.max_blocks = max_blocks;
  a.w_tokens = w_tokens;
  a.B = B;
  a.R = R;
  a.Hq = Hq;
  a.G = Hq / cache->heads;
  a.causal = causal != 0;
  a.scale = scale * 1.4426950408889634f;
  a.decay = decay;
  const int64_t units = (tokens + kKeys - 1) / kKeys, M = (int64_t)R * a.G;
  // several steps a CTA, so that its queries and block numbers are brought in once for them, where steps are many: of
  // few rows as many as leave 16 CTAs an SM, of many, which take longer to bring in, 6 (window of 33 rows: 34.1 us with 4,
  // 33.6 with 6, 36.5 with 10; lifelong: 52.5 with 16, 55.3 with 12)
  a.steps = (int)std::max<int64_t>(1, std::min<int64_t>(kMostSteps, units * B * cache->heads / (sm_count() * (M > 16 ? 6 : 16))));
  cudaError_t err = cudaSuccess;
  for_dim(cache->dim, [&](auto dv) {
    constexpr int D = decltype(dv)::value;
    // query rows in shared memory at once: all, or as many as leave an SM two CTAs (one of 128 dims in 8 bits, whose ring
    // is the largest, from some 170 rows on)
    constexpr int kRowBytes = 2 * D + 12, kRowsAtOnce = 60 * 1024 / kRowBytes / 8 * 8;
    a.rows_at_once = (int)std::min<int64_t>((M + 7) / 8 * 8, kRowsAtOnce);
    auto typed = [&](auto ev) {
      using E = typename decltype(ev)::type;
      for_format(cache->format, [&](auto fv) {
        constexpr int FMT = decltype(fv)::value;
        auto kern = k_kv_weights<E, D, FMT>;
        const int smem = WeightShape<D, FMT>::kRing + a.rows_at_once * kRowBytes;
        // the limit is the kernel's, not the call's: the most that any call asks for, so that calls of several threads agree
        constexpr int kMostSmem = WeightShape<D, FMT>::kRing + kRowsAtOnce * kRowBytes;
        if (smem > 40 * 1024) err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (err == cudaSuccess)
          err = launch_early(kern, dim3((unsigned)((units + a.steps - 1) / a.steps), cache->heads, B), 32 * kWarps, smem,
                             static_cast<cudaStream_t>(stream), a, rows_of<E>(q));
      });
    };
    if (q->dtype == ZG_BF16) typed(Elem<__nv_bfloat16>{});
    else typed(Elem<__half>{});
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "attention weights launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}
