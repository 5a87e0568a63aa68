// Attention over a history cache held in 8 bits.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q . k_j)
//
// in one pass over the cache.  Codes enter the products exactly as halves.  A
// key block's scale multiplies its scores; a value block's scale s enters the
// exponent: with z the score in log2 units,
//
//   w_j = exp2(z_j + log2 s_j - m),  out = sum_j w_j code_j / sum_j w_j / s_j
//
// so one running reference m a row, the largest z + log2 s, keeps the weights
// inside a half whatever the scales are, and a scale costs nothing an
// element.  The reference moves only when a tile exceeds it by 2^8, so that
// accumulators are rescaled rarely; a weight stays below 2^8.
#include <cmath>
#include <string>

#include "kv_attn.cuh"

namespace zg {
namespace {

__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of halves held one row a group of four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr int kFewThreads = 128;

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

// Dynamic shared memory of k_attn_few: each warp's ring of two steps (two
// tiles of keys, two of values each), then (in its place) the warps' sums.
template <int D, int NT>
constexpr int few_smem() {
  const int ring = 4 * 2 * 4 * Tile16<D>::kBytes, sums = 4 * 8 * NT * (D + 2) * 4;
  return ring > sums ? ring : sums;
}

// Keys go to the CTAs of k_attn_few by the unit of 128 (a step a warp), all
// items (request, key head, 8 NT rows) in a row and the same share for each
// CTA, however the histories' lengths differ: an item may lie in several CTAs
// (the join adds their parts up), and a CTA may hold the end of one item,
// whole ones and the beginning of another.
constexpr int kUnit = 128;
__device__ __forceinline__ int item_keys(const AttnArgs& a, const Seen& s, int m, int nr) {
  // later rows see no less: the item sees what its last row does, or its request's last
  const int last = min(min(m * nr + nr, a.R * a.G) - 1, s.rows * a.G - 1);
  return last < m * nr ? 0 : visible(a, s, last / a.G);
}
// A row of items that see nothing takes one unit too: somebody has to write its outputs.
__device__ __forceinline__ int item_units(const AttnArgs& a, const Seen& s, int m, int nr) {
  return max(1, (item_keys(a, s, m, nr) + kUnit - 1) / kUnit);
}
__device__ __forceinline__ int request_units(const AttnArgs& a, const Seen& s, int nr) {
  int n = 0;
  for (int m = 0; m < a.mt; ++m) n += item_units(a, s, m, nr);
  return n * a.heads;
}

// Few query rows: a row is (token, query head of the group).  Each warp walks
// its own keys, two tiles of 16 a step (a tile a step left the warps waiting
// for their own shuffles and products), brought by bulk copies one step ahead
// (16-byte copies a lane, in the order of the fragments, stopped at 4.9 TB/s
// without any work behind them).  Keys and dims are the long side of the
// products (S^T = K Q^T, O^T = V^T P^T), so that eight rows fill an instruction
// that sixteen keys or dims by eight rows make.  Bound by memory: 8 requests of
// up to 131,072 tokens (4 heads of 128, int8, 645 MB) take 107 us, some 103 of
// them here (6.3 TB/s) and the rest the join; 64 requests of up to 4,096 tokens
// (85 MB) 26 us, some 6 of them the chain from the lengths to the first codes.
constexpr uint32_t kFewSpin = 1u << 20;  // polls of a wait at most

template <typename T, int D, bool INT8, int NT>
__global__ void __launch_bounds__(kFewThreads, NT == 1 ? 3 : 2) k_attn_few(const __grid_constant__ AttnArgs a,
                                                                                const Rows<T> q, const Rows<T> out,
                                                                                uint32_t spin) {
  using Tl = Tile16<D>;
  constexpr int KW = Tl::KW, VW = Tl::VW, NR = 8 * NT;
  __shared__ float sm_m[4][NR], sm_l[4][NR];
  extern __shared__ __align__(128) uint8_t ring[];  // [warp][step][side][tile]; then float [4][NR][D + 2]
  __shared__ uint64_t full[4][2];  // [warp][step]: its copies have landed
  auto sm_o = reinterpret_cast<float (*)[NR][D + 2]>(ring);
  __shared__ int sm_sum[4], sm_b, sm_first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int M = a.R * a.G;

  if (threadIdx.x < 8) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&full[0][0] + threadIdx.x)));
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  uint32_t issued = 0, taken = 0;  // steps of this warp, over all its items
  bool good = true;
  after_predecessor();

  // every request's units, their sum, and the request in which this CTA's share begins (a thread a request; over
  // again for the second only where there are more requests than threads)
  int total = 0, n = 0, before = 0;  // of the thread's request
  auto scan = [&](int b0, bool report) -> int {
    const int b = b0 + threadIdx.x;
    n = b < a.B ? request_units(a, seen_of(a, b, report), NR) : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm_sum[warp] = x;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) x += sm_sum[w];
      all += sm_sum[w];
    }
    before = x - n;
    return all;
  };
  for (int b0 = 0; b0 < a.B; b0 += kFewThreads) {
    if (b0) __syncthreads();
    total += scan(b0, blockIdx.x == 0);
  }
  const int share = (total + gridDim.x - 1) / gridDim.x;
  int u = blockIdx.x * share;
  const int u_end = min(total, u + share);
  if (u >= u_end) return;
  int sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += kFewThreads) {
    int all = total;
    if (a.B > kFewThreads) {
      __syncthreads();
      all = scan(b0, false);
    }
    if (sum + before <= u && u < sum + before + n) {
      sm_b = b0 + threadIdx.x;
      sm_first = sum + before;
    }
    sum += all;
  }
  __syncthreads();
  int b = sm_b, first = sm_first;  // `first`: units before request b, then before the item
  Seen s = seen_of(a, b, false);
  // the item: (head, rows)
  const int per_head = request_units(a, s, NR) / a.heads;
  int h = (u - first) / per_head, m = 0, units = item_units(a, s, 0, NR);
  first += h * per_head;
  while (first + units <= u) {
    first += units;
    units = item_units(a, s, ++m, NR);
  }

  auto next_item = [&]() {
    first += units;
    if (++m == a.mt) m = 0, ++h;
    if (h == a.heads) {
      h = 0;
      s = seen_of(a, ++b, false);
    }
    units = item_units(a, s, m, NR);
  };

  while (u < u_end) {
    const int vmax = item_keys(a, s, m, NR);
    const int v_end = min(u_end, first + units);  // units [u, v_end) of this item are ours
    // steps of 32 keys, in turn to the warps
    const int t0 = (u - first) * (kUnit / 32) + warp, t1 = min((vmax + 31) / 32, (v_end - first) * (kUnit / 32));
    const bool whole = u == first && v_end == first + units;
    const int slot = 2 * blockIdx.x + (u > (int)blockIdx.x * share ? 1 : 0);
    if (a.info && u == first && threadIdx.x == 0)  // for the join: the item's first slot, and in how many CTAs it lies
      a.info[((int64_t)b * a.heads + h) * a.mt + m] = make_int2(slot, (first + units - 1) / share - blockIdx.x + 1);

    auto block_of = [&](int t, int half) -> int {
      const int key = t * 32 + half * 16;
      if (t >= t1 || key >= vmax) return -1;
      const int blk = a.table[(int64_t)b * a.max_blocks + (key >> a.bt_log2)];
      if (blk >= 0 && blk < a.n_blocks) return blk;
      if (lane == 0) atomicOr(a.status, kStatusCache);
      return -1;
    };
    // the tiles of step t into the warp's next slot: lanes 0-3 a copy each, (half, side)
    uint8_t* mine = ring + warp * (2 * 4 * Tl::kBytes);
    auto fetch = [&](int t, int b0, int b1) {
      if (t >= t1) return;
      const uint32_t bar = smem_u32(&full[warp][issued & 1]);
      const int blk = lane & 1 ? b1 : b0, key = t * 32 + (lane & 1) * 16;
      const uint32_t bytes = ((b0 >= 0) + (b1 >= 0)) * 2 * Tl::kBytes;
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
      __syncwarp();
      if (lane < 4 && blk >= 0) {
        const int64_t from = (((int64_t)blk * a.heads + h) * a.bt + (key & (a.bt - 1))) * D;
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_u32(mine + ((issued & 1) * 4 + lane) * Tl::kBytes)),
            "l"((lane & 2 ? a.vc : a.kc) + from), "r"(Tl::kBytes), "r"(bar)
            : "memory");
      }
      ++issued;
    };
    auto scales = [&](int blk, float& ks, float& vs) {
      ks = blk < 0 ? 0.f : a.ks[(int64_t)blk * a.heads + h];
      vs = blk < 0 ? 0.f : a.vs[(int64_t)blk * a.heads + h];
    };
    int b0 = block_of(t0, 0), b1 = block_of(t0, 1);
    fetch(t0, b0, b1);
    float ks[2], vs[2];
    scales(b0, ks[0], vs[0]);
    scales(b1, ks[1], vs[1]);
    bool ok0 = b0 >= 0, ok1 = b1 >= 0;
    const bool small = small_scale(vs[0]);
    float last_lv = kNoScale;
    b0 = block_of(t0 + 4, 0), b1 = block_of(t0 + 4, 1);

    // the rows: lane (g, c) the dims of its words of row g; then the sight and the scale of rows 2c, 2c + 1
    uint32_t qb[NT][KW][2];
    int vis[NT][2];
    float fz[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int i = m * NR + n * 8 + g;
      const int row = i / a.G;
      const int sees = i < M ? visible(a, s, row) : 0;
      float x[KW][4], top = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[w][k] = 0.f;
        if (sees > 0) load4(q.at(b, row, h * a.G + i % a.G) + Tl::dim_of(w, c), x[w]);
      }
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(x[w][k]));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int ex = row_exponent(top);
      const float dn = __uint_as_float((uint32_t)(127 - ex) << 23), up = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        qb[n][w][0] = pack_half2(x[w][0] * dn, x[w][1] * dn);
        qb[n][w][1] = pack_half2(x[w][2] * dn, x[w][3] * dn);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        vis[n][e] = __shfl_sync(0xFFFFFFFFu, sees, (2 * c + e) * 4);
        fz[n][e] = __shfl_sync(0xFFFFFFFFu, up, (2 * c + e) * 4);
      }
    }

    int vmin = 0x7FFFFFFF;  // of the rows there are: keys before it need no mask
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (m * NR + n * 8 + 2 * c + e < M) vmin = min(vmin, vis[n][e]);
    vmin = min(vmin, __shfl_xor_sync(0xFFFFFFFFu, vmin, 1));
    vmin = min(vmin, __shfl_xor_sync(0xFFFFFFFFu, vmin, 2));

    float o[NT][D / 16][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mx[n][0] = mx[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;
    }

    for (int t = t0; t < t1; t += 4) {
      const int b0n = block_of(t + 8, 0), b1n = block_of(t + 8, 1);
      fetch(t + 4, b0, b1);
      float ksn[2], vsn[2];
      scales(b0, ksn[0], vsn[0]);
      scales(b1, ksn[1], vsn[1]);
      const uint8_t* tiles = mine + (taken & 1) * 4 * Tl::kBytes;
      good = warp_wait(&full[warp][taken & 1], (taken >> 1) & 1, spin);
      if (!good) break;
      ++taken;
      const int key0 = t * 32;
      float z[2][NT][4], lv[2], iv[2];
      if (last_lv == kNoScale) last_lv = scale_log2(vs[0], scale_log2(vs[1], kNoScale));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t k[2][KW];
        Tl::keys(tiles + half * Tl::kBytes, g, c, k);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[half][n][j] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t ka[4];
          codes_half4<INT8>(k[0][w], ka[0], ka[2]);
          codes_half4<INT8>(k[1][w], ka[1], ka[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816(z[half][n], ka, qb[n][w][0], qb[n][w][1]);
        }
        last_lv = lv[half] = scale_log2(vs[half], last_lv);
        iv[half] = sum_weight(lv[half], small);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = fz[n][e] * ks[half];
            z[half][n][e] = fmaf(z[half][n][e], f, lv[half]);
            z[half][n][2 + e] = fmaf(z[half][n][2 + e], f, lv[half]);
          }
      }
      // keys that a row does not see, and tiles that are not there
      if (!ok0 || !ok1 || key0 + 32 > vmin) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (key0 + 16 * (j >> 1) + 8 * (j & 1) + g >= vis[n][e] || !(j >> 1 ? ok1 : ok0))
                z[j >> 1][n][2 * (j & 1) + e] = -INFINITY;
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // whether any score passes the reference: each lane asks for its own, the largest is found only then
        float tm[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          tm[e] = fmaxf(fmaxf(z[0][n][e], z[0][n][2 + e]), fmaxf(z[1][n][e], z[1][n][2 + e]));
        if (__any_sync(0xFFFFFFFFu, tm[0] > mx[n][0] + 8.f || tm[1] > mx[n][1] + 8.f)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xFFFFFFFFu, tm[e], x));
            const float nm = fmaxf(mx[n][e], tm[e]);
            const float f = mx[n][e] == -INFINITY ? 0.f : exp2_fast(mx[n][e] - nm);
            l[n][e] = moved_sum(l[n][e], mx[n][e], nm);
            mx[n][e] = nm;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[n][j][e] *= f;
              o[n][j][2 + e] *= f;
            }
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mu = mx[n][e] == -INFINITY ? 0.f : mx[n][e];
            p[e] = exp2_fast(z[half][n][e] - mu);
            p[2 + e] = exp2_fast(z[half][n][2 + e] - mu);
            l[n][e] = fmaf(p[e] + p[2 + e], iv[half], l[n][e]);
          }
          pb[half][n][0] = transpose8(pack_half2(p[0], p[1]));  // (key, rows) -> (row, keys)
          pb[half][n][1] = transpose8(pack_half2(p[2], p[3]));
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t vw[4][VW];
        Tl::values(tiles + (2 + half) * Tl::kBytes, g, c, vw);
        const bool some = (half ? ok1 : ok0) && has_scale(vs[half]);
        if (key0 + 16 * half + 16 > vmax || !some) {  // behind what is seen: not defined, may be NaN
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (key0 + 16 * half + 2 * c + (j & 1) + (j >> 1) * 8 >= vmax || !some)
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[j][w] = 0;
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t x[4], y[4];  // of four dims: keys 2c, 2c + 1, and 8 on
          codes_half4<INT8>(__byte_perm(vw[0][w], vw[1][w], 0x5140), x[0], x[1]);
          codes_half4<INT8>(__byte_perm(vw[0][w], vw[1][w], 0x7362), x[2], x[3]);
          codes_half4<INT8>(__byte_perm(vw[2][w], vw[3][w], 0x5140), y[0], y[1]);
          codes_half4<INT8>(__byte_perm(vw[2][w], vw[3][w], 0x7362), y[2], y[3]);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t va[4] = {x[2 * v], x[2 * v + 1], y[2 * v], y[2 * v + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(o[n][2 * w + v], va, pb[half][n][0], pb[half][n][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the slot: the next fetch may fill it
      ok0 = b0 >= 0, ok1 = b1 >= 0;
      b0 = b0n, b1 = b1n;
#pragma unroll
      for (int half = 0; half < 2; ++half) ks[half] = ksn[half], vs[half] = vsn[half];
    }
    if (!good) {  // a copy has not come: recorded; what is still on its way lands before the CTA ends
      if (lane == 0) atomicOr(a.status, kStatusTimeout);
      for (; taken < issued; ++taken) warp_wait(&full[warp][taken & 1], (taken >> 1) & 1, kFewSpin);
    }
    __syncthreads();  // the sums take the ring's place
    // join the warps: accumulator tile j, element (e, row g or g + 8) is row 2c + e, dim g * D/8 + 2 j (+ 1)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], x);
        const int r = n * 8 + 2 * c + e;
        const PartEnd end = part_end(mx[n][e], l[n][e], small);
        if (g == 0) {
          sm_m[warp][r] = end.m;
          sm_l[warp][r] = end.l;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          *reinterpret_cast<float2*>(&sm_o[warp][r][g * (D / 8) + 2 * j]) = make_float2(o[n][j][e] * end.down, o[n][j][2 + e] * end.down);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < NR * (D / 4); i += kFewThreads) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      const int ri = m * NR + r;
      if (ri >= M) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, sm_m[w][r]);
      float sum = 0.f, x[4] = {};
      if (top != -INFINITY) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = exp2_fast(sm_m[w][r] - top);
          sum = fmaf(f, sm_l[w][r], sum);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = fmaf(f, sm_o[w][r][d + k], x[k]);
        }
      }
      if (!whole) {
        const int64_t pi = (int64_t)slot * NR + r;
        store4(a.part + pi * D + d, x);
        if (d == 0) {
          float* ml = a.part + a.slots * NR * D + pi * 2;
          ml[0] = top;
          ml[1] = sum;
        }
      } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int tr = ri / a.G, th = h * a.G + ri % a.G;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] *= inv;
        store4(out.at(b, tr, th) + d, x);
        if (a.lse && d == 0)
          a.lse[((int64_t)b * a.R + tr) * a.Hq + th] =
              top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    const bool gone = __syncthreads_or(!good);  // the joined warps' buffers are free again
    u = v_end;
    if (u < u_end) next_item();
    if (gone) {
      // the items that begin in the rest of the share are left out: one part, which the join passes by (their outputs are
      // not defined), since it would follow whatever the workspace holds there
      while (u < u_end) {
        if (a.info && threadIdx.x == 0) a.info[((int64_t)b * a.heads + h) * a.mt + m] = make_int2(0, 1);
        u = first + units;
        if (u < u_end) next_item();
      }
      return;
    }
  }
}

// Joins the parts of the keys, WARPS warps a (request, row, query head), each
// every WARPS-th part, eight of them in flight.  Items of one part have their
// outputs already.  Bound by latency: the item's parts, then the sums.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ AttnArgs a, const Rows<T> out) {
  constexpr int kLanes = D / 4;  // lanes that hold four dims
  __shared__ float sm_m[8], sm_l[8], sm_x[8][D];
  after_predecessor();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % WARPS;
  const int64_t total = (int64_t)a.B * a.R * a.Hq;
  const int64_t id = (int64_t)blockIdx.x * (8 / WARPS) + warp / WARPS;
  const int64_t rid = min(id, total - 1);
  const int qh = (int)(rid % a.Hq);
  const int64_t br = rid / a.Hq;
  const int r = (int)(br % a.R), b = (int)(br / a.R);
  const int i = r * a.G + qh % a.G, m = i / a.tile;
  const int64_t item = ((int64_t)b * a.heads + qh / a.G) * a.mt + m;
  int parts;
  int64_t slot0, later, step;  // slots of the parts: slot0, then later + step, later + 2 step, ...
  if (a.info) {
    const int2 e = a.info[item];
    parts = e.y;
    slot0 = e.x, later = e.x & ~1, step = 2;
    if (e.x < 0 || parts < 1 || (e.x >> 1) + (int64_t)parts > a.slots / 2) {  // another call has written the workspace
      if (lane == 0) atomicOr(a.status, kStatusCache);
      parts = 1;
    }
  } else {
    const Seen s = seen_of(a, b, false);
    parts = parts_of(a, item_keys(a, s, m, a.tile));
    slot0 = later = item * a.splits, step = 1;
  }
  const float* ml = a.part + a.slots * a.tile * D;
  float top = -INFINITY, sum = 0.f, x[4] = {};
  if (parts > 1) {
    for (int s0 = w; s0 < parts; s0 += 8 * WARPS) {
      float2 e[8];
      float y[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int sp = s0 + WARPS * j;
        e[j] = make_float2(-INFINITY, 0.f);
        y[j][0] = y[j][1] = y[j][2] = y[j][3] = 0.f;
        if (sp < parts) {
          const int64_t at = (sp ? later + sp * step : slot0) * a.tile + i % a.tile;
          e[j] = *reinterpret_cast<const float2*>(ml + at * 2);
          if (lane < kLanes) load4(a.part + at * D + 4 * lane, y[j]);
        }
      }
      float nt = top;
#pragma unroll
      for (int j = 0; j < 8; ++j) nt = fmaxf(nt, e[j].x);
      if (nt == -INFINITY) continue;
      const float f0 = exp2_fast(top - nt);
      top = nt;
      sum *= f0;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= f0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = exp2_fast(e[j].x - nt);
        sum = fmaf(f, e[j].y, sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = fmaf(f, y[j][k], x[k]);
      }
    }
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) sm_m[warp] = top, sm_l[warp] = sum;
    if (lane < kLanes) store4(&sm_x[warp][4 * lane], x);
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) top = fmaxf(top, sm_m[warp + k]);
    const float f0 = top == -INFINITY ? 0.f : exp2_fast(sm_m[warp] - top);
    sum *= f0;
#pragma unroll
    for (int d = 0; d < 4; ++d) x[d] *= f0;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) {
      const float f = top == -INFINITY ? 0.f : exp2_fast(sm_m[warp + k] - top);
      sum = fmaf(f, sm_l[warp + k], sum);
      float y[4] = {};
      if (lane < kLanes) load4(&sm_x[warp + k][4 * lane], y);
#pragma unroll
      for (int d = 0; d < 4; ++d) x[d] = fmaf(f, y[d], x[d]);
    }
  }
  if (id >= total || parts <= 1) return;
  if (lane < kLanes) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= inv;
    store4(out.at(b, r, qh) + 4 * lane, x);
  }
  if (a.lse && lane == 0)
    a.lse[rid] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

// ---------------------------------------------------------------- host side

// Rows up to which the join has four warps a row, not one.  Measured (us a call of
// single tokens, four warps against one): 128 rows of some 14 parts 108.3/111.7,
// 512 of some 4 27.1/27.8; 1,024 rows (32 requests of 4,000 tokens, 32 heads over
// 4) 35.0/33.7, 4,096 (of 1,000) 41.0/35.6, 16,384 (of 300) 81.2/64.7.  Eight
// warps take 108.1 and 28.9 for the first two.
constexpr int64_t kJoinRows = 512;

struct AttnPlan {
  bool tc;
  int tile, mt, splits, chunk, ctas;
  int64_t items, slots;
  size_t bytes;
};

// Query rows a key head up to which k_attn_few is taken.  Measured (us, few
// against many rows; 4 heads, e4m3), at 16, 24, 32 and 48 rows:
//   32 requests of  2,000 tokens, 64 dims: 20.8/33.1  27.8/33.0  30.9/33.1  43.3/33.0
//                                128 dims: 26.8/37.7  36.9/37.1  40.4/37.1  59.7/37.2
//    4 requests of 30,000 tokens, 64 dims: 31.0/55.7  45.3/55.6  47.4/55.6  53.4/55.9
//                                128 dims: 41.1/59.7  61.1/59.8  63.7/59.7  70.8/60.2
inline int few_rows(int dim) { return dim <= 64 ? 32 : 24; }

// Few rows: as many CTAs as are resident, or one for each unit that the
// histories may have.  Many rows: one CTA an item, its keys in parts only where
// items leave SMs idle, 512 keys each at least; the longest history may have
// `splits`.
AttnPlan attn_plan(const zg_kv_cache* c, int max_blocks, int B, int R, int Hq) {
  AttnPlan p = {};
  const int64_t M = (int64_t)R * (Hq / c->heads);
  p.tc = M > few_rows(c->dim);
  p.tile = p.tc ? attn_tc_tile(M) : M > 8 ? 16 : 8;
  p.mt = (int)((M + p.tile - 1) / p.tile);
  p.items = (int64_t)B * c->heads * p.mt;
  const int64_t keys = (int64_t)max_blocks * c->block_tokens;
  if (p.tc) {
    const int64_t parts = std::max<int64_t>(1, p.items ? sm_count() / p.items : 1);
    p.chunk = (int)std::min<int64_t>(std::max<int64_t>(512, ((keys + parts - 1) / parts + 511) / 512 * 512), 1 << 30);
    p.splits = (int)((keys + p.chunk - 1) / p.chunk);
    p.slots = p.splits > 1 ? p.items * p.splits : 0;
  } else {
    const int resident = p.tile == 16 ? 2 : 3;
    p.ctas = (int)std::min<int64_t>((int64_t)sm_count() * resident, p.items * ((keys + 127) / 128));
    p.slots = p.ctas > 1 && keys > 128 ? 2 * (int64_t)p.ctas : 0;
  }
  p.bytes = p.slots ? ((size_t)p.slots * p.tile * (c->dim + 2) + (p.tc ? 0 : 2 * p.items)) * 4 : 0;
  return p;
}

zg_status check_attn(const zg_kv_cache* c, int32_t max_blocks, int32_t B, int32_t R, int32_t Hq, const char* call) {
  if (B < 0 || R < 0) return bad_arg(call, "B and R must be >= 0");
  if (Hq < 1 || Hq > 1024 || Hq % c->heads) return bad_arg(call, "Hq must be a multiple of cache.heads, at most 1024");
  if ((int64_t)B * R >= 0x80000000LL / Hq) return bad_arg(call, "B * R * Hq must be below 2^31");
  if ((int64_t)max_blocks * c->block_tokens > kMostTokens)
    return fail(ZG_ERR_UNSUPPORTED, std::string(call) + ": more than 2^31 - 2^20 tokens in a table");
  return ZG_OK;
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zg_status zg_kv_attention_workspace_size(const zg_kv_cache* cache, int32_t max_blocks, int32_t B, int32_t R,
                                         int32_t Hq, size_t* bytes) try {
  const char* call = "zg_kv_attention_workspace_size";
  static const int32_t no_table = 0;
  zg_status st;
  if (!bytes) return bad_arg(call, "bytes is NULL");
  if ((st = check_cache(cache, &no_table, max_blocks, call)) != ZG_OK) return st;
  if ((st = check_attn(cache, max_blocks, B, R, Hq, call)) != ZG_OK) return st;
  // what this batch and every smaller one needs: of many rows a small batch is split into parts where a large one,
  // with an item for every SM, is not
  *bytes = attn_plan(cache, max_blocks, B, R, Hq).bytes;
  for (int b = 1; b < std::min(B, sm_count()); ++b) *bytes = std::max(*bytes, attn_plan(cache, max_blocks, b, R, Hq).bytes);
  return ZG_OK;
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

zg_status zg_kv_attention(const zg_kv_cache* cache, const int32_t* table, int32_t max_blocks, const int32_t* length,
                          const int32_t* n_rows, const zg_rows* q, const zg_rows* out, float* lse, int32_t B,
                          int32_t R, int32_t Hq, float scale, int32_t causal, void* workspace, size_t ws_bytes,
                          void* stream) try {
  const char* call = "zg_kv_attention";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if ((st = check_attn(cache, max_blocks, B, R, Hq, call)) != ZG_OK) return st;
  if (B == 0 || R == 0) return ZG_OK;
  if ((st = check_rows(q, "q", -1, call)) != ZG_OK) return st;
  if (q->dtype == ZG_F32) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_attention: q must be ZG_BF16 or ZG_F16");
  if ((st = check_rows(out, "out", q->dtype, call)) != ZG_OK) return st;
  if (!length) return bad_arg(call, "length is NULL");
  if (!(scale > 0.f && std::isfinite(scale))) return bad_arg(call, "scale must be finite and > 0");
  if (lse && reinterpret_cast<uintptr_t>(lse) % 4) return bad_arg(call, "lse must be 4-byte aligned");
  const AttnPlan p = attn_plan(cache, max_blocks, B, R, Hq);
  if (p.bytes && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < p.bytes))
    return bad_arg(call, "workspace must hold zg_kv_attention_workspace_size bytes, 256-byte aligned");
  if (p.items * std::max<int64_t>(p.tc ? p.splits : ((int64_t)max_blocks * cache->block_tokens + 127) / 128, 1) > kMostUnits)
    return fail(ZG_ERR_UNSUPPORTED, "zg_kv_attention: more than 2^31 - 2^20 units of work (B * heads * keys of a table / 128)");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  AttnArgs a = {};
  a.kc = static_cast<const uint8_t*>(cache->k_codes);
  a.vc = static_cast<const uint8_t*>(cache->v_codes);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.table = table;
  a.length = length;
  a.n_rows = n_rows;
  a.status = status;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.n_blocks = cache->n_blocks;
  a.heads = cache->heads;
  a.bt = cache->block_tokens;
  while ((1 << a.bt_log2) < a.bt) ++a.bt_log2;
  a.max_blocks = max_blocks;
  a.B = B;
  a.R = R;
  a.Hq = Hq;
  a.G = Hq / cache->heads;
  a.tile = p.tile;
  a.mt = p.mt;
  a.splits = p.splits;
  a.slots = p.slots;
  if (!p.tc && p.slots)  // an even count of floats: 8-byte aligned
    a.info = reinterpret_cast<int2*>(a.part + (size_t)p.slots * p.tile * (cache->dim + 2));
  a.chunk = p.chunk;
  a.causal = causal != 0;
  a.scale = scale * 1.4426950408889634f;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  auto launch = [&](auto ev, auto dv, auto iv) {
    using E = typename decltype(ev)::type;
    constexpr int D = decltype(dv)::value;
    if (!p.tc) {
      auto kern = p.tile == 8 ? k_attn_few<E, D, decltype(iv)::value, 1> : k_attn_few<E, D, decltype(iv)::value, 2>;
      const int smem = p.tile == 8 ? few_smem<D, 1>() : few_smem<D, 2>();
      if (smem > 40 * 1024) err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err != cudaSuccess) return;
      err = launch_early(kern, p.ctas, kFewThreads, smem, sm, a, rows_of<E>(q), rows_of<E>(out),
                         std::min(wait_limit(), kFewSpin));
      if (err != cudaSuccess) return;
    }
    if (p.slots) {
      // several warps a row where the rows alone would leave SMs idle
      const int64_t rows = (int64_t)B * R * Hq;
      const int warps = rows <= kJoinRows ? 4 : 1;
      err = launch_early(warps == 4 ? k_attn_join<E, D, 4> : k_attn_join<E, D, 1>, (rows * warps + 7) / 8, 256, 0, sm, a,
                         rows_of<E>(out));
    }
  };
  if (p.tc) {
    const cudaError_t e = launch_attn_tc(a, q, out, cache->dim, cache->format == ZG_KV_INT8, p.items * p.splits, sm);
    if (e != cudaSuccess) return cuda_fail(e, "cache attention launch");
  }
  for_dim(cache->dim, [&](auto dv) {
    auto typed = [&](auto ev) {
      if (cache->format == ZG_KV_INT8) launch(ev, dv, std::true_type{});
      else launch(ev, dv, std::false_type{});
    };
    if (q->dtype == ZG_BF16) typed(Elem<__nv_bfloat16>{});
    else typed(Elem<__half>{});
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "cache attention launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

}  // extern "C"
