// Eviction from a history cache by what its tokens have collected of attention:
// a request that holds more than `keep` tokens keeps, each key head for
// itself, its last `recent` ones and the keep - recent others of largest
// weight, moved to the front in their order.
//
// One cluster of CTAs a (request, key head), in one launch:
//   select  the weight of the last one kept, 11 + 11 + 10 bits at a time from
//           histograms of order-preserving integers (the CTAs' histograms added
//           through distributed shared memory), then the kept numbers in
//           order.  Weights are read once and stay in shared memory, 32,768 a
//           CTA at most; those behind them are read again by every pass.
//           Integer counts alone: nothing hangs on an order of atomics.
//   move    row i comes from kept[i] >= i, and kept[] ascends: the cluster reads
//           a batch of rows into its shared memory, all its CTAs wait for one
//           another, then it is written; what a later batch reads lies behind
//           all that is written by then.
//
// Measured: 64 histories of up to 2,047 tokens (2 heads of 64, int8) cut to 500
// 11.3 us; 8 of up to 131,072 (4 heads of 128, 4 bits) cut to 8,192 39 us, of
// which the longest spends some 20 with its selection, the rest with two
// batches of rows.  Bound by latency: barriers, and the chain kept number ->
// block -> row (no warp is ready in 61 % of cycles).  As two launches 27 and 45
// us.  A head has eight CTAs at most: one history of one head of 128, 100,000
// tokens cut to 50,000, takes 65 us in 4 bits and 108 in e4m3.
//
// In 8 bits a block's new scale is the largest of its rows' old ones, and rows
// of a smaller one are coded again.  In 4 bits rows carry their scales along
// and nothing is rounded.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
static_assert(2 * kThreads == kBins, "two bins a thread");
constexpr int kHists = 6;
constexpr int kStrip = 128;              // tokens that a warp looks at at once, four a lane
constexpr int kMostRanks = 8;            // CTAs of a cluster, at most
constexpr int kMostSmem = 128 * 1024;    // weights of a CTA, then rows of a batch

struct EvictArgs {
  CacheView c;
  const int32_t* length;
  float* w;
  int32_t *new_length, *kept;
  int32_t w_tokens, keep, recent;
  int32_t bt_log2;     // of a block's tokens
  int32_t smem;        // bytes before the histograms
  int32_t held, rows;  // strips that a warp keeps in shared memory; rows of a CTA's share of a batch, whole blocks
};

// Larger numbers for larger weights; NaN (1) below everything, both zeros the
// same; 0 stands for no token.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int held(const EvictArgs& a, int b, bool report) {
  const int n = a.length[b], most = a.c.max_blocks * a.c.bt;
  if (n >= 0 && n <= most) return n;
  if (report) atomicOr(a.c.status, kStatusCache);
  return min(max(n, 0), most);
}

// The scale bytes of a row, as wide as they are aligned.
template <int D>
struct ScaleBytes {
  using type = std::conditional_t<D == 128, uint2, std::conditional_t<D == 64, uint32_t, uint16_t>>;
  static constexpr int kCount = Row4<D>::kScales / sizeof(type);
};

template <int D, int FMT>
struct EvictShape {
  static constexpr bool k4 = FMT == ZG_KV_E2M1;
  static constexpr int kRow = k4 ? Row4<D>::kCodes : D, kUnits = kRow / 16;
  static constexpr int kScales = Row4<D>::kScales;  // scale bytes of a row in 4 bits
  // rows of keys and of values in shared memory, a thread each for what is small of them
  static constexpr int kRows = kMostSmem / (2 * kRow) / 128 * 128 < kThreads ? kMostSmem / (2 * kRow) / 128 * 128 : kThreads;
};

// Four codes of a row coded again by another scale, as the write does it.
template <bool INT8>
__device__ __forceinline__ uint32_t code_again(uint32_t w, float s0, float inv) {
  float y[4];
  codes_float4<INT8>(w, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] *= s0;
  return float4_codes<INT8>(y, inv);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_evict(const __grid_constant__ EvictArgs a) {
  using Sh = EvictShape<D, FMT>;
  using Bytes = typename ScaleBytes<D>::type;
  constexpr int kBytes = ScaleBytes<D>::kCount;
  constexpr bool INT8 = FMT == ZG_KV_INT8;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  extern __shared__ __align__(16) uint8_t smem[];
  // a histogram a pass, so that none is written while another CTA reads it; of the first, in which most weights fall into
  // few bins, one for every fourth lane, of which hist[0] is the sum
  uint32_t(*hist)[kBins] = reinterpret_cast<uint32_t(*)[kBins]>(smem + a.smem);
  __shared__ uint32_t sums[kWarps], found[3][3];
  __shared__ int mine[2];  // of this CTA's tokens: above the last weight, equal to it
  __shared__ int warp_above[kWarps], warp_equal[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / ranks, b = bh / a.c.heads, h = bh % a.c.heads;
  for (int i = tid; i < kHists * kBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  auto all = [&]() {  // every thread of the cluster
    if (ranks > 1) cl.sync();
    else __syncthreads();
  };
  after_predecessor();
  const int n = held(a, b, tid == 0 && rank == 0 && h == 0);
  int32_t* kept = a.kept + (int64_t)bh * a.keep;
  if (tid == 0 && rank == 0 && h == 0) a.new_length[b] = min(n, a.keep);
  if (n <= a.keep) {  // stays as it is
    for (int i = rank * kThreads + tid; i < a.keep; i += ranks * kThreads) kept[i] = i < n ? i : -1;
    return;
  }
  float* w = a.w + (int64_t)bh * a.w_tokens;
  const int m = n - a.recent, want = a.keep - a.recent;  // `want` of the first m
  for (int i = rank * kThreads + tid; i < a.recent; i += ranks * kThreads) kept[want + i] = m + i;

  if (want > 0) {
    // ------------------------------------------------------------- select
    // this warp's tokens, whole strips of them, and its place in shared memory
    uint32_t* mem = reinterpret_cast<uint32_t*>(smem) + warp * a.held * kStrip;
    const int per = ((m + ranks * kWarps - 1) / (ranks * kWarps) + kStrip - 1) / kStrip * kStrip;
    const int64_t from = (int64_t)(rank * kWarps + warp) * per;
    const int lo = (int)min((int64_t)m, from), hi = (int)min((int64_t)m, from + per);
    const int strips = (hi - lo + kStrip - 1) / kStrip;
    auto key_at = [&](int i) -> uint32_t { return i < hi ? order_key(w[i]) : 0; };
    // they come in sixteen a lane at a time, and are counted by their first bits at once
    __syncthreads();  // the histograms are zero
    uint32_t* counts = hist[lane & 3 ? 2 + (lane & 3) : 0];
    for (int j0 = lane; j0 < (hi - lo); j0 += 16 * 32) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = j0 + 32 * k < hi - lo ? w[lo + j0 + 32 * k] : 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int j = j0 + 32 * k;
        const uint32_t u = j < hi - lo ? order_key(x[k]) : 0;
        if (u && j < a.held * kStrip) mem[j] = u;
        if (u) atomicAdd(&counts[u >> (32 - 11)], 1u);
      }
    }
    for (int j = hi - lo + lane; j < min(a.held, strips) * kStrip; j += 32) mem[j] = 0;  // no tokens
    __syncwarp();
    // a lane's four neighbours of a strip
    auto strip = [&](int s) -> uint4 {
      if (s < a.held) return reinterpret_cast<const uint4*>(mem)[s * 32 + lane];
      const int i = lo + s * kStrip + 4 * lane;
      return make_uint4(key_at(i), key_at(i + 1), key_at(i + 2), key_at(i + 3));
    };
    uint32_t key = 0;  // what is known of the last kept weight
    int above = 0;     // weights above what is known of it
    int left = 32;     // bits not known yet
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = left - bits, bins = 1 << bits;
      if (pass == 0) {
        __syncthreads();
        for (int i = tid; i < kBins; i += kThreads) hist[0][i] += hist[3][i] + hist[4][i] + hist[5][i];
      } else {
#pragma unroll 2
        for (int s = 0; s < strips; ++s) {
          const uint4 x4 = strip(s);
          const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (x[k] >> left == key >> left) atomicAdd(&hist[pass][(x[k] >> shift) & (bins - 1)], 1u);
        }
      }
      all();
      // two bins a thread, the largest first; the bin in which the count passes what is wanted
      uint32_t t[2] = {};
      const int bin0 = bins - 1 - 2 * tid;
      if (bin0 >= 1) {
        if (ranks == 1) {
          t[0] = hist[pass][bin0];
          t[1] = hist[pass][bin0 - 1];
        } else {
#pragma unroll
          for (int r = 0; r < kMostRanks; ++r) {
            if (r < ranks) {
              const uint2 x = *reinterpret_cast<const uint2*>(cl.map_shared_rank(&hist[pass][bin0 - 1], r));
              t[0] += x.y;
              t[1] += x.x;
            }
          }
        }
      }
      const uint32_t s = t[0] + t[1];
      uint32_t run = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      uint32_t before = run - s + (uint32_t)above + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[lane] : 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (before < (uint32_t)want && before + t[j] >= (uint32_t)want) {
          found[pass][0] = bin0 - j;
          found[pass][1] = before;
          found[pass][2] = before + t[j];
        }
        before += t[j];
      }
      __syncthreads();
      key |= found[pass][0] << shift;
      above = (int)found[pass][1];
      left = shift;
      if (found[pass][2] == (uint32_t)want) {  // all of the bin are kept: as if the last weight were the next below it,
        key -= 1;                              // and none equal to it kept
        above = want;
        break;
      }
    }
    // kept before this warp's tokens: all above the last weight, and of those equal to it the first ones
    int na = 0, ne = 0;
#pragma unroll 2
    for (int s = 0; s < strips; ++s) {
      const uint4 x = strip(s);
      na += (x.x > key) + (x.y > key) + (x.z > key) + (x.w > key);
      ne += (x.x == key) + (x.y == key) + (x.z == key) + (x.w == key);
    }
    na = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)na);
    ne = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)ne);
    if (lane == 0) warp_above[warp] = na, warp_equal[warp] = ne;
    __syncthreads();
    int over = lane < warp ? warp_above[lane] : 0, equal = lane < warp ? warp_equal[lane] : 0;
    if (ranks > 1) {
      if (warp == 0) {
        const int all_above = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)warp_above[lane]),
                  all_equal = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)warp_equal[lane]);
        if (lane == 0) mine[0] = all_above, mine[1] = all_equal;
      }
      cl.sync();
      if (lane < rank) {
        over += *cl.map_shared_rank(&mine[0], lane);
        equal += *cl.map_shared_rank(&mine[1], lane);
      }
    }
    over = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)over);
    equal = (int)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)equal);
    const int ties = want - above;  // kept of those equal
    const uint32_t below = (1u << lane) - 1;
    for (int s = 0; s < strips; ++s) {
      const uint4 x4 = strip(s);
      const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
      int my_over = over, my_equal = equal;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t ba = __ballot_sync(0xFFFFFFFFu, x[k] > key), be = __ballot_sync(0xFFFFFFFFu, x[k] == key);
        my_over += __popc(ba & below);
        my_equal += __popc(be & below);
        over += __popc(ba);
        equal += __popc(be);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x[k] > key || (x[k] == key && my_equal < ties)) kept[my_over + min(my_equal, ties)] = lo + s * kStrip + 4 * lane + k;
        my_over += x[k] > key;
        my_equal += x[k] == key;
      }
    }
  }
  all();  // the kept numbers are there; nobody reads another's shared memory from here on

  // ----------------------------------------------------------------- move
  __shared__ float row_scale[2][Sh::k4 ? 1 : Sh::kRows], new_scale[2][Sh::k4 ? 1 : Sh::kRows / 16];
  const int bt = a.c.bt, sh = a.bt_log2;
  const int32_t* table = a.c.table + (int64_t)b * a.c.max_blocks;
  auto good = [&](int blk) { return blk >= 0 && blk < a.c.n_blocks; };
  auto row_of = [&](int blk, int token) -> int64_t { return (((int64_t)blk * a.c.heads + h) << sh) + (token & (bt - 1)); };
  auto codes = [&](int side) { return side ? a.c.vc : a.c.kc; };
  auto scales = [&](int side) { return side ? a.c.vs : a.c.ks; };
  auto bytes = [&](int side, int blk, int token) {
    return reinterpret_cast<Bytes*>(reinterpret_cast<uint8_t*>(scales(side)) + row_of(blk, token) * Sh::kScales);
  };
  for (int64_t first = 0; first < a.keep; first += (int64_t)ranks * a.rows) {
    const int64_t r0 = first + (int64_t)rank * a.rows;
    const int count = (int)max((int64_t)0, min((int64_t)a.rows, a.keep - r0)), base = (int)r0;
    const int units = count * Sh::kUnits;  // of 16 bytes, of each side
    // the codes of both sides, four chains (kept number, block, row) at a time
    for (int x0 = tid; x0 < units; x0 += 4 * kThreads) {
      int from[4], blk[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = x0 + k * kThreads;
        from[k] = x < units ? __ldcg(kept + base + x / Sh::kUnits) : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) blk[k] = from[k] >= 0 ? table[from[k] >> sh] : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = x0 + k * kThreads;
        if (x >= units) continue;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          uint4* to = reinterpret_cast<uint4*>(smem) + side * a.rows * Sh::kUnits + x;
          if (good(blk[k])) {
            const uint4* p = reinterpret_cast<const uint4*>(codes(side) + row_of(blk[k], from[k]) * Sh::kRow) + x % Sh::kUnits;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(p)
                         : "memory");
          } else {
            *to = make_uint4(0, 0, 0, 0);
          }
        }
      }
    }
    // what is small of a row stays with its thread
    float weight = 0.f;
    Bytes u[2][Sh::k4 ? kBytes : 1];
    int to_blk = -1;
    if (tid < count) {
      to_blk = table[(base + tid) >> sh];
      const int from = __ldcg(kept + base + tid), blk = table[from >> sh];
      if (!good(blk) || !good(to_blk)) atomicOr(a.c.status, kStatusCache);
      weight = __ldcg(w + from);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        if constexpr (Sh::k4) {
          const Bytes* p = bytes(side, good(blk) ? blk : 0, from);
#pragma unroll
          for (int j = 0; j < kBytes; ++j) u[side][j] = good(blk) ? p[j] : Bytes{};
        } else {
          row_scale[side][tid] = good(blk) ? scales(side)[(int64_t)blk * a.c.heads + h] : 0.f;
        }
      }
    }
    if constexpr (!Sh::k4) {  // the new scales of the rows' blocks
      __syncthreads();
      for (int j = warp; j << sh < count; j += kWarps) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          float s = 0.f;
          for (int r = lane; r < bt; r += 32)
            if ((j << sh) + r < count) s = fmaxf(s, row_scale[side][(j << sh) + r]);
#pragma unroll
          for (int o = 16; o; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
          if (lane == 0) new_scale[side][j] = s;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    all();  // all of the batch has been read
    if (tid < count) {
      const int row = base + tid;
      w[row] = weight;
      if (good(to_blk)) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          if constexpr (Sh::k4) {
            Bytes* p = bytes(side, to_blk, row);
#pragma unroll
            for (int j = 0; j < kBytes; ++j) p[j] = u[side][j];
          } else if ((row & (bt - 1)) == 0) {
            scales(side)[(int64_t)to_blk * a.c.heads + h] = new_scale[side][tid >> sh];
          }
        }
      }
    }
#pragma unroll 2
    for (int x = tid; x < units; x += kThreads) {
      const int i = x / Sh::kUnits, row = base + i, blk = table[row >> sh];
      if (!good(blk)) continue;  // recorded above
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint4 y = reinterpret_cast<const uint4*>(smem)[side * a.rows * Sh::kUnits + x];
        if constexpr (!Sh::k4) {
          const float s0 = row_scale[side][i], s1 = new_scale[side][i >> sh];
          if (s0 != s1) {
            const float inv = s1 > 0.f ? __frcp_rn(s1) : 0.f;
            y = make_uint4(code_again<INT8>(y.x, s0, inv), code_again<INT8>(y.y, s0, inv), code_again<INT8>(y.z, s0, inv),
                           code_again<INT8>(y.w, s0, inv));
          }
        }
        reinterpret_cast<uint4*>(codes(side) + row_of(blk, row) * Sh::kRow)[x % Sh::kUnits] = y;
      }
    }
    __syncthreads();  // shared memory is free again
  }
}

// A kernel in clusters of `ranks` CTAs along x, started early as by launch_early.
cudaError_t launch_clusters(void (*kern)(EvictArgs), dim3 grid, int ranks, int threads, size_t smem, cudaStream_t st,
                            const EvictArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" zg_status zg_kv_evict(const zg_kv_cache* cache, const int32_t* table, int32_t max_blocks, const int32_t* length,
                                 float* weights, int32_t w_tokens, int32_t keep, int32_t recent, int32_t* new_length,
                                 int32_t* kept, int32_t B, void* stream) try {
  const char* call = "zg_kv_evict";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if (B < 0 || keep < 1) return bad_arg(call, "B must be >= 0 and keep >= 1");
  if ((int64_t)B * cache->heads > 65535) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_evict: more than 65,535 (request, key head)s");
  if (keep > 0x40000000) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_evict: keep above 2^30");
  if (recent < 0 || recent > keep) return bad_arg(call, "recent must be in [0, keep]");
  const int64_t tokens = (int64_t)max_blocks * cache->block_tokens;
  if (tokens > 0x7FF00000) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_evict: more than 2^31 - 2^20 tokens in a table");
  if (w_tokens < tokens) return bad_arg(call, "w_tokens must be at least max_blocks * block_tokens");
  if (B == 0) return ZG_OK;
  if (!length || !new_length || !kept || !weights) return bad_arg(call, "length, weights, new_length or kept is NULL");
  if ((reinterpret_cast<uintptr_t>(length) | reinterpret_cast<uintptr_t>(new_length) | reinterpret_cast<uintptr_t>(kept) |
       reinterpret_cast<uintptr_t>(weights)) % 4)
    return bad_arg(call, "length, weights, new_length and kept must be 4-byte aligned");
  if (length == new_length) return bad_arg(call, "new_length must not be length");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  const int bhs = B * cache->heads;
  EvictArgs a = {{static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->v_codes), cache->k_scale,
                  cache->v_scale, cache->n_blocks, cache->heads, cache->block_tokens, max_blocks, table, status},
                 length, weights, new_length, kept, w_tokens, keep, recent, 0, 0, 0, 0};
  while (1 << a.bt_log2 < cache->block_tokens) ++a.bt_log2;
  // as many CTAs a head as hold its weights four a thread (or its kept rows in a batch), and as fit the SMs at once (8 x
  // 4 heads of up to 131,072 tokens: one CTA a head 143 us, two 76, four 39, eight, which the SMs do not hold, 58)
  int ranks = 1;
  while (ranks < kMostRanks && (tokens > (int64_t)ranks * 4 * kThreads || keep > ranks * 512) && bhs * ranks * 2 <= sm_count())
    ranks *= 2;
  cudaError_t err = cudaSuccess;
  for_dim(cache->dim, [&](auto dv) {
    for_format(cache->format, [&](auto fv) {
      using Sh = EvictShape<decltype(dv)::value, decltype(fv)::value>;
      auto kern = k_evict<decltype(dv)::value, decltype(fv)::value>;
      const int64_t share = (keep + ranks - 1) / ranks;
      a.rows = (int)std::min<int64_t>(Sh::kRows, (share + 127) / 128 * 128);
      constexpr int kStripBytes = 4 * kStrip * kWarps;
      const int64_t strips = (tokens + ranks * kWarps * kStrip - 1) / (ranks * kWarps * kStrip);  // a warp
      const int smem = std::max((int)std::min<int64_t>(strips * kStripBytes, kMostSmem), a.rows * 2 * Sh::kRow);
      a.held = smem / kStripBytes;
      a.smem = smem;
      // the limit is the kernel's, not the call's: the most that any call asks for, so that calls of several threads agree
      constexpr int kHistBytes = kHists * kBins * 4;
      static_assert(Sh::kRows * 2 * Sh::kRow <= kMostSmem, "a batch of rows fits too");
      err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem + kHistBytes);
      if (err == cudaSuccess)
        err = launch_clusters(kern, dim3(bhs * ranks), ranks, kThreads, smem + kHistBytes, static_cast<cudaStream_t>(stream), a);
    });
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "cache eviction launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}
