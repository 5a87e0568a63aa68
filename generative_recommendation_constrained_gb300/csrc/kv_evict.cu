// Eviction from a history cache by what its tokens have collected of attention:
// a request that holds more than `keep` tokens keeps, each key head for
// itself, its last `recent` ones and the keep - recent others of largest
// weight, moved to the front in their order.
//
//   k_evict_select  finds them: the weight of the last one kept, 11 + 11 + 10
//                   bits at a time from histograms of order-preserving integers
//                   (a cluster of CTAs a head, their histograms added through
//                   distributed shared memory), then their numbers in order.
//                   Integer counts alone: nothing hangs on an order of atomics.
//   k_evict_move    moves rows in place.  Row i comes from kept[i] >= i, and
//                   kept[] ascends.  Rows whose source lies in the first `keep`
//                   places, where rows are also written, are moved first, in
//                   order, each batch read before it and all before it are
//                   written; then the others, whose sources nothing writes, by
//                   as many CTAs as there are.  Each CTA has 32-byte columns of
//                   its own, so none waits for another.
//
// In 8 bits a block's new scale is the largest of its rows' old ones, and rows
// of a smaller one are coded again.  In 4 bits rows carry their scales along
// and nothing is rounded.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048, kCopies = 4;  // histograms of a CTA, one for every fourth warp: neighbours often meet in a bin

struct EvictArgs {
  CacheView c;
  const int32_t* length;
  float* w;
  int32_t *new_length, *kept;
  int32_t* front;    // [B][heads]: kept tokens whose numbers are below `keep`
  float* row_scale;  // 8 bits: [side][B][heads][keep] scale of each kept row as it was
  int32_t B, w_tokens, keep, recent;
};

// Larger numbers for larger weights; NaN below everything, both zeros the same.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int held(const EvictArgs& a, int b, bool report) {
  const int n = a.length[b], most = a.c.max_blocks * a.c.bt;
  if (n >= 0 && n <= most) return n;
  if (report) atomicOr(a.c.status, kStatusCache);
  return min(max(n, 0), most);
}

// A token's block, -1 (recorded) outside the cache.
__device__ __forceinline__ int block_at(const EvictArgs& a, int b, int token) {
  const int blk = a.c.table[(int64_t)b * a.c.max_blocks + token / a.c.bt];
  if (blk >= 0 && blk < a.c.n_blocks) return blk;
  atomicOr(a.c.status, kStatusCache);
  return -1;
}

// One cluster a (request, key head).
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  __shared__ uint32_t hist[kCopies][kBins];
  __shared__ uint32_t sums[kSelWarps], found[2];
  __shared__ int mine[2], front;                     // of this CTA's tokens: above the last weight, equal to it
  __shared__ int warp_above[kSelWarps], warp_equal[kSelWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / ranks, b = bh / a.c.heads, h = bh % a.c.heads;
  after_predecessor();
  const int n = held(a, b, tid == 0 && rank == 0 && h == 0);
  int32_t* kept = a.kept + (int64_t)bh * a.keep;
  if (tid == 0 && rank == 0 && h == 0) a.new_length[b] = min(n, a.keep);
  if (n <= a.keep) {  // stays as it is
    for (int i = rank * kSelThreads + tid; i < a.keep; i += ranks * kSelThreads) kept[i] = i < n ? i : -1;
    if (tid == 0 && rank == 0) a.front[bh] = 0;
    return;
  }
  const int m = n - a.recent, want = a.keep - a.recent;  // `want` of the first m
  const float* w = a.w + (int64_t)bh * a.w_tokens;
  // this CTA's tokens, this warp's among them
  const int per = (m + ranks * kSelWarps - 1) / (ranks * kSelWarps);
  const int64_t from = (int64_t)(rank * kSelWarps + warp) * per;
  const int lo = (int)min((int64_t)m, from), hi = (int)min((int64_t)m, from + per);
  uint32_t key = 0;  // what is known of the last kept weight
  int above = 0, above_mine = 0, equal_mine = 0;
  if (tid == 0) front = 0;
  if (want > 0) {
    int left = 32;  // bits not known yet
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = left - bits, bins = 1 << bits;
      for (int i = tid; i < kCopies * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
      __syncthreads();
      for (int i0 = lo; i0 < hi; i0 += 4 * 32) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i0 + 32 * j + lane < hi ? w[i0 + 32 * j + lane] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = order_key(x[j]);
          if (i0 + 32 * j + lane < hi && (pass == 0 || u >> left == key >> left))
            atomicAdd(&hist[warp % kCopies][(u >> shift) & (bins - 1)], 1u);
        }
      }
      __syncthreads();
      for (int i = tid; i < bins; i += kSelThreads) {
        uint32_t s = 0;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) s += hist[k][i];
        hist[0][i] = s;
      }
      cl.sync();
      // four bins a thread, the largest first; the bin in which the count passes what is wanted
      uint32_t t[4], s = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t[j] = 0;
        const int bin = bins - 1 - (4 * tid + j);
        if (bin >= 0)
          for (int r = 0; r < ranks; ++r) t[j] += *cl.map_shared_rank(&hist[0][bin], r);
        s += t[j];
      }
      uint32_t run = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      uint32_t before = run - s;
      for (int k = 0; k < warp; ++k) before += sums[k];
      before += (uint32_t)above;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < (uint32_t)want && before + t[j] >= (uint32_t)want) found[0] = bins - 1 - (4 * tid + j), found[1] = before;
        before += t[j];
      }
      __syncthreads();
      const uint32_t bin = found[0];
      above = (int)found[1];
      key |= bin << shift;
      left = shift;
      // this CTA's own: those in larger bins are above for good
      uint32_t over = 0;
      for (int i = (int)bin + 1 + tid; i < bins; i += kSelThreads) over += hist[0][i];
#pragma unroll
      for (int o = 16; o; o >>= 1) over += __shfl_xor_sync(0xFFFFFFFFu, over, o);
      if (lane == 0) sums[warp] = over;
      __syncthreads();
      for (int k = 0; k < kSelWarps; ++k) above_mine += (int)sums[k];
      equal_mine = (int)hist[0][bin];
      cl.sync();  // every CTA has read the histograms
    }
  }
  // kept before this CTA's tokens: all above the last weight, and of those equal to it the first ones
  if (tid == 0) mine[0] = above_mine, mine[1] = equal_mine;
  cl.sync();
  int over = 0, equal = 0;
  for (int r = 0; r < rank; ++r) {
    over += *cl.map_shared_rank(&mine[0], r);
    equal += *cl.map_shared_rank(&mine[1], r);
  }
  const int ties = want - above;  // kept of those equal
  int in_front = 0;
  if (want > 0) {
    int na = 0, ne = 0;
    for (int i0 = lo; i0 < hi; i0 += 4 * 32) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i0 + 32 * j + lane < hi ? w[i0 + 32 * j + lane] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = order_key(x[j]);
        const bool in = i0 + 32 * j + lane < hi;
        na += __popc(__ballot_sync(0xFFFFFFFFu, in && u > key));
        ne += __popc(__ballot_sync(0xFFFFFFFFu, in && u == key));
      }
    }
    if (lane == 0) warp_above[warp] = na, warp_equal[warp] = ne;
    __syncthreads();
    for (int k = 0; k < warp; ++k) over += warp_above[k], equal += warp_equal[k];
    for (int i0 = lo; i0 < hi; i0 += 4 * 32) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i0 + 32 * j + lane < hi ? w[i0 + 32 * j + lane] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j + lane;
        const uint32_t u = order_key(x[j]), ba = __ballot_sync(0xFFFFFFFFu, i < hi && u > key),
                       be = __ballot_sync(0xFFFFFFFFu, i < hi && u == key), below = (1u << lane) - 1;
        const int my_over = over + __popc(ba & below), my_equal = equal + __popc(be & below);
        if (i < hi && (u > key || (u == key && my_equal < ties))) {
          kept[my_over + min(my_equal, ties)] = i;
          in_front += i < a.keep;
        }
        over += __popc(ba);
        equal += __popc(be);
      }
    }
  }
  for (int i = rank * kSelThreads + tid; i < a.recent; i += ranks * kSelThreads) {
    kept[want + i] = m + i;
    in_front += m + i < a.keep;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) in_front += __shfl_xor_sync(0xFFFFFFFFu, in_front, o);
  __syncthreads();
  if (lane == 0 && in_front) atomicAdd(&front, in_front);
  cl.sync();
  if (rank == 0 && tid == 0) {
    int all = 0;
    for (int r = 0; r < ranks; ++r) all += *cl.map_shared_rank(&front, r);
    a.front[bh] = all;
  }
  cl.sync();  // nobody leaves while its shared memory is read
}

// 8 bits: the scale of every kept row as it was, before blocks get new ones.
__global__ void __launch_bounds__(256) k_evict_scales(const __grid_constant__ EvictArgs a) {
  after_predecessor();
  const int bh = blockIdx.y, b = bh / a.c.heads, h = bh % a.c.heads;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.keep || held(a, b, false) <= a.keep) return;
  const int blk = block_at(a, b, a.kept[(int64_t)bh * a.keep + i]);
  const int64_t at = (int64_t)bh * a.keep + i, side = (int64_t)a.B * a.c.heads * a.keep;
  a.row_scale[at] = blk < 0 ? 0.f : a.c.ks[(int64_t)blk * a.c.heads + h];
  a.row_scale[side + at] = blk < 0 ? 0.f : a.c.vs[(int64_t)blk * a.c.heads + h];
}

constexpr int kMoveThreads = 256, kUnits = 4;  // 16-byte units a thread and batch

// What a CTA moves: units [first, first + count) of 16 bytes of each row of
// codes; or the scale bytes of 4-bit codes, in units of two; or the weights.
struct Part {
  int kind, side, first, count;  // kind 0: codes, 1: scale bytes, 2: weights
};

template <int D, int FMT>
struct MoveShape {
  static constexpr bool k4 = FMT == ZG_KV_E2M1;
  static constexpr int kRow = k4 ? Row4<D>::kCodes : D;
  static constexpr int kRowUnits = kRow / 16;
  static constexpr int kSplit = kRowUnits % 2 == 0 ? kRowUnits / 2 : 1;  // CTAs over a row's columns: sectors of 32 bytes
  static constexpr int kParts = 2 * kSplit + (k4 ? 2 : 0) + 1;
  static __device__ __forceinline__ Part part(int p) {
    if (p < 2 * kSplit) return {0, p / kSplit, p % kSplit * (kRowUnits / kSplit), kRowUnits / kSplit};
    if (k4 && p < 2 * kSplit + 2) return {1, p - 2 * kSplit, 0, D / 32};
    return {2, 0, 0, 1};
  }
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

// LATE false: rows whose sources lie in the first `keep` places, in order, one
// CTA a part.  LATE true: the others, a batch a CTA.
template <int D, int FMT, bool LATE>
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const __grid_constant__ EvictArgs a) {
  using Sh = MoveShape<D, FMT>;
  __shared__ float block_scale[2][kUnits * kMoveThreads / 16];  // 8 bits: new scales of the batch's blocks
  after_predecessor();
  const int bh = blockIdx.z, b = bh / a.c.heads, h = bh % a.c.heads, tid = threadIdx.x;
  const Part p = Sh::part(blockIdx.y);
  if (held(a, b, false) <= a.keep) return;
  const int front = a.front[bh], bt = a.c.bt;
  // rows of a batch: whole blocks, all its units in the threads' registers
  const int rows = max(kUnits * kMoveThreads / p.count / 128 * 128, 128);
  const int first = LATE ? front / rows + (int)blockIdx.x : 0;
  const int last = LATE ? first + 1 : (front + rows - 1) / rows;  // batches
  if (first * (int64_t)rows >= a.keep) return;
  const int32_t* kept = a.kept + (int64_t)bh * a.keep;
  const float* row_scale = a.row_scale + ((int64_t)p.side * a.B * a.c.heads + bh) * a.keep;
  uint8_t* codes = p.side ? a.c.vc : a.c.kc;
  float* scales = p.side ? a.c.vs : a.c.ks;
  float* w = a.w + (int64_t)bh * a.w_tokens;

  struct Batch {
    uint4 x[kUnits];
    float s[kUnits];
  };
  // unit u of a batch: row u / count, its place in the row first + u % count.  The rows' columns of 16 bytes and the
  // two narrow kinds share the registers.
  auto mine = [&](int batch, int k, int& row, int& col) -> bool {
    const int u = tid + k * kMoveThreads;
    row = batch * rows + u / p.count;
    col = p.first + u % p.count;
    return u < rows * p.count && row < a.keep && (LATE ? row >= front : row < front);
  };
  auto load = [&](int batch, Batch& x) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int row, col;
      x.x[k] = make_uint4(0, 0, 0, 0);
      x.s[k] = 0.f;
      if (batch >= last || !mine(batch, k, row, col)) continue;
      const int from = kept[row];
      if (p.kind == 2) {
        x.x[k].x = __float_as_uint(w[from]);
        continue;
      }
      const int blk = block_at(a, b, from);
      if (blk < 0) continue;  // zeros
      const int64_t at = ((int64_t)blk * a.c.heads + h) * bt + from % bt;
      if (p.kind == 1) {
        x.x[k].x = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(scales) + at * Row4<D>::kScales)[col];
      } else {
        x.x[k] = reinterpret_cast<const uint4*>(codes + at * Sh::kRow)[col];
        if constexpr (!Sh::k4) x.s[k] = row_scale[row];
      }
    }
  };
  // 8 bits: the new scales of the batch's blocks, the largest of their rows'
  auto new_scales = [&](int batch, int buf) {
    if constexpr (!Sh::k4) {
      if (p.kind) return;
      const int per = rows / bt;
      for (int j = tid >> 5; j < per; j += kMoveThreads / 32) {
        float s = 0.f;
        for (int r = tid & 31; r < bt; r += 32) {
          const int row = batch * rows + j * bt + r;
          if (row < a.keep) s = fmaxf(s, row_scale[row]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        if ((tid & 31) == 0) block_scale[buf][j] = s;
      }
    }
  };
  auto store = [&](int batch, int buf, const Batch& x) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int row, col;
      if (!mine(batch, k, row, col)) continue;
      if (p.kind == 2) {
        w[row] = __uint_as_float(x.x[k].x);
        continue;
      }
      const int blk = block_at(a, b, row);
      if (blk < 0) continue;
      const int64_t bhb = (int64_t)blk * a.c.heads + h, at = bhb * bt + row % bt;
      if (p.kind == 1) {
        reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(scales) + at * Row4<D>::kScales)[col] = (uint16_t)x.x[k].x;
        continue;
      }
      uint4 y = x.x[k];
      if constexpr (!Sh::k4) {
        const float s1 = block_scale[buf][(row - batch * rows) / bt];
        if (x.s[k] != s1) {
          const float inv = s1 > 0.f ? __frcp_rn(s1) : 0.f;
          constexpr bool INT8 = FMT == ZG_KV_INT8;
          y = make_uint4(code_again<INT8>(y.x, x.s[k], inv), code_again<INT8>(y.y, x.s[k], inv),
                         code_again<INT8>(y.z, x.s[k], inv), code_again<INT8>(y.w, x.s[k], inv));
        }
        if (col == 0) scales[bhb] = s1;  // the first column's CTA; its rows write the same
      }
      reinterpret_cast<uint4*>(codes + at * Sh::kRow)[col] = y;
    }
  };
  Batch x[2];
  load(first, x[0]);
  if (!LATE && last <= first) return;
  for (int i = first, buf = 0; i < last; ++i, buf ^= 1) {
    // the next batch is read before this one is written: their sources lie behind what is written before
    if (!LATE) load(i + 1, x[1]);
    new_scales(i, buf);
    __syncthreads();
    store(i, buf, x[0]);
    if (!LATE) x[0] = x[1];
  }
}

}  // namespace
}  // namespace zg

using namespace zg;

namespace {

// Rows' scales (8 bits), and a count a (request, key head).
size_t evict_bytes(const zg_kv_cache* c, int64_t B, int64_t keep) {
  const int64_t heads = B * c->heads;
  return (size_t)((c->format == ZG_KV_E2M1 ? 0 : 2 * heads * keep) + heads) * 4;
}

zg_status check_evict(const zg_kv_cache* c, int32_t B, int32_t keep, const char* call) {
  if (B < 0 || keep < 1) return bad_arg(call, "B must be >= 0 and keep >= 1");
  if ((int64_t)B * c->heads > 65535) return fail(ZG_ERR_UNSUPPORTED, std::string(call) + ": more than 65,535 (request, key head)s");
  if (keep > 0x40000000) return fail(ZG_ERR_UNSUPPORTED, std::string(call) + ": keep above 2^30");
  return ZG_OK;
}

}  // namespace

extern "C" {

zg_status zg_kv_evict_workspace_size(const zg_kv_cache* cache, int32_t B, int32_t keep, size_t* bytes) try {
  const char* call = "zg_kv_evict_workspace_size";
  static const int32_t no_table = 0;
  zg_status st;
  if (!bytes) return bad_arg(call, "bytes is NULL");
  if ((st = check_cache(cache, &no_table, 1, call)) != ZG_OK) return st;
  if ((st = check_evict(cache, B, keep, call)) != ZG_OK) return st;
  *bytes = evict_bytes(cache, B, keep);
  return ZG_OK;
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

zg_status zg_kv_evict(const zg_kv_cache* cache, const int32_t* table, int32_t max_blocks, const int32_t* length,
                      float* weights, int32_t w_tokens, int32_t keep, int32_t recent, int32_t* new_length, int32_t* kept,
                      int32_t B, void* workspace, size_t ws_bytes, void* stream) try {
  const char* call = "zg_kv_evict";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if ((st = check_evict(cache, B, keep, call)) != ZG_OK) return st;
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
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < evict_bytes(cache, B, keep))
    return bad_arg(call, "workspace must hold zg_kv_evict_workspace_size bytes, 256-byte aligned");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  const int bhs = B * cache->heads;
  EvictArgs a = {};
  a.c = {static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->v_codes), cache->k_scale, cache->v_scale,
         cache->n_blocks, cache->heads, cache->block_tokens, max_blocks, table, status};
  a.length = length;
  a.w = weights;
  a.new_length = new_length;
  a.kept = kept;
  a.front = static_cast<int32_t*>(workspace);
  a.row_scale = static_cast<float*>(workspace) + bhs;
  a.B = B;
  a.w_tokens = w_tokens;
  a.keep = keep;
  a.recent = recent;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);

  // a cluster for every head, as large as leaves every SM a CTA, with 1,024 tokens for each at least
  int ranks = 1;
  while (ranks < 8 && bhs * ranks * 2 <= 2 * sm_count() && tokens / (2 * ranks) >= 1024) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(bhs * ranks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = sm;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t err = cudaLaunchKernelEx(&cfg, k_evict_select, a);
  if (err == cudaSuccess && cache->format != ZG_KV_E2M1)
    err = launch_early(k_evict_scales, dim3((keep + 255) / 256, bhs), 256, 0, sm, a);
  for_dim(cache->dim, [&](auto dv) {
    for_format(cache->format, [&](auto fv) {
      constexpr int D = decltype(dv)::value, FMT = decltype(fv)::value;
      using Sh = MoveShape<D, FMT>;
      if (err == cudaSuccess) err = launch_early(k_evict_move<D, FMT, false>, dim3(1, Sh::kParts, bhs), kMoveThreads, 0, sm, a);
      // batches of the part with the smallest ones, and one more since the first may begin inside one
      const int most = std::max(Sh::kRowUnits / Sh::kSplit, D / 32);
      const int rows = std::max(kUnits * kMoveThreads / most / 128 * 128, 128);
      if (err == cudaSuccess)
        err = launch_early(k_evict_move<D, FMT, true>, dim3((keep + rows - 1) / rows + 1, Sh::kParts, bhs), kMoveThreads, 0, sm, a);
    });
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "cache eviction launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

}  // extern "C"
