// Attention over whole prompts: packed sequences of different lengths, each
// row over its own sequence, causal or not, on the 5th-generation tensor cores.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q . k_j)
//
// One CTA takes up to 128 query rows (token, query head of the group) of one
// sequence and key head through 128 keys a step:
//   one warp    brings keys and values in by TMA, as they lie in memory;
//   one warp    issues S = Q K^T and O += P V (tcgen05, one thread);
//   four warps  one thread a row: scores out of tensor memory, running
//               maximum, p = exp2, rounded to the rows' type back to tensor
//               memory, in halves of 64 keys so that the product starts early;
//   two warps   look over the values of tiles that some row does not see whole.
// Two CTAs share an SM, each with half of its tensor memory, and fill one
// another's waits, beginnings and ends (one CTA with two tiles an SM: 8 x 4,000
// rows of 8 heads over 2 take 181 us against 164 at 64 dims, 239 against 228 at
// 128).  Up to 64 dims P has columns of its own, beyond it lies over S.  The
// rows of a group's heads share the keys.
//
// A weight of 0 times an infinity or a NaN would be a NaN, so values that a row
// does not see must not meet it: rows of the tile behind the sequence are made
// zero, and so are rows inside it that hold something not finite, where not all
// rows of the CTA see them; what those give the rows that do see them is added
// at the end, from memory, a key and a row at a time: with no finite value at
// all a causal call takes up to some 200 times as long (4,000 rows, 16 heads over
// 4 of 128: 59 us and 11.7 ms).
//
// Measured: four sequences of up to 11,000 rows (16 heads over 4 of 128, bf16,
// causal, 1.14 TFLOP) 804 to 822 us, 1.4 PFLOP/s or 72 % of the measured rate,
// bound by the chain scores -> softmax -> product of a step (1.8 us a CTA, two
// CTAs an SM, of which the tensor cores need 0.65 for each); 64 of up to 500
// rows (8 heads over 2 of 64, f16) 41 us, bound by the beginnings and ends of
// CTAs of some 8 us (queries 1.3, a step 1.1, rows out 1.2, the rest the item's
// search and the first keys).  A version of CTAs that stay and take items in
// turn (the next one's queries and keys fetched ahead) took 45 us, and 920 for
// the long ones; it spilled registers and had a ring of two entries.
// Not causal the same take 1,565 us (1.46 PFLOP/s) and 45.
//
// Every wait is bounded; on expiry kStatusTimeout is recorded, what was issued
// is drained, tensor memory is freed and the kernel returns.
#include <cmath>

#include <cuda.h>

#include "tc.cuh"

namespace zg {
namespace {

constexpr int kNK = 128, kItem = 128;  // keys a step, query rows a CTA
constexpr int kMmaWarp = 4, kLoadWarp = 5, kFixWarps = 2, kThreads = 256;
// Registers a thread: 128 at launch, 256 threads; 128 x 200 + 128 x 56 = 256 x 128.
constexpr int kSoftRegs = 200, kOtherRegs = 56;
constexpr uint32_t kSpin = 1u << 20;
constexpr uint32_t kColumns = 256;  // of tensor memory
constexpr int kEdges = 4;           // tiles of an item that not all its rows see whole: two at most
// Sequences whose tiles each CTA counts, at most, so that those with the most keys begin first.  Of more the item is looked
// up by its place (128 sequences of 20 to 300 rows, 8 heads over 2 of 64: 38.9 us counted, 41.8 looked up; 512: 158 both).
constexpr int kCounted = 128;

template <int D>
struct PromptShape {
  static constexpr bool kApart = D <= 64;       // P beside S
  static constexpr int kSub = (D + 63) / 64;    // 64-dim subtiles (128-byte rows)
  static constexpr int kTile = kSub * 128 * 128;
  static constexpr int kRing = kApart ? 5 : 2;  // entries, each the keys or values of a step
  static constexpr size_t kSmem = (1 + kRing) * kTile + 1024;
  static constexpr uint32_t kP = kApart ? kNK : 0, kO = kColumns - D;  // S in front
  static_assert((kApart ? kNK + 64 : kNK) <= kO, "S, P and O fit");
  static_assert(kSmem <= 111 * 1024, "with the barriers inside 227 KiB an SM");
  // Ring entries in the order of their use.  Apart: keys 0, keys 1, values 0, keys 2, values 1, ..., one entry for
  // the keys behind the last step empty.  Else: keys 0, values 0, keys 1, ...
  static __device__ __forceinline__ int entries(int steps) { return kApart && steps ? 2 * steps + 1 : 2 * steps; }
  static __device__ __forceinline__ int keys(int t) { return kApart ? (t ? 2 * t - 1 : 0) : 2 * t; }
  static __device__ __forceinline__ int values(int t) { return kApart ? 2 * t + 2 : 2 * t + 1; }
  static __device__ __forceinline__ int side(int n) { return kApart ? (n > 0 && !(n & 1)) : n & 1; }
  static __device__ __forceinline__ int step(int n) { return kApart ? (n & 1 ? (n + 1) / 2 : n ? n / 2 - 1 : 0) : n / 2; }
};

struct PromptArgs {
  const int32_t* starts;
  float* lse;
  uint32_t* status;
  int32_t B, T_, Hq, Hk, G, causal;
  float scale;  // scale * log2(e)
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Whether a pair of elements holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  constexpr uint32_t m = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  return (w & m) == m || (w & (m << 16)) == (m << 16);
}

// A sequence's rows, held inside what there is.
struct Seq {
  int first, n;
};
__device__ __forceinline__ Seq seq_of(const PromptArgs& a, int b, bool report) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  Seq s;
  s.first = min(max(s0, 0), a.T_);
  s.n = min(max(s1, s.first), a.T_) - s.first;
  if (report && (s.first != s0 || s.first + s.n != s1)) atomicOr(a.status, kStatusCache);
  return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
    k_prompt(const __grid_constant__ PromptArgs a, const Rows<T> q, const Rows<T> k, const Rows<T> v, const Rows<T> out,
             const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, uint32_t spin) {
  using Sh = PromptShape<D>;
  constexpr int kRing = Sh::kRing;
  constexpr uint32_t kBf16 = std::is_same<T, __half>::value ? 0u : 1u;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;               // the query tile
  uint8_t* ring = sq + Sh::kTile;  // keys and values
  // The barriers of the scores have one phase a step, and none is passed twice before all who wait for it have seen
  // it; the fixing warps pass every entry of the ring too, so that none of its barriers leaves them behind.
  __shared__ uint64_t full[kRing], empty[kRing];
  __shared__ uint64_t q_full, s_full, s_free, p_full[2], o_done, fixed[kEdges], drained;
  __shared__ uint32_t s_bad[kEdges][4];  // keys of an edge tile whose values are not finite
  __shared__ int2 s_item;  // sequence, tile of rows
  __shared__ uint32_t tmem_base;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1 + kFixWarps);
    }
    bar_init(&s_full, 1);
    bar_init(&s_free, 4);
    bar_init(&p_full[0], 4);
    bar_init(&p_full[1], 4);
    bar_init(&o_done, 1);
    for (int i = 0; i < kEdges; ++i) bar_init(&fixed[i], kFixWarps);
    bar_init(&q_full, 4);
    bar_init(&drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  after_predecessor();
  if (warp == kMmaWarp) {  // only now: a CTA of the predecessor that waits for tensor memory must not wait for this one
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // CTAs start in the order of their numbers.  One warp looks for this one's item.
  const int p = blockIdx.x / a.Hk, h = blockIdx.x % a.Hk;
  auto tiles_of = [&](int b, bool report) -> int {
    const Seq s = seq_of(a, b, report);
    return (int)(((int64_t)s.n * a.G + kItem - 1) / kItem);
  };
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kThreads) tiles_of(b, true);
  if (warp == 0) {
    if (lane == 0) s_item = make_int2(-1, 0);
    __syncwarp();
    if (a.B <= kCounted) {
      // Those with the most keys before them first.  Item p is the (p - F(m + 1))-th of the sequences with more than m
      // tiles, where F(x) counts the tiles of numbers x and on, and m is the largest with F(m) > p.
      int held[kCounted / 32];  // of sequences lane, lane + 32, ...
#pragma unroll
      for (int j = 0; j < kCounted / 32; ++j) held[j] = lane + 32 * j < a.B ? tiles_of(lane + 32 * j, false) : 0;
      auto count = [&](int x) -> int {  // F(x)
        int c = 0;
#pragma unroll
        for (int j = 0; j < kCounted / 32; ++j) c += max(0, held[j] - x);
        return __reduce_add_sync(0xFFFFFFFFu, c);
      };
      if (count(0) > p) {
        int most = 0;
#pragma unroll
        for (int j = 0; j < kCounted / 32; ++j) most = max(most, held[j]);
        int lo = 0, hi = __reduce_max_sync(0xFFFFFFFFu, most), f_hi = 0;  // F(lo) > p >= F(hi)
#pragma unroll 1
        while (hi - lo > 1) {
          const int mid = lo + (hi - lo) / 2, f = count(mid);
          if (f > p) lo = mid;
          else hi = mid, f_hi = f;
        }
        int rank = p - f_hi;  // among the sequences with more than `lo` tiles
#pragma unroll
        for (int j = 0; j < kCounted / 32; ++j) {
          const uint32_t has = __ballot_sync(0xFFFFFFFFu, held[j] > lo);
          if (((has >> lane) & 1) && __popc(has & ((1u << lane) - 1)) == rank) s_item = make_int2(32 * j + lane, lo);
          rank -= __popc(has);
        }
      }
    } else {
      // Numbers from the last sequence's end to the first's beginning: sequence b has those from first * G / 128 +
      // min(b, first) on, `first` its first row.  They do not fall, and there is room for its tiles before those of
      // b + 1: floor((first + n) G / 128) - floor(first G / 128) + 1 is n G / 128 rounded up at least.
      const int n = (int)(gridDim.x / a.Hk) - 1 - p;
      auto number = [&](int b) -> int64_t {
        const int first = seq_of(a, b, false).first;
        return (int64_t)first * a.G / kItem + min(b, first);
      };
      int lo = 0, hi = a.B, below = 1;  // number(lo) <= n < number(hi): thirty-two ways at a time
#pragma unroll 1
      while (hi - lo > 1 && below) {
        const int step = (hi - lo - 1) / 32 + 1, at = min(lo + (int64_t)lane * step, (int64_t)hi);
        below = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && number(at) <= n));
        hi = (int)min((int64_t)hi, lo + (int64_t)below * step);
        lo += max(below - 1, 0) * step;
      }
      if (below && lane == 0) {
        const int64_t m = n - number(lo);
        if (m >= 0 && m < tiles_of(lo, false)) s_item = make_int2(lo, (int)m);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  auto give_up = [&]() { atomicOr(a.status, kStatusTimeout); };
  const int b = s_item.x, m = s_item.y;
  const Seq s = b < 0 ? Seq{0, 0} : seq_of(a, b, false);  // fewer items than CTAs: nothing to do
  const int row0 = m * kItem, mine = min((int)min((int64_t)s.n * a.G, (int64_t)0x7FFFFFFF) - row0, kItem);  // query rows
  auto sees = [&](int row) -> int { return a.causal ? row / a.G + 1 : s.n; };
  const int steps = __shfl_sync(0xFFFFFFFFu, mine > 0 ? (sees(row0 + mine - 1) + kNK - 1) / kNK : 0, 0);
  const int edge = sees(row0) / kNK;  // the first tile that not all rows see whole

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
      // ----------------------------------------------------------- products
      const uint32_t types = (kBf16 << 7) | (kBf16 << 10);
      const uint32_t id_s = (1u << 4) | types | ((uint32_t)(kNK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | types | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint64_t q0 = desc_k(smem_u32(sq)), k0 = desc_k(smem_u32(ring)), v0 = desc_mn(smem_u32(ring), kNK * 128);
      auto scores = [&](int t) -> bool {
        const int n = Sh::keys(t), ws = n % kRing;
        if (!spin_wait(&full[ws], (n / kRing) & 1, spin)) return false;
        // apart: every warp has the last scores in registers; else the product that reads P in their place is over
        if (t > 0 && !spin_wait(Sh::kApart ? &s_free : &o_done, (t - 1) & 1, spin)) return false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t kd = k0 + ws * (Sh::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = (c / 4) * (128 * 128 >> 4) + (c % 4) * 2;
            mma_ss(tmem, q0 + off, kd + off, id_s, c > 0);
          }
          commit(&s_full);
          commit(&empty[ws]);
        }
        __syncwarp();
        return true;
      };
      auto values = [&](int t) -> bool {
        const int n = Sh::values(t), ws = n % kRing;
        if (!spin_wait(&full[ws], (n / kRing) & 1, spin)) return false;
        if (t >= edge && !spin_wait(&fixed[t - edge], 0, spin)) return false;
        const uint64_t vd = v0 + ws * (Sh::kTile >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!spin_wait(&p_full[half], t & 1, spin)) return false;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
#pragma unroll
            for (int j = half * 4; j < half * 4 + 4; ++j)
              mma_ts(tmem + Sh::kO, tmem + Sh::kP + (uint32_t)(j * 8), vd + j * (2048 >> 4), id_o, (t > 0 || j > 0) ? 1u : 0u);
            if (half) {
              commit(&o_done);
              commit(&empty[ws]);
            }
          }
          __syncwarp();
        }
        return true;
      };
      bool good = spin_wait(&q_full, 0, spin) && (steps == 0 || scores(0));
      for (int t = 0; t < steps && good; ++t) {
        const bool more = t + 1 < steps;
        if constexpr (Sh::kApart) good = (!more || scores(t + 1)) && values(t);
        else good = values(t) && (!more || scores(t + 1));
      }
      if (!good && lane == 0) give_up();
      if (elect_one()) commit(&drained);
      __syncwarp();
      if (!spin_wait(&drained, 0, kSpin) && lane == 0) give_up();
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------- keys and values
      int issued = 0;
      bool good = true;
      for (int n = 0; n < Sh::entries(steps); ++n) {
        const int ws = n % kRing, t = Sh::step(n), side = Sh::side(n);
        if (n >= kRing && !warp_wait(&empty[ws], ((n / kRing) - 1) & 1, spin)) {
          good = false;
          break;
        }
        if (elect_one()) {
          const uint32_t bytes = t < steps ? (uint32_t)Sh::kTile : 0;  // the keys behind the last step: none
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&full[ws])), "r"(bytes)
                       : "memory");
          if (t < steps)
#pragma unroll
            for (int c = 0; c < Sh::kSub; ++c)
              tma_load_3d(ring + ws * Sh::kTile + c * (128 * 128), side ? &map_v : &map_k, &full[ws], 64 * c, h,
                          s.first + t * kNK);
        }
        __syncwarp();
        issued = n + 1;
      }
      if (!good && lane == 0) give_up();
      // every copy has landed before the CTA may end
      for (int n = max(0, issued - kRing); n < issued; ++n)
        if (!warp_wait(&full[n % kRing], (n / kRing) & 1, kSpin) && lane == 0) give_up();
    } else {
      // -------------------------------------------- values of the edge tiles
      const int w = warp - kLoadWarp - 1;
      for (int n = 0; n < Sh::entries(steps); ++n) {
        const int ws = n % kRing, t = Sh::step(n);
        if (!warp_wait(&full[ws], (n / kRing) & 1, spin)) {
          if (lane == 0) give_up();
          break;
        }
        if (Sh::side(n) && t >= edge) {
          uint8_t* tile = ring + ws * Sh::kTile;
          for (int r0 = 32 * w; r0 < kNK; r0 += 32 * kFixWarps) {
            const int r = r0 + lane, key = t * kNK + r;
            uint8_t* row = tile + r * 128;
            bool zero = key >= s.n;
            if (a.causal && !zero) {
#pragma unroll 4
              for (int c = 0; c < D / 8; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(row + c / 8 * (128 * 128) + (((c % 8) ^ (r & 7)) << 4));
                zero |= not_finite2<T>(x.x) || not_finite2<T>(x.y) || not_finite2<T>(x.z) || not_finite2<T>(x.w);
              }
            }
            const uint32_t bad = __ballot_sync(0xFFFFFFFFu, zero && key < s.n);
            if (zero)
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(row + c / 8 * (128 * 128) + (((c % 8) ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            if (lane == 0) s_bad[t - edge][r0 / 32] = bad;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(&fixed[t - edge]);
        }
        if (lane == 0) bar_arrive(&empty[ws]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // -------------------------------------------------------------- softmax
    const int r = threadIdx.x, ri = row0 + r;  // row of the tile, of the sequence
    const bool live = (int)threadIdx.x < mine;
    const int token = live ? ri / a.G : 0, qh = h * a.G + (live ? ri % a.G : 0);
    const int vis = live ? sees(ri) : 0;
    // lanes of a row when a warp moves its 32 rows: four elements each, kAt rows at a time
    constexpr int kLanes = D / 4, kSlot = D == 96 ? 32 : kLanes, kAt = 32 / kSlot;
    const int l4 = lane % kSlot, e = 4 * l4;
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, live);
    {
      // the warp's 32 rows into its query tile: a group of lanes a row, four elements a lane; where a row is comes from
      // the lane that it belongs to
      const int64_t q_row = (int64_t)(s.first + token) * q.st + qh * q.sh;
      uint8_t* tile = sq + (e / 64) * (128 * 128) + (e & 4) * 2;
      uint2 w[32 / kAt];  // every load in flight before the first is used
#pragma unroll
      for (int c = 0; c < 32 / kAt; ++c) {
        const int rw = c * kAt + lane / kSlot;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, q_row, rw);
        w[c] = make_uint2(0, 0);
        if (((some >> rw) & 1) && l4 < kLanes) w[c] = *reinterpret_cast<const uint2*>(q.data + at + e);
      }
#pragma unroll
      for (int c = 0; c < 32 / kAt; ++c) {
        const int rr = warp * 32 + c * kAt + lane / kSlot;  // row of the tile
        if (l4 < kLanes) *reinterpret_cast<uint2*>(tile + rr * 128 + ((((e % 64) / 8) ^ (rr & 7)) << 4)) = w[c];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&q_full);
    }
    const uint32_t s_at = tmem + ((uint32_t)(warp * 32) << 16), p_at = s_at + Sh::kP, o_at = s_at + Sh::kO;
    const float f = a.scale;
    float mx = -INFINITY, l = 0.f;
    bool good = true;
    for (int t = 0; t < steps; ++t) {
      if (!warp_wait(&s_full, t & 1, spin)) {
        good = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      uint32_t sr[kNK];
      tmem_load128(s_at, sr);
      if constexpr (Sh::kApart) {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&s_free);
      }
      float* z = reinterpret_cast<float*>(sr);
      const int left = vis - t * kNK;  // keys of this step that the row sees
      if (__any_sync(0xFFFFFFFFu, left < kNK)) {
#pragma unroll
        for (int j = 0; j < kNK; ++j) z[j] = j < left ? z[j] : -INFINITY;
      }
      float g[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        g[c] = max3(z[32 * c], z[32 * c + 1], z[32 * c + 2]);
#pragma unroll
        for (int j = 3; j + 1 < 32; j += 2) g[c] = max3(g[c], z[32 * c + j], z[32 * c + j + 1]);
        g[c] = fmaxf(g[c], z[32 * c + 31]);
      }
      const float tm = fmaxf(max3(g[0], g[1], g[2]), g[3]) * f;
      float al = 1.f;
      const bool move = __any_sync(0xFFFFFFFFu, tm > mx + 8.f);
      if (move) {
        const float nm = fmaxf(mx, tm);
        if (nm != mx) {
          al = exp2_fast(mx - nm);
          l *= al;
        }
        mx = nm;
      }
      const float mu = mx == -INFINITY ? 0.f : mx;
      // A score enters the exponent unrounded and mu rounded, so that a row's weights are off by a common factor, up to
      // 2^(ulp(mu)); from 2^26 on that could leave a half's range, and scores are taken times a power of two that keeps
      // it within 2^4.  There scores that differ by their last bit lie 8 apart or more.
      const int far = (int)((__float_as_uint(mu) >> 23) & 0xFF) - (127 + 25);
      const float down = power_of_2(-max(far, 0)), fd = f * down, md = -mu * down;
      // the product of the last step has read its probabilities, and is in the sums (with P over S the scores have
      // waited for it)
      if (Sh::kApart && t > 0) {
        if (!warp_wait(&o_done, (t - 1) & 1, spin)) {
          good = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      if (move && t > 0) {
#pragma unroll
        for (int d = 0; d < D; d += 16) {  // few at a time: the scores stay in registers
          uint32_t o[16];
          tmem_load16(o_at + d, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
          tmem_store16(o_at + d, o);
        }
      }
      const uint64_t f2 = pair(fd, fd), m2 = pair(md, md);
      uint64_t sum[2] = {0, 0};  // 0.f, 0.f
#pragma unroll
      for (int c = 0; c < kNK / 32; ++c) {
        uint32_t pr[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float x0, x1;
          unpair(fma2(pair(z[32 * c + 2 * j], z[32 * c + 2 * j + 1]), f2, m2), x0, x1);
          const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
          sum[j & 1] = add2(sum[j & 1], pair(p0, p1));
          pr[j] = pack2<T>(p0, p1);
        }
        tmem_store16(p_at + 16 * c, pr);
        if (c & 1) {
          tmem_store_wait();
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(&p_full[c >> 1]);
        }
      }
      float s0, s1;
      unpair(add2(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
    }
    if (good && steps > 0) good = warp_wait(&o_done, (steps - 1) & 1, spin);
    // what the fixing warps have left out
    bool bad = false;
    if (a.causal && good)
      for (int t = edge; t < steps; ++t) {
        good = good && warp_wait(&fixed[t - edge], 0, spin);
        for (int w = 0; w < 4 && good; ++w) bad |= s_bad[t - edge][w] != 0;
      }
    if (!good && lane == 0) give_up();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (good && steps > 0) {
      const float inv = 1.f / l;
      uint8_t* tile = sq;  // every product that reads the queries is complete
#pragma unroll
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        tmem_load(o_at + d, o);
        float* x = reinterpret_cast<float*>(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] *= inv;
        if (bad) {  // of all lanes or none
          if (live) {
            for (int t = edge; t < steps; ++t)
              for (int key = t * kNK; key < min((t + 1) * kNK, vis); ++key) {
                if (!((s_bad[t - edge][(key % kNK) / 32] >> (key % 32)) & 1)) continue;
                const T* qr = q.data + (int64_t)(s.first + token) * q.st + qh * q.sh;
                const T* kr = k.data + (int64_t)(s.first + key) * k.st + h * k.sh;
                const T* vr = v.data + (int64_t)(s.first + key) * v.st + h * v.sh + d;
                float z = 0.f;
                for (int c = 0; c < D; ++c) z = fmaf((float)qr[c], (float)kr[c], z);
                const float pw = exp2_fast(fmaf(z, f, -mx)) * inv;
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = fmaf(pw, (float)vr[j], x[j]);
              }
          }
          __syncwarp();  // lanes see different numbers of keys, and the next load of tensor memory takes the whole warp
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          *reinterpret_cast<uint4*>(tile + ((d + j) / 64) * (128 * 128) + r * 128 + (((((d + j) % 64) / 8) ^ (r & 7)) << 4)) =
              make_uint4(pack2<T>(x[j], x[j + 1]), pack2<T>(x[j + 2], x[j + 3]), pack2<T>(x[j + 4], x[j + 5]),
                         pack2<T>(x[j + 6], x[j + 7]));
      }
      // whole rows out, as the queries came in
      const int64_t out_row = (int64_t)(s.first + token) * out.st + qh * out.sh;
      __syncwarp();
#pragma unroll 8
      for (int c = 0; c < 32 / kAt; ++c) {
        const int rw = c * kAt + lane / kSlot, rr = warp * 32 + rw;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, out_row, rw);
        if (((some >> rw) & 1) && l4 < kLanes)
          *reinterpret_cast<uint2*>(out.data + at + e) = *reinterpret_cast<const uint2*>(
              tile + (e / 64) * (128 * 128) + rr * 128 + ((((e % 64) / 8) ^ (rr & 7)) << 4) + (e & 4) * 2);
      }
      if (live && a.lse) a.lse[(int64_t)(s.first + token) * a.Hq + qh] = (mx + log2f(l)) * 0.693147180559945f;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns) : "memory");
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r);
    return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

// Rows [tokens][heads][dim], boxes of 128 tokens of one head and 64 dims (zeros behind the dims and the tokens),
// 128-byte swizzle.
bool make_map(CUtensorMap* m, const zg_rows* r, int dim, int heads, int tokens) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)r->stride_h * 2, (cuuint64_t)r->stride_t * 2};
  const cuuint32_t box[3] = {64, 1, kNK}, step[3] = {1, 1, 1};
  return fn(m, r->dtype == ZG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, r->data, dims,
            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" zg_status zg_prompt_attention(const zg_rows* q, const zg_rows* k, const zg_rows* v, const zg_rows* out,
                                         float* lse, const int32_t* starts, int32_t B, int32_t T, int32_t Hq, int32_t Hk,
                                         int32_t dim, float scale, int32_t causal, void* stream) try {
  const char* call = "zg_prompt_attention";
  zg_status st;
  if (dim != 32 && dim != 64 && dim != 96 && dim != 128)
    return fail(ZG_ERR_UNSUPPORTED, "zg_prompt_attention: dim must be 32, 64, 96 or 128");
  if (B < 0 || T < 0) return bad_arg(call, "B and T must be >= 0");
  if (Hk < 1 || Hq < 1 || Hq > 1024 || Hq % Hk) return bad_arg(call, "Hq must be a multiple of Hk, at most 1024");
  if ((int64_t)T >= 0x80000000LL / Hq) return bad_arg(call, "T * Hq must be below 2^31");
  if (!(scale > 0.f && std::isfinite(scale))) return bad_arg(call, "scale must be finite and > 0");
  if (B == 0 || T == 0) return ZG_OK;
  if ((st = check_rows(q, "q", -1, call)) != ZG_OK) return st;
  if (q->dtype == ZG_F32) return fail(ZG_ERR_UNSUPPORTED, "zg_prompt_attention: q must be ZG_BF16 or ZG_F16");
  if ((st = check_rows(k, "k", q->dtype, call)) != ZG_OK || (st = check_rows(v, "v", q->dtype, call)) != ZG_OK ||
      (st = check_rows(out, "out", q->dtype, call)) != ZG_OK)
    return st;
  for (const zg_rows* r : {k, v}) {
    if (reinterpret_cast<uintptr_t>(r->data) % 16 || r->stride_t % 8 || (Hk > 1 && r->stride_h % 8))
      return bad_arg(call, "k and v must be 16-byte aligned, their strides multiples of 8");
  }
  if (!starts || reinterpret_cast<uintptr_t>(starts) % 4) return bad_arg(call, "starts is NULL or not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(lse) % 4) return bad_arg(call, "lse must be 4-byte aligned");
  // items of 128 rows at most: a part-filled one a sequence beside the full ones
  const int64_t G = Hq / Hk, items = (int64_t)T * G / kItem + std::min<int64_t>(B, (int64_t)T);
  if (items * Hk > 0x7FFFFFFF || (int64_t)B > 0x7FFFFFFF - kThreads)
    return fail(ZG_ERR_UNSUPPORTED, "zg_prompt_attention: more than 2^31 CTAs");
  zg_rows kk = *k, vv = *v;
  if (Hk == 1) kk.stride_h = vv.stride_h = dim;  // of one head: any
  CUtensorMap mk, mv;
  if (!make_map(&mk, &kk, dim, Hk, T) || !make_map(&mv, &vv, dim, Hk, T))
    return fail(ZG_ERR_UNSUPPORTED, "zg_prompt_attention: k or v cannot be described (strides of 0, or of 2^40 bytes and more)");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  const PromptArgs a = {starts, lse, status, B, T, Hq, Hk, (int32_t)G, causal != 0, scale * 1.4426950408889634f};
  cudaError_t err = cudaSuccess;
  for_dim(dim, [&](auto dv) {
    constexpr int D = decltype(dv)::value;
    auto typed = [&](auto ev) {
      using E = typename decltype(ev)::type;
      auto kern = k_prompt<E, D>;
      err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PromptShape<D>::kSmem);
      if (err == cudaSuccess)
        err = launch_early(kern, items * Hk, kThreads, PromptShape<D>::kSmem, static_cast<cudaStream_t>(stream), a,
                           rows_of<E>(q), rows_of<E>(k), rows_of<E>(v), rows_of<E>(out), mk, mv,
                           std::min(wait_limit(), kSpin));
    };
    if (q->dtype == ZG_BF16) typed(Elem<__nv_bfloat16>{});
    else typed(Elem<__half>{});
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "prompt attention launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}
