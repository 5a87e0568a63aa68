// Attention of many query rows over a history cache, on the 5th-generation
// tensor cores.
//
// One CTA takes up to two tiles of 128 query rows (of one request and key
// head) through 128 keys a step:
//   warp 13     brings codes into a ring of shared buffers by bulk copies, 16
//               keys (always inside one block) a copy;
//   warps 8-11  widen them to halves, exactly, into a ring of
//               128-byte-swizzled operands;
//   warp 12     issues S = Q K^T and O += P V (tcgen05, one thread);
//   warps 0-7   one thread a row: scores out of tensor memory, running
//               maximum, p = exp2, halves back to tensor memory.
// A step has 128 keys: a product of 128 rows reads its 128 x 16 slice of Q
// from shared memory whatever its width, some 80 cycles an instruction, so
// narrower steps cost the tensor cores as much for less.  Tensor memory holds
// S and O of both tiles.  Up to 64 dims P has a place of its own and the
// scores of the next step are made as soon as this step's are in registers;
// beyond, P lies over S and they wait for the product that reads it.  While
// one tile's softmax runs the tensor cores work for the other.  P is handed
// over in halves of 64 keys, so that its product starts during the softmax.
// An item of one query tile takes both places: each has the same queries and
// every other step, and their sums are joined at the end.
// Measured: causal chunks of 2,048 rows over up to 16,384 tokens (2 requests, 16
// heads over 4 of 128) 387 us, 1.05 PFLOP/s or 55 % of the measured bf16 rate;
// 256 rows each for 64 requests over up to 2,048 tokens 61 us.  By the counters
// the tensor pipe is active 42 % of the chunk's time and 58 % of the cycles in
// which an SM has a CTA (28 % pass without one: 256 items on 152 SMs), 25 % and
// 32 % of the 256 rows'.  Bound by the waits in the chain softmax -> product ->
// scores of a tile: with the widening, the exponentials and the maxima all left
// out a chunk took 379 us (of 399 then), with seven eighths of the products 380,
// with all of them 349.  The loader of the codes is on that chain too: what it
// does before it asks for a step's codes costs the whole kernel (scales after
// the copies 431 us, divisions by the block's size 392, shifts 387).
//
// Of 4-bit codes (whose scales come with them and are applied by the widening
// warps, exactly) 256 rows each for 64 requests take 64 us.
//
// A key block's scale multiplies its scores, a value block's scale enters the
// exponent (kv_attention.cu has the formula), so neither costs anything an
// element.
//
// Every wait is bounded; on expiry kStatusTimeout is recorded, what was
// issued is drained, tensor memory is freed and the kernel returns.
#include "kv_attn.cuh"
#include "tc.cuh"

namespace zg {
namespace {

constexpr int kSoftWarps = 8, kWidenWarps = 4;
constexpr int kThreads = 512;       // four warpgroups, two of them softmax; warps 14 and 15 only lend registers
constexpr int kNK = 128;            // keys a step
constexpr int kGroups = kNK / 16;   // groups of 16 keys: one block, one scale each
// Registers a thread: 128 at launch, 512 threads, all of an SM's 65,536; moved between warpgroups to 256 x 184 +
// 256 x 72 = 65,536, since a softmax thread holds its row's scores of a step.
constexpr int kSoftRegs = 184, kOtherRegs = 72;
constexpr uint32_t kSpin = 1u << 20;  // polls of a wait at most; of those before exit always

template <int D, int FMT>
struct TcShape {
  static constexpr bool kApart = D <= 64;              // P beside S
  static constexpr int kWide = kApart ? 6 : 3;         // ring entries of halves, each the keys or values of a step
  static constexpr int kRaw = kApart ? 6 : 4;          // ring entries of codes
  static constexpr int kSub = (D + 63) / 64;           // 64-dim subtiles (128-byte rows)
  static constexpr int kTile = kSub * 128 * 128;       // bytes of 128 rows of halves: a query tile, a ring entry
  static constexpr bool k4 = FMT == ZG_KV_E2M1;        // 4 bits: the scale bytes lie behind a ring entry's codes
  static constexpr int kRow = k4 ? Row4<D>::kCodes : D;
  static constexpr int kCodes = kNK * (kRow + (k4 ? Row4<D>::kScales : 0));  // bytes of a ring entry of codes
  static constexpr size_t kSmem = (2 + kWide) * kTile + kRaw * kCodes + 1024;
  // columns of tensor memory; tile i at i * kNK, i * kPStep, i * D of them
  static constexpr uint32_t kS = 0, kP = kApart ? 256 : 0, kPStep = kApart ? 64 : kNK, kO = 512 - 2 * D;
  static_assert((kApart ? 256 + 128 : 256) <= kO, "S, P and O fit");
  static_assert(kSmem <= 225 * 1024, "with the barriers inside 227 KiB");
  // Ring entries in the order of their use.  Apart: keys 0, keys 1, values 0, keys 2, values 1, ..., one entry for
  // the keys behind the last step empty.  Else: keys 0, values 0, keys 1, ...
  static __device__ __forceinline__ int entries(int steps) { return kApart && steps ? 2 * steps + 1 : 2 * steps; }
  static __device__ __forceinline__ int keys(int t) { return kApart ? (t ? 2 * t - 1 : 0) : 2 * t; }
  static __device__ __forceinline__ int values(int t) { return kApart ? 2 * t + 2 : 2 * t + 1; }
  static __device__ __forceinline__ int side(int n) { return kApart ? (n > 0 && !(n & 1)) : n & 1; }
  static __device__ __forceinline__ int step(int n) { return kApart ? (n & 1 ? (n + 1) / 2 : n ? n / 2 - 1 : 0) : n / 2; }
};

// `bytes` from global into shared memory, counted on `bar`; both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(to)),
               "l"(from), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The codes of a block outside the cache, and the values of one without a scale.
__device__ __align__(16) uint8_t g_no_codes[16 * 128];

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a, const Rows<T> q, const Rows<T> out, uint32_t spin) {
  using Sh = TcShape<D, FMT>;
  constexpr int kRaw = Sh::kRaw, kWide = Sh::kWide;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;                        // two query tiles
  uint8_t* wide = sq + 2 * Sh::kTile;           // the ring of halves
  uint8_t* raw = wide + kWide * Sh::kTile;   // the ring of codes
  // The barriers of a query tile have one phase a step, and none is passed twice before all who wait for it have seen
  // it: scores of t + 1 come after every warp has taken those of t, probabilities of t + 1 after the product of t.
  __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw], wide_full[kWide], wide_empty[kWide];
  __shared__ uint64_t q_full, s_full[2], s_free[2], p_full[2][2], o_done[2], drained;  // [tile], p_full [tile][half]
  // of 16 keys each, a ring of 16 steps (the codes of step t + 10 come only after the softmax of step t): key scale,
  // log2 of the value scale, and what a weight counts for in the row's sum
  __shared__ float s_ks[16][kGroups], s_lv[16][kGroups], s_iv[16][kGroups];
  __shared__ uint32_t tmem_base;
  __shared__ bool s_small;  // of this part's sums (kv_attn.cuh)
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  after_predecessor();

  // CTAs start in the order of their numbers: the requests with most to read first, the last rows of each first
  int it = blockIdx.x;
  const int split = it % a.splits;
  it /= a.splits;
  const int m = a.mt - 1 - it % a.mt;
  it /= a.mt;
  const int h = it % a.heads;
  int b = it / a.heads;
  if (a.B > 1 && a.B <= kThreads) {
    __shared__ int s_b;
    int* s_len = reinterpret_cast<int*>(sq);
    if (threadIdx.x < a.B) s_len[threadIdx.x] = a.length[threadIdx.x];
    __syncthreads();
    if (threadIdx.x < a.B) {
      const int mylen = s_len[threadIdx.x];
      int rank = 0;
      for (int j = 0; j < a.B; ++j) rank += s_len[j] > mylen || (s_len[j] == mylen && j < (int)threadIdx.x);
      if (rank == b) s_b = threadIdx.x;
    }
    __syncthreads();
    b = s_b;
  }
  const int item = (b * a.heads + h) * a.mt + m;
  const Seen s = seen_of(a, b, threadIdx.x == 0);
  const int M = a.R * a.G;
  const int mine = min(M - m * a.tile, a.tile);  // query rows of this item
  const int tiles = (mine + 127) / 128;          // query tiles
  const bool twice = tiles == 1;                 // one tile: both places have it, and every other step
  // later rows see no less: the item sees what its last row does, or its request's last
  const int last = min((m * a.tile + mine - 1) / a.G, s.rows - 1);
  const int vmax = last < m * a.tile / a.G ? 0 : visible(a, s, last);
  const int parts = parts_of(a, vmax);
  if (split >= parts) return;  // the join does not look for it
  const int t0 = split * (a.chunk / kNK), t1 = min((vmax + kNK - 1) / kNK, t0 + a.chunk / kNK);
  const int steps = __shfl_sync(0xFFFFFFFFu, t1 - t0, 0);  // uniform, for the compiler too

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      bar_init(&raw_full[i], 1);
      bar_init(&raw_empty[i], kWidenWarps);
    }
    for (int i = 0; i < kWide; ++i) {
      bar_init(&wide_full[i], kWidenWarps);
      bar_init(&wide_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&s_full[i], 1);
      bar_init(&s_free[i], 4);
      bar_init(&p_full[i][0], 4);
      bar_init(&p_full[i][1], 4);
      bar_init(&o_done[i], 1);
    }
    bar_init(&q_full, 8);
    bar_init(&drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  auto give_up = [&]() { atomicOr(a.status, kStatusTimeout); };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kSoftWarps + kWidenWarps) {
      // ----------------------------------------------------------- widening
      constexpr int C16 = Sh::kRow / 16;  // 16-byte pieces of a code row
      constexpr int N = kNK * C16 / 128;  // pieces a thread: tid, tid + 128, ...
      constexpr int NB = N % 4 ? 2 : 4;   // of them at a time
      const int tid = threadIdx.x - 32 * kSoftWarps;
      // where a piece goes; 128 pieces on are a multiple of 8 rows, so the place moves and the swizzle stays (a head
      // of 96 has six pieces a row: there it is worked out each time)
      auto place = [&](int idx, uint32_t& first, uint32_t& second) {
        const int r = idx / C16, c = idx % C16, j = (c % 4) * 2;
        const uint32_t at = (uint32_t)((c / 4) * (kNK * 128) + r * 128);
        first = at + ((j ^ (r & 7)) << 4);
        second = at + (((j + 1) ^ (r & 7)) << 4);
      };
      uint32_t p1, p2;
      place(tid, p1, p2);
      // the pieces of both subtiles fall on the same banks: one half of the lanes stores its second piece first
      const bool swap = D == 128 && tid % C16 >= 4;
      for (int n = 0; n < Sh::entries(steps); ++n) {
        const int rs = n % kRaw, ws = n % kWide;
        const int held = s.len - (t0 + Sh::step(n)) * kNK;
        if (!warp_wait(&raw_full[rs], (n / kRaw) & 1, spin) ||
            (n >= kWide && !warp_wait(&wide_empty[ws], ((n / kWide) - 1) & 1, spin))) {
          if (lane == 0) give_up();
          break;
        }
        const uint8_t* codes = raw + rs * Sh::kCodes + tid * 16;
        uint8_t* to = wide + ws * Sh::kTile;
        if constexpr (Sh::k4) {
          // a piece is 32 elements: four stores, of which lanes of the second subtile begin two on (they fall on the
          // same banks as the first's)
          const uint8_t* scales = raw + rs * Sh::kCodes + kNK * Sh::kRow;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int idx = tid + 128 * i, r = idx / C16, c = idx % C16, j = (c & 1) * 4;
            const uint4 w = *reinterpret_cast<const uint4*>(codes + 128 * i * 16);
            uint32_t u = *reinterpret_cast<const uint16_t*>(scales + r * Row4<D>::kScales + 2 * c);
            if (r >= held) u = 0;  // behind the history: not defined, may be NaN
            const bool second = c >= 2;
            const uint32_t s0 = scale_twice(second ? u >> 8 : u & 0xFF), s1 = scale_twice(second ? u & 0xFF : u >> 8);
            uint4 h[4];
            e2m1_half8(second ? w.z : w.x, s0, &h[0].x);
            e2m1_half8(second ? w.w : w.y, s0, &h[1].x);
            e2m1_half8(second ? w.x : w.z, s1, &h[2].x);
            e2m1_half8(second ? w.y : w.w, s1, &h[3].x);
            uint8_t* at = to + (c / 2) * (kNK * 128) + r * 128;
#pragma unroll
            for (int p = 0; p < 4; ++p) *reinterpret_cast<uint4*>(at + (((j + (second ? p ^ 2 : p)) ^ (r & 7)) << 4)) = h[p];
          }
        } else {
#pragma unroll
          for (int i0 = 0; i0 < N; i0 += NB) {
            uint4 w[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) w[i] = *reinterpret_cast<const uint4*>(codes + 128 * (i0 + i) * 16);
            if (held < kNK) {  // behind the history: not defined, may be NaN
#pragma unroll
              for (int i = 0; i < NB; ++i)
                if ((tid + 128 * (i0 + i)) / C16 >= held) w[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              uint32_t a1 = p1 + (i0 + i) * (128 / C16) * 128, a2 = p2 + (i0 + i) * (128 / C16) * 128;
              if constexpr (D == 96) place(tid + 128 * (i0 + i), a1, a2);
              uint4 lo, hi;
              codes_half4<FMT == ZG_KV_INT8>(w[i].x, lo.x, lo.y);
              codes_half4<FMT == ZG_KV_INT8>(w[i].y, lo.z, lo.w);
              codes_half4<FMT == ZG_KV_INT8>(w[i].z, hi.x, hi.y);
              codes_half4<FMT == ZG_KV_INT8>(w[i].w, hi.z, hi.w);
              *reinterpret_cast<uint4*>(to + (swap ? a2 : a1)) = swap ? hi : lo;
              *reinterpret_cast<uint4*>(to + (swap ? a1 : a2)) = swap ? lo : hi;
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&wide_full[ws]);
          bar_arrive(&raw_empty[rs]);
        }
      }
    } else if (warp == 12 && steps > 0) {
      // ----------------------------------------------------------- products
      // The whole warp walks the loop and one elected thread issues, so that descriptors stay in uniform registers
      // (from one diverged thread an instruction took some 100 cycles to issue).
      const uint32_t id_s = (1u << 4) | ((uint32_t)(kNK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint64_t q0 = desc_k(smem_u32(sq)), k0 = desc_k(smem_u32(wide)), v0 = desc_mn(smem_u32(wide), kNK * 128);
      // scores, products of step t in place i; `k`: how many that place has had before
      auto scores = [&](int t, int i, int k) -> bool {
        const int n = Sh::keys(t), ws = n % kWide;
        if ((twice || i == 0) && !spin_wait(&wide_full[ws], (n / kWide) & 1, spin)) return false;
        // apart: every warp has the last scores in registers; else the product that reads P in their place is over
        if (k > 0 && !spin_wait(Sh::kApart ? &s_free[i] : &o_done[i], (k - 1) & 1, spin)) return false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t kd = k0 + ws * (Sh::kTile >> 4), qd = q0 + i * (Sh::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * (128 * 128 >> 4) + (k % 4) * 2;
            mma_ss(tmem + Sh::kS + (uint32_t)(i * kNK), qd + off, kd + off, id_s, k > 0);
          }
          commit(&s_full[i]);
          if (twice || i == 1) commit(&wide_empty[ws]);
        }
        __syncwarp();
        return true;
      };
      auto values = [&](int t, int i, int k) -> bool {
        const int n = Sh::values(t), ws = n % kWide;
        if ((twice || i == 0) && !spin_wait(&wide_full[ws], (n / kWide) & 1, spin)) return false;
        const uint64_t vd = v0 + ws * (Sh::kTile >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!spin_wait(&p_full[i][half], k & 1, spin)) return false;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
#pragma unroll
            for (int j = half * 4; j < half * 4 + 4; ++j)
              mma_ts(tmem + Sh::kO + (uint32_t)(i * D), tmem + Sh::kP + i * Sh::kPStep + (uint32_t)(j * 8),
                     vd + j * (2048 >> 4), id_o, (k > 0 || j > 0) ? 1u : 0u);
            if (half) {
              commit(&o_done[i]);
              if (twice || i == 1) commit(&wide_empty[ws]);
            }
          }
          __syncwarp();
        }
        return true;
      };
      bool good = spin_wait(&q_full, 0, spin);
      if (twice) {
        for (int t = 0; t < 2 && t < steps && good; ++t) good = scores(t, t, 0);
        for (int t = 0; t < steps && good; ++t) {
          const int i = t & 1, k = t >> 1;
          const bool more = t + 2 < steps;
          if constexpr (Sh::kApart) good = (!more || scores(t + 2, i, k + 1)) && values(t, i, k);
          else good = values(t, i, k) && (!more || scores(t + 2, i, k + 1));
        }
      } else {
        for (int i = 0; i < 2 && good; ++i) good = scores(0, i, 0);
        for (int t = 0; t < steps && good; ++t) {
          if constexpr (Sh::kApart)
            for (int i = 0; i < 2 && good && t + 1 < steps; ++i) good = scores(t + 1, i, t + 1);
          for (int i = 0; i < 2 && good; ++i)
            good = values(t, i, t) && (Sh::kApart || t + 1 == steps || scores(t + 1, i, t + 1));
        }
      }
      if (!good && lane == 0) give_up();
      if (elect_one()) commit(&drained);
      __syncwarp();
      if (!spin_wait(&drained, 0, kSpin) && lane == 0) give_up();
    } else if (warp == 13) {
      // -------------------------------------------------------------- codes
      // Lane g brings keys 16 g .. 16 g + 15 of a step.  Block numbers and scales are read a step or more ahead of
      // their use.
      const int g = lane % kGroups;
      auto block_of = [&](int t) -> int {  // -1: behind the history; -2: outside the cache (recorded)
        const int key = (t0 + t) * kNK + 16 * g;
        if (t >= steps || key >= s.len) return -1;
        const int blk = a.table[(int64_t)b * a.max_blocks + (key >> a.bt_log2)];
        if (blk >= 0 && blk < a.n_blocks) return blk;
        if (lane < kGroups) atomicOr(a.status, kStatusCache);
        return -2;
      };
      // blocks of the step whose values come next and of the three behind it; scales of the step whose keys come next
      int tv = 0, b0 = block_of(0), b1 = block_of(1), b2 = block_of(2), b3 = block_of(3);
      // of 4-bit codes, whose scales are in the halves already: 1
      auto scale_of = [&](const float* scales, int blk) -> float {
        if constexpr (Sh::k4) return 1.f;
        return blk < 0 ? 0.f : scales[(int64_t)blk * a.heads + h];
      };
      float ks = scale_of(a.ks, b0), vs = scale_of(a.vs, b0);
      const bool small = __shfl_sync(0xFFFFFFFFu, small_scale(vs), 0);
      if (lane == 0) s_small = small;  // seen by all who see the first codes
      float last_lv = kNoScale;      // of this lane's group, in the step before
      bool none0 = false, none1 = false;  // its values have no scale: in the step whose values come next, and behind it
      int issued = 0;
      bool good = true;
      for (int n = 0; n < Sh::entries(steps); ++n) {
        const int rs = n % kRaw, side = Sh::side(n), t = Sh::step(n);
        const int blk = t == tv ? b0 : b1;
        if (n >= kRaw && !warp_wait(&raw_empty[rs], ((n / kRaw) - 1) & 1, spin)) {
          good = false;
          break;
        }
        const uint32_t bytes =
            __popc(__ballot_sync(0xFFFFFFFFu, lane < kGroups && blk != -1)) * (uint32_t)(Sh::kCodes / kGroups);
        if (!side) {
          float lv = log2_fast(vs), iv = sum_weight(lv, small);
          const uint32_t some = __ballot_sync(0xFFFFFFFFu, has_scale(vs)) & ((1u << kGroups) - 1);
          if (some != (1u << kGroups) - 1) {  // rare, and at the end: where a scale of 0 stands (kv_attn.cuh)
            const uint32_t upto = some & ((2u << g) - 1);
            const float before = __shfl_sync(0xFFFFFFFFu, last_lv, kGroups - 1);
            const float first = __shfl_sync(0xFFFFFFFFu, lv, some ? __ffs(some) - 1 : 0);
            const float near = __shfl_sync(0xFFFFFFFFu, lv, upto ? 31 - __clz(upto) : 0);
            last_lv = lv = upto ? near : some && before == kNoScale ? first : before;
            iv = sum_weight(lv, small);
            if (blk == -2) lv = -INFINITY, iv = 0.f;  // outside the cache: no score, no part in a sum
          } else {
            last_lv = lv;
          }
          if (Sh::k4 && blk == -2) lv = -INFINITY, iv = 0.f;
          if (lane < kGroups && t < steps) {
            s_ks[t & 15][g] = ks;
            s_lv[t & 15][g] = lv;
            s_iv[t & 15][g] = iv;
          }
          (t == tv ? none0 : none1) = !has_scale(vs);
          const int nb = t == tv ? b1 : b2;
          ks = scale_of(a.ks, nb);
          vs = scale_of(a.vs, nb);
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&raw_full[rs])),
                       "r"(bytes)
                       : "memory");
        __syncwarp();
        const int64_t row = ((int64_t)blk * a.heads + h) * a.bt + (((t0 + t) * kNK + 16 * g) & (a.bt - 1));
        if (lane < kGroups && blk != -1) {
          bulk_load(raw + rs * Sh::kCodes + 16 * g * Sh::kRow,
                    blk < 0 || (side && none0) ? g_no_codes : (side ? a.vc : a.kc) + row * Sh::kRow, 16 * Sh::kRow,
                    &raw_full[rs]);
          if constexpr (Sh::k4)
            bulk_load(raw + rs * Sh::kCodes + kNK * Sh::kRow + 16 * g * Row4<D>::kScales,
                      blk < 0 ? g_no_codes : (side ? a.vg : a.kg) + row * Row4<D>::kScales, 16 * Row4<D>::kScales,
                      &raw_full[rs]);
        }
        issued = n + 1;
        if (side) {
          ++tv;
          none0 = none1;
          b0 = b1, b1 = b2, b2 = b3, b3 = block_of(tv + 3);
        }
      }
      if (!good && lane == 0) give_up();
      // every copy has landed before the CTA may end
      for (int n = max(0, issued - kRaw); n < issued; ++n)
        if (!warp_wait(&raw_full[n % kRaw], (n / kRaw) & 1, kSpin) && lane == 0) give_up();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int i = warp >> 2;  // the place
    {
      // ------------------------------------------------------------ softmax
      const int r = threadIdx.x & 127, ir = twice ? r : threadIdx.x, ri = m * a.tile + ir;  // row of the tile, item, call
      const bool live = ir < mine;
      const int row = ri / a.G, qh = h * a.G + ri % a.G;
      const int vis = live ? visible(a, s, row) : 0;
      const int first = twice ? i : 0, stride = twice ? 2 : 1;  // steps of this place
      const int turns = first < steps ? (steps - first + stride - 1) / stride : 0;
      // lanes of a row when a warp moves its 32 rows: four elements each, kAt rows at a time
      constexpr int kLanes = D / 4, kSlot = D == 96 ? 32 : kLanes, kAt = 32 / kSlot;
      const int l4 = lane % kSlot, e = 4 * l4;
      const int64_t q_row = b * q.sb + row * q.st + qh * q.sh;
      float fz;
      {
        // the warp's 32 rows into its query tile as halves, each scaled by a power of two: a group of lanes a row,
        // four elements a lane; where a row is comes from the lane that it belongs to
        uint8_t* tile = sq + i * Sh::kTile + (e / 64) * (128 * 128) + (e & 4) * 2;
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, vis > 0);
        uint2 w[32 / kAt];  // every load in flight before the first is used
#pragma unroll
        for (int k = 0; k < 32 / kAt; ++k) {
          const int rw = k * kAt + lane / kSlot;
          const int64_t at = __shfl_sync(0xFFFFFFFFu, q_row, rw);
          w[k] = make_uint2(0, 0);
          if (((some >> rw) & 1) && l4 < kLanes) w[k] = *reinterpret_cast<const uint2*>(q.data + at + e);
        }
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 32 / kAt; ++k) {
          const int rr = (warp & 3) * 32 + k * kAt + lane / kSlot;  // row of the tile
          float x[4];
          load4(reinterpret_cast<const T*>(&w[k]), x);
          float tp = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
          for (int o = kSlot / 2; o; o >>= 1) tp = fmaxf(tp, __shfl_xor_sync(0xFFFFFFFFu, tp, o));
          const float dn = __uint_as_float((uint32_t)(127 - row_exponent(tp)) << 23);
          if (l4 < kLanes)
            *reinterpret_cast<uint2*>(tile + rr * 128 + ((((e % 64) / 8) ^ (rr & 7)) << 4)) =
                make_uint2(pack_half2(x[0] * dn, x[1] * dn), pack_half2(x[2] * dn, x[3] * dn));
          const float own = __shfl_sync(0xFFFFFFFFu, tp, (lane % kAt) * kSlot);
          if (lane / kAt == k) top = own;
        }
        fz = a.scale * __uint_as_float((uint32_t)(127 + row_exponent(top)) << 23);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&q_full);
      }
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + Sh::kS + (uint32_t)(i * kNK) + lanes;
      const uint32_t p_at = tmem + Sh::kP + i * Sh::kPStep + lanes;
      const uint32_t o_at = tmem + Sh::kO + (uint32_t)(i * D) + lanes;
      float mx = -INFINITY, l = 0.f;
      bool good = true;
      for (int k = 0; k < turns; ++k) {
        const int t = first + k * stride;
        if (!warp_wait(&s_full[i], k & 1, spin)) {
          good = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        uint32_t sr[kNK];
        tmem_load128(s_at, sr);
        if constexpr (Sh::kApart) {
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(&s_free[i]);
        }
        float* z = reinterpret_cast<float*>(sr);
        const int left = vis - (t0 + t) * kNK;  // keys of this step that the row sees
        if (__any_sync(0xFFFFFFFFu, left < kNK)) {
#pragma unroll
          for (int j = 0; j < kNK; ++j) z[j] = j < left ? z[j] : -INFINITY;
        }
        float tm = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          float gm = max3(z[16 * g], z[16 * g + 1], z[16 * g + 2]);
#pragma unroll
          for (int j = 3; j + 1 < 16; j += 2) gm = max3(gm, z[16 * g + j], z[16 * g + j + 1]);
          gm = fmaxf(gm, z[16 * g + 15]);
          // a key scale of 0 must not meet an infinite score
          tm = fmaxf(tm, fmaf(gm, fmaxf(fz * s_ks[t & 15][g], 1e-37f), s_lv[t & 15][g]));
        }
        float al = 1.f;
        const bool move = __any_sync(0xFFFFFFFFu, tm > mx + 8.f);
        if (move) {
          const float nm = fmaxf(mx, tm);
          if (nm != mx) {
            al = exp2_fast(mx - nm);
            l = moved_sum(l, mx, nm);
          }
          mx = nm;
        }
        const float mu = mx == -INFINITY ? 0.f : mx;
        // A score enters the exponent unrounded and mu rounded, so that a row's weights are off by a common factor, up to
        // 2^(ulp(mu)); from 2^26 on that could leave a half's range, and scores are taken times a power of two that
        // keeps it within 2^4.  There scores that differ by their last bit lie 8 apart or more.
        const int far = (int)((__float_as_uint(mu) >> 23) & 0xFF) - (127 + 25);
        const float down = power_of_2(-max(far, 0)), fd = fz * down, md = mu * down;
        // the product of the last step has read its probabilities, and is in the sums (with P over S the scores have
        // waited for it)
        if (Sh::kApart && k > 0) {
          if (!warp_wait(&o_done[i], (k - 1) & 1, spin)) {
            good = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
        if (move && k > 0) {
#pragma unroll
          for (int d = 0; d < D; d += 16) {  // few at a time: the scores stay in registers
            uint32_t o[16];
            tmem_load16(o_at + d, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
            tmem_store16(o_at + d, o);
          }
        }
#pragma unroll
        for (int g2 = 0; g2 < kGroups; g2 += 2) {
          uint32_t pr[16];
#pragma unroll
          for (int g = g2; g < g2 + 2; ++g) {
            const float f = fmaxf(fd * s_ks[t & 15][g], 1e-37f), c = fmaf(s_lv[t & 15][g], down, -md);
            const uint64_t f2 = pair(f, f), c2 = pair(c, c);
            uint64_t sum = 0;  // 0.f, 0.f
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float x0, x1;
              unpair(fma2(pair(z[16 * g + 2 * j], z[16 * g + 2 * j + 1]), f2, c2), x0, x1);
              const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
              sum = add2(sum, pair(p0, p1));
              pr[8 * (g - g2) + j] = pack_half2(p0, p1);
            }
            float a0, a1;
            unpair(sum, a0, a1);
            l = fmaf(a0 + a1, s_iv[t & 15][g], l);
          }
          tmem_store16(p_at + 8 * g2, pr);
          if (g2 % (kGroups / 2) == kGroups / 2 - 2) {
            tmem_store_wait();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) bar_arrive(&p_full[i][g2 / (kGroups / 2)]);
          }
        }
      }
      if (good && turns > 0) good = warp_wait(&o_done[i], (turns - 1) & 1, spin);
      if (!good && lane == 0) give_up();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const PartEnd end = part_end(mx, l, turns > 0 && good && s_small);
      mx = end.m;
      l = end.l;
      float own = end.down, other = 0.f;  // factors of the two places' sums
      float* sum1 = reinterpret_cast<float*>(wide);  // [D + 2][128]: place 1's sums, reference and row sum
      if (twice) {
        if (i == 1) {
          // every product is complete in both places before the ring is written over
          asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
          for (int d = 0; d < D; d += 16) {
            uint32_t o[16];
            if (turns > 0) tmem_load16(o_at + d, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum1[(d + j) * 128 + r] = turns > 0 ? __uint_as_float(o[j]) * own : 0.f;
          }
          sum1[D * 128 + r] = mx;
          sum1[(D + 1) * 128 + r] = l;
          asm volatile("bar.sync 1, 256;" ::: "memory");
        } else {
          asm volatile("bar.sync 1, 256;" ::: "memory");
          asm volatile("bar.sync 1, 256;" ::: "memory");
          const float m1 = sum1[D * 128 + r], l1 = sum1[(D + 1) * 128 + r], top = fmaxf(mx, m1);
          const float f = mx == -INFINITY ? 0.f : exp2_fast(mx - top);
          own *= f;
          other = m1 == -INFINITY ? 0.f : exp2_fast(m1 - top);
          mx = top;
          l = l * f + l1 * other;
        }
      }
      if (parts == 1) {  // no join: outputs
        const float inv = l == 0.f ? 0.f : 1.f / l;
        own *= inv;
        other *= inv;
      }
      const int64_t pi = ((int64_t)item * a.splits + split) * a.tile + ir;
      if (good && !(twice && i == 1)) {
        uint8_t* tile = sq + i * Sh::kTile;  // every product that reads the queries is complete
#pragma unroll
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          if (turns > 0) {
            tmem_load(o_at + d, o);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * own);
          if (twice) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) + sum1[(d + j) * 128 + r] * other);
          }
          const float* x = reinterpret_cast<const float*>(o);
          if (parts > 1) {
            if (live)
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(a.part + pi * D + d + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4*>(tile + ((d + j) / 64) * (128 * 128) + r * 128 +
                                        (((((d + j) % 64) / 8) ^ (r & 7)) << 4)) =
                  make_uint4(pack2<T>(x[j], x[j + 1]), pack2<T>(x[j + 2], x[j + 3]), pack2<T>(x[j + 4], x[j + 5]),
                             pack2<T>(x[j + 6], x[j + 7]));
          }
        }
        if (parts == 1) {  // whole rows out, as the queries came in
          const int64_t out_row = b * out.sb + row * out.st + qh * out.sh;
          const uint32_t mine_of = __ballot_sync(0xFFFFFFFFu, live);
          __syncwarp();
#pragma unroll 8
          for (int k = 0; k < 32 / kAt; ++k) {
            const int rw = k * kAt + lane / kSlot, rr = (warp & 3) * 32 + rw;
            const int64_t at = __shfl_sync(0xFFFFFFFFu, out_row, rw);
            if (((mine_of >> rw) & 1) && l4 < kLanes)
              *reinterpret_cast<uint2*>(out.data + at + e) = *reinterpret_cast<const uint2*>(
                  tile + (e / 64) * (128 * 128) + rr * 128 + ((((e % 64) / 8) ^ (rr & 7)) << 4) + (e & 4) * 2);
          }
        }
        if (live && parts > 1) {
          float* ml = a.part + a.slots * a.tile * D + pi * 2;
          ml[0] = mx;
          ml[1] = l;
        } else if (live && a.lse) {
          a.lse[((int64_t)b * a.R + row) * a.Hq + qh] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.693147180559945f;
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 12) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace

int attn_tc_tile(int64_t rows) { return rows > 128 ? 256 : 128; }

cudaError_t launch_attn_tc(const AttnArgs& a, const zg_rows* q, const zg_rows* out, int dim, int format,
                           int64_t items, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  auto go = [&](auto ev, auto dv, auto iv) {
    using E = typename decltype(ev)::type;
    constexpr int D = decltype(dv)::value;
    constexpr int FMT = decltype(iv)::value;
    auto kern = k_attn_tc<E, D, FMT>;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TcShape<D, FMT>::kSmem);
    if (err != cudaSuccess) return;
    err = launch_early(kern, items, kThreads, TcShape<D, FMT>::kSmem, st, a, rows_of<E>(q), rows_of<E>(out),
                       std::min(wait_limit(), kSpin));
  };
  for_dim(dim, [&](auto dv) {
    auto typed = [&](auto ev) { for_format(format, [&](auto fv) { go(ev, dv, fv); }); };
    if (q->dtype == ZG_BF16) typed(Elem<__nv_bfloat16>{});
    else typed(Elem<__half>{});
  });
  return err;
}

}  // namespace zg
