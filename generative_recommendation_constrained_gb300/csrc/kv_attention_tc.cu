// Attention of many query rows over a history cache, on the 5th-generation
// tensor cores.
//
// One CTA takes up to two tiles of 128 query rows (of one request and key
// head) through 64 keys at a time:
//   warp 13     brings the codes of 64 keys a step into a ring of four by bulk
//               copies, 16 keys (always inside one block) a copy;
//   warps 8-11  widen the codes of keys and values to halves, exactly, into
//               two 128-byte-swizzled shared buffers;
//   warp 12     issues S = Q K^T and O += P V (tcgen05, one thread): S and O
//               live in tensor memory, P is read from there;
//   warps 0-7   one thread a row: scores out of tensor memory, running
//               maximum, p = exp2, halves back over the scores.
// Two score buffers a tile let the next scores be made while this tile's
// probabilities are; the two tiles' softmaxes overlap each other's products.
//
// A key block's scale multiplies its scores, a value block's scale enters the
// exponent (kv_attention.cu has the formula), so neither costs anything an
// element.
//
// Every wait is bounded; on expiry kStatusTimeout is recorded, what was
// issued is drained, tensor memory is freed and the kernel returns.
#include "kv_attn.cuh"

namespace zg {
namespace {

constexpr int kNK = 64;             // keys a step
constexpr int kSoftWarps = 8, kWidenWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kWidenWarps + 2);
constexpr int kRing = 4;            // steps of codes in flight
constexpr uint32_t kSpin = 1u << 20;  // polls of a wait at most; of those before exit always

template <int D>
struct TcShape {
  static constexpr int kSub = (D + 63) / 64;          // 64-dim subtiles (128-byte rows)
  static constexpr int kQ = kSub * 128 * 128;         // bytes of one query tile
  static constexpr int kKV = kSub * kNK * 128;        // bytes of one widened key or value buffer
  static constexpr int kRaw = 2 * kNK * D;            // codes of one step, keys then values
  static constexpr size_t kSmem = 2 * kQ + 4 * kKV + kRing * kRaw + 1024;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
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

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// K-major operand, 128-byte swizzle: rows of 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Transposed operand (rows are the contraction's index): 64 columns a row of
// 128 bytes, the next 64 columns `lead` bytes on, 8 rows 1024 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

#define ZG_R32(r)                                                                                                    \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),        \
      "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),         \
      "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),        \
      "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define ZG_I32(r)                                                                                                    \
  "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),      \
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),    \
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),    \
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])

// 32 columns of this warp's 32 lanes; the values are there when it returns.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : ZG_R32(r)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}
// 64 columns.
__device__ __forceinline__ void tmem_load64(uint32_t addr, uint32_t* r) {
  uint32_t* r2 = r + 32;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : ZG_R32(r), ZG_R32(r2)
      : "r"(addr), "r"(addr + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::ZG_I32(r),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// `bytes` from global into shared memory, counted on `bar`; both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(to)),
               "l"(from), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return pack_half2(a, b);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a, const Rows<T> q, const Rows<T> out, uint32_t spin) {
  using Sh = TcShape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;                       // two query tiles
  uint8_t* sk = sq + 2 * Sh::kQ;            // two key buffers
  uint8_t* sv = sk + 2 * Sh::kKV;           // two value buffers
  uint8_t* raw = sv + 2 * Sh::kKV;          // the ring of codes
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], drained, raw_full[kRing], raw_empty[kRing];
  // [query tile][step parity]: one phase of each is never passed before all its waits are over, because step t + 2
  // of a kind starts only after the warps that wait for step t have done their part of it
  __shared__ uint64_t s_full[2][2], p_full[2][2], o_done[2][2];
  // of 16 keys each, a ring of eight steps (the codes of step t + 8 come only after the softmax of step t): key
  // scale, log2 of the value scale, and 2^-that
  __shared__ float s_ks[8][4], s_lv[8][4], s_iv[8][4];
  __shared__ uint32_t tmem_base;
  __shared__ int s_vmax;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  int it = blockIdx.x;
  const int split = it % a.splits;
  it /= a.splits;
  const int item = it;
  const int m = it % a.mt;
  it /= a.mt;
  const int h = it % a.heads, b = it / a.heads;
  const Seen s = seen_of(a, b, threadIdx.x == 0);
  const int M = a.R * a.G;
  const int tiles = (min(M - m * a.tile, a.tile) + 127) / 128;  // query tiles in use

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&k_full[i], kWidenWarps);
      bar_init(&v_full[i], kWidenWarps);
      bar_init(&k_empty[i], 1);
      bar_init(&v_empty[i], 1);
      for (int j = 0; j < 2; ++j) {
        bar_init(&s_full[i][j], 1);
        bar_init(&p_full[i][j], 4);
        bar_init(&o_done[i][j], 1);
      }
    }
    bar_init(&drained, 1);
    for (int i = 0; i < kRing; ++i) {
      bar_init(&raw_full[i], 1);
      bar_init(&raw_empty[i], kWidenWarps);
    }
    s_vmax = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();

  // the rows: one thread each, scaled by a power of two into halves
  int vis = 0, row = 0, qh = 0;
  float fz = 0.f;
  const int ri = m * a.tile + threadIdx.x;  // row of a softmax thread
  if (warp < kSoftWarps) {
    row = ri / a.G;
    qh = h * a.G + ri % a.G;
    if (ri < M && (int)threadIdx.x < a.tile) vis = visible(a, s, row);
    uint8_t* tile = sq + (warp >> 2) * Sh::kQ;
    const int r = threadIdx.x & 127;
    float top = 0.f;
    if (vis > 0) {
      const T* p = q.at(b, row, qh);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float x[4];
        load4(p + d, x);
        top = fmaxf(fmaxf(top, fmaxf(fabsf(x[0]), fabsf(x[1]))), fmaxf(fabsf(x[2]), fabsf(x[3])));
      }
    }
    const int ex = row_exponent(top);
    const float dn = __uint_as_float((uint32_t)(127 - ex) << 23);
    fz = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
    if ((warp >> 2) < tiles) {
#pragma unroll 4
      for (int d = 0; d < D; d += 8) {
        float x[8] = {};
        if (vis > 0) {
          load4(q.at(b, row, qh) + d, x);
          load4(q.at(b, row, qh) + d + 4, x + 4);
        }
        const uint4 w = make_uint4(pack_half2(x[0] * dn, x[1] * dn), pack_half2(x[2] * dn, x[3] * dn),
                                   pack_half2(x[4] * dn, x[5] * dn), pack_half2(x[6] * dn, x[7] * dn));
        *reinterpret_cast<uint4*>(tile + (d / 64) * (128 * 128) + r * 128 + ((((d % 64) / 8) ^ (r & 7)) << 4)) = w;
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    int vm = vis;
#pragma unroll
    for (int o = 16; o; o >>= 1) vm = max(vm, __shfl_xor_sync(0xFFFFFFFFu, vm, o));
    if (lane == 0) atomicMax(&s_vmax, vm);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  const uint32_t t_o = tmem + 256;  // columns: S of tile 0 (two buffers), of tile 1, then O of each
  const int steps_all = (s_vmax + kNK - 1) / kNK;
  const int per = (steps_all + a.splits - 1) / a.splits;
  const int t0 = min(steps_all, split * per);
  const int steps = __shfl_sync(0xFFFFFFFFu, min(steps_all, t0 + per) - t0, 0);  // uniform, for the compiler too

  auto give_up = [&]() { atomicOr(a.status, kStatusTimeout); };

  if (warp >= kSoftWarps && warp < kSoftWarps + kWidenWarps) {
    // ------------------------------------------------------------- widening
    constexpr int C16 = D / 16;                // 16-byte pieces of a code row
    constexpr int N = kNK * C16 / 128;         // pieces a thread and side
    const int tid = threadIdx.x - 32 * kSoftWarps;
    auto widen = [&](uint8_t* buf, const uint8_t* codes, int held) {
      uint4 w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint4*>(codes + (tid + 128 * i) * 16);
      if (held < kNK) {  // behind the history: not defined, may be NaN
#pragma unroll
        for (int i = 0; i < N; ++i)
          if ((tid + 128 * i) / C16 >= held) w[i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int idx = tid + 128 * i, r = idx / C16, c = idx % C16;
        uint4 lo, hi;
        codes_half4<INT8>(w[i].x, lo.x, lo.y);
        codes_half4<INT8>(w[i].y, lo.z, lo.w);
        codes_half4<INT8>(w[i].z, hi.x, hi.y);
        codes_half4<INT8>(w[i].w, hi.z, hi.w);
        uint8_t* p = buf + (c / 4) * (kNK * 128) + r * 128;
        const int j = (c % 4) * 2;
        // the pieces of both subtiles fall on the same banks: one half of the lanes stores its second piece first
        const bool swap = c >= 4;
        *reinterpret_cast<uint4*>(p + (((j + (swap ? 1 : 0)) ^ (r & 7)) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(p + (((j + (swap ? 0 : 1)) ^ (r & 7)) << 4)) = swap ? lo : hi;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    for (int t = 0; t < steps; ++t) {
      const int buf = t & 1, slot = t % kRing;
      const int held = s.len - (t0 + t) * kNK;
      const uint8_t* codes = raw + slot * Sh::kRaw;
      if (!warp_wait(&raw_full[slot], (t / kRing) & 1, spin) ||
          (t >= 2 && !warp_wait(&k_empty[buf], ((t >> 1) - 1) & 1, spin))) {
        if (lane == 0) give_up();
        break;
      }
      widen(sk + buf * Sh::kKV, codes, held);
      if (lane == 0) bar_arrive(&k_full[buf]);
      if (t >= 2 && !warp_wait(&v_empty[buf], ((t >> 1) - 1) & 1, spin)) {
        if (lane == 0) give_up();
        break;
      }
      widen(sv + buf * Sh::kKV, codes + kNK * D, held);
      if (lane == 0) {
        bar_arrive(&v_full[buf]);
        bar_arrive(&raw_empty[slot]);
      }
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------------- codes
    // Lane g of four brings keys 16 g .. 16 g + 15 of a step.  Block numbers are read two steps and scales one step
    // ahead of their use.
    const int g = lane & 3;
    auto block_of = [&](int t) -> int {  // -1: behind the history, or outside the cache (recorded)
      const int key = (t0 + t) * kNK + 16 * g;
      if (t >= steps || key >= s.len) return -1;
      const int blk = a.table[(int64_t)b * a.max_blocks + key / a.bt];
      if (blk >= 0 && blk < a.n_blocks) return blk;
      if (lane < 4) atomicOr(a.status, kStatusCache);
      return -1;
    };
    int blk = block_of(0), blk1 = block_of(1);
    float ks = blk < 0 ? 0.f : a.ks[(int64_t)blk * a.heads + h], vs = blk < 0 ? 0.f : a.vs[(int64_t)blk * a.heads + h];
    int issued = 0;
    for (int t = 0; t < steps; ++t) {
      const int blk2 = block_of(t + 2);
      const float ks1 = blk1 < 0 ? 0.f : a.ks[(int64_t)blk1 * a.heads + h];
      const float vs1 = blk1 < 0 ? 0.f : a.vs[(int64_t)blk1 * a.heads + h];
      const int slot = t % kRing;
      if (t >= kRing && !warp_wait(&raw_empty[slot], ((t / kRing) - 1) & 1, spin)) {
        if (lane == 0) give_up();
        break;
      }
      if (lane < 4) {
        s_ks[t & 7][g] = ks;
        s_lv[t & 7][g] = scale_log2(vs);
        s_iv[t & 7][g] = exp2_fast(-scale_log2(vs));
      }
      const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, lane < 4 && blk >= 0));
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&raw_full[slot])),
                     "r"(n * 2u * 16u * (uint32_t)D)
                     : "memory");
      __syncwarp();
      if (lane < 4 && blk >= 0) {
        const int row = ((t0 + t) * kNK + 16 * g) % a.bt;
        const int64_t at = (((int64_t)blk * a.heads + h) * a.bt + row) * D;
        uint8_t* to = raw + slot * Sh::kRaw + 16 * g * D;
        bulk_load(to, a.kc + at, 16 * D, &raw_full[slot]);
        bulk_load(to + kNK * D, a.vc + at, 16 * D, &raw_full[slot]);
      }
      issued = t + 1;
      blk = blk1, ks = ks1, vs = vs1, blk1 = blk2;
    }
    // every copy has landed before the CTA may end
    for (int t = max(0, issued - kRing); t < issued; ++t)
      if (!warp_wait(&raw_full[t % kRing], (t / kRing) & 1, kSpin) && lane == 0) give_up();
  } else if (warp == 12) {
    // ------------------------------------------------------------- products
    // The whole warp walks the loop and one elected thread issues, so that descriptors stay in uniform registers
    // (from one diverged thread an instruction took some 100 cycles to issue: 3,900 a step, 1,000 of them work).
    if (steps > 0) {
      const uint32_t id_s = (1u << 4) | ((uint32_t)(kNK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint64_t q0 = desc_k(smem_u32(sq)), k0 = desc_k(smem_u32(sk)), v0 = desc_mn(smem_u32(sv), kNK * 128);
      bool good = true;
      for (int t = 0; t <= steps && good; ++t) {
        if (t < steps) {
          const uint32_t par = t & 1, ph = (t >> 1) & 1;
          const uint64_t kd = k0 + par * (Sh::kKV >> 4);
          good = warp_wait(&k_full[par], ph, spin);
          for (int i = 0; i < tiles && good; ++i) {
            // the scores go where step t - 2 had its probabilities
            if (t >= 2) good = warp_wait(&o_done[i][par], ph ^ 1, spin);
            if (!good) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + (uint32_t)(i * 128 + par * kNK);
            const uint64_t qd = q0 + i * (Sh::kQ >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_ss(d, qd + (k / 4) * (128 * 128 >> 4) + (k % 4) * 2, kd + (k / 4) * (kNK * 128 >> 4) + (k % 4) * 2,
                       id_s, k > 0);
              commit(&s_full[i][par]);
              if (i == tiles - 1) commit(&k_empty[par]);
            }
            __syncwarp();
          }
        }
        if (t > 0 && good) {
          const int u = t - 1;
          const uint32_t par = u & 1, ph = (u >> 1) & 1;
          const uint64_t vd = v0 + par * (Sh::kKV >> 4);
          good = warp_wait(&v_full[par], ph, spin);
          for (int i = 0; i < tiles && good; ++i) {
            good = warp_wait(&p_full[i][par], ph, spin);
            if (!good) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t p = tmem + (uint32_t)(i * 128 + par * kNK), o = t_o + (uint32_t)(i * 128);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kNK / 16; ++k) mma_ts(o, p + k * 8, vd + k * (2048 >> 4), id_o, (u > 0 || k > 0) ? 1u : 0u);
              commit(&o_done[i][par]);
              if (i == tiles - 1) commit(&v_empty[par]);
            }
            __syncwarp();
          }
        }
      }
      if (!good && lane == 0) give_up();
      if (elect_one()) commit(&drained);
      __syncwarp();
      if (!warp_wait(&drained, 0, kSpin) && lane == 0) give_up();
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------------- codes
    // Lane g of four brings keys 16 g .. 16 g + 15 of a step.  Block numbers are read two steps and scales one step
    // ahead of their use.
    const int g = lane & 3;
    auto block_of = [&](int t) -> int {  // -1: behind the history, or outside the cache (recorded)
      const int key = (t0 + t) * kNK + 16 * g;
      if (t >= steps || key >= s.len) return -1;
      const int blk = a.table[(int64_t)b * a.max_blocks + key / a.bt];
      if (blk >= 0 && blk < a.n_blocks) return blk;
      if (lane < 4) atomicOr(a.status, kStatusCache);
      return -1;
    };
    int blk = block_of(0), blk1 = block_of(1);
    float ks = blk < 0 ? 0.f : a.ks[(int64_t)blk * a.heads + h], vs = blk < 0 ? 0.f : a.vs[(int64_t)blk * a.heads + h];
    int issued = 0;
    for (int t = 0; t < steps; ++t) {
      const int blk2 = block_of(t + 2);
      const float ks1 = blk1 < 0 ? 0.f : a.ks[(int64_t)blk1 * a.heads + h];
      const float vs1 = blk1 < 0 ? 0.f : a.vs[(int64_t)blk1 * a.heads + h];
      const int slot = t % kRing;
      if (t >= kRing && !warp_wait(&raw_empty[slot], ((t / kRing) - 1) & 1, spin)) {
        if (lane == 0) give_up();
        break;
      }
      if (lane < 4) {
        s_ks[t & 7][g] = ks;
        s_lv[t & 7][g] = scale_log2(vs);
        s_iv[t & 7][g] = exp2_fast(-scale_log2(vs));
      }
      const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, lane < 4 && blk >= 0));
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&raw_full[slot])),
                     "r"(n * 2u * 16u * (uint32_t)D)
                     : "memory");
      __syncwarp();
      if (lane < 4 && blk >= 0) {
        const int row = ((t0 + t) * kNK + 16 * g) % a.bt;
        const int64_t at = (((int64_t)blk * a.heads + h) * a.bt + row) * D;
        uint8_t* to = raw + slot * Sh::kRaw + 16 * g * D;
        bulk_load(to, a.kc + at, 16 * D, &raw_full[slot]);
        bulk_load(to + kNK * D, a.vc + at, 16 * D, &raw_full[slot]);
      }
      issued = t + 1;
      blk = blk1, ks = ks1, vs = vs1, blk1 = blk2;
    }
    // every copy has landed before the CTA may end
    for (int t = max(0, issued - kRing); t < issued; ++t)
      if (!warp_wait(&raw_full[t % kRing], (t / kRing) & 1, kSpin) && lane == 0) give_up();
  } else if (warp == 12) {
    // ------------------------------------------------------------- products
    if (lane == 0 && steps > 0) {
      const uint32_t id_s = (1u << 4) | ((uint32_t)(kNK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t q0 = smem_u32(sq), k0 = smem_u32(sk), v0 = smem_u32(sv);
      bool good = true;
      for (int t = 0; t <= steps && good; ++t) {
        if (t < steps) {
          good = bar_wait(&k_full[t & 1], (t >> 1) & 1, spin);
          if (!good) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int i = 0; i < tiles; ++i) {
            // the scores go where step t - 2 had its probabilities
            if (t >= 2 && !(good = bar_wait(&o_done[i][t & 1], ((t >> 1) - 1) & 1, spin))) break;
            const uint32_t d = tmem + (uint32_t)(i * 128 + (t & 1) * kNK);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (uint32_t)((k % 4) * 32);
              mma_ss(d, desc_k(q0 + i * Sh::kQ + (k / 4) * (128 * 128) + off),
                     desc_k(k0 + (t & 1) * Sh::kKV + (k / 4) * (kNK * 128) + off), id_s, k > 0);
            }
            commit(&s_full[i][t & 1]);
          }
          if (!good) break;
          commit(&k_empty[t & 1]);
        }
        if (t > 0) {
          const int u = t - 1;
          good = bar_wait(&v_full[u & 1], (u >> 1) & 1, spin);
          for (int i = 0; i < tiles && good; ++i) {
            good = bar_wait(&p_full[i][u & 1], (u >> 1) & 1, spin);
            if (!good) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t p = tmem + (uint32_t)(i * 128 + (u & 1) * kNK);
#pragma unroll
            for (int k = 0; k < kNK / 16; ++k)
              mma_ts(t_o + (uint32_t)(i * 128), p + k * 8, desc_mn(v0 + (u & 1) * Sh::kKV + k * 2048, kNK * 128), id_o,
                     (u > 0 || k > 0) ? 1u : 0u);
            commit(&o_done[i][u & 1]);
          }
          if (good) commit(&v_empty[u & 1]);
        }
      }
      if (!good) give_up();
      commit(&drained);
      if (!bar_wait(&drained, 0, kSpin)) atomicOr(a.status, kStatusTimeout);
    }
  } else if ((warp >> 2) < tiles) {
    // -------------------------------------------------------------- softmax
    const int i = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_at = t_o + (uint32_t)(i * 128) + lanes;
    float mx = -INFINITY, l = 0.f;
    bool good = true;
    for (int t = 0; t < steps; ++t) {
      if (!warp_wait(&s_full[i][t & 1], (t >> 1) & 1, spin)) {
        good = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t s_at = tmem + (uint32_t)(i * 128 + (t & 1) * kNK) + lanes;
      uint32_t sr[kNK];
      tmem_load64(s_at, sr);
      float* z = reinterpret_cast<float*>(sr);
      const int left = vis - (t0 + t) * kNK;  // keys of this step that the row sees
      if (__any_sync(0xFFFFFFFFu, left < kNK)) {
#pragma unroll
        for (int j = 0; j < kNK; ++j) z[j] = j < left ? z[j] : -INFINITY;
      }
      float f[4], lv[4], tm = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f[g] = fmaxf(fz * s_ks[t & 7][g], 1e-37f);  // a scale of 0 must not meet an infinite score
        lv[g] = s_lv[t & 7][g];
        float gm = z[16 * g];
#pragma unroll
        for (int j = 1; j < 16; ++j) gm = fmaxf(gm, z[16 * g + j]);
        tm = fmaxf(tm, fmaf(gm, f[g], lv[g]));
      }
      if (__any_sync(0xFFFFFFFFu, tm > mx + 8.f)) {
        const float nm = fmaxf(mx, tm);
        const float al = nm == mx ? 1.f : exp2_fast(mx - nm);
        mx = nm;
        l *= al;
        if (t > 0) {
          // the sums so far: the product of step t - 1 has to be in them
          if (!warp_wait(&o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1, spin)) {
            good = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
          for (int d = 0; d < D; d += 16) {  // few at a time: the scores stay in registers
            uint32_t r[16];
            tmem_load16(o_at + d, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al);
            tmem_store16(o_at + d, r);
          }
          tmem_store_wait();
        }
      }
      const float mu = mx == -INFINITY ? 0.f : mx;
      uint32_t pr[kNK / 2];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float c = lv[g] - mu;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float p0 = exp2_fast(fmaf(z[16 * g + j], f[g], c)), p1 = exp2_fast(fmaf(z[16 * g + j + 1], f[g], c));
          sum += p0 + p1;
          pr[8 * g + j / 2] = pack_half2(p0, p1);
        }
        l = fmaf(sum, s_iv[t & 7][g], l);
      }
      tmem_store(s_at, pr);
      tmem_store_wait();
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&p_full[i][t & 1]);
    }
    if (good && steps > 0) {
      good = warp_wait(&o_done[i][(steps - 1) & 1], ((steps - 1) >> 1) & 1, spin);
    }
    if (!good && lane == 0) give_up();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const bool live = ri < M && (int)threadIdx.x < a.tile;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t pi = ((int64_t)item * a.splits + split) * a.tile + threadIdx.x;
    if (good) {
#pragma unroll
      for (int d = 0; d < D; d += 32) {
        uint32_t r[32];
        if (steps > 0) {
          tmem_load(o_at + d, r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        if (!live) continue;
        const float* x = reinterpret_cast<const float*>(r);
        if (a.splits > 1) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(a.part + pi * D + d + j) =
                make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        } else {
          T* o = out.at(b, row, qh) + d;
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint2*>(o + j) =
                make_uint2(pack2<T>(x[j] * inv, x[j + 1] * inv), pack2<T>(x[j + 2] * inv, x[j + 3] * inv));
        }
      }
      if (live && a.splits > 1) {
        float* ml = a.part + (int64_t)a.B * a.heads * a.mt * a.splits * a.tile * D + pi * 2;
        ml[0] = l > 0.f ? mx : -INFINITY;
        ml[1] = l;
      } else if (live && a.lse) {
        a.lse[((int64_t)b * a.R + row) * a.Hq + qh] = l > 0.f ? (mx + log2f(l)) * 0.693147180559945f : -INFINITY;
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

cudaError_t launch_attn_tc(const AttnArgs& a, const zg_rows* q, const zg_rows* out, int dim, bool int8,
                           int64_t items, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  auto go = [&](auto ev, auto dv, auto iv) {
    using E = typename decltype(ev)::type;
    constexpr int D = decltype(dv)::value;
    auto kern = k_attn_tc<E, D, decltype(iv)::value>;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TcShape<D>::kSmem);
    if (err != cudaSuccess) return;
    kern<<<(unsigned)items, kThreads, TcShape<D>::kSmem, st>>>(a, rows_of<E>(q), rows_of<E>(out), std::min(wait_limit(), kSpin));
    err = cudaGetLastError();
  };
  for_dim(dim, [&](auto dv) {
    auto typed = [&](auto ev) {
      if (int8) go(ev, dv, std::true_type{});
      else go(ev, dv, std::false_type{});
    };
    if (q->dtype == ZG_BF16) typed(Elem<__nv_bfloat16>{});
    else typed(Elem<__half>{});
  });
  return err;
}

}  // namespace zg
