// Attention of many query rows over a history cache, on the 5th-generation
// tensor cores.
//
// One CTA takes up to two tiles of 128 query rows (of one request and key
// head) through 128 keys a step:
//   warp 13     brings codes into a ring of shared buffers by bulk copies, 16
//               keys (always inside one block) a copy;
//   warps 8-11  widen them to halves, exactly, into a ring of three
//               128-byte-swizzled operands: keys, values, keys, ...;
//   warp 12     issues S = Q K^T and O += P V (tcgen05, one thread): S and O
//               live in tensor memory, P replaces S there and is read there;
//   warps 0-7   one thread a row: scores out of tensor memory, running
//               maximum, p = exp2, halves back over the scores.
// The two tiles alternate: one's softmax runs beside the other's products.
// Steps of 128 keys, not 64: a product of 128 rows reads its 128 x 16 slice of
// Q whatever its width, and at 64 columns shared memory, not the tensor
// cores, set its time (80 cycles an instruction of 32).
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

constexpr int kNK = 128;            // keys a step
constexpr int kSoftWarps = 8, kWidenWarps = 4;
constexpr int kThreads = 512;       // four warpgroups, two of them softmax; warps 14 and 15 only lend registers
constexpr int kGroups = kNK / 16;   // groups of 16 keys a step: one block, one scale each
constexpr int kRaw = 4, kWide = 3;  // ring entries, each the keys or the values of a step: codes, halves
// Registers a thread: 128 at launch, 512 threads, all of an SM's 65,536; moved between warpgroups to
// 256 x 184 + 256 x 72 = 65,536, since a softmax thread holds its row of 128 scores.
constexpr int kSoftRegs = 184, kOtherRegs = 72;
constexpr uint32_t kSpin = 1u << 20;  // polls of a wait at most; of those before exit always

template <int D>
struct TcShape {
  static constexpr int kSub = (D + 63) / 64;          // 64-dim subtiles (128-byte rows)
  static constexpr int kTile = kSub * 128 * 128;      // bytes of 128 rows of halves: a query tile, a ring entry
  static constexpr int kCodes = kNK * D;              // bytes of a ring entry of codes
  static constexpr size_t kSmem = (2 + kWide) * kTile + kRaw * kCodes + 1024;
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
// 128 columns.
__device__ __forceinline__ void tmem_load128(uint32_t addr, uint32_t* r) {
  uint32_t *r1 = r + 32, *r2 = r + 64, *r3 = r + 96;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : ZG_R32(r), ZG_R32(r1), ZG_R32(r2), ZG_R32(r3)
      : "r"(addr), "r"(addr + 32), "r"(addr + 64), "r"(addr + 96)
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Largest of three; pairs of floats in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

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
  uint8_t* sq = smem;                        // two query tiles
  uint8_t* wide = sq + 2 * Sh::kTile;        // the ring of halves
  uint8_t* raw = wide + kWide * Sh::kTile;   // the ring of codes
  // Entry n of the rings is the keys (n = 2 t) or the values (n = 2 t + 1) of step t.  s_full, p_full and o_done
  // ([query tile]) have one phase a step; none is passed twice before all who wait for it have seen it, because the
  // scores of step t + 1 come after the products of step t, and those after every warp's probabilities.
  __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw], wide_full[kWide], wide_empty[kWide];
  __shared__ uint64_t q_full, s_full[2], p_full[2], o_done[2], drained;
  // of 16 keys each, a ring of four steps (the codes of step t + 4 come only after the softmax of step t): key
  // scale, log2 of the value scale, and 2^-that
  __shared__ float s_ks[4][kGroups], s_lv[4][kGroups], s_iv[4][kGroups];
  __shared__ uint32_t tmem_base;
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
  const int mine = min(M - m * a.tile, a.tile);  // query rows of this item
  const int tiles = (mine + 127) / 128;          // query tiles in use
  // later rows see no less: the item sees what its last row does, or its request's last
  const int last = min((m * a.tile + mine - 1) / a.G, s.rows - 1);
  const int vmax = last < m * a.tile / a.G ? 0 : visible(a, s, last);
  const int steps_all = (vmax + kNK - 1) / kNK;
  const int per = (steps_all + a.splits - 1) / a.splits;
  const int t0 = min(steps_all, split * per);
  const int steps = __shfl_sync(0xFFFFFFFFu, min(steps_all, t0 + per) - t0, 0);  // uniform, for the compiler too

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
      bar_init(&p_full[i], 4);
      bar_init(&o_done[i], 1);
    }
    bar_init(&q_full, 4 * tiles);
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
  const uint32_t t_o = tmem + 256;  // columns: S of each tile, then O of each
  auto give_up = [&]() { atomicOr(a.status, kStatusTimeout); };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kSoftWarps + kWidenWarps) {
      // ----------------------------------------------------------- widening
      constexpr int C16 = D / 16;         // 16-byte pieces of a code row
      constexpr int N = kNK * C16 / 128;  // pieces a thread
      constexpr int NB = N < 4 ? N : 4;   // of them at a time
      static_assert(N % NB == 0 || D == 96, "");
      const int tid = threadIdx.x - 32 * kSoftWarps;
      for (int n = 0; n < 2 * steps; ++n) {
        const int rs = n % kRaw, ws = n % kWide;
        const int held = s.len - (t0 + n / 2) * kNK;
        if (!warp_wait(&raw_full[rs], (n / kRaw) & 1, spin) ||
            (n >= kWide && !warp_wait(&wide_empty[ws], ((n / kWide) - 1) & 1, spin))) {
          if (lane == 0) give_up();
          break;
        }
        const uint8_t* codes = raw + rs * Sh::kCodes;
        uint8_t* to = wide + ws * Sh::kTile;
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += NB) {
          uint4 w[NB];
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (i0 + i < N) w[i] = *reinterpret_cast<const uint4*>(codes + (tid + 128 * (i0 + i)) * 16);
          if (held < kNK) {  // behind the history: not defined, may be NaN
#pragma unroll
            for (int i = 0; i < NB; ++i)
              if ((tid + 128 * (i0 + i)) / C16 >= held) w[i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            if (i0 + i >= N) continue;
            const int idx = tid + 128 * (i0 + i), r = idx / C16, c = idx % C16;
            uint4 lo, hi;
            codes_half4<INT8>(w[i].x, lo.x, lo.y);
            codes_half4<INT8>(w[i].y, lo.z, lo.w);
            codes_half4<INT8>(w[i].z, hi.x, hi.y);
            codes_half4<INT8>(w[i].w, hi.z, hi.w);
            uint8_t* p = to + (c / 4) * (kNK * 128) + r * 128;
            const int j = (c % 4) * 2;
            // the pieces of both subtiles fall on the same banks: one half of the lanes stores its second piece first
            const bool swap = c >= 4;
            *reinterpret_cast<uint4*>(p + (((j + (swap ? 1 : 0)) ^ (r & 7)) << 4)) = swap ? hi : lo;
            *reinterpret_cast<uint4*>(p + (((j + (swap ? 0 : 1)) ^ (r & 7)) << 4)) = swap ? lo : hi;
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
      // scores of step t for tile i; they replace the probabilities of step t - 1
      auto scores = [&](int t, int i) -> bool {
        const int ws = (2 * t) % kWide;
        if (i == 0 && !warp_wait(&wide_full[ws], ((2 * t) / kWide) & 1, spin)) return false;
        if (t > 0 && !warp_wait(&o_done[i], (t - 1) & 1, spin)) return false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t kd = k0 + ws * (Sh::kTile >> 4), qd = q0 + i * (Sh::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * (128 * 128 >> 4) + (k % 4) * 2;
            mma_ss(tmem + (uint32_t)(i * 128), qd + off, kd + off, id_s, k > 0);
          }
          commit(&s_full[i]);
          if (i == tiles - 1) commit(&wide_empty[ws]);
        }
        __syncwarp();
        return true;
      };
      auto values = [&](int t, int i) -> bool {
        const int ws = (2 * t + 1) % kWide;
        if (i == 0 && !warp_wait(&wide_full[ws], ((2 * t + 1) / kWide) & 1, spin)) return false;
        if (!warp_wait(&p_full[i], t & 1, spin)) return false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t vd = v0 + ws * (Sh::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kNK / 16; ++k)
            mma_ts(t_o + (uint32_t)(i * 128), tmem + (uint32_t)(i * 128 + k * 8), vd + k * (2048 >> 4), id_o,
                   (t > 0 || k > 0) ? 1u : 0u);
          commit(&o_done[i]);
          if (i == tiles - 1) commit(&wide_empty[ws]);
        }
        __syncwarp();
        return true;
      };
      bool good = warp_wait(&q_full, 0, spin);
      for (int i = 0; i < tiles && good; ++i) good = scores(0, i);
      for (int t = 0; t < steps && good; ++t)
        for (int i = 0; i < tiles && good; ++i) good = values(t, i) && (t + 1 == steps || scores(t + 1, i));
      if (!good && lane == 0) give_up();
      if (elect_one()) commit(&drained);
      __syncwarp();
      if (!warp_wait(&drained, 0, kSpin) && lane == 0) give_up();
    } else if (warp == 13) {
      // -------------------------------------------------------------- codes
      // Lane g of eight brings keys 16 g .. 16 g + 15 of a step.  Block numbers are read two steps and scales one step
      // ahead of their use.
      const int g = lane & (kGroups - 1);
      auto block_of = [&](int t) -> int {  // -1: behind the history, or outside the cache (recorded)
        const int key = (t0 + t) * kNK + 16 * g;
        if (t >= steps || key >= s.len) return -1;
        const int blk = a.table[(int64_t)b * a.max_blocks + key / a.bt];
        if (blk >= 0 && blk < a.n_blocks) return blk;
        if (lane < kGroups) atomicOr(a.status, kStatusCache);
        return -1;
      };
      int blk = block_of(0), blk1 = block_of(1);
      float ks = blk < 0 ? 0.f : a.ks[(int64_t)blk * a.heads + h];
      float vs = blk < 0 ? 0.f : a.vs[(int64_t)blk * a.heads + h];
      int issued = 0;
      bool good = true;
      for (int t = 0; t < steps && good; ++t) {
        const int blk2 = block_of(t + 2);
        const float ks1 = blk1 < 0 ? 0.f : a.ks[(int64_t)blk1 * a.heads + h];
        const float vs1 = blk1 < 0 ? 0.f : a.vs[(int64_t)blk1 * a.heads + h];
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, lane < kGroups && blk >= 0)) * (16u * (uint32_t)D);
        const int64_t at = (((int64_t)blk * a.heads + h) * a.bt + ((t0 + t) * kNK + 16 * g) % a.bt) * D;
        for (int side = 0; side < 2; ++side) {
          const int n = 2 * t + side, rs = n % kRaw;
          if (n >= kRaw && !warp_wait(&raw_empty[rs], ((n / kRaw) - 1) & 1, spin)) {
            good = false;
            break;
          }
          if (side == 0 && lane < kGroups) {
            s_ks[t & 3][g] = ks;
            s_lv[t & 3][g] = scale_log2(vs);
            s_iv[t & 3][g] = exp2_fast(-scale_log2(vs));
          }
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&raw_full[rs])),
                         "r"(bytes)
                         : "memory");
          __syncwarp();
          if (lane < kGroups && blk >= 0)
            bulk_load(raw + rs * Sh::kCodes + 16 * g * D, (side ? a.vc : a.kc) + at, 16 * D, &raw_full[rs]);
          issued = n + 1;
        }
        blk = blk1, ks = ks1, vs = vs1, blk1 = blk2;
      }
      if (!good && lane == 0) give_up();
      // every copy has landed before the CTA may end
      for (int n = max(0, issued - kRaw); n < issued; ++n)
        if (!warp_wait(&raw_full[n % kRaw], (n / kRaw) & 1, kSpin) && lane == 0) give_up();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int i = warp >> 2;
    if (i < tiles) {
      // ------------------------------------------------------------ softmax
      const int r = threadIdx.x & 127, ri = m * a.tile + threadIdx.x;
      const bool live = (int)threadIdx.x < mine;
      const int row = ri / a.G, qh = h * a.G + ri % a.G;
      const int vis = live ? visible(a, s, row) : 0;
      float fz;
      {
        // the row, scaled by a power of two, into its query tile as halves
        const T* p = q.at(b, row, qh);
        float x[D / 8][8], top = 0.f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[d][k] = 0.f;
          if (vis > 0) {
            load4(p + 8 * d, x[d]);
            load4(p + 8 * d + 4, x[d] + 4);
          }
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
          for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[d][k]));
        const int ex = row_exponent(top);
        const float dn = __uint_as_float((uint32_t)(127 - ex) << 23);
        fz = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          *reinterpret_cast<uint4*>(sq + i * Sh::kTile + (d / 8) * (128 * 128) + r * 128 + (((d % 8) ^ (r & 7)) << 4)) =
              make_uint4(pack_half2(x[d][0] * dn, x[d][1] * dn), pack_half2(x[d][2] * dn, x[d][3] * dn),
                         pack_half2(x[d][4] * dn, x[d][5] * dn), pack_half2(x[d][6] * dn, x[d][7] * dn));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&q_full);
      }
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + (uint32_t)(i * 128) + lanes, o_at = t_o + (uint32_t)(i * 128) + lanes;
      float mx = -INFINITY, l = 0.f;
      bool good = true;
      for (int t = 0; t < steps; ++t) {
        if (!warp_wait(&s_full[i], t & 1, spin)) {
          good = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        uint32_t sr[kNK];
        tmem_load128(s_at, sr);
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
          tm = fmaxf(tm, fmaf(gm, fmaxf(fz * s_ks[t & 3][g], 1e-37f), s_lv[t & 3][g]));
        }
        if (__any_sync(0xFFFFFFFFu, tm > mx + 8.f)) {
          const float nm = fmaxf(mx, tm);
          const float al = nm == mx ? 1.f : exp2_fast(mx - nm);
          mx = nm;
          l *= al;
          if (t > 0) {  // the sums so far are complete: these scores were made after them
#pragma unroll
            for (int d = 0; d < D; d += 16) {  // few at a time: the scores stay in registers
              uint32_t o[16];
              tmem_load16(o_at + d, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
              tmem_store16(o_at + d, o);
            }
          }
        }
        const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int g2 = 0; g2 < kGroups; g2 += 2) {
          uint32_t pr[16];
#pragma unroll
          for (int g = g2; g < g2 + 2; ++g) {
            const float f = fmaxf(fz * s_ks[t & 3][g], 1e-37f), c = s_lv[t & 3][g] - mu;
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
            l = fmaf(a0 + a1, s_iv[t & 3][g], l);
          }
          tmem_store16(s_at + 8 * g2, pr);
        }
        tmem_store_wait();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&p_full[i]);
      }
      if (good && steps > 0) good = warp_wait(&o_done[i], (steps - 1) & 1, spin);
      if (!good && lane == 0) give_up();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t pi = ((int64_t)item * a.splits + split) * a.tile + threadIdx.x;
      if (good) {
#pragma unroll
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_load(o_at + d, o);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          }
          if (!live) continue;
          const float* x = reinterpret_cast<const float*>(o);
          if (a.splits > 1) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(a.part + pi * D + d + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          } else {
            T* y = out.at(b, row, qh) + d;
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint2*>(y + j) =
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
