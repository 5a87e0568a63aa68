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

template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b);
template <>
__device__ __forceinline__ void store2<__half>(__half* p, float a, float b) {
  *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
}
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

constexpr int kFewThreads = 128;

// Few query rows: one CTA an item (request, key head, 16 rows, part of the
// keys); a row is (token, query head of the group).  Each warp walks its own
// 16-key tiles straight from global memory into matrix fragments: the order
// of the dims inside a product is free, so a lane reads neighbouring bytes.
template <typename T, int D, bool INT8>
__global__ void __launch_bounds__(kFewThreads) k_attn_few(const __grid_constant__ AttnArgs a, const Rows<T> q,
                                                          const Rows<T> out) {
  constexpr int U = D / 32;  // 8-byte units of a key row a lane reads; words of a value row
  __shared__ float sm_m[4][16], sm_l[4][16];
  __shared__ float sm_o[4][16][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  int it = blockIdx.x;
  const int split = it % a.splits;
  it /= a.splits;
  const int item = it;
  const int m = it % a.mt;
  it /= a.mt;
  const int h = it % a.heads, b = it / a.heads;
  const Seen s = seen_of(a, b, threadIdx.x == 0);
  const int M = a.R * a.G;

  int vis[2], row[2], qh[2];
  uint32_t qa[2 * U][4];
  float fz[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = m * 16 + g + 8 * e;
    row[e] = i / a.G;
    qh[e] = h * a.G + i % a.G;
    vis[e] = i < M ? visible(a, s, row[e]) : 0;
    float x[U][8];
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[u][k] = 0.f;
      if (vis[e] > 0) {
        load4(q.at(b, row[e], qh[e]) + u * 32 + c * 8, x[u]);
        load4(q.at(b, row[e], qh[e]) + u * 32 + c * 8 + 4, x[u] + 4);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[u][k]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int ex = row_exponent(top);
    const float dn = __uint_as_float((uint32_t)(127 - ex) << 23);
    fz[e] = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qa[2 * u + k][e] = pack_half2(x[u][4 * k] * dn, x[u][4 * k + 1] * dn);
        qa[2 * u + k][2 + e] = pack_half2(x[u][4 * k + 2] * dn, x[u][4 * k + 3] * dn);
      }
  }
  int vmax = max(vis[0], vis[1]);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) vmax = max(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, o));
  const int tiles = (vmax + 15) / 16;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int t0 = split * per, t1 = min(tiles, t0 + per);

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
  float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int t = t0 + warp; t < t1; t += 4) {
    const int key0 = t * 16;
    const int blk = a.table[(int64_t)b * a.max_blocks + key0 / a.bt];
    if (blk < 0 || blk >= a.n_blocks) {
      if (lane == 0) atomicOr(a.status, kStatusCache);
      continue;
    }
    const int64_t bh = (int64_t)blk * a.heads + h;
    const uint8_t* kp = a.kc + (bh * a.bt + key0 % a.bt) * D;
    const uint8_t* vp = a.vc + (bh * a.bt + key0 % a.bt) * D;
    const float ks = a.ks[bh], lv = scale_log2(a.vs[bh]), iv = exp2_fast(-lv);
    uint2 kw[2][U];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int u = 0; u < U; ++u) kw[n][u] = *reinterpret_cast<const uint2*>(kp + (n * 8 + g) * D + u * 32 + c * 8);
    uint32_t vw[4][U];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = 2 * c + (k & 1) + (k >> 1) * 8;
#pragma unroll
      for (int u = 0; u < U; ++u)
        vw[k][u] = *reinterpret_cast<const uint32_t*>(vp + key * D + g * (D / 8) + 4 * u);
      if (key0 + key >= s.len) {  // behind the history: not defined, may be NaN
#pragma unroll
        for (int u = 0; u < U; ++u) vw[k][u] = 0;
      }
    }
    float z[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t b0, b1;
        codes_half4<INT8>(kw[n][u].x, b0, b1);
        mma_16816(z[n], qa[2 * u], b0, b1);
        codes_half4<INT8>(kw[n][u].y, b0, b1);
        mma_16816(z[n], qa[2 * u + 1], b0, b1);
      }
    float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = key0 + n * 8 + 2 * c + (k & 1);
        z[n][k] = key < vis[k >> 1] ? fmaf(z[n][k], fz[k >> 1] * ks, lv) : -INFINITY;
        tm[k >> 1] = fmaxf(tm[k >> 1], z[n][k]);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xFFFFFFFFu, tm[e], 1));
      tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xFFFFFFFFu, tm[e], 2));
    }
    if (__any_sync(0xFFFFFFFFu, tm[0] > mx[0] + 8.f || tm[1] > mx[1] + 8.f)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float nm = fmaxf(mx[e], tm[e]);
        const float f = mx[e] == -INFINITY ? 0.f : exp2_fast(mx[e] - nm);
        mx[e] = nm;
        l[e] *= f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * e] *= f;
          o[j][2 * e + 1] *= f;
        }
      }
    }
    uint32_t pa[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float mu = mx[e] == -INFINITY ? 0.f : mx[e];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = exp2_fast(z[n][2 * e] - mu), p1 = exp2_fast(z[n][2 * e + 1] - mu);
        l[e] = fmaf(p0 + p1, iv, l[e]);
        pa[2 * n + e] = pack_half2(p0, p1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t b0[4], b1[4];  // four dims: (key 2c, key 2c + 1), and 8 keys on
      codes_half4<INT8>(__byte_perm(vw[0][u], vw[1][u], 0x5140), b0[0], b0[1]);
      codes_half4<INT8>(__byte_perm(vw[0][u], vw[1][u], 0x7362), b0[2], b0[3]);
      codes_half4<INT8>(__byte_perm(vw[2][u], vw[3][u], 0x5140), b1[0], b1[1]);
      codes_half4<INT8>(__byte_perm(vw[2][u], vw[3][u], 0x7362), b1[2], b1[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_16816(o[4 * u + k], pa, b0[k], b1[k]);
    }
  }

  // join the warps: column j of accumulator tile jj is dim (2c + j) * D/8 + jj
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
    l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
    if (c == 0) {
      sm_m[warp][g + 8 * e] = mx[e];
      sm_l[warp][g + 8 * e] = l[e];
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      sm_o[warp][g + 8 * e][2 * c * (D / 8) + j] = o[j][2 * e];
      sm_o[warp][g + 8 * e][(2 * c + 1) * (D / 8) + j] = o[j][2 * e + 1];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * (D / 2); i += kFewThreads) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2));
    const int ri = m * 16 + r;
    if (ri >= M) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, sm_m[w][r]);
    float sum = 0.f, x0 = 0.f, x1 = 0.f;
    if (top != -INFINITY) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2_fast(sm_m[w][r] - top);
        sum = fmaf(f, sm_l[w][r], sum);
        x0 = fmaf(f, sm_o[w][r][d], x0);
        x1 = fmaf(f, sm_o[w][r][d + 1], x1);
      }
    }
    if (a.splits > 1) {
      const int64_t pi = ((int64_t)item * a.splits + split) * 16 + r;
      *reinterpret_cast<float2*>(a.part + pi * D + d) = make_float2(x0, x1);
      if (d == 0) {
        float* ml = a.part + (int64_t)a.B * a.heads * a.mt * a.splits * 16 * D + pi * 2;
        ml[0] = top;
        ml[1] = sum;
      }
    } else {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int tr = ri / a.G, th = h * a.G + ri % a.G;
      store2(out.at(b, tr, th) + d, x0 * inv, x1 * inv);
      if (a.lse && d == 0)
        a.lse[((int64_t)b * a.R + tr) * a.Hq + th] =
            top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
    }
  }
}

// Joins the parts of the keys: one warp a (request, row, query head).
template <typename T, int D>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ AttnArgs a, const Rows<T> out) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.B * a.R * a.Hq) return;
  const int qh = (int)(w % a.Hq);
  const int64_t br = w / a.Hq;
  const int r = (int)(br % a.R), b = (int)(br / a.R);
  const int i = r * a.G + qh % a.G;
  const int64_t item = ((int64_t)b * a.heads + qh / a.G) * a.mt + i / a.tile;
  const float* ml = a.part + (int64_t)a.B * a.heads * a.mt * a.splits * a.tile * D;
  const int64_t p0 = item * a.splits * a.tile + i % a.tile;
  float top = -INFINITY;
  for (int sp = lane; sp < a.splits; sp += 32) top = fmaxf(top, ml[(p0 + (int64_t)sp * a.tile) * 2]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.f, x[D / 32] = {};
  if (top != -INFINITY) {
    for (int sp = 0; sp < a.splits; ++sp) {
      const int64_t pi = p0 + (int64_t)sp * a.tile;
      const float f = exp2_fast(ml[pi * 2] - top);
      sum = fmaf(f, ml[pi * 2 + 1], sum);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) x[k] = fmaf(f, a.part[pi * D + lane + 32 * k], x[k]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  T* p = out.at(b, r, qh);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) p[lane + 32 * k] = (T)(x[k] * inv);
  if (a.lse && lane == 0)
    a.lse[w] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

// ---------------------------------------------------------------- host side

struct AttnPlan {
  bool tc;
  int tile, mt, splits;
  int64_t items;
  size_t bytes;
};

constexpr int kFewRows = 32;  // query rows a key head up to which k_attn_few is the faster

// Few rows: items for every SM several times over, 256 keys a part at least.
// Many rows: parts only where items leave SMs idle, 512 keys each at least.
AttnPlan attn_plan(const zg_kv_cache* c, int max_blocks, int B, int R, int Hq) {
  AttnPlan p;
  const int64_t M = (int64_t)R * (Hq / c->heads);
  p.tc = M > kFewRows;
  p.tile = p.tc ? attn_tc_tile(M) : 16;
  p.mt = (int)((M + p.tile - 1) / p.tile);
  p.items = (int64_t)B * c->heads * p.mt;
  const int64_t keys = (int64_t)max_blocks * c->block_tokens;
  const int64_t most = std::max<int64_t>(1, keys / (p.tc ? 512 : 256));
  int64_t want = 1;
  if (p.items) want = p.tc ? sm_count() / p.items : ((int64_t)sm_count() * 8 + p.items - 1) / p.items;
  p.splits = (int)std::max<int64_t>(1, std::min(want, most));
  p.bytes = p.splits > 1 ? (size_t)p.items * p.splits * p.tile * (c->dim + 2) * 4 : 0;
  return p;
}

zg_status check_attn(const zg_kv_cache* c, int32_t max_blocks, int32_t B, int32_t R, int32_t Hq, const char* call) {
  if (B < 0 || R < 0) return bad_arg(call, "B and R must be >= 0");
  if (Hq < 1 || Hq > 1024 || Hq % c->heads) return bad_arg(call, "Hq must be a multiple of cache.heads, at most 1024");
  if ((int64_t)B * R >= 0x80000000LL / Hq) return bad_arg(call, "B * R * Hq must be below 2^31");
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
  *bytes = attn_plan(cache, max_blocks, B, R, Hq).bytes;
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
  if ((st = check_rows(q, "q", -1, call)) != ZG_OK) return st;
  if (q->dtype == ZG_F32) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_attention: q must be ZG_BF16 or ZG_F16");
  if ((st = check_rows(out, "out", q->dtype, call)) != ZG_OK) return st;
  if (!length) return bad_arg(call, "length is NULL");
  if (!(scale > 0.f && std::isfinite(scale))) return bad_arg(call, "scale must be finite and > 0");
  if (lse && reinterpret_cast<uintptr_t>(lse) % 4) return bad_arg(call, "lse must be 4-byte aligned");
  if (B == 0 || R == 0) return ZG_OK;
  const AttnPlan p = attn_plan(cache, max_blocks, B, R, Hq);
  if (p.bytes && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < p.bytes))
    return bad_arg(call, "workspace must hold zg_kv_attention_workspace_size bytes, 256-byte aligned");
  if (p.items * p.splits > 0x7FFFFFFF) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_attention: more than 2^31 CTAs");
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
  a.max_blocks = max_blocks;
  a.B = B;
  a.R = R;
  a.Hq = Hq;
  a.G = Hq / cache->heads;
  a.tile = p.tile;
  a.mt = p.mt;
  a.splits = p.splits;
  a.causal = causal != 0;
  a.scale = scale * 1.4426950408889634f;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto ev, auto dv, auto iv) {
    using E = typename decltype(ev)::type;
    constexpr int D = decltype(dv)::value;
    if (!p.tc)
      k_attn_few<E, D, decltype(iv)::value>
          <<<(unsigned)(p.items * p.splits), kFewThreads, 0, sm>>>(a, rows_of<E>(q), rows_of<E>(out));
    if (p.splits > 1) {
      const int64_t warps = (int64_t)B * R * Hq;
      k_attn_join<E, D><<<(unsigned)((warps + 7) / 8), 256, 0, sm>>>(a, rows_of<E>(out));
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
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ZG_OK : cuda_fail(e, "cache attention launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

}  // extern "C"
