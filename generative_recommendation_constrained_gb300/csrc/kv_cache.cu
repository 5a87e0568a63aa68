// The history cache's writes: per-head norm and rotation, quantised writes,
// reads.  All are bound by memory; each input element is loaded once and each
// output written once, with 32-bit arithmetic between.
//
//   norm     y = x / sqrt(mean(x^2) + eps) * gain over a head
//   rotation (a, b) -> (a cos - b sin, a sin + b cos) by position * frequency
//   code     rne(y * inv), scale = max |y| of a (block, head) / Q, and inv the
//            reciprocal of max |y| * (1 / Q), which differs from the scale's
//            in its last bits at most: a tensor divided by a number is a
//            product with the number's reciprocal in torch, and the codes
//            equal those of elementary float32 operations bit for bit
//
// A lane holds eight elements of a head as two vectors of four that make four
// whole rotation pairs, so the rotation needs no exchange between lanes and
// the norm one short shuffle sum.
#include <cfloat>
#include <cmath>
#include <string>

#include "kv.cuh"

namespace zg {
namespace {

// ---------------------------------------------------------- norm + rotation

template <typename T>
struct RotateArgs {
  Rows<T> q, k, qo, ko;
  const int32_t* pos;
  int32_t B, T_, Hq, Hk, chunk, nchunk;  // heads a group of lanes walks; such chunks a token
  NormRopeArgs nr;
};

constexpr int kAhead = 4;  // heads that a lane group has in flight

// `n` heads of one token through a lane group, kAhead of them in flight in
// shared memory (each thread waits for its own elements alone; `ring`: this
// thread's first four, `step` elements to the next).  Every lane of the warp
// takes part `most` times.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void turn_heads(const NormRopeArgs& a, const LaneMap& m, const Turn& t, const T* from,
                                           int64_t from_step, T* to, int64_t to_step, int n, int most, T* ring,
                                           int step) {
  from += m.e0;
  to += m.e0;
  const int d = m.e1 - m.e0;
  auto fetch = [&](int i) {
    if (i < n) {
      T* s = ring + (i % kAhead) * 2 * step;
      copy4_async(s, from);
      copy4_async(s + step, from + d);
    }
    from += from_step;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch(i);
  for (int i = 0; i < most; ++i) {
    fetch(i + kAhead - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    float x[8] = {};
    if (i < n) {
      const T* s = ring + (i % kAhead) * 2 * step;
      load4(s, x);
      load4(s + step, x + 4);
    }
    norm_rotate<D, INTER>(a, t, x);
    if (i < n) {
      store4(to, x);
      store4(to + d, x + 4);
    }
    to += to_step;
  }
}

// One group of lanes a (token, chunk of heads): the angles are computed once
// for the chunk.  Bound by memory: 32 x 4,096 tokens of 20 heads of 128 (bf16,
// 1.34 GB in and out) take 203 us, 6.6 TB/s of 6.75 copied; with a head at a
// time in registers 338 us, with four 571 (94 registers).  Heads 0..Hq-1 are the queries, Hq..Hq+Hk-1 the keys.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256) k_norm_rope(const __grid_constant__ RotateArgs<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  __shared__ __align__(16) T ring[kAhead * 2 * 256 * 4];
  after_predecessor();
  const int l = threadIdx.x % GS;
  const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS;
  const int64_t token = g / a.nchunk;
  const bool live = token < (int64_t)a.B * a.T_;
  const int b = live ? (int)(token / a.T_) : 0, t = live ? (int)(token % a.T_) : 0;
  const int h0 = (int)(g % a.nchunk) * a.chunk, h1 = min(h0 + a.chunk, a.Hq + a.Hk);
  const LaneMap m = lane_map<D, INTER>(a.nr, l);
  const bool on = live && m.used;
  float sn[4], cs[4];
  lane_angles(a.nr, m, l, live && a.nr.rot ? a.pos[token] : 0, sn, cs);
  T* mine = ring + threadIdx.x * 4;
  // a warp's lane groups may hold different chunks: each side as often as the largest needs
  if (a.Hq) {
    const Turn tq = turn_of(sn, cs, lane_gain<INTER>(a.nr.q_gain, m));
    turn_heads<T, D, INTER>(a.nr, m, tq, a.q.at(b, t, h0), a.q.sh, a.qo.at(b, t, h0), a.qo.sh,
                            on ? min(h1, a.Hq) - h0 : 0, min(a.chunk, a.Hq), mine, 256 * 4);
  }
  if (a.Hk) {
    const Turn tk = turn_of(sn, cs, lane_gain<INTER>(a.nr.k_gain, m));
    const int k0 = max(h0, a.Hq);
    turn_heads<T, D, INTER>(a.nr, m, tk, a.k.at(b, t, k0 - a.Hq), a.k.sh, a.ko.at(b, t, k0 - a.Hq), a.ko.sh,
                            on ? h1 - k0 : 0, min(a.chunk, a.Hk), mine, 256 * 4);
  }
}

// ------------------------------------------------------------------- append

struct CacheView {
  uint8_t *kc, *vc;
  float *ks, *vs;
  int32_t n_blocks, heads, bt, max_blocks;
  const int32_t* table;
  uint32_t* status;
};

template <typename T>
struct AppendArgs {
  CacheView c;
  Rows<T> k, v, q, qo;
  const int32_t *start, *n_new;
  int32_t B, T_, Hq, jmax;      // jmax: blocks that T_ tokens may touch
  int32_t pieces, kv_ctas, chunk, nchunk;
  int32_t has_nr;
  NormRopeArgs nr;
};

constexpr int kPasses = 8;  // rows a lane group keeps in registers

// What a CTA writes at a time: one side and head of one block.
struct Piece {
  int b, h, side, bj, blk, lo, hi, start;  // rows lo..hi-1 of the block; hi <= lo: none
};

// Persistent CTAs, one piece after the other: the rows of the next piece come
// into shared memory (each thread its own elements, so only it waits) while
// this one's are turned, kept in registers between the maximum and the codes,
// and written.  CTAs past kv_ctas turn the queries.  Bound by issue and the
// chains of its shuffles: 32 x 2,048 tokens, 16 + 4 heads of 128, bf16 to e4m3
// with norm and rotation take 156 us (738 MB, 4.7 TB/s); a piece a CTA, loaded
// into registers, took 387.
template <typename T, int D, bool INT8, bool INTER>
__global__ void __launch_bounds__(256, 2) k_kv_append(const __grid_constant__ AppendArgs<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  constexpr float Q = INT8 ? 127.f : 448.f;
  extern __shared__ __align__(16) uint8_t stage_raw[];  // [2][kPasses][2][threads][4]
  __shared__ float red[2][8];
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS, rpp = blockDim.x / GS;
  const LaneMap m = lane_map<D, INTER>(a.nr, l);
  after_predecessor();

  if (blockIdx.x >= a.kv_ctas) {
    const int64_t g = (int64_t)(blockIdx.x - a.kv_ctas) * rpp + grp;
    const int64_t token = g / a.nchunk;
    const bool live = token < (int64_t)a.B * a.T_;
    const int b = live ? (int)(token / a.T_) : 0, t = live ? (int)(token % a.T_) : 0;
    const int h0 = (int)(g % a.nchunk) * a.chunk;
    float sn[4], cs[4];
    lane_angles(a.nr, m, l, live ? a.start[b] + t : 0, sn, cs);
    const Turn tq = turn_of(sn, cs, lane_gain<INTER>(a.nr.q_gain, m));
    turn_heads<T, D, INTER>(a.nr, m, tq, a.q.at(b, t, h0), a.q.sh, a.qo.at(b, t, h0), a.qo.sh,
                            live && m.used ? min(a.chunk, a.Hq - h0) : 0, a.chunk,
                            reinterpret_cast<T*>(stage_raw) + threadIdx.x * 4, blockDim.x * 4);
    return;
  }

  const int step = blockDim.x * 4;
  auto piece_of = [&](int it) -> Piece {
    Piece p;
    p.h = it % a.c.heads;
    it /= a.c.heads;
    p.side = it & 1;
    it >>= 1;
    const int j = it % a.jmax;
    p.b = it / a.jmax;
    p.start = a.start[p.b];
    p.lo = p.hi = 0;
    p.blk = -1;
    const int n = a.n_new ? a.n_new[p.b] : a.T_;
    if (p.start < 0 || n < 0 || n > a.T_ || (int64_t)p.start + n > (int64_t)a.c.max_blocks * a.c.bt) {
      if (threadIdx.x == 0) atomicOr(a.c.status, kStatusCache);
      return p;
    }
    p.bj = p.start / a.c.bt + j;
    const int64_t left = (int64_t)p.start + n - (int64_t)p.bj * a.c.bt;
    p.lo = j ? 0 : p.start - p.bj * a.c.bt;
    const int hi = left < a.c.bt ? (int)left : a.c.bt;
    if (n == 0 || hi <= p.lo) return p;
    p.blk = a.c.table[(int64_t)p.b * a.c.max_blocks + p.bj];
    if (p.blk < 0 || p.blk >= a.c.n_blocks) {
      if (threadIdx.x == 0) atomicOr(a.c.status, kStatusCache);
      return p;
    }
    p.hi = hi;
    return p;
  };
  auto fetch = [&](const Piece& p, int buf) {
    const Rows<T>& src = p.side ? a.v : a.k;
    T* to = reinterpret_cast<T*>(stage_raw) + buf * kPasses * 2 * step + threadIdx.x * 4;
    const T* s = src.at(p.b, p.bj * a.c.bt + p.lo + grp - p.start, p.h) + m.e0;
    const int64_t down = rpp * src.st;
#pragma unroll
    for (int i = 0; i < kPasses; ++i, s += down) {
      if (m.used && p.lo + i * rpp + grp < p.hi) {
        copy4_async(to + 2 * i * step, s);
        copy4_async(to + (2 * i + 1) * step, s + (m.e1 - m.e0));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  const LaneGain gk = lane_gain<INTER>(a.has_nr ? a.nr.k_gain : nullptr, m);
  float ds[4], dc[4];
  lane_angles(a.nr, m, l, rpp, ds, dc);
  Piece cur = piece_of(blockIdx.x);
  fetch(cur, 0);
  int buf = 0, red_of = 0;  // `red` alternates over the pieces that use it
  for (int it = blockIdx.x; it < a.pieces; it += a.kv_ctas, buf ^= 1) {
    Piece nxt = cur;
    if (it + a.kv_ctas < a.pieces) {
      nxt = piece_of(it + a.kv_ctas);
      fetch(nxt, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (cur.hi > cur.lo) {  // uniform over the CTA
      const int lo = cur.lo, hi = cur.hi;
      const int64_t bh = (int64_t)cur.blk * a.c.heads + cur.h;
      float* scale = (cur.side ? a.c.vs : a.c.ks) + bh;
      uint8_t* codes = (cur.side ? a.c.vc : a.c.kc) + bh * a.c.bt * D;
      const bool turn = !cur.side && a.has_nr;
      const float s0 = lo ? *scale : 0.f;
      const T* from = reinterpret_cast<const T*>(stage_raw) + buf * kPasses * 2 * step + threadIdx.x * 4;
      float x[kPasses][8], sn[4], cs[4];
      float top = 0.f;
      bool bad = false;
      // four passes at a time without a branch between them, so that their chains of shuffles and roots overlap
#pragma unroll
      for (int p0 = 0; p0 < kPasses; p0 += 4) {
        const bool some = lo + p0 * rpp < hi;  // uniform over the CTA
#pragma unroll
        for (int p = p0; p < p0 + 4; ++p) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[p][i] = 0.f;
          if (m.used && lo + p * rpp + grp < hi) {
            load4(from + 2 * p * step, x[p]);
            load4(from + (2 * p + 1) * step, x[p] + 4);
          }
        }
        if (!some) continue;
        if (turn) {
#pragma unroll
          for (int p = p0; p < p0 + 4; ++p) {
            // rows rpp apart: the next angle by one complex product (at most 7 of them, each within 2^-23)
            if (p == 0) {
              lane_angles(a.nr, m, l, cur.bj * a.c.bt + lo + grp, sn, cs);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float s = sn[i] * dc[i] + cs[i] * ds[i];
                cs[i] = cs[i] * dc[i] - sn[i] * ds[i];
                sn[i] = s;
              }
            }
            norm_rotate<D, INTER>(a.nr, turn_of(sn, cs, gk), x[p]);
          }
        }
        float big = 0.f;
        uint64_t all2 = 0;  // 0.f, 0.f
#pragma unroll
        for (int p = p0; p < p0 + 4; ++p) {  // rows that are not there are zero
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            big = fmaxf(big, fmaxf(fabsf(x[p][i]), fabsf(x[p][i + 1])));
            all2 = add2(all2, pair(x[p][i], x[p][i + 1]));
          }
        }
        float all, all1;
        unpair(all2, all, all1);
        if (!(fabsf(all + all1) <= FLT_MAX)) {  // a NaN or an infinity (or a sum past the range)
          big = 0.f;
#pragma unroll
          for (int p = p0; p < p0 + 4; ++p)
            if (m.used && lo + p * rpp + grp < hi) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (fabsf(x[p][i]) <= FLT_MAX) {
                  big = fmaxf(big, fabsf(x[p][i]));
                } else {  // NaN -> 0; an infinity saturates
                  bad = true;
                  x[p][i] = isnan(x[p][i]) ? 0.f : copysignf(FLT_MAX, x[p][i]);
                }
              }
            }
        }
        top = fmaxf(top, big);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      if (blockDim.x > 32) {
        if ((threadIdx.x & 31) == 0) red[red_of][threadIdx.x >> 5] = top;
        __syncthreads();  // also: every thread has read the old scale
        for (int w = 0; w < (int)blockDim.x / 32; ++w) top = fmaxf(top, red[red_of][w]);
      } else {
        __syncwarp();
      }
      red_of ^= 1;
      float s1 = fmaxf(s0, __fdiv_rn(top, Q));
      if (s1 < FLT_MIN) s1 = 0.f;  // 1 / s1 stays finite
      const float inv = s1 > 0.f ? __frcp_rn(fmaxf(s0, top * (1.f / Q))) : 0.f;
      if (threadIdx.x == 0) *scale = s1;
      if (bad) atomicOr(a.c.status, kStatusNonFinite);
      if (s1 > s0 && m.used) {
        for (int r = grp; r < lo; r += rpp) {  // rows held already: the scale has grown
          uint32_t* w0 = reinterpret_cast<uint32_t*>(codes + r * D + m.e0);
          uint32_t* w1 = reinterpret_cast<uint32_t*>(codes + r * D + m.e1);
          float y[8];
          codes_float4<INT8>(*w0, y);
          codes_float4<INT8>(*w1, y + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= s0;
          *w0 = float4_codes<INT8>(y, inv);
          *w1 = float4_codes<INT8>(y + 4, inv);
        }
      }
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = lo + p * rpp + grp;
        if (m.used && r < hi) {
          *reinterpret_cast<uint32_t*>(codes + r * D + m.e0) = float4_codes<INT8>(x[p], inv);
          *reinterpret_cast<uint32_t*>(codes + r * D + m.e1) = float4_codes<INT8>(x[p] + 4, inv);
        }
      }
    }
    cur = nxt;
  }
}

// --------------------------------------------------------------------- read

template <typename T>
struct ReadArgs {
  CacheView c;
  Rows<T> ko, vo;
  const int32_t *start, *n;
  int32_t B, T_, sides, side0, chunk, nchunk;  // heads a group walks; such chunks a (token, side)
};

// One group of lanes a (token, side, chunk of heads), eight codes a lane and
// head, four heads in flight.  16 x 1,000 tokens of 4 heads of 64 written and
// read back: 17 us (a group a head, with its divisions, 4 us more).
template <typename T, int D, bool INT8>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ ReadArgs<T> a) {
  constexpr int GS = HeadLanes<D>::kGroup;
  after_predecessor();
  const int l = threadIdx.x % GS;
  const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / GS;
  if (g >= (int64_t)a.B * a.T_ * a.sides * a.nchunk || l >= HeadLanes<D>::kUsed) return;
  uint32_t x = (uint32_t)g;  // below 2^31 / GS CTAs of 256 / GS groups
  const int h0 = (int)(x % a.nchunk) * a.chunk, h1 = min(h0 + a.chunk, a.c.heads);
  x /= a.nchunk;
  const int side = a.side0 + (int)(x % a.sides);
  x /= a.sides;
  const int t = (int)(x % a.T_), b = (int)(x / a.T_);
  const int n = a.n ? a.n[b] : a.T_, start = a.start[b];
  int blk = -1, row = 0;
  if (t < n) {
    const int64_t p = (int64_t)start + t;
    if (start >= 0 && p < (int64_t)a.c.max_blocks * a.c.bt) {
      blk = a.c.table[(int64_t)b * a.c.max_blocks + (uint32_t)p / a.c.bt];
      row = (uint32_t)p % a.c.bt;
    }
    if (blk < 0 || blk >= a.c.n_blocks) {
      if (l == 0) atomicOr(a.c.status, kStatusCache);
      blk = -1;
    }
  }
  const Rows<T>& out = side ? a.vo : a.ko;
  T* o = out.at(b, t, h0) + 8 * l;
  const int64_t bh = (int64_t)max(blk, 0) * a.c.heads + h0;
  const float* scale = (side ? a.c.vs : a.c.ks) + bh;
  const uint8_t* codes = (side ? a.c.vc : a.c.kc) + (bh * a.c.bt + row) * D + 8 * l;
  for (int h = h0; h < h1; h += 4, scale += 4, codes += 4 * a.c.bt * D) {
    uint2 w[4];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = make_uint2(0, 0);
      s[i] = 0.f;
      if (blk >= 0 && h + i < h1) {
        w[i] = *reinterpret_cast<const uint2*>(codes + i * a.c.bt * D);
        s[i] = scale[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + i >= h1) break;
      float y[8];
      codes_float4<INT8>(w[i].x, y);
      codes_float4<INT8>(w[i].y, y + 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= s[i];
      store4(o, y);
      store4(o + 4, y + 4);
      o += out.sh;
    }
  }
}

// ---------------------------------------------------------------- host side

// Tokens (rows) of a call at most, so that products with heads and lanes (2^11 and 2^4
// at most) stay inside 64 bits.
constexpr int64_t kMostRows = (int64_t)1 << 40;
// Pieces of a write and CTAs at most: a CTA that steps past the last piece
// stays below 2^31.
constexpr int64_t kMostPieces = 0x7FF00000;

bool dim_ok(int d) { return d == 32 || d == 64 || d == 96 || d == 128; }

// zg_norm_rope (NULL: neither norm nor rotation) as a kernel argument.
zg_status nr_args(const zg_norm_rope* nr, int dim, const char* call, NormRopeArgs* o) {
  *o = {};
  if (!nr) return ZG_OK;
  if (nr->rot_dim < 0 || nr->rot_dim > dim || nr->rot_dim % 8)
    return bad_arg(call, "rot_dim must be a multiple of 8 in [0, dim]");
  if (nr->norm && !(nr->eps >= 0.f && std::isfinite(nr->eps))) return bad_arg(call, "eps must be finite and >= 0");
  if ((reinterpret_cast<uintptr_t>(nr->q_gain) | reinterpret_cast<uintptr_t>(nr->k_gain)) % 4)
    return bad_arg(call, "gains must be aligned to 4 bytes");
  if (nr->rot_dim && !nr->freq && !(nr->theta >= 1.0 && std::isfinite(nr->theta)))
    return bad_arg(call, "theta must be finite and >= 1 (or freq given)");
  o->norm = nr->norm != 0;
  o->rot = nr->rot_dim;
  o->inter = nr->interleaved != 0;
  o->eps = nr->eps;
  if (o->norm) {  // the gains belong to the norm
    o->q_gain = nr->q_gain;
    o->k_gain = nr->k_gain;
  }
  // theta^(-2i/rot_dim) by doubling: seven powers and one product each (seven roundings at most) instead of 64 powers
  double f[64] = {1.0};
  const int n = nr->rot_dim / 2;
  if (nr->freq)
    for (int i = 0; i < n; ++i) f[i] = nr->freq[i];
  else
    for (int w = 1; w < n; w *= 2) {
      const double r = std::pow(nr->theta, -2.0 * w / nr->rot_dim);
      for (int i = w; i < std::min(2 * w, n); ++i) f[i] = f[i - w] * r;
    }
  for (int i = 0; i < n; ++i) {
    if (!(f[i] >= 0.0 && f[i] <= 4.0)) return bad_arg(call, "freq must be in [0, 4]");
    o->turns[i] = (uint64_t)(f[i] / 6.283185307179586476925 * 18446744073709551616.0);
  }
  return ZG_OK;
}

CacheView view(const zg_kv_cache* c, const int32_t* table, int32_t max_blocks, uint32_t* status) {
  return {static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scale, c->v_scale,
          c->n_blocks, c->heads, c->block_tokens, max_blocks, table, status};
}

template <typename F>
void for_type(int dtype, F&& f) {
  if (dtype == ZG_F32) f(Elem<float>{});
  else if (dtype == ZG_BF16) f(Elem<__nv_bfloat16>{});
  else f(Elem<__half>{});
}

int group_lanes(int dim) { return dim == 96 ? 16 : dim / 8; }

// Heads a lane group walks: all of a token's when there are tokens enough for
// every SM, fewer when there are not.
int head_chunk(int64_t tokens, int heads, int lanes) {
  const int64_t room = (int64_t)sm_count() * 1024;  // threads that keep the memory busy
  const int64_t all = tokens * heads * lanes;
  return (int)std::max<int64_t>(1, std::min<int64_t>(heads, all / room));
}

}  // namespace

zg_status bad_arg(const char* call, const std::string& what) {
  return fail(ZG_ERR_INVALID_ARG, std::string(call) + ": " + what);
}

zg_status check_rows(const zg_rows* r, const char* name, int dtype, const char* call) {
  if (!r || !r->data) return bad_arg(call, std::string(name) + " is NULL");
  if (r->dtype != ZG_F32 && r->dtype != ZG_BF16 && r->dtype != ZG_F16)
    return bad_arg(call, std::string(name) + ".dtype must be ZG_F32, ZG_BF16 or ZG_F16");
  if (dtype >= 0 && r->dtype != dtype) return bad_arg(call, std::string(name) + " must have the type of the other rows");
  if (r->stride_b < 0 || r->stride_t < 0 || r->stride_h < 0 || (r->stride_b | r->stride_t | r->stride_h) % 4)
    return bad_arg(call, std::string(name) + " strides must be non-negative multiples of 4");
  if (reinterpret_cast<uintptr_t>(r->data) % (r->dtype == ZG_F32 ? 16 : 8))
    return bad_arg(call, std::string(name) + ".data must be aligned to 4 elements");
  return ZG_OK;
}

zg_status check_cache(const zg_kv_cache* c, const int32_t* table, int32_t max_blocks, const char* call) {
  if (!c) return bad_arg(call, "cache is NULL");
  if (c->format != ZG_KV_E4M3 && c->format != ZG_KV_INT8)
    return bad_arg(call, "cache.format must be ZG_KV_E4M3 or ZG_KV_INT8");
  if (c->n_blocks < 1 || c->heads < 1 || c->heads > 1024)
    return bad_arg(call, "cache needs n_blocks >= 1 and heads in [1, 1024]");
  const int t = c->block_tokens;
  if (t != 16 && t != 32 && t != 64 && t != 128)
    return bad_arg(call, "cache.block_tokens must be 16, 32, 64 or 128");
  if (!dim_ok(c->dim)) return fail(ZG_ERR_UNSUPPORTED, std::string(call) + ": cache.dim must be 32, 64, 96 or 128");
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return bad_arg(call, "cache pointer is NULL");
  if ((reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes)) % 16)
    return bad_arg(call, "cache codes must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) % 4)
    return bad_arg(call, "cache scales must be 4-byte aligned");
  if (!table || reinterpret_cast<uintptr_t>(table) % 4) return bad_arg(call, "table is NULL or not 4-byte aligned");
  if (max_blocks < 1 || (int64_t)max_blocks * c->block_tokens > 0x7FFFFFFF)
    return bad_arg(call, "max_blocks must be >= 1 with max_blocks * block_tokens below 2^31");
  return ZG_OK;
}

}  // namespace zg

using namespace zg;

extern "C" {

zg_status zg_qk_norm_rope(const zg_norm_rope* nr, const zg_rows* q, const zg_rows* k, const zg_rows* q_out,
                          const zg_rows* k_out, const int32_t* positions, int32_t B, int32_t T, int32_t Hq,
                          int32_t Hk, int32_t dim, void* stream) try {
  const char* call = "zg_qk_norm_rope";
  zg_status st;
  if (!nr) return bad_arg(call, "norm_rope is NULL");
  if (!dim_ok(dim)) return fail(ZG_ERR_UNSUPPORTED, "zg_qk_norm_rope: dim must be 32, 64, 96 or 128");
  if (B < 0 || T < 0) return bad_arg(call, "B and T must be >= 0");
  if (B == 0 || T == 0) return ZG_OK;
  if (Hq < 0 || Hk < 0 || Hq > 1024 || Hk > 1024) return bad_arg(call, "Hq and Hk must be in [0, 1024]");
  if ((!q) != (Hq == 0) || (!k) != (Hk == 0))
    return bad_arg(call, "q and k are NULL exactly when their head count is 0");
  if (Hq + Hk == 0) return bad_arg(call, "neither q nor k given");
  const int dt = q ? q->dtype : k->dtype;
  if (q && ((st = check_rows(q, "q", dt, call)) != ZG_OK || (st = check_rows(q_out, "q_out", dt, call)) != ZG_OK))
    return st;
  if (k && ((st = check_rows(k, "k", dt, call)) != ZG_OK || (st = check_rows(k_out, "k_out", dt, call)) != ZG_OK))
    return st;
  NormRopeArgs na;
  if ((st = nr_args(nr, dim, call, &na)) != ZG_OK) return st;
  if (na.rot && !positions) return bad_arg(call, "positions is NULL");
  const int64_t tokens = (int64_t)B * T;
  if (tokens > kMostRows) return fail(ZG_ERR_UNSUPPORTED, "zg_qk_norm_rope: more than 2^40 tokens");
  const int lanes = group_lanes(dim), heads = Hq + Hk;
  const int chunk = head_chunk(tokens, heads, lanes), nchunk = (heads + chunk - 1) / chunk;
  const int64_t ctas = (tokens * nchunk * lanes + 255) / 256;
  if (ctas > 0x7FFFFFFF) return fail(ZG_ERR_UNSUPPORTED, "zg_qk_norm_rope: more than 2^31 CTAs");
  cudaError_t err = cudaSuccess;
  for_type(dt, [&](auto e) {
    using E = typename decltype(e)::type;
    const RotateArgs<E> a = {rows_of<E>(q), rows_of<E>(k), rows_of<E>(q_out), rows_of<E>(k_out), positions,
                             B, T, Hq, Hk, chunk, nchunk, na};
    for_dim(dim, [&](auto dv) {
      auto kern = na.inter ? k_norm_rope<E, decltype(dv)::value, true> : k_norm_rope<E, decltype(dv)::value, false>;
      err = launch_early(kern, ctas, 256, 0, static_cast<cudaStream_t>(stream), a);
    });
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "norm and rotation launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

zg_status zg_kv_append(const zg_kv_cache* cache, const zg_norm_rope* nr, const zg_rows* k, const zg_rows* v,
                       const zg_rows* q, const zg_rows* q_out, int32_t Hq, const int32_t* table, int32_t max_blocks,
                       const int32_t* start, const int32_t* n_new, int32_t B, int32_t T, void* stream) try {
  const char* call = "zg_kv_append";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if (B < 0 || T < 0) return bad_arg(call, "B and T must be >= 0");
  if (B == 0 || T == 0) return ZG_OK;
  if ((st = check_rows(k, "k", -1, call)) != ZG_OK || (st = check_rows(v, "v", k->dtype, call)) != ZG_OK) return st;
  if (Hq < 0 || Hq > 1024 || (!q) != (Hq == 0))
    return bad_arg(call, "Hq must be in [0, 1024], and 0 exactly when q is NULL");
  if (q) {
    if (!nr) return bad_arg(call, "q given without a norm_rope");
    if ((st = check_rows(q, "q", k->dtype, call)) != ZG_OK ||
        (st = check_rows(q_out, "q_out", k->dtype, call)) != ZG_OK)
      return st;
  }
  if (!start) return bad_arg(call, "start is NULL");
  NormRopeArgs na;
  if ((st = nr_args(nr, cache->dim, call, &na)) != ZG_OK) return st;
  const int bt = cache->block_tokens, lanes = group_lanes(cache->dim);
  const int64_t tokens = (int64_t)B * T, jmax = ((int64_t)T + bt - 2) / bt + 1;
  if (tokens > kMostRows) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_append: more than 2^40 tokens");
  // eight rows a lane group at most: groups for min(T, bt) rows, whole warps
  int groups = 1;
  while (groups * kPasses < std::min(T, bt)) groups *= 2;
  const int threads = std::max(32, groups * lanes);
  const int64_t pieces = (int64_t)B * jmax * 2 * cache->heads;
  const int chunk = Hq ? head_chunk(tokens, Hq, lanes) : 1, nchunk = Hq ? (Hq + chunk - 1) / chunk : 0;
  const int64_t qc = (tokens * nchunk * lanes + threads - 1) / threads;
  if (pieces + qc > kMostPieces) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_append: more than 2^31 - 2^20 pieces and CTAs");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  // resident CTAs (128 registers a thread: 512 threads an SM; their buffers inside 200 KB) walk the pieces; where there
  // are queries too, half of each SM is theirs from the start (32 x 2,048 tokens: 156 us against 160)
  const size_t smem = 2 * (size_t)kPasses * threads * 8 * (k->dtype == ZG_F32 ? 4 : 2);
  const int64_t resident = std::max<int64_t>(1, std::min<int64_t>((Hq ? 256 : 512) / threads, (200 << 10) / smem));
  const int64_t kv = std::min<int64_t>(pieces, resident * sm_count());
  cudaError_t err = cudaSuccess;
  for_type(k->dtype, [&](auto e) {
    using E = typename decltype(e)::type;
    const AppendArgs<E> a = {view(cache, table, max_blocks, status), rows_of<E>(k), rows_of<E>(v), rows_of<E>(q),
                             rows_of<E>(q_out), start, n_new, B, T, Hq, (int32_t)jmax, (int32_t)pieces, (int32_t)kv,
                             chunk, nchunk, nr != nullptr, na};
    for_dim(cache->dim, [&](auto dv) {
      constexpr int D = decltype(dv)::value;
      auto kern = cache->format == ZG_KV_INT8
                      ? (na.inter ? k_kv_append<E, D, true, true> : k_kv_append<E, D, true, false>)
                      : (na.inter ? k_kv_append<E, D, false, true> : k_kv_append<E, D, false, false>);
      if (smem > 40 * 1024) err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err == cudaSuccess) err = launch_early(kern, kv + qc, threads, smem, static_cast<cudaStream_t>(stream), a);
    });
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "cache append launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

zg_status zg_kv_read(const zg_kv_cache* cache, const int32_t* table, int32_t max_blocks, const int32_t* start,
                     const int32_t* n, int32_t B, int32_t T, const zg_rows* k_out, const zg_rows* v_out,
                     void* stream) try {
  const char* call = "zg_kv_read";
  zg_status st;
  if ((st = check_cache(cache, table, max_blocks, call)) != ZG_OK) return st;
  if (B < 0 || T < 0) return bad_arg(call, "B and T must be >= 0");
  if (B == 0 || T == 0) return ZG_OK;
  if (!k_out && !v_out) return bad_arg(call, "neither k_out nor v_out given");
  const int dt = k_out ? k_out->dtype : v_out->dtype;
  if (k_out && (st = check_rows(k_out, "k_out", dt, call)) != ZG_OK) return st;
  if (v_out && (st = check_rows(v_out, "v_out", dt, call)) != ZG_OK) return st;
  if (!start) return bad_arg(call, "start is NULL");
  if ((int64_t)B * T > kMostRows) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_read: more than 2^40 tokens");
  const int sides = (k_out ? 1 : 0) + (v_out ? 1 : 0);
  const int lanes = group_lanes(cache->dim);
  const int chunk = head_chunk((int64_t)B * T * sides, cache->heads, lanes), nchunk = (cache->heads + chunk - 1) / chunk;
  const int64_t groups = (int64_t)B * T * sides * nchunk, ctas = (groups * lanes + 255) / 256;
  if (groups > 0x7FFFFFFF) return fail(ZG_ERR_UNSUPPORTED, "zg_kv_read: more than 2^31 (token, side, head chunk)s");
  uint32_t* status = nullptr;
  if ((st = get_status_ptr(&status)) != ZG_OK) return st;
  cudaError_t err = cudaSuccess;
  for_type(dt, [&](auto e) {
    using E = typename decltype(e)::type;
    const ReadArgs<E> a = {view(cache, table, max_blocks, status), rows_of<E>(k_out), rows_of<E>(v_out), start, n,
                           B, T, sides, k_out ? 0 : 1, chunk, nchunk};
    for_dim(cache->dim, [&](auto dv) {
      constexpr int D = decltype(dv)::value;
      auto kern = cache->format == ZG_KV_INT8 ? k_kv_read<E, D, true> : k_kv_read<E, D, false>;
      err = launch_early(kern, ctas, 256, 0, static_cast<cudaStream_t>(stream), a);
    });
  });
  return err == cudaSuccess ? ZG_OK : cuda_fail(err, "cache read launch");
} catch (...) {
  return ZG_ERR_OUT_OF_MEMORY;
}

}  // extern "C"
