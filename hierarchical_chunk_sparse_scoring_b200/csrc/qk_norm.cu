// RMS norm of every query and key head and the rotary position code, one pass; its backward; and
// the serving form that writes keys and values to their slots of a paged cache.
//
//   r = 1 / sqrt(mean(x^2) + eps),   y = R_p (w * x r)
// with R_p turning the pairs (a, b) of the first rot dimensions by p freq[m]:
// (a c - b s, a s + b c).  With cw = w c and sw = -+ w_partner s this is, per element,
// y_i = r (x_i cw_i + x_partner sw_i): two products per element once a lane holds cw and sw.
// Backward: g = R_p^T dy (the same with s negated), dw = sum g x r,
// dx = r (w g - x r^2 mean(w g x)).
//
// Bound: HBM (a row is read once and written once, about ten flops an element).
// Layout: eight elements per lane (16 bytes of bf16), LPR lanes per row (8, 16 or 32 by the head
// dim), so a warp reads whole rows in one or two wide loads.  A lane group keeps one token and
// walks its heads: its eight cosines and sines are computed once and serve every head.  The angle
// is position times a 64-bit fraction of a turn, modulo 2^64: exact, so far positions lose
// nothing, and two integer products where fp64 arithmetic took a fifth of the kernel's time.  In the half layout the
// partner of a lane's eight elements is another lane's eight (rot is a multiple of 16), one
// shuffle per word; in the interleaved layout it is in the lane.
#include <type_traits>

#include "common.cuh"
#include "qk_norm.h"

namespace hils {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkBlocks = 3;   // blocks per SM (forward)
// heads of a lane group loaded together (forward); as many more are on their way
template <typename T>
constexpr int kQkRows = sizeof(T) == 2 ? 4 : 2;

// Eight elements of a row as the words they are stored in.
template <typename T>
struct Raw8 {
  static constexpr int W = sizeof(T) * 8 / 4;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  // (read once: streaming loads leave the cache to the outputs)
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 t = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    }
  }
  // the same words of lane `src` of the lane group
  template <int LPR>
  __device__ __forceinline__ Raw8 from_lane(int src) const {
    Raw8 r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], src, LPR);
    return r;
  }
};

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a lane needs to turn its eight elements 8p .. 8p + 7 of a head at one position: cosine
// and signed sine per element (element i becomes x_i c_i + x_partner s_i).
struct LaneTurn {
  float c[8], s[8];
  int partner;   // lane of the group that holds the partners (half layout; else this lane)
  bool on;       // this lane's elements turn
  bool cross;    // the partners are another lane's (uniform over the warp)

  // cosine and sine of pair m at the position: the nearest quarter turn, and the Taylor polynomials
  // of the rest (at most an eighth turn, where their next terms are below 2^-28)
  __device__ __forceinline__ void pair(const RopeTable& R, int64_t pos, int m, float& co,
                                       float& si) const {
    const uint64_t turns = (uint64_t)pos * R.turn[m];
    const uint32_t hi = (uint32_t)(turns >> 32), quarter = (hi + 0x20000000u) >> 30;
    const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));   // below 2^61
    const float x = (float)(int32_t)(rest >> 30) * (6.2831853071795865f / 17179869184.f);
    const float z = x * x;
    const float sn =
        x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
    const float cs = fmaf(
        z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24),
                -0.5f), 1.f);
    // quarters 1 and 3 exchange the two, 1 and 2 negate the cosine, 2 and 3 the sine
    co = R.mscale * ((quarter & 1) ? sn : cs);
    si = R.mscale * ((quarter & 1) ? cs : sn);
    if ((quarter + 1) & 2) co = -co;
    if (quarter & 2) si = -si;
  }
  __device__ __forceinline__ void init(const RopeTable& R, int p, bool live, int64_t position) {
    const int half = R.rot / 2;
    on = 8 * p < R.rot;
    cross = !R.interleaved;
    partner = !cross || !on ? p : (8 * p < half ? p + half / 8 : p - half / 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
    if (!on || !live) return;
    const int64_t pos = position;
    if (cross) {
      const int m0 = 8 * p < half ? 8 * p : 8 * p - half;
      const float sign = 8 * p < half ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pair(R, pos, m0 + i, c[i], s[i]);
        s[i] *= sign;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pair(R, pos, 4 * p + i, c[2 * i], s[2 * i + 1]);
        c[2 * i + 1] = c[2 * i];
        s[2 * i] = -s[2 * i + 1];
      }
    }
  }
};

// This lane's eight norm weights and those of its partners (ones without a weight vector).
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, int e0, int d, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.f;
  if (w && e0 < d) {
    Raw8<T> r;
    r.load(static_cast<const T*>(w) + e0);
    r.get(v);
  }
}

__device__ __forceinline__ int64_t token_offset(const QkArgs& a, const int64_t (&st)[3],
                                                int64_t t) {
  const int64_t b = t / a.N;
  return b * st[0] + (t - b * a.N) * st[2];
}

// Rows h0 + (i0 + u) hs, u < kQkRows<T>, of one token's H rows (zeros past the end).
template <typename T>
__device__ __forceinline__ void load_rows(Raw8<T> (&x)[kQkRows<T>], bool act, const T* src,
                                          int64_t sh, int H, int h0, int hs, int i0) {
#pragma unroll
  for (int u = 0; u < kQkRows<T>; ++u) {
    const int h = (i0 + u) * hs + h0;
    x[u].zero();
    if (act && h < H) x[u].load(src + h * sh);
  }
}

// Norm and rotation of rows h0, h0 + hs, ... < H of one token: src + h sh -> dst + h dh.  `x` holds
// the first rows; the rows after next are on their way while the present ones are turned.
template <typename T, int LPR>
__device__ __forceinline__ void turn_rows(const QkArgs& a, const LaneTurn& L, int p, bool act,
                                          Raw8<T> (&x)[kQkRows<T>], const T* src, int64_t sh, T* dst,
                                          int64_t dh, int H, int h0, int hs, const void* w) {
  float cw[8], sw[8];
  {
    float own[8], other[8];
    load_weights<T>(w, 8 * p, a.d, own);
    load_weights<T>(w, 8 * L.partner, a.d, other);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cw[i] = own[i] * L.c[i];
      sw[i] = (L.cross ? other[i] : own[i ^ 1]) * L.s[i];
    }
  }
  const float inv_d = 1.f / (float)a.d;
  for (int i0 = 0; i0 * hs < H; i0 += kQkRows<T>) {
    Raw8<T> ahead[kQkRows<T>];
    load_rows<T>(ahead, act, src, sh, H, h0, hs, i0 + kQkRows<T>);
#pragma unroll
    for (int u = 0; u < kQkRows<T>; ++u) {
      const int h = (i0 + u) * hs + h0;
      float v[8], o[8];
      x[u].get(v);
      float r = 1.f;
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        r = __frsqrt_rn(group_sum<LPR>(ss) * inv_d + a.eps);
      }
      if (L.cross) {
        x[u].template from_lane<LPR>(L.partner).get(o);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i ^ 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = v[i] * cw[i];
        v[i] = r * (L.on ? fmaf(o[i], sw[i], y) : y);
      }
      if (act && h < H) {
        x[u].put(v);
        x[u].store(dst + h * dh);
      }
      x[u] = ahead[u];
    }
  }
}

// grid: blocks of 2^tbl tokens; a lane group holds token (group mod 2^tbl) and the heads
// (group / 2^tbl) mod the groups per token.
template <typename T, int LPR, bool PAGED>
__global__ void __launch_bounds__(kQkThreads, kQkBlocks)
    qk_norm_rope_kernel(const __grid_constant__ QkArgs a, int tbl) {
  constexpr int NLG = kQkThreads / LPR;
  const int lg = threadIdx.x / LPR, p = threadIdx.x % LPR;
  const int64_t t = ((int64_t)blockIdx.x << tbl) + (lg & ((1 << tbl) - 1));
  const int h0 = lg >> tbl, hs = NLG >> tbl;
  bool live = t < a.tokens;
  int64_t slot = 0;
  if constexpr (PAGED) {
    if (live) slot = a.slot[t];
    if (slot >= a.n_slots) {
      record_status(a.status, kStatusDeviceCheck);
      live = false;
    }
    live = live && slot >= 0;
  }
  const bool act = live && 8 * p < a.d;
  int64_t position = 0;
  if (live) position = a.pos ? (int64_t)a.pos[t] : a.pos0 + t % a.N;
  const int64_t tt = live ? t : 0;
  const T* q = static_cast<const T*>(a.q) + token_offset(a, a.qs, tt) + 8 * p;
  const T* k = static_cast<const T*>(a.k) + token_offset(a, a.ks, tt) + 8 * p;
  Raw8<T> x[kQkRows<T>];
  load_rows<T>(x, act, q, a.qs[1], a.Hq, h0, hs, 0);
  LaneTurn L;
  L.init(a.rope, p, live, position);
  turn_rows<T, LPR>(a, L, p, act, x, q, a.qs[1],
                    static_cast<T*>(a.qo) + token_offset(a, a.qos, tt) + 8 * p, a.qos[1], a.Hq,
                    h0, hs, a.wq);
  load_rows<T>(x, act, k, a.ks[1], a.Hkv, h0, hs, 0);
  if constexpr (PAGED) {
    const int64_t page = live ? slot / a.page_size : 0;
    const int64_t off = page * a.cs[0] + (live ? slot - page * a.page_size : 0) * a.cs[2] + 8 * p;
    Raw8<T> y[kQkRows<T>];
    const T* v = static_cast<const T*>(a.v) + token_offset(a, a.vs, tt) + 8 * p;
    load_rows<T>(y, act, v, a.vs[1], a.Hkv, h0, hs, 0);
    turn_rows<T, LPR>(a, L, p, act, x, k, a.ks[1], static_cast<T*>(a.Kc) + off, a.cs[1], a.Hkv,
                      h0, hs, a.wk);
    for (int i0 = 0; i0 * hs < a.Hkv; i0 += kQkRows<T>) {
      if (i0 > 0) load_rows<T>(y, act, v, a.vs[1], a.Hkv, h0, hs, i0);
#pragma unroll
      for (int u = 0; u < kQkRows<T>; ++u) {
        const int h = (i0 + u) * hs + h0;
        if (act && h < a.Hkv) y[u].store(static_cast<T*>(a.Vc) + off + h * a.cs[1]);
      }
    }
  } else {
    turn_rows<T, LPR>(a, L, p, act, x, k, a.ks[1],
                      static_cast<T*>(a.ko) + token_offset(a, a.kos, tt) + 8 * p, a.kos[1], a.Hkv,
                      h0, hs, a.wk);
  }
}

// ---------------------------------------------------------------------------------- backward

// Gradients of rows h0, h0 + hs, ... < H of one token; dw gains their share of this lane's eight
// weight gradients.
template <typename T, typename GT, int LPR>
__device__ __forceinline__ void grad_rows(const QkArgs& a, const LaneTurn& L, int p, bool act,
                                          const T* src, int64_t sh, const GT* dy, int64_t gh,
                                          GT* dst, int64_t dh, int H, int h0, int hs,
                                          const float (&w)[8], float (&dw)[8]) {
  constexpr int U = 2;   // heads in flight together
  const float inv_d = 1.f / (float)a.d;
  for (int hb = 0; hb < H; hb += hs * U) {
    Raw8<T> xr[U];
    Raw8<GT> gr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * hs + h0;
      xr[u].zero();
      gr[u].zero();
      if (act && h < H) {
        if (a.norm) xr[u].load(src + h * sh);
        gr[u].load(dy + h * gh);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * hs + h0;
      float x[8], g[8], o[8];
      gr[u].get(g);
      if (L.cross) {
        gr[u].template from_lane<LPR>(L.partner).get(o);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = g[i ^ 1];
      }
      if (L.on) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = fmaf(-o[i], L.s[i], g[i] * L.c[i]);
      }
      if (a.norm) {
        xr[u].get(x);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          dot = fmaf(g[i] * w[i], x[i], dot);
        }
        ss = group_sum<LPR>(ss);
        dot = group_sum<LPR>(dot);
        const float r = __frsqrt_rn(ss * inv_d + a.eps);
        const float f = r * r * dot * inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[i] = fmaf(g[i] * r, x[i], dw[i]);
          g[i] = r * fmaf(-x[i], f, g[i] * w[i]);
        }
      }
      if (act && h < H) {
        gr[u].put(g);
        gr[u].store(dst + h * dh);
      }
    }
  }
}

template <typename T, typename GT, int LPR>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a, int tbl) {
  constexpr int NLG = kQkThreads / LPR;
  __shared__ float sDw[NLG][2][LPR * 8];
  const int lg = threadIdx.x / LPR, p = threadIdx.x % LPR;
  const int h0 = lg >> tbl, hs = NLG >> tbl;
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weights<T>(a.wq, 8 * p, a.d, wq);
  load_weights<T>(a.wk, 8 * p, a.d, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x << tbl; t0 < a.tokens; t0 += (int64_t)gridDim.x << tbl) {
    const int64_t t = t0 + (lg & ((1 << tbl) - 1));
    const bool live = t < a.tokens;
    const bool act = live && 8 * p < a.d;
    int64_t position = 0;
    if (live) position = a.pos ? (int64_t)a.pos[t] : a.pos0 + t % a.N;
    LaneTurn L;
    L.init(a.rope, p, live, position);
    const int64_t tt = live ? t : 0;
    if (a.Hq > 0)
      grad_rows<T, GT, LPR>(a, L, p, act,
                            static_cast<const T*>(a.q) + token_offset(a, a.qs, tt) + 8 * p,
                            a.qs[1],
                            static_cast<const GT*>(a.gq) + token_offset(a, a.gqs, tt) + 8 * p,
                            a.gqs[1], static_cast<GT*>(a.qo) + token_offset(a, a.qos, tt) + 8 * p,
                            a.qos[1], a.Hq, h0, hs, wq, dwq);
    if (a.Hkv > 0)
      grad_rows<T, GT, LPR>(a, L, p, act,
                            static_cast<const T*>(a.k) + token_offset(a, a.ks, tt) + 8 * p,
                            a.ks[1],
                            static_cast<const GT*>(a.gk) + token_offset(a, a.gks, tt) + 8 * p,
                            a.gks[1], static_cast<GT*>(a.ko) + token_offset(a, a.kos, tt) + 8 * p,
                            a.kos[1], a.Hkv, h0, hs, wk, dwk);
  }
  if (!a.dw_part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sDw[lg][0][8 * p + i] = dwq[i];
    sDw[lg][1][8 * p + i] = dwk[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * a.d; e += kQkThreads) {
    const int which = e / a.d, i = e - which * a.d;
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < NLG; ++g) v += sDw[g][which][i];
    a.dw_part[(int64_t)blockIdx.x * 2 * a.d + e] = v;
  }
}

// dw[e] = sum of the blocks' partials in a fixed order; 32 columns x 32 slices per block.
__global__ void __launch_bounds__(1024)
    qk_dw_join_kernel(const float* __restrict__ part, int blocks, int d, float* __restrict__ dw_q,
                      float* __restrict__ dw_k) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  float v = 0.f;
  if (e < 2 * d)
    for (int b = sl; b < blocks; b += 32) v += part[(int64_t)b * 2 * d + e];
  s[sl][c] = v;
  __syncthreads();
  v = warp_sum(s[c][sl]);   // column sl of the block, over the 32 slices
  const int o = blockIdx.x * 32 + sl;
  if (c == 0 && o < 2 * d) {
    float* dst = o < d ? dw_q : dw_k;
    if (dst) dst[o < d ? o : o - d] = v;
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Tokens of a block, log2: as many as it has lane groups, halved while the grid would leave SMs
// without two blocks (a few tokens then spread their heads over the lane groups instead).
int tokens_log2(int64_t tokens, int groups, int sms) {
  int l = 0;
  while ((1 << (l + 1)) <= groups && (tokens >> (l + 1)) >= 2 * (int64_t)sms) ++l;
  return l;
}

template <typename T, int LPR>
cudaError_t launch_fwd(const QkArgs& a, bool paged, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int tbl = tokens_log2(a.tokens, kQkThreads / LPR, sms);
  const int64_t grid = (a.tokens + (1 << tbl) - 1) >> tbl;
  if (paged)
    qk_norm_rope_kernel<T, LPR, true><<<(unsigned)grid, kQkThreads, 0, st>>>(a, tbl);
  else
    qk_norm_rope_kernel<T, LPR, false><<<(unsigned)grid, kQkThreads, 0, st>>>(a, tbl);
  return cudaGetLastError();
}

template <typename T, typename GT, int LPR>
cudaError_t launch_bwd(const QkArgs& a, float* dw_q, float* dw_k, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int tbl = tokens_log2(a.tokens, kQkThreads / LPR, sms);
  int64_t grid = (a.tokens + (1 << tbl) - 1) >> tbl;
  if (grid > kQkBwdBlocks) grid = kQkBwdBlocks;
  if (grid > 0)
    qk_norm_rope_bwd_kernel<T, GT, LPR><<<(unsigned)grid, kQkThreads, 0, st>>>(a, tbl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dw_part) return e;
  qk_dw_join_kernel<<<(2 * a.d + 31) / 32, 1024, 0, st>>>(a.dw_part, (int)grid, a.d, dw_q, dw_k);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs& a, bool bf16, bool paged, cudaStream_t st) {
  if (bf16)
    return a.d <= 64    ? launch_fwd<__nv_bfloat16, 8>(a, paged, st)
           : a.d <= 128 ? launch_fwd<__nv_bfloat16, 16>(a, paged, st)
                        : launch_fwd<__nv_bfloat16, 32>(a, paged, st);
  return a.d <= 64    ? launch_fwd<float, 8>(a, paged, st)
         : a.d <= 128 ? launch_fwd<float, 16>(a, paged, st)
                      : launch_fwd<float, 32>(a, paged, st);
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, bool bf16, bool grad_bf16, float* dw_q,
                                    float* dw_k, cudaStream_t st) {
  auto go = [&](auto t, auto g) -> cudaError_t {
    using T = decltype(t);
    using GT = decltype(g);
    return a.d <= 64    ? launch_bwd<T, GT, 8>(a, dw_q, dw_k, st)
           : a.d <= 128 ? launch_bwd<T, GT, 16>(a, dw_q, dw_k, st)
                        : launch_bwd<T, GT, 32>(a, dw_q, dw_k, st);
  };
  if (!bf16) return go(float(), float());
  return grad_bf16 ? go(__nv_bfloat16(), __nv_bfloat16()) : go(__nv_bfloat16(), float());
}

}  // namespace hils
