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
// Bound: HBM, and close behind it instruction issue: a row of 128 bf16 is read and written once
// (512 bytes, 12 ns of one SM's share of HBM), so that 140 instructions for a warp's step of two
// rows already take as long as the copies.  (32768 tokens of 40 heads: 119 us, 5.7 TB/s, issue
// slots 62% used; the copies alone 104 us.)  Hence:
//   - a lane holds eight elements as two pieces of four, which in the half layout are both members
//     of four pairs (dims 4p .. and rot/2 + 4p ..): a rotation never leaves its lane, and the only
//     exchange is the sum of squares over the row's LPR lanes (8, 16 or 32 by the head dim);
//   - products and sums go two at a time (f32x2);
//   - a lane group keeps one token and walks its heads: the token's four cosines and sines per
//     lane are computed once.  The angle is position times a 64-bit fraction of a turn, modulo
//     2^64: exact, so far positions lose nothing, and two integer products;
//   - the next heads' rows are loaded while the present ones are turned.
#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "qk_norm.h"

namespace hils {
namespace {

// Blocks per SM and heads that a lane group loads together (as many more are on their way): what
// the registers hold.  32768 tokens of 40 heads, 128 bf16, forward / 16301 tokens, append:
// 119 / 74 us; two heads at eight blocks 126 / 81, six blocks (spilling) 121 / 84; 256 threads
// and three blocks, whose ends leave more of an SM idle, 125 / 89.  Backward of 2 x 8192 tokens:
// 146 us; one head 176, five blocks 186.
constexpr int kQkThreads = 128;
constexpr int kQkBlocks = 5;    // forward
constexpr int kBwdBlocks = 4;
constexpr int kBwdRows = 2;
template <typename T>
constexpr int kQkRows = sizeof(T) == 2 ? 4 : 2;

// A lane's eight elements as they are stored: pieces of four at element offsets e0 and e1.
template <typename T>
struct Raw8 {
  static constexpr int W = sizeof(T);   // words per piece: 2 (bf16) or 4
  uint32_t w[2][W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[0][i] = w[1][i] = 0u;
  }
  // (read once: streaming loads leave the cache to the outputs)
  __device__ __forceinline__ void load(const T* row, int e0, int e1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const T* p = row + (h ? e1 : e0);
      if constexpr (sizeof(T) == 2) {
        const uint2 t = __ldcs(reinterpret_cast<const uint2*>(p));
        w[h][0] = t.x; w[h][1] = t.y;
      } else {
        const uint4 t = __ldcs(reinterpret_cast<const uint4*>(p));
        w[h][0] = t.x; w[h][1] = t.y; w[h][2] = t.z; w[h][3] = t.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int e0, int e1) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      T* p = row + (h ? e1 : e0);
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[h][0], w[h][1]);
      else
        *reinterpret_cast<uint4*>(p) = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
    }
  }
  // v[0], v[1]: the first piece; v[2], v[3]: the second
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        v[i] = pack2(bf16_lo(w[i / 2][i % 2]), bf16_hi(w[i / 2][i % 2]));
      else
        v[i] = pack2(__uint_as_float(w[i / 2][2 * (i % 2)]),
                     __uint_as_float(w[i / 2][2 * (i % 2) + 1]));
    }
  }
  __device__ __forceinline__ void put(const f2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack2(v[i]);
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(t.x, t.y);
        w[i / 2][i % 2] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i / 2][2 * (i % 2)] = __float_as_uint(t.x);
        w[i / 2][2 * (i % 2) + 1] = __float_as_uint(t.y);
      }
    }
  }
};

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ... of the products a_i b_i of every lane's eight elements
template <int LPR>
__device__ __forceinline__ float group_dot(const f2 (&a)[4], const f2 (&b)[4]) {
  f2 s = mul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(a[i], b[i], s);
  const float2 t = unpack2(s);
  return group_sum<LPR>(t.x + t.y);
}

// The partners of a lane's elements, in the same order.
template <bool IL>   // interleaved layout (else half)
__device__ __forceinline__ void partners(const f2 (&v)[4], f2 (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (IL) {
      const float2 t = unpack2(v[i]);
      o[i] = pack2(t.y, t.x);
    } else {
      o[i] = v[i ^ 2];
    }
  }
}

// What a lane needs to turn its eight elements at one position: where they are, and cosine and
// signed sine per element (element i becomes x_i c_i + x_partner s_i).
struct LaneTurn {
  int e0, e1;     // first elements of its pieces
  bool on;        // they turn
  f2 c[4], s[4];

  __device__ __forceinline__ void place(const RopeTable& R, int p) {
    on = 8 * p < R.rot;
    e0 = 8 * p;
    e1 = 8 * p + 4;
    if (on && !R.interleaved) {
      e0 = 4 * p;
      e1 = R.rot / 2 + 4 * p;
    }
  }
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
  __device__ __forceinline__ void turn_to(const RopeTable& R, int64_t pos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { c[i] = pack2(1.f, 1.f); s[i] = 0ull; }
    if (!on) return;
    float co[4], si[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pair(R, pos, (R.interleaved ? e0 / 2 : e0) + i, co[i], si[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (R.interleaved) {
        c[i] = pack2(co[i], co[i]);
        s[i] = pack2(-si[i], si[i]);
      } else {
        const int j = 2 * (i & 1);
        c[i] = pack2(co[j], co[j + 1]);
        s[i] = i < 2 ? pack2(-si[j], -si[j + 1]) : pack2(si[j], si[j + 1]);
      }
    }
  }
};

// This lane's eight norm weights (ones without a weight vector).
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, const LaneTurn& L, bool in_row,
                                             f2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(1.f, 1.f);
  if (w && in_row) {
    Raw8<T> r;
    r.load(static_cast<const T*>(w), L.e0, L.e1);
    r.get(v);
  }
}

// Offset of token t (fewer than 2^31) by strides (batch, head, token).
__device__ __forceinline__ int64_t token_offset(const QkArgs& a, const int64_t (&st)[3],
                                                int64_t t) {
  if (t < a.N) return t * st[2];
  const uint32_t b = (uint32_t)t / (uint32_t)a.N;
  return b * st[0] + (t - b * a.N) * st[2];
}

__device__ __forceinline__ int64_t position_of(const QkArgs& a, int64_t t) {
  if (a.pos) return a.pos[t];
  return a.pos0 + (t < a.N ? t : (int64_t)((uint32_t)t % (uint32_t)a.N));
}

// Rows of the heads h, h + hs, ... below H of one token, R of them (zeros past the end).
template <typename T, int R>
__device__ __forceinline__ void load_rows(Raw8<T> (&x)[R], bool act, const T* src, int64_t sh,
                                          int H, int h, int hs, const LaneTurn& L) {
#pragma unroll
  for (int u = 0; u < R; ++u) {
    x[u].zero();
    if (act && h + u * hs < H) x[u].load(src + (h + u * hs) * sh, L.e0, L.e1);
  }
}

// Norm and rotation of the heads h0, h0 + hs, ... < H of one token: src + h sh -> dst + h dh.  `x`
// holds the first rows.
template <typename T, int LPR, bool IL>
__device__ __forceinline__ void turn_rows(const QkArgs& a, const LaneTurn& L, bool act,
                                          Raw8<T> (&x)[kQkRows<T>], const T* src, int64_t sh,
                                          T* dst, int64_t dh, int H, int h0, int hs,
                                          const void* w, bool in_row) {
  constexpr int R = kQkRows<T>;
  f2 cw[4], sw[4];
  load_weights<T>(w, L, in_row, cw);
  partners<IL>(cw, sw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cw[i] = mul2(cw[i], L.c[i]);
    sw[i] = mul2(sw[i], L.s[i]);
  }
  const float inv_d = 1.f / (float)a.d;
  for (int hb = 0; hb < H; hb += R * hs) {   // (as many rounds for every lane of the warp)
    const int h1 = hb + h0;
    Raw8<T> ahead[R];
    load_rows<T, R>(ahead, act, src, sh, H, h1 + R * hs, hs, L);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int h = h1 + u * hs;
      f2 v[4], o[4];
      x[u].get(v);
      partners<IL>(v, o);
      f2 r = pack2(1.f, 1.f);
      if (a.norm) {
        const float t = rsqrtf(fmaf(group_dot<LPR>(v, v), inv_d, a.eps));
        r = pack2(t, t);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], cw[i]);
      if (L.on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma2(o[i], sw[i], v[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], r);
      if (act && h < H) {
        x[u].put(v);
        x[u].store(dst + h * dh, L.e0, L.e1);
      }
      x[u] = ahead[u];
    }
  }
}

// grid: blocks of 2^tbl tokens; a lane group holds token (group mod 2^tbl) and the heads
// (group / 2^tbl) mod the groups per token.
template <typename T, int LPR, bool IL, bool PAGED>
__global__ void __launch_bounds__(kQkThreads, kQkBlocks)
    qk_norm_rope_kernel(const __grid_constant__ QkArgs a, int tbl) {
  constexpr int NLG = kQkThreads / LPR;
  const int lg = threadIdx.x / LPR, p = threadIdx.x % LPR;
  const int64_t t = ((int64_t)blockIdx.x << tbl) + (lg & ((1 << tbl) - 1));
  const int h0 = lg >> tbl, hs = NLG >> tbl;
  bool live = t < a.tokens;
  int64_t slot = -1;
  if constexpr (PAGED) {
    if (live) slot = a.slot[t];
    if (slot >= a.n_slots) {
      record_status(a.status, kStatusDeviceCheck);
      live = false;
    }
    live = live && slot >= 0;
  }
  constexpr int R = kQkRows<T>;
  const bool in_row = 8 * p < a.d, act = live && in_row;
  const int64_t tt = live ? t : 0;
  LaneTurn L;
  L.place(a.rope, p);
  const T* q = static_cast<const T*>(a.q) + token_offset(a, a.qs, tt);
  const T* k = static_cast<const T*>(a.k) + token_offset(a, a.ks, tt);
  Raw8<T> x[R];
  load_rows<T, R>(x, act, q, a.qs[1], a.Hq, h0, hs, L);
  L.turn_to(a.rope, live ? position_of(a, t) : 0);
  turn_rows<T, LPR, IL>(a, L, act, x, q, a.qs[1],
                    static_cast<T*>(a.qo) + token_offset(a, a.qos, tt), a.qos[1], a.Hq, h0, hs,
                    a.wq, in_row);
  load_rows<T, R>(x, act, k, a.ks[1], a.Hkv, h0, hs, L);
  if constexpr (PAGED) {
    const uint32_t page = live ? (uint32_t)slot / (uint32_t)a.page_size : 0;
    const int64_t off =
        page * a.cs[0] + (live ? slot - (int64_t)page * a.page_size : 0) * a.cs[2];
    Raw8<T> y[R];
    const T* v = static_cast<const T*>(a.v) + token_offset(a, a.vs, tt);
    load_rows<T, R>(y, act, v, a.vs[1], a.Hkv, h0, hs, L);
    turn_rows<T, LPR, IL>(a, L, act, x, k, a.ks[1], static_cast<T*>(a.Kc) + off, a.cs[1], a.Hkv, h0,
                      hs, a.wk, in_row);
    for (int h = h0; h < a.Hkv; h += R * hs) {
      if (h > h0) load_rows<T, R>(y, act, v, a.vs[1], a.Hkv, h, hs, L);
#pragma unroll
      for (int u = 0; u < R; ++u)
        if (act && h + u * hs < a.Hkv)
          y[u].store(static_cast<T*>(a.Vc) + off + (h + u * hs) * a.cs[1], L.e0, L.e1);
    }
  } else {
    turn_rows<T, LPR, IL>(a, L, act, x, k, a.ks[1],
                      static_cast<T*>(a.ko) + token_offset(a, a.kos, tt), a.kos[1], a.Hkv, h0, hs,
                      a.wk, in_row);
  }
}

// ---------------------------------------------------------------------------------- backward

// Gradients of the heads h0, h0 + hs, ... < H of one token.  `sum` (shared memory, element i at
// i LPR; null: no weight) gains their share of this lane's eight weight gradients: a token's heads
// are added in 32 bits, tokens in 64, so that the error does not grow with their number.
template <typename T, typename GT, int LPR, bool IL>
__device__ __forceinline__ void grad_rows(const QkArgs& a, const LaneTurn& L, bool act,
                                          const T* src, int64_t sh, const GT* dy, int64_t gh,
                                          GT* dst, int64_t dh, int H, int h0, int hs,
                                          const f2 (&w)[4], double* sum) {
  constexpr int R = kBwdRows;
  f2 dw[4] = {0ull, 0ull, 0ull, 0ull};
  const float inv_d = 1.f / (float)a.d;
  const bool actx = act && a.norm;
  Raw8<T> x[R];
  Raw8<GT> g[R];
  load_rows<T, R>(x, actx, src, sh, H, h0, hs, L);
  load_rows<GT, R>(g, act, dy, gh, H, h0, hs, L);
  for (int hb = 0; hb < H; hb += R * hs) {
    const int h1 = hb + h0;
    Raw8<T> xn[R];
    Raw8<GT> gn[R];
    load_rows<T, R>(xn, actx, src, sh, H, h1 + R * hs, hs, L);
    load_rows<GT, R>(gn, act, dy, gh, H, h1 + R * hs, hs, L);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int h = h1 + u * hs;
      f2 v[4], o[4];
      g[u].get(v);
      if (L.on) {   // (turned back: L is at the negated position)
        partners<IL>(v, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma2(o[i], L.s[i], mul2(v[i], L.c[i]));
      }
      if (a.norm) {
        f2 xv[4], wv[4];
        x[u].get(xv);
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[i] = mul2(v[i], w[i]);
        const float ss = group_dot<LPR>(xv, xv), dot = group_dot<LPR>(wv, xv);
        // (places without a row hold zeros: without eps their norm would be infinite)
        const float r = act && h < H ? rsqrtf(fmaf(ss, inv_d, a.eps)) : 0.f;
        const float f = -r * r * dot * inv_d;
        const f2 rr = pack2(r, r), ff = pack2(f, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw[i] = fma2(mul2(v[i], rr), xv[i], dw[i]);
          v[i] = mul2(rr, fma2(xv[i], ff, wv[i]));
        }
      }
      if (act && h < H) {
        g[u].put(v);
        g[u].store(dst + h * dh, L.e0, L.e1);
      }
      x[u] = xn[u];
      g[u] = gn[u];
    }
  }
  if (sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack2(dw[i]);
      sum[2 * i * LPR] += t.x;
      sum[(2 * i + 1) * LPR] += t.y;
    }
  }
}

// Blocks walk the token groups; each leaves its lanes' shares of the weight gradients, added over
// its lane groups, in dw_part.
template <typename T, typename GT, int LPR, bool IL>
__global__ void __launch_bounds__(kQkThreads, kBwdBlocks)
    qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a, int tbl) {
  constexpr int NLG = kQkThreads / LPR;
  __shared__ double sDw[NLG][2][LPR * 8];   // element i of lane p at i LPR + p
  const int lg = threadIdx.x / LPR, p = threadIdx.x % LPR;
  const int h0 = lg >> tbl, hs = NLG >> tbl;
  const bool in_row = 8 * p < a.d;
  LaneTurn L;
  L.place(a.rope, p);
  f2 wq[4], wk[4];
  load_weights<T>(a.wq, L, in_row, wq);
  load_weights<T>(a.wk, L, in_row, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) sDw[lg][0][i * LPR + p] = sDw[lg][1][i * LPR + p] = 0.0;
  double* const sum_q = a.dw_part ? &sDw[lg][0][p] : nullptr;
  double* const sum_k = a.dw_part ? &sDw[lg][1][p] : nullptr;
  for (int64_t t0 = (int64_t)blockIdx.x << tbl; t0 < a.tokens; t0 += (int64_t)gridDim.x << tbl) {
    const int64_t t = t0 + (lg & ((1 << tbl) - 1));
    const bool live = t < a.tokens, act = live && in_row;
    const int64_t tt = live ? t : 0;
    L.turn_to(a.rope, live ? -position_of(a, t) : 0);   // the transposed rotation turns back
    grad_rows<T, GT, LPR, IL>(a, L, act, static_cast<const T*>(a.q) + token_offset(a, a.qs, tt),
                          a.qs[1], static_cast<const GT*>(a.gq) + token_offset(a, a.gqs, tt),
                          a.gqs[1], static_cast<GT*>(a.qo) + token_offset(a, a.qos, tt),
                          a.qos[1], a.Hq, h0, hs, wq, sum_q);
    grad_rows<T, GT, LPR, IL>(a, L, act, static_cast<const T*>(a.k) + token_offset(a, a.ks, tt),
                          a.ks[1], static_cast<const GT*>(a.gk) + token_offset(a, a.gks, tt),
                          a.gks[1], static_cast<GT*>(a.ko) + token_offset(a, a.kos, tt),
                          a.kos[1], a.Hkv, h0, hs, wk, sum_k);
  }
  if (!a.dw_part) return;
  __syncthreads();
  for (int x = threadIdx.x; x < 2 * LPR * 8; x += kQkThreads) {
    const int which = x / (LPR * 8), i = x / LPR % 8, lane = x % LPR;
    if (8 * lane >= a.d) continue;
    double v = 0.0;
#pragma unroll
    for (int g = 0; g < NLG; ++g) v += sDw[g][which][x % (LPR * 8)];
    LaneTurn P;
    P.place(a.rope, lane);
    const int e = (i < 4 ? P.e0 : P.e1) + i % 4;
    a.dw_part[((int64_t)blockIdx.x * 2 + which) * a.d + e] = v;
  }
}

// dw[e] = sum of the blocks' partials in a fixed order, rounded once; 32 columns x 32 slices per
// block.
__global__ void __launch_bounds__(1024)
    qk_dw_join_kernel(const double* __restrict__ part, int blocks, int d, float* __restrict__ dw_q,
                      float* __restrict__ dw_k) {
  __shared__ double s[32][33];
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  double v = 0.0;
  if (e < 2 * d)
    for (int b = sl; b < blocks; b += 32) v += part[(int64_t)b * 2 * d + e];
  s[sl][c] = v;
  __syncthreads();
  v = s[c][sl];   // column sl of the block, over the 32 slices
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int o = blockIdx.x * 32 + sl;
  if (c == 0 && o < 2 * d) {
    float* dst = o < d ? dw_q : dw_k;
    if (dst) dst[o < d ? o : o - d] = (float)v;
  }
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
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int tbl = tokens_log2(a.tokens, kQkThreads / LPR, sms);
  const int64_t grid = (a.tokens + (1 << tbl) - 1) >> tbl;
  auto kern = a.rope.interleaved ? (paged ? qk_norm_rope_kernel<T, LPR, true, true>
                                          : qk_norm_rope_kernel<T, LPR, true, false>)
                                 : (paged ? qk_norm_rope_kernel<T, LPR, false, true>
                                          : qk_norm_rope_kernel<T, LPR, false, false>);
  kern<<<(unsigned)grid, kQkThreads, 0, st>>>(a, tbl);
  return cudaGetLastError();
}

template <typename T, typename GT, int LPR>
cudaError_t launch_bwd(const QkArgs& a, float* dw_q, float* dw_k, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int tbl = tokens_log2(a.tokens, kQkThreads / LPR, sms);
  int64_t grid = (a.tokens + (1 << tbl) - 1) >> tbl;
  if (grid > kQkBwdBlocks) grid = kQkBwdBlocks;
  auto kern = a.rope.interleaved ? qk_norm_rope_bwd_kernel<T, GT, LPR, true>
                                 : qk_norm_rope_bwd_kernel<T, GT, LPR, false>;
  if (grid > 0) kern<<<(unsigned)grid, kQkThreads, 0, st>>>(a, tbl);
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
