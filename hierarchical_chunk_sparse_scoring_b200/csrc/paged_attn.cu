// Attention of single tokens over a paged cache, split over the cache's length and joined.
//
//   out[t, h] = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale q.K_j - m),  lse = m + ln sum_j p_j
// over the tokens j the row sees, one pass with a running maximum m and sum (both fp32).
// Bound: HBM; every seen key and value row is read once for all G heads of its KV head, 4 G d
// flops for 2 d elements.
//
// Work split.  A unit is a (row, KV head); its tokens are cut into tiles of 16 (bf16) or 8 (fp32).
// All units in order (row, head) form one list in which a unit takes one place for its own cost
// (queries, output) and one per tile.  Every CTA (one per SM, all of its shared memory) takes an
// equal stretch of the list and every warp an equal stretch of its CTA's, whatever the rows'
// lengths; CTAs sum the rows' tiles themselves, so nothing about the lengths is needed on the
// host.  (Short units are not cut; they go with their first place.)  A warp walks its stretch with
// its own ring of cp.async stages, across unit boundaries, and its own running maximum and sum,
// and writes units that lie within it: no block barrier until every warp is done.  Then the parts
// (m, sum, O) of units cut by a warp boundary are added in shared memory, and those of units cut by
// a CTA boundary go to the workspace, where the join kernel adds them, always in the list's order.
// The 128 KB a CTA has in flight cover the latency of HBM; a tile's page id is read one tile ahead
// of its copy.
// Measured (bf16, 32/8 heads, d = 128): 8 rows of 120K tokens 577 us = 6.7 TB/s, 64 ragged rows of
// 500 to 15K tokens 183 us = 6.1 TB/s; one row of 1000 tokens 11 us, a chain of latencies (the
// plan of the split 1.8 us, first data 3 us, one tile 0.5 us, adding the parts 1.2 us, the join 3).
//
//   bf16  S^T = K Q^T and O^T += V^T P^T by m16n8k16 products: the tokens (then the head
//         dimension) are the 16 rows, the G heads the 8 columns, so no row of a product is
//         padding at G = 8 and P^T is S^T transposed in registers (movmatrix).  (A tile is 16
//         tokens of one warp; the 128-row products of tcgen05 would tie four warps to each tile
//         and pass its scores through tensor memory, for arithmetic that HBM leaves idle anyway.)
//   fp32  each lane holds D/32 dimensions of q and O for all heads; a tile's dot products are
//         summed over the lanes by halving exchanges that leave each lane its own (head, token).
#include "block_scan.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "paged.h"

namespace hils {
namespace {

constexpr int kPaCtas = 148;      // CTAs at most (one per SM of 148)
constexpr int kPaMinPer = 4;      // places of the list a CTA takes at least
// Units of up to this many places (and not longer than a warp's stretch) are not cut: joining the
// parts costs about as much as the tiles that a warp may get too many (2048 units of four tiles:
// 15.7 us uncut, 20.2 us cut; without this bound ragged rows of up to 1000 tiles lose 20%).
constexpr int kPaSmall = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The unit at the start of a CTA's stretch, for the join: the start's place in the unit, the
// unit's places, and the places per stretch (n = 0: no stretch, or a unit that is not cut).
struct PaRec {
  int64_t off, n, per;
  int32_t row, head;
};

struct PaWs {
  PaRec* rec;    // [ctas]
  float* ml;     // [ctas][2][G][2] running maximum (base 2) and sum
  float* o;      // [ctas][2][G][d]
  float* first;  // [ctas][8 warps][G][d], if shared memory does not hold them
};

__host__ __device__ inline size_t pa_align(size_t x) { return (x + 255) / 256 * 256; }

__host__ __device__ inline PaWs pa_carve(char* ws, int64_t G, int64_t d) {
  PaWs w;
  w.rec = reinterpret_cast<PaRec*>(ws);
  ws += pa_align(kPaCtas * sizeof(PaRec));
  w.ml = reinterpret_cast<float*>(ws);
  ws += pa_align((size_t)kPaCtas * 2 * G * 2 * sizeof(float));
  w.o = reinterpret_cast<float*>(ws);
  ws += pa_align((size_t)kPaCtas * 2 * G * d * sizeof(float));
  w.first = reinterpret_cast<float*>(ws);
  return w;
}

// What row t sees: tokens lo .. hi - 1 of sequence seq (seq < 0: padding).
struct PaRow {
  int seq, lo, hi;
  template <int KT>
  __device__ __forceinline__ int tiles() const {
    return hi > lo ? (hi - 1) / KT - lo / KT + 1 : 0;
  }
  // places of one of its units in the list
  template <int KT>
  __device__ __forceinline__ int places() const {
    return hi > lo ? tiles<KT>() + 1 : 0;
  }
};

__device__ __forceinline__ PaRow pa_row(const PagedAttnArgs& a, int t, bool& bad) {
  PaRow r;
  r.seq = a.seq ? a.seq[t] : t;
  r.lo = r.hi = 0;
  const int pos = a.pos[t];
  if (r.seq < 0) return r;
  if (r.seq >= a.B || pos < -1 || pos >= a.max_len) {
    bad = true;
    r.seq = 0;
    return r;
  }
  r.hi = pos + 1;
  r.lo = a.window > 0 && r.hi > a.window ? r.hi - a.window : 0;
  return r;
}

// ... nothing past the last row.
__device__ __forceinline__ PaRow pa_row_or_none(const PagedAttnArgs& a, int t, bool& bad) {
  return t < a.T ? pa_row(a, t, bad) : PaRow{-1, 0, 0};
}

// Where a stretch of the list begins: row `row`, whose first unit starts at place `at`, holds
// place `begin` (begin >= total, the places of the list: no stretch).
struct PaStretch {
  int64_t begin, total, at;
  int row;
};

// x / n, in 32 bits where they do.
__device__ __forceinline__ int pa_head(int64_t x, int n) {
  return x < n ? 0 : x < INT32_MAX ? (int)((uint32_t)x / (uint32_t)n) : (int)(x / n);
}

// Places per CTA and per warp, and where the stretches of this CTA's warps begin (in shared memory,
// sS [NW]).
struct PaPlan {
  int64_t per, per_warp;
};
template <int NW, int KT>
__device__ __forceinline__ PaPlan pa_schedule(const PagedAttnArgs& a, PaStretch* sS, bool& bad) {
  constexpr int NT = NW * 32;
  __shared__ int64_t sWarp[NW];
  const int chunk = (a.T + NT - 1) / NT;
  const int t0 = threadIdx.x * chunk;
  const int t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  int64_t mine = 0;
  for (int t = t0; t < t1; ++t) mine += pa_row(a, t, bad).places<KT>();
  mine *= a.Hkv;
  int64_t total;
  int64_t at = block_scan<NT>(mine, sWarp, total);
  // enough for every place (rounded up in doubles: 2^-53 of a total below 2^48 is no place)
  PaPlan P;
  P.per = (int64_t)((double)total * a.inv_ctas) + 1;
  if (P.per < kPaMinPer) P.per = kPaMinPer;
  P.per_warp = (P.per + NW - 1) / NW;
  const int64_t begin = P.per * blockIdx.x;
  if (threadIdx.x < NW) {
    sS[threadIdx.x].begin = begin + threadIdx.x * P.per_warp;
    sS[threadIdx.x].total = total;
  }
  if (begin < at + mine && begin + P.per > at) {   // a stretch may begin among this thread's rows
    int w = 0;
    while (w < NW && begin + w * P.per_warp < at) ++w;
    for (int t = t0; t < t1 && w < NW; ++t) {
      const int64_t next = at + (int64_t)pa_row(a, t, bad).places<KT>() * a.Hkv;
      for (; w < NW && begin + w * P.per_warp < next; ++w) {
        sS[w].row = t;
        sS[w].at = at;
      }
      at = next;
    }
  }
  __syncthreads();
  return P;
}

template <typename T>
__device__ __forceinline__ void store_out(T* p, float v) { *p = Elem<T>::from_f(v); }

// ln of the sum, from its maximum (base 2) and the sum relative to it.
__device__ __forceinline__ float pa_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros instead when `take` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shape of a CTA.  GM bounds the heads of a KV group.
template <typename T, int D, int GM>
struct PaShape {
  static constexpr int KT = sizeof(T) == 2 ? 16 : 8;        // tokens per tile
  static constexpr int ROW = D * (int)sizeof(T);            // bytes of a token's row
  static constexpr int CH = ROW / 16;                       // its 16-byte pieces
  static constexpr int HALF = KT * ROW;                     // K (or V) of a tile
  static constexpr int STAGE = 2 * HALF;
  // Warps, and the stages of each one's ring.  The first part of a warp (G D floats) waits in
  // shared memory where that fits beside the rings, else in the workspace.  (bf16 of 16 heads: as
  // many warps as fit with their parts.  32 rows of 16384 tokens, d = 128: 68 us with seven, 76 with
  // six, 73 with eight and the parts in the workspace; d = 64: 49 us with eight, 52 with seven, 58
  // with six.  fp32, bound by instructions, wants the eight.)
  static constexpr int NW = GM > 8 && sizeof(T) == 2 && D > 64 ? 7 : 8;
  static constexpr int ST = 24576 / STAGE;
  static constexpr bool FIRST_SMEM = GM <= 4 || sizeof(T) == 2 || (GM <= 8 && D == 64);
  static constexpr int FIRST = FIRST_SMEM ? GM * D : 0;
  static constexpr int THREADS = NW * 32;
  static constexpr int SCRATCH = sizeof(T) == 2 ? 0 : KT * GM + GM;   // fp32: weights, factors
  static int smem(int G) {
    return NW * ST * STAGE + NW * ((FIRST_SMEM ? G * D : 0) + 4 * G + SCRATCH) * (int)sizeof(float);
  }
  static_assert(NW * (ST * STAGE + (FIRST + 4 * GM + SCRATCH) * 4) + 1024 <= 227 * 1024,
                "fits an SM");
  static_assert(GM * D * 4 <= ST * STAGE, "a part fits a warp's ring");
  static_assert(ST >= 3, "two tiles in flight while one is used");
  static_assert(CH == 8 || CH == 16 || CH == 32, "whole rows per copy");
};

// A softmax weight w > 0 as three numbers >= 0 whose upper 16 bits, as bf16, add up to it: eight
// bits of the mantissa each, cut off and not rounded, so that none is negative.  A part that would
// be zero is w 2^-30 instead, which changes the sum by less than its rounding: with all three above
// zero an infinite value times the weight is that infinity (a weight from 2^-96 on, below which the
// small part has no normal bf16), where parts of both signs or zero would give NaN.
__device__ __forceinline__ float upper16(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
__device__ __forceinline__ void split_weight(float w, float (&part)[3]) {
  const float least = w * 0x1p-30f;
  part[0] = w;
  part[1] = fmaxf(w - upper16(w), least);
  part[2] = fmaxf(part[1] - upper16(part[1]), least);
}
// The upper 16 bits of two numbers, a's below.
__device__ __forceinline__ uint32_t pack_upper16(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// The softmax and products of one warp over its tiles of a unit.  load(q) reads the unit's
// queries, tile() takes one tile, finish() leaves (m, sum, O) of every head in shared memory.
template <typename T, int D, int GM>
struct PaWarp;

template <int D, int GM>
struct PaWarp<__nv_bfloat16, D, GM> {
  using S = PaShape<__nv_bfloat16, D, GM>;
  static constexpr int NB = (GM + 7) / 8;   // columns of 8 heads
  uint32_t q[NB][D / 16][2];
  float o[NB][D / 16][4], m[NB][2], l[NB][2];

  __device__ __forceinline__ void load(const __nv_bfloat16* src, int G, int lane) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int g = nb * 8 + lane / 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[nb][k][e] = g < G ? *reinterpret_cast<const uint32_t*>(src + g * D + k * 16 + e * 8 +
                                                                   (lane % 4) * 2)
                              : 0u;
    }
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nb][i][e] = 0.f;
    }
  }
  // mask: bit j set if token j of the tile is seen
  __device__ __forceinline__ void tile(uint32_t sK, uint32_t sV, uint32_t mask, float sc, int lane,
                                       float*) {
    float s[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[4];
      const int r = lane & 15;
      ldsm4(a, sK + r * S::ROW + (((2 * k + (lane >> 4)) ^ (r & 7)) << 4));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], a, q[nb][k][0], q[nb][k][1]);
    }
    const bool see0 = (mask >> (lane / 4)) & 1, see1 = (mask >> (lane / 4 + 8)) & 1;
    // The weights as three bf16 each, all 24 bits of them.  (One alone would add as much error as
    // the rounding of the output, two leave 16 bits.  Three cost nothing: 64 ragged rows 181 us with
    // two or three.)
    uint32_t p[NB][3][2];
    float f[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[nb][e] = see0 ? s[nb][e] * sc : -INFINITY;
        s[nb][2 + e] = see1 ? s[nb][2 + e] * sc : -INFINITY;
        float t = fmaxf(s[nb][e], s[nb][2 + e]);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, w));
        t = fmaxf(t, m[nb][e]);
        f[nb][e] = 1.f;
        if (t > m[nb][e]) {
          f[nb][e] = exp2f(m[nb][e] - t);
          m[nb][e] = t;
        }
        // (a maximum of -inf: nothing seen yet, all weights are zero)
        const float base = t == -INFINITY ? 0.f : t;
        s[nb][e] = exp2f(s[nb][e] - base);
        s[nb][2 + e] = exp2f(s[nb][2 + e] - base);
        l[nb][e] = fmaf(l[nb][e], f[nb][e], s[nb][e] + s[nb][2 + e]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float a[3], b[3];
        split_weight(s[nb][2 * h], a);
        split_weight(s[nb][2 * h + 1], b);
#pragma unroll
        for (int k = 0; k < 3; ++k) p[nb][k][h] = transpose8x8(pack_upper16(a[k], b[k]));
      }
    }
    // The tile's sums apart, smallest parts first, then added to O: the products cut their sums off
    // and do not round to nearest, which over thousands of tiles in one accumulator leaned the
    // output towards zero by 2e-4 (rows of 65536 tokens).  (It costs nothing up to 8 heads of
    // d = 128, 64 ragged rows 181 us either way, and 2% at d = 64, 64 rows of 16384 tokens.)
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      const int r = (lane & 7) + ((lane >> 4) << 3);
      ldsm4_t(a, sV + r * S::ROW + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 2; k >= 0; --k) mma16816(t, a, p[nb][k][0], p[nb][k][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nb][i][e] = fmaf(o[nb][i][e], f[nb][e & 1], t[e]);
      }
    }
  }
  // the sums over the tokens' lanes
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1)
          l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], w);
  }
  // a whole unit: out [G][D] and lse [G] (nullable)
  __device__ __forceinline__ void emit(__nv_bfloat16* out, float* lse, int G, int lane) {
    close();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float inv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = nb * 8 + (lane % 4) * 2 + e;
        inv[e] = l[nb][e] > 0.f ? 1.f / l[nb][e] : l[nb][e];   // (0 and NaN stay)
        if (lse && lane < 4 && g < G) lse[g] = pa_lse(m[nb][e], l[nb][e]);
      }
      const int g = nb * 8 + lane / 4;   // after the transposition: lane / 4 is the head
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __nv_bfloat162 w =
              __floats2bfloat162_rn(o[nb][i][2 * h] * inv[0], o[nb][i][2 * h + 1] * inv[1]);
          const uint32_t t = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
          if (g < G)
            *reinterpret_cast<uint32_t*>(out + g * D + i * 16 + h * 8 + (lane % 4) * 2) = t;
        }
    }
  }
  // a part of a unit, to shared memory
  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, int G, int lane) {
    close();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = nb * 8 + (lane % 4) * 2 + e;
        if (g >= G) continue;
        if (lane < 4) {
          sM[g] = m[nb][e];
          sL[g] = l[nb][e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          sO[g * D + i * 16 + lane / 4] = o[nb][i][e];
          sO[g * D + i * 16 + lane / 4 + 8] = o[nb][i][2 + e];
        }
      }
  }
};

// Sums V values per lane over the warp; lane i keeps values i V/32 .. (V >= 32), or value
// i V/32 (V < 32, each in 32 / V lanes).
template <int V>
__device__ __forceinline__ void scatter_sum(float (&v)[V], int lane) {
  int n = V;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    if (n > 1) {
      const bool up = lane & w;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (i >= n / 2) break;
        const float keep = up ? v[n / 2 + i] : v[i], give = up ? v[i] : v[n / 2 + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
      n /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
    }
  }
}

template <int D, int GM>
struct PaWarp<float, D, GM> {
  using S = PaShape<float, D, GM>;
  static constexpr int EPL = D / 32;            // dimensions of a lane
  static constexpr int KG = GM > 8 ? 4 : 8;     // tokens summed together
  static constexpr int V = KG * GM;             // their (head, token) logits, head-major
  static constexpr int NV = V > 32 ? V / 32 : 1;       // logits of a lane: tokens of one head
  static constexpr int SPAN = V >= 32 ? 1 : 32 / V;    // lanes that hold the same logit
  static constexpr int LPH = 32 / GM;           // lanes that hold a head's logits
  static_assert(NV <= KG, "a lane's logits belong to one head");
  static constexpr int PL = EPL / 2;            // ... in pairs
  f2 q[GM][PL], o[GM][PL];
  float m, l;                                   // of head lane / LPH

  static __device__ __forceinline__ void get_row(f2 (&v)[PL], uint32_t addr) {
    if constexpr (PL == 2)
      asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];"
                   : "=l"(v[0]), "=l"(v[1])
                   : "r"(addr)
                   : "memory");
    else
      asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v[0]) : "r"(addr) : "memory");
  }
  // one value per head (the scratch of GM > 1 lies on 16-byte boundaries)
  static __device__ __forceinline__ void get_heads(float (&v)[GM], const float* p) {
    if constexpr (GM >= 4) {
#pragma unroll
      for (int i = 0; i < GM / 4; ++i) {
        const float4 t = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
      }
    } else {
      v[0] = p[0];
    }
  }
  __device__ __forceinline__ void load(const float* src, int G, int lane) {
#pragma unroll
    for (int g = 0; g < GM; ++g) {
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        q[g][e] = 0ull;
        if (g < G) q[g][e] = reinterpret_cast<const f2*>(src + g * D + lane * EPL)[e];
      }
    }
  }
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int g = 0; g < GM; ++g)
#pragma unroll
      for (int e = 0; e < PL; ++e) o[g][e] = 0ull;
  }
  __device__ __forceinline__ void tile(uint32_t sK, uint32_t sV, uint32_t mask, float sc, int lane,
                                       float* scratch) {
    float* sP = scratch;               // [KT][GM]
    float* sF = scratch + S::KT * GM;  // [GM]
#pragma unroll
    for (int k0 = 0; k0 < S::KT; k0 += KG) {
      float x[V];
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        f2 kv[PL];
        get_row(kv, sK + (k0 + k) * S::ROW + lane * EPL * 4);
#pragma unroll
        for (int g = 0; g < GM; ++g) {
          f2 t = mul2(q[g][0], kv[0]);
#pragma unroll
          for (int e = 1; e < PL; ++e) t = fma2(q[g][e], kv[e], t);
          const float2 u = unpack2(t);
          x[g * KG + k] = u.x + u.y;
        }
      }
      scatter_sum<V>(x, lane);
      const int first = (lane / SPAN) * NV;        // of the logits
      const int tok = first % KG, head = first / KG;
      float t = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = (mask >> (k0 + tok + i)) & 1 ? x[i] * sc : -INFINITY;
        t = fmaxf(t, x[i]);
      }
#pragma unroll
      for (int w = 1; w < LPH; w <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, w));
      t = fmaxf(t, m);
      const bool moved = t > m;
      const float f = moved ? exp2f(m - t) : 1.f;
      m = t;
      const float base = t == -INFINITY ? 0.f : t;
      l *= f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = exp2f(x[i] - base);
        if (lane % SPAN == 0) {
          l += x[i];
          sP[(k0 + tok + i) * GM + head] = x[i];
        }
      }
      const bool any = __any_sync(0xffffffffu, moved);
      if (any && lane % LPH == 0) sF[head] = f;
      __syncwarp();
      if (any) {
#pragma unroll
        for (int g = 0; g < GM; ++g) {
          const f2 r = pack2(sF[g], sF[g]);
#pragma unroll
          for (int e = 0; e < PL; ++e) o[g][e] = mul2(o[g][e], r);
        }
      }
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        f2 vv[PL];
        get_row(vv, sV + (k0 + k) * S::ROW + lane * EPL * 4);
        float w[GM];
        get_heads(w, sP + (k0 + k) * GM);
#pragma unroll
        for (int g = 0; g < GM; ++g)
#pragma unroll
          for (int e = 0; e < PL; ++e) o[g][e] = fma2(pack2(w[g], w[g]), vv[e], o[g][e]);
      }
      __syncwarp();   // the scratch is written again
    }
  }
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int w = 1; w < LPH; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  }
  __device__ __forceinline__ void emit(float* out, float* lse, int G, int lane) {
    close();
    const int head = lane / LPH;
    const float inv = l > 0.f ? 1.f / l : l;   // (0 and NaN stay)
    if (lse && lane % LPH == 0 && head < G) lse[head] = pa_lse(m, l);
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      const float f = __shfl_sync(0xffffffffu, inv, g * LPH);
      if (g < G) {
#pragma unroll
        for (int e = 0; e < PL; ++e)
          reinterpret_cast<f2*>(out + g * D + lane * EPL)[e] = mul2(o[g][e], pack2(f, f));
      }
    }
  }
  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, int G, int lane) {
    close();
    const int head = lane / LPH;
    if (lane % LPH == 0 && head < G) {
      sM[head] = m;
      sL[head] = l;
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      if (g >= G) break;
#pragma unroll
      for (int e = 0; e < PL; ++e) reinterpret_cast<f2*>(sO + g * D + lane * EPL)[e] = o[g][e];
    }
  }
};

// A warp's walk over the units of its stretch: of the present one it takes tiles i0, i0 + step, ...
// below i1 (of n; the row's tile t0 is the unit's first).  Its lanes walk together.  starts / ends:
// the stretch holds the unit's first / last tile.
template <int KT, int NW>
struct PaWalk {
  int64_t end, unit;   // end of the stretch, place of the unit
  int64_t small;       // a unit of up to this many places is not cut: it goes with its first place
  int row, head, n, i0, i1, t0, step, turn;
  bool starts, ends;
  PaRow R;

  __device__ __forceinline__ void here(int64_t begin) {
    n = R.template tiles<KT>();
    t0 = R.lo / KT;
    i0 = begin > unit ? (int)(begin - unit - 1) : 0;
    i1 = end - unit - 1 < n ? (int)(end - unit - 1) : n;
    if (n < small) {
      i0 = begin > unit ? n : 0;
      i1 = n;
    }
    starts = i0 == 0;
    ends = i1 == n;
    if (step > 1) {   // the tiles go round the warps; `turn` is this warp's distance to its next
      const int mine = i0 + turn, count = i1 - i0;
      turn = (turn + NW - count % NW) % NW;
      i0 = mine;
    }
  }
  __device__ __forceinline__ void next_unit(const PagedAttnArgs& a, bool& bad) {
    unit += n + 1;
    if (++head == a.Hkv) {
      head = 0;
      R = pa_row_or_none(a, ++row, bad);
      // (idle rows are passed 32 at a time: 1000 between two live ones 27 us in all, 174 us with one
      // dependent read after another; 20000 0.55 and 4.2 ms)
      while (R.hi <= R.lo && row < a.T) {
        const PaRow r = pa_row_or_none(a, row + 1 + (threadIdx.x & 31), bad);
        const uint32_t live = __ballot_sync(0xffffffffu, r.hi > r.lo);
        const int k = live ? __ffs(live) - 1 : 31;
        row += 1 + k;
        R.seq = __shfl_sync(0xffffffffu, r.seq, k);
        R.lo = __shfl_sync(0xffffffffu, r.lo, k);
        R.hi = __shfl_sync(0xffffffffu, r.hi, k);
      }
    }
    here(unit);
  }
  // the next unit begins in the stretch
  __device__ __forceinline__ bool more() const { return unit + n + 1 < end; }
  // ends the stretch that begins at `begin` before place e
  __device__ __forceinline__ void limit(int64_t begin, int64_t e) {
    if (e < end) {
      end = e;
      here(begin);
    }
  }
  // to the first unit from here on with a tile for this warp; false if there is none
  __device__ __forceinline__ bool settle(const PagedAttnArgs& a, bool& bad) {
    while (i0 >= i1) {
      if (!more()) return false;
      next_unit(a, bad);
    }
    return true;
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs& a, bool& bad) {
    if (!more()) return false;
    next_unit(a, bad);
    return settle(a, bad);
  }
  __device__ __forceinline__ void open(const PagedAttnArgs& a, const PaStretch& s, int64_t e,
                                       int64_t uncut, bool& bad) {
    end = e;
    small = uncut;
    step = 1;
    turn = 0;
    row = s.row;
    R = pa_row(a, row, bad);
    n = R.template tiles<KT>();
    head = pa_head(s.begin - s.at, n + 1);
    unit = s.at + (int64_t)head * (n + 1);
    here(s.begin);
  }
};

// A part of a unit left in shared memory by a warp.
struct PaPart {
  int row, head;      // row < 0: none
  int starts, ends;   // it holds the unit's first / last tile
};

template <typename T, int D, int GM>
__global__ void __launch_bounds__(PaShape<T, D, GM>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using S = PaShape<T, D, GM>;
  constexpr int KT = S::KT, NW = S::NW, ST = S::ST, NT = S::THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t sMask[NW][ST];
  __shared__ PaStretch sStretch[NW];
  __shared__ PaPart sPart[NW][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G;
  uint8_t* ring = smem + warp * (ST * S::STAGE);
  float* sO = reinterpret_cast<float*>(smem + NW * ST * S::STAGE);   // [NW][G][D]
  float* sM = sO + (S::FIRST_SMEM ? NW * G * D : 0);               // [NW][2][G]
  float* sL = sM + NW * 2 * G;
  float* scratch = sL + NW * 2 * G + warp * S::SCRATCH;
  bool bad = false;
  const PaPlan P = pa_schedule<NW, KT>(a, sStretch, bad);
  const PaWs W = pa_carve(a.ws, G, D);

  float* const firsts_at = S::FIRST_SMEM ? sO : W.first + (int64_t)blockIdx.x * NW * G * D;

  // ---- copies of this warp's tiles.  Where the CTA's stretch lies in at most two units its tiles
  // go round the warps, so that the CTA reads consecutive rows (long rows: 563 us against 592 us
  // with one stretch per warp, 8 rows of 120K tokens); else each warp has a stretch of its own
  // and writes the units within it alone (fp32, 37 rows of up to 2048 tokens, 592 units: 53 us
  // against 138 us with every unit shared by the warps)
  PaWalk<KT, NW> w;
  bool more = sStretch[0].begin < sStretch[0].total;
  bool round = false;
  const int64_t total = sStretch[0].total;
  const int64_t cta_end = sStretch[0].begin + P.per < total ? sStretch[0].begin + P.per : total;
  const int64_t uncut = P.per_warp < kPaSmall ? P.per_warp : kPaSmall;
  PaRec rec = {};
  rec.per = P.per;
  if (more) {
    w.open(a, sStretch[0], cta_end, uncut, bad);
    rec.off = sStretch[0].begin - w.unit;
    rec.n = w.n < w.small ? 0 : w.n + 1;
    rec.row = w.row;
    rec.head = w.head;
    PaWalk<KT, NW> next = w;
    if (next.more()) next.next_unit(a, bad);
    round = !next.more();
    if (round) {
      w.step = NW;
      w.turn = warp;
      w.here(sStretch[0].begin);
    } else if (warp > 0) {
      more = sStretch[warp].begin < cta_end;
      if (more) w.open(a, sStretch[warp], cta_end, uncut, bad);
    }
    if (!round && more) w.limit(sStretch[warp].begin, sStretch[warp].begin + P.per_warp);
    if (more) more = w.settle(a, bad);
  }
  if (threadIdx.x == 0) W.rec[blockIdx.x] = rec;
  PaWalk<KT, NW> u = w;   // the same walk, for the products
  bool go = more;
  int page = -1;
  bool want = false;
  // j / page_size (see launch_both)
  auto page_of = [&](int j) { return (int)((uint64_t)(uint32_t)j * a.page_mul >> a.page_shift); };
  // the page of this lane's token of tile w.i0 (read here, used when the tile is copied)
  auto look = [&]() {
    const int j = (w.t0 + w.i0) * KT + lane;
    want = lane < KT && j >= w.R.lo && j < w.R.hi;
    if (want) page = a.table[w.R.seq * a.max_pages + page_of(j)];
  };
  auto copy = [&](int stage) {
    if (more) {
      int64_t at = -1;
      if (want) {
        if (page >= 0 && page < a.n_pages) {
          const int j = (w.t0 + w.i0) * KT + lane;
          at = page * a.cs[0] + w.head * a.cs[1] +
               (int64_t)(j - page_of(j) * a.page_size) * a.cs[2];
        } else {
          bad = true;
        }
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, at >= 0);
      if (lane == 0) sMask[warp][stage] = mask;
      const uint32_t sK = smem_addr(ring + stage * S::STAGE);
      constexpr int RPI = 32 / S::CH;   // rows per instruction
#pragma unroll
      for (int i = 0; i < KT / RPI; ++i) {
        const int r = i * RPI + lane / S::CH, c = lane % S::CH;
        const int64_t ro = __shfl_sync(0xffffffffu, at, r);
        // bf16 rows are read eight at a time by ldmatrix: pieces swizzled by the row
        const uint32_t dst = sK + r * S::ROW + ((sizeof(T) == 2 ? c ^ (r & 7) : c) << 4);
        const int64_t eo = ro < 0 ? 0 : ro + c * (16 / (int)sizeof(T));
        copy16(dst, static_cast<const T*>(a.K) + eo, ro >= 0);
        copy16(dst + S::HALF, static_cast<const T*>(a.V) + eo, ro >= 0);
      }
      w.i0 += w.step;
      if (w.i0 >= w.i1) more = w.next(a, bad);
      if (more) look();
    }
    copy_commit();
  };
  if (more) look();
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) copy(s);

  // ---- rows that see nothing; what the join needs
  // (found 32 at a time by every warp, filled by the whole block)
  for (int64_t t0 = blockIdx.x; t0 < a.T; t0 += (int64_t)32 * gridDim.x) {
    const int64_t mine = t0 + (int64_t)lane * gridDim.x;
    const PaRow r = mine < a.T ? pa_row(a, (int)mine, bad) : PaRow{-1, 0, 0};
    for (uint32_t left = __ballot_sync(0xffffffffu, r.seq >= 0 && r.hi <= r.lo); left;
         left &= left - 1) {
      const int64_t t = t0 + (int64_t)(__ffs(left) - 1) * gridDim.x;
      for (int e = threadIdx.x; e < a.Hq * D; e += NT)
        store_out(static_cast<T*>(a.out) + t * a.Hq * D + e, 0.f);
      if (a.lse)
        for (int h = threadIdx.x; h < a.Hq; h += NT) a.lse[t * a.Hq + h] = -INFINITY;
    }
  }
  if (threadIdx.x < 2 * NW) sPart[threadIdx.x / 2][threadIdx.x % 2].row = -1;
  __syncthreads();

  // ---- the units of the stretch
  const float sc = a.scale * kLog2e;
  PaWarp<T, D, GM> c;
  int stage = 0;
  while (go) {
    c.load(static_cast<const T*>(a.q) + ((int64_t)u.row * a.Hq + u.head * G) * D, G, lane);
    c.reset();
    for (int i = u.i0; i < u.i1; i += u.step) {
      copy_wait<ST - 2>();
      __syncwarp();   // every lane's copies have landed, and the stage before is read
      copy(stage == 0 ? ST - 1 : stage - 1);
      const uint32_t sK = smem_addr(ring + stage * S::STAGE);
      c.tile(sK, sK + S::HALF, sMask[warp][stage], sc, lane, scratch);
      stage = stage + 1 == ST ? 0 : stage + 1;
    }
    const bool starts = u.starts, ends = u.ends;
    const int row = u.row, head = u.head;
    go = u.next(a, bad);
    if (starts && ends && !round) {
      const int64_t h = (int64_t)row * a.Hq + head * G;
      c.emit(static_cast<T*>(a.out) + h * D, a.lse ? a.lse + h : nullptr, G, lane);
    } else {
      // the first part waits beside the rings, the last one in this warp's own, then unused
      const int k = go ? 0 : 1;
      __syncwarp();
      c.finish(go ? firsts_at + warp * G * D : reinterpret_cast<float*>(ring),
               sM + (warp * 2 + k) * G, sL + (warp * 2 + k) * G, G, lane);
      if (lane == 0) sPart[warp][k] = PaPart{row, head, starts, ends};
    }
  }
  copy_wait<0>();
  if (bad) record_status(a.status, kStatusDeviceCheck);
  __syncthreads();

  // ---- the parts, unit by unit.  Lane p of every warp holds part p; a warp adds whole heads
  static_assert(2 * NW <= 32, "a part per lane");
  const PaPart f = lane < 2 * NW ? sPart[lane / 2][lane % 2] : PaPart{-1, 0, 0, 0};
  const uint32_t mem = __match_any_sync(
      0xffffffffu, f.row < 0 ? ~0ull : ((unsigned long long)f.row << 32 | (uint32_t)f.head));
  const uint32_t starts = __ballot_sync(0xffffffffu, f.starts);
  const uint32_t ends = __ballot_sync(0xffffffffu, f.ends);
  const uint32_t firsts = __ballot_sync(0xffffffffu, f.row >= 0 && __ffs(mem) - 1 == lane);
  constexpr int EPL = D / 32;   // dimensions of a lane
  const int pairs = __popc(firsts) * G;
  for (int x = warp; x < pairs; x += NW) {
    const int g = x % G;
    uint32_t left = firsts;
    for (int k = x / G; k > 0; --k) left &= left - 1;
    const int p = __ffs(left) - 1;
    const uint32_t unit = __shfl_sync(0xffffffffu, mem, p);
    const int row = __shfl_sync(0xffffffffu, f.row, p), head = __shfl_sync(0xffffffffu, f.head, p);
    const bool whole = (starts & unit) && (ends & unit), in = unit >> lane & 1;
    // the CTA's first unit goes to slot 0, another one that is cut to slot 1
    const int slot = blockIdx.x * 2 + (row == rec.row && head == rec.head ? 0 : 1);
    const float m = in ? sM[lane * G + g] : -INFINITY;
    const float M = warp_max(m);
    const float r = in ? exp2f(m - (M == -INFINITY ? 0.f : M)) : 0.f;
    const float L = warp_sum(in ? r * sL[lane * G + g] : 0.f);
    float O[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) O[e] = 0.f;
    for (uint32_t of = unit; of; of &= of - 1) {
      const int o = __ffs(of) - 1;
      const float ro = __shfl_sync(0xffffffffu, r, o);
      const float* v = (o % 2 ? reinterpret_cast<const float*>(smem + (o / 2) * (ST * S::STAGE))
                              : firsts_at + (o / 2) * G * D) + g * D + lane * EPL;
#pragma unroll
      for (int e = 0; e < EPL; ++e) O[e] = fmaf(ro, v[e], O[e]);
    }
    if (whole) {
      const int64_t h = (int64_t)row * a.Hq + head * G + g;
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        store_out(static_cast<T*>(a.out) + h * D + lane * EPL + e, O[e] * inv);
      if (a.lse && lane == 0) a.lse[h] = pa_lse(M, L);
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e) W.o[((int64_t)slot * G + g) * D + lane * EPL + e] = O[e];
      if (lane == 0) *reinterpret_cast<float2*>(W.ml + (slot * G + g) * 2) = make_float2(M, L);
    }
  }
}

// Block (x, g) adds head g of a cut unit: of the unit that boundary c = x + 1 cuts (BY_UNIT
// false), or of unit x (true; fewer blocks when there are fewer units than boundaries).  A unit's
// first boundary is the first behind one of its tiles (its place 0 is none); its parts are those
// of CTAs c - 1, c, ..., added in that order by slices of the block, slice s taking every
// (NT / D)th from the sth.
template <typename T, int D, int NT, bool BY_UNIT>
__global__ void __launch_bounds__(NT)
    paged_attn_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas) {
  constexpr int NS = NT / D;
  __shared__ float sF[kPaCtas], sRed[NT / 32], sO[NS][D];
  __shared__ int sC;
  const int g = blockIdx.y, G = a.G;
  const PaWs W = pa_carve(a.ws, G, D);
  int c = blockIdx.x + 1;
  if constexpr (BY_UNIT) {
    if (threadIdx.x == 0) sC = 0;
    __syncthreads();
    const int t = threadIdx.x;
    if (t >= 1 && t < ctas) {
      const PaRec r = W.rec[t];
      if (r.n && (int64_t)r.row * a.Hkv + r.head == blockIdx.x && r.off > 1 && r.off <= r.per + 1)
        sC = t;
    }
    __syncthreads();
    c = sC;
    if (c == 0) return;
  }
  const PaRec r = W.rec[c];
  if (r.n == 0 || r.off <= 1 || r.off > r.per + 1) return;
  // the part before the boundary is of CTA c - 1's first unit if its stretch begins in the unit
  const int first = 2 * (c - 1) + (r.off >= r.per ? 0 : 1);
  const int parts = 1 + (int)((r.n - r.off + r.per - 1) / r.per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // factors and sum
  float m = -INFINITY, l = 0.f;
  const int k0 = threadIdx.x;   // (parts <= ctas <= 148 <= NT)
  if (k0 < parts) {
    const int part = k0 == 0 ? first : 2 * (c - 1 + k0);
    const float2 t = *reinterpret_cast<const float2*>(W.ml + (part * G + g) * 2);
    m = t.x;
    l = t.y;
  }
  float M = warp_max(m);
  if (lane == 0) sRed[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) M = fmaxf(M, sRed[w]);
  const float f = k0 < parts ? exp2f(m - (M == -INFINITY ? 0.f : M)) : 0.f;
  if (k0 < parts) sF[k0] = f;
  l = warp_sum(f * l);
  __syncthreads();
  if (lane == 0) sRed[warp] = l;
  __syncthreads();
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) L += sRed[w];
  const int sl = threadIdx.x / D, i = threadIdx.x - sl * D;
  float O = 0.f;
#pragma unroll 8
  for (int k = sl; k < parts; k += NS) {
    const int part = k == 0 ? first : 2 * (c - 1 + k);
    O = fmaf(sF[k], W.o[((int64_t)part * G + g) * D + i], O);
  }
  sO[sl][i] = O;
  __syncthreads();
  if (sl != 0) return;
#pragma unroll
  for (int s = 1; s < NS; ++s) O += sO[s][i];
  const int64_t h = (int64_t)r.row * a.Hq + r.head * G + g;
  store_out(static_cast<T*>(a.out) + h * D + i, L == 0.f ? 0.f : O / L);
  if (a.lse && i == 0) a.lse[h] = pa_lse(M, L);
}

template <typename T, int D, int GM>
cudaError_t launch_one(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  using S = PaShape<T, D, GM>;
  auto kern = paged_attn_kernel<T, D, GM>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::smem(GM));
  if (e != cudaSuccess) return e;
  kern<<<grid, S::THREADS, S::smem(a.G), st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_both(const PagedAttnArgs& a, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  cudaError_t e;
  const int grid = sms < kPaCtas ? sms : kPaCtas;
  PagedAttnArgs b = a;
  b.inv_ctas = 1.0 / grid;
  // j / page_size as j mul >> shift, exact below 2^31: with 2^s >= page_size and
  // mul = ceil(2^(31+s) / page_size) the error j (mul page_size - 2^(31+s)) stays below 2^(31+s)
  int s = 0;
  while (((int64_t)1 << s) < a.page_size) ++s;
  b.page_mul = (((uint64_t)1 << (31 + s)) + a.page_size - 1) / a.page_size;
  b.page_shift = 31 + s;
  // (bf16: up to 8 heads are the columns of one product, so one bound serves them)
  if constexpr (sizeof(T) == 2)
    e = a.G <= 8 ? launch_one<T, D, 8>(b, grid, st) : launch_one<T, D, 16>(b, grid, st);
  else
    e = a.G <= 1   ? launch_one<T, D, 1>(b, grid, st)
        : a.G <= 4 ? launch_one<T, D, 4>(b, grid, st)
        : a.G <= 8 ? launch_one<T, D, 8>(b, grid, st)
                   : launch_one<T, D, 16>(b, grid, st);
  if (e != cudaSuccess || grid < 2) return e;
  const int64_t units = (int64_t)a.T * a.Hkv;
  // (launched early by programmatic dependent launch the join gained nothing: one row of 1000
  // tokens 11.0 us against 10.2 us)
  // (few units have many parts each: wide blocks while they all fit one per SM)
  if (units * a.G <= grid)
    paged_attn_join_kernel<T, D, 1024, true>
        <<<dim3((unsigned)units, a.G), 1024, 0, st>>>(b, grid);
  else if (units < grid - 1)
    paged_attn_join_kernel<T, D, 256, true><<<dim3((unsigned)units, a.G), 256, 0, st>>>(b, grid);
  else
    paged_attn_join_kernel<T, D, 256, false><<<dim3(grid - 1, a.G), 256, 0, st>>>(b, grid);
  return cudaGetLastError();
}

}  // namespace

bool paged_attn_supported(int64_t d, int64_t G) { return (d == 64 || d == 128) && G <= 16; }

size_t paged_attn_ws(int64_t d, int64_t G) {
  const PaWs w = pa_carve(nullptr, G, d);
  // (first parts: wherever a kernel for more than four heads may leave them there)
  return reinterpret_cast<size_t>(w.first) +
         (G > 4 ? pa_align((size_t)kPaCtas * 8 * G * d * sizeof(float)) : 0);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, bool bf16, cudaStream_t st) {
  if (bf16)
    return a.d == 64 ? launch_both<__nv_bfloat16, 64>(a, st) : launch_both<__nv_bfloat16, 128>(a, st);
  return a.d == 64 ? launch_both<float, 64>(a, st) : launch_both<float, 128>(a, st);
}

}  // namespace hils
