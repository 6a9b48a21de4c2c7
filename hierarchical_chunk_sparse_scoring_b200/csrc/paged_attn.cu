// Attention of single tokens over a paged cache, split over the cache's length and joined.
//
//   out[t, h] = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale q.K_j - m),  lse = m + ln sum_j p_j
// over the tokens j the row sees, one pass with a running maximum m and sum (both fp32).
// Bound: HBM; every seen key and value row is read once for all G heads of its KV head, 4 G d
// flops for 2 d elements.
//
// Work split.  A unit is a (row, KV head); its tokens are cut into tiles of 16 (bf16) or 8 (fp32).
// The tiles of all units in order (row, head, tile) form one list, and every CTA (one per SM, all
// of its shared memory) takes an equal stretch of it, whatever the rows' lengths; CTAs sum the
// rows' tile counts themselves, so nothing about the lengths is needed on the host.  A CTA writes
// units that lie within its stretch; the part of a unit that crosses a boundary goes to the
// workspace as (m, sum, unnormalised output), and the join kernel adds the parts in order.
//
// Inside a CTA tile f of the stretch is warp f mod 8's, and each warp runs its own ring of cp.async
// stages over its tiles, across unit boundaries, with its own running maximum and sum: no block
// barrier while a unit lasts, two where one ends and the warps' results are added.  The 128 KB a
// CTA has in flight cover the latency of HBM; a tile's page id is read one tile ahead of its copy.
//   bf16  S^T = K Q^T and O^T += V^T P^T by m16n8k16 products: the tokens (then the head
//         dimension) are the 16 rows, the G heads the 8 columns, so no row of a product is
//         padding at G = 8 and P^T is S^T transposed in registers (movmatrix).
//   fp32  each lane holds D/32 dimensions of q and O for all heads; a tile's dot products are
//         summed over the lanes by halving exchanges that leave each lane its own (head, token).
#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace hils {
namespace {

constexpr int kPaCtas = 148;      // CTAs at most (one per SM of 148)
constexpr int kPaMinTiles = 8;    // tiles a CTA takes at least: one per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The first unit of a CTA's stretch, for the join: offset of the stretch in the unit, the unit's
// tiles, and the tiles per stretch (n = 0: no stretch).
struct PaRec {
  int64_t off, n, per;
  int32_t row, head;
};

struct PaWs {
  PaRec* rec;    // [ctas]
  float* ml;     // [ctas][2][G][2] running maximum (base 2) and sum
  float* o;      // [ctas][2][G][d]
};

__host__ __device__ inline size_t pa_align(size_t x) { return (x + 255) / 256 * 256; }

__host__ __device__ inline PaWs pa_carve(char* ws, int64_t G, int64_t d) {
  PaWs w;
  w.rec = reinterpret_cast<PaRec*>(ws);
  ws += pa_align(kPaCtas * sizeof(PaRec));
  w.ml = reinterpret_cast<float*>(ws);
  ws += pa_align((size_t)kPaCtas * 2 * G * 2 * sizeof(float));
  w.o = reinterpret_cast<float*>(ws);
  return w;
}

// What row t sees: tokens lo .. hi - 1 of sequence seq (seq < 0: padding).
struct PaRow {
  int seq, lo, hi;
  template <int KT>
  __device__ __forceinline__ int tiles() const {
    return hi > lo ? (hi - 1) / KT - lo / KT + 1 : 0;
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

// Where the CTA's stretch of the tile list begins.
struct PaStart {
  int64_t begin, end, per;   // tiles of the list
  int64_t off;               // of the first unit before `begin`
  int row, head;
};

template <int NT, int KT>
__device__ __forceinline__ PaStart pa_schedule(const PagedAttnArgs& a, bool& bad) {
  __shared__ int64_t sWarp[NT / 32];
  __shared__ int64_t sOff;
  __shared__ int sRow, sHead;
  const int chunk = (a.T + NT - 1) / NT;
  const int t0 = threadIdx.x * chunk;
  const int t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  int64_t mine = 0;
  for (int t = t0; t < t1; ++t) mine += pa_row(a, t, bad).tiles<KT>();
  mine *= a.Hkv;
  int64_t total;
  int64_t at = block_scan<NT>(mine, sWarp, total);
  PaStart s;
  s.per = (total + gridDim.x - 1) / gridDim.x;
  if (s.per < kPaMinTiles) s.per = kPaMinTiles;
  s.begin = s.per * blockIdx.x;
  s.end = s.begin + s.per < total ? s.begin + s.per : total;
  if (s.begin < total && s.begin >= at && s.begin < at + mine) {
    for (int t = t0; t < t1; ++t) {
      const int64_t n = pa_row(a, t, bad).tiles<KT>();
      if (s.begin < at + n * a.Hkv) {
        sRow = t;
        sHead = (int)((s.begin - at) / n);
        sOff = (s.begin - at) - sHead * n;
        break;
      }
      at += n * a.Hkv;
    }
  }
  __syncthreads();
  s.row = sRow;
  s.head = sHead;
  s.off = sOff;
  return s;
}

template <typename T>
__device__ __forceinline__ void store_out(T* p, float v) { *p = Elem<T>::from_f(v); }

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
  // warps and the bytes of each one's ring: what fits beside the merge (G (D + 4) floats a warp)
  static constexpr int NW = GM <= 4 || (GM <= 8 && sizeof(T) == 2) ? 8 : 6;
  static constexpr int ST = (GM <= 8 && NW == 6 ? 32768 : 24576) / STAGE;
  static constexpr int THREADS = NW * 32;
  static constexpr int OS = D + 4;                          // floats per head of the merge
  static constexpr int SCRATCH = sizeof(T) == 2 ? 0 : KT * GM + GM;   // fp32: weights, factors
  static int smem(int G) {
    return NW * ST * STAGE + NW * (G * OS + 2 * G + SCRATCH) * (int)sizeof(float);
  }
  static_assert(NW * (ST * STAGE + (GM * OS + 2 * GM + SCRATCH) * 4) <= 226 * 1024, "fits an SM");
  static_assert(ST >= 3, "two tiles in flight while one is used");
  static_assert(CH == 8 || CH == 16 || CH == 32, "whole rows per copy");
};

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
    uint32_t p[NB][2];
    float f[NB][2];
    bool moved = false;
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
          moved = true;
        }
        // (a maximum of -inf: nothing seen yet, all weights are zero)
        const float base = t == -INFINITY ? 0.f : t;
        s[nb][e] = exp2f(s[nb][e] - base);
        s[nb][2 + e] = exp2f(s[nb][2 + e] - base);
        l[nb][e] = fmaf(l[nb][e], f[nb][e], s[nb][e] + s[nb][2 + e]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(s[nb][2 * h], s[nb][2 * h + 1]);
        p[nb][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nb][i][e] *= f[nb][e & 1];
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      const int r = (lane & 7) + ((lane >> 4) << 3);
      ldsm4_t(a, sV + r * S::ROW + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][i], a, p[nb][0], p[nb][1]);
    }
  }
  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, int G, int lane) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = nb * 8 + (lane % 4) * 2 + e;
        float t = l[nb][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
        if (g >= G) continue;
        if (lane < 4) {
          sM[g] = m[nb][e];
          sL[g] = t;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          sO[g * S::OS + i * 16 + lane / 4] = o[nb][i][e];
          sO[g * S::OS + i * 16 + lane / 4 + 8] = o[nb][i][2 + e];
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
  float q[GM][EPL], o[GM][EPL], m, l;   // m, l: of head lane / LPH

  static __device__ __forceinline__ void get(float (&v)[EPL], const float* p) {
    if constexpr (EPL == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(p);
      v[0] = t.x; v[1] = t.y;
    }
  }
  static __device__ __forceinline__ void get_row(float (&v)[EPL], uint32_t addr) {
    if constexpr (EPL == 4)
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                   : "r"(addr)
                   : "memory");
    else
      asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                   : "=f"(v[0]), "=f"(v[1])
                   : "r"(addr)
                   : "memory");
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
      for (int e = 0; e < EPL; ++e) q[g][e] = 0.f;
      if (g < G) get(q[g], src + g * D + lane * EPL);
    }
  }
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int g = 0; g < GM; ++g)
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[g][e] = 0.f;
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
        float kv[EPL];
        get_row(kv, sK + (k0 + k) * S::ROW + lane * EPL * 4);
#pragma unroll
        for (int g = 0; g < GM; ++g) {
          float t = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) t = fmaf(q[g][e], kv[e], t);
          x[g * KG + k] = t;
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
          const float r = sF[g];
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[g][e] *= r;
        }
      }
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        float vv[EPL];
        get_row(vv, sV + (k0 + k) * S::ROW + lane * EPL * 4);
        float w[GM];
        get_heads(w, sP + (k0 + k) * GM);
#pragma unroll
        for (int g = 0; g < GM; ++g)
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[g][e] = fmaf(w[g], vv[e], o[g][e]);
      }
      __syncwarp();   // the scratch is written again
    }
  }
  __device__ __forceinline__ void finish(float* sO, float* sM, float* sL, int G, int lane) {
#pragma unroll
    for (int w = 1; w < LPH; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    const int head = lane / LPH;
    if (lane % LPH == 0 && head < G) {
      sM[head] = m;
      sL[head] = l;
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      if (g >= G) break;
#pragma unroll
      for (int e = 0; e < EPL; ++e) sO[g * S::OS + lane * EPL + e] = o[g][e];
    }
  }
};

// A warp's walk over the tiles of its CTA's stretch, for the copies: tile f of the stretch lies in
// the unit part f0 .. f1 - 1, whose first tile is the row's tile t0.
template <int KT>
struct PaWalk {
  int64_t f, f0, f1, len;
  int row, head;
  int64_t t0;
  PaRow R;

  __device__ __forceinline__ void start(const PagedAttnArgs& a, const PaStart& s, int64_t at,
                                        bool& bad) {
    f = at;
    f0 = 0;
    len = s.end > s.begin ? s.end - s.begin : 0;
    f1 = 0;
    if (len == 0) return;
    row = s.row;
    head = s.head;
    R = pa_row(a, row, bad);
    t0 = R.lo / KT + s.off;
    const int64_t n = R.template tiles<KT>() - s.off;
    f1 = n < len ? n : len;
  }
  // to the next unit (there is one: f1 < len)
  __device__ __forceinline__ void next_unit(const PagedAttnArgs& a, bool& bad) {
    f0 = f1;
    if (++head == a.Hkv) {
      head = 0;
      do {
        ++row;
        R = pa_row(a, row, bad);
      } while (R.template tiles<KT>() == 0);
    }
    t0 = R.lo / KT;
    const int64_t n = R.template tiles<KT>();
    f1 = f0 + n < len ? f0 + n : len;
  }
};

template <typename T, int D, int GM>
__global__ void __launch_bounds__(PaShape<T, D, GM>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using S = PaShape<T, D, GM>;
  constexpr int KT = S::KT, NW = S::NW, ST = S::ST, NT = S::THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t sMask[NW][ST];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G;
  uint8_t* ring = smem + warp * (ST * S::STAGE);
  float* sO = reinterpret_cast<float*>(smem + NW * ST * S::STAGE);   // [NW][G][OS]
  float* sM = sO + NW * G * S::OS;                                   // [NW][G]
  float* sL = sM + NW * G;
  float* scratch = sL + NW * G + warp * S::SCRATCH;
  bool bad = false;
  const PaStart P = pa_schedule<NT, KT>(a, bad);
  const PaWs W = pa_carve(a.ws, G, D);

  // ---- copies of this warp's tiles
  PaWalk<KT> w;
  w.start(a, P, warp, bad);
  int page = -1;
  bool want = false;
  // the page of this lane's token of tile w.f (read here, used when the tile is copied)
  auto look = [&]() {
    want = false;
    if (w.f >= w.len) return;
    while (w.f >= w.f1) w.next_unit(a, bad);
    const int64_t j = (w.t0 + w.f - w.f0) * KT + lane;
    want = lane < KT && j >= w.R.lo && j < w.R.hi;
    if (want) page = a.table[w.R.seq * a.max_pages + (int)j / a.page_size];
  };
  auto copy = [&](int stage) {
    if (w.f < w.len) {
      int64_t at = -1;
      if (want) {
        if (page >= 0 && page < a.n_pages) {
          const int j = (int)(w.t0 + w.f - w.f0) * KT + lane;
          at = page * a.cs[0] + w.head * a.cs[1] + (int64_t)(j % a.page_size) * a.cs[2];
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
      w.f += NW;
      look();
    }
    copy_commit();
  };
  look();
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) copy(s);

  // ---- rows that see nothing; what the join needs
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const PaRow r = pa_row(a, t, bad);
    if (r.seq < 0 || r.tiles<KT>() > 0) continue;
    for (int e = threadIdx.x; e < a.Hq * D; e += NT)
      store_out(static_cast<T*>(a.out) + (int64_t)t * a.Hq * D + e, 0.f);
    if (a.lse)
      for (int h = threadIdx.x; h < a.Hq; h += NT) a.lse[(int64_t)t * a.Hq + h] = -INFINITY;
  }
  PaWalk<KT> u;
  u.start(a, P, warp, bad);
  if (threadIdx.x == 0) {
    PaRec rec = {};
    rec.per = P.per;
    if (u.len > 0) {
      rec.off = P.off;
      rec.n = u.R.template tiles<KT>();
      rec.row = u.row;
      rec.head = u.head;
    }
    W.rec[blockIdx.x] = rec;
  }

  // ---- the units of the stretch
  const float sc = a.scale * kLog2e;
  PaWarp<T, D, GM> c;
  bool first = true;
  int64_t off = P.off;
  int stage = 0;
  while (u.f0 < u.len) {
    c.load(static_cast<const T*>(a.q) + ((int64_t)u.row * a.Hq + u.head * G) * D, G, lane);
    c.reset();
    for (; u.f < u.f1; u.f += NW) {
      copy_wait<ST - 2>();
      __syncwarp();   // every lane's copies have landed, and the stage before is read
      copy(stage == 0 ? ST - 1 : stage - 1);
      const uint32_t sK = smem_addr(ring + stage * S::STAGE);
      c.tile(sK, sK + S::HALF, sMask[warp][stage], sc, lane, scratch);
      stage = stage + 1 == ST ? 0 : stage + 1;
    }
    c.finish(sO + warp * G * S::OS, sM + warp * G, sL + warp * G, G, lane);
    __syncthreads();
    const int n = u.R.template tiles<KT>();
    const bool whole = off == 0 && u.f1 - u.f0 == n;
    const int part = blockIdx.x * 2 + (first ? 0 : 1);
    for (int e = threadIdx.x; e < G * D; e += NT) {
      const int g = e / D, i = e - g * D;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < NW; ++k) M = fmaxf(M, sM[k * G + g]);
      float L = 0.f, O = 0.f;
      if (M > -INFINITY) {
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          const float f = exp2f(sM[k * G + g] - M);
          L = fmaf(f, sL[k * G + g], L);
          O = fmaf(f, sO[(k * G + g) * S::OS + i], O);
        }
      }
      if (whole) {
        const int64_t h = (int64_t)u.row * a.Hq + u.head * G + g;
        store_out(static_cast<T*>(a.out) + h * D + i, L > 0.f ? O / L : 0.f);
        if (a.lse && i == 0) a.lse[h] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
      } else {
        W.o[((int64_t)part * G + g) * D + i] = O;
        if (i == 0) {
          W.ml[(part * G + g) * 2] = M;
          W.ml[(part * G + g) * 2 + 1] = L;
        }
      }
    }
    __syncthreads();
    first = false;
    off = 0;
    if (u.f1 >= u.len) break;
    u.next_unit(a, bad);
  }
  copy_wait<0>();
  if (bad) record_status(a.status, kStatusDeviceCheck);
}

// Block (c, g): head g of the unit that boundary c = 1 .. ctas - 1 cuts, if c is the unit's first
// boundary: the parts of CTAs c - 1, c, ... in that order.
template <typename T, int D>
__global__ void __launch_bounds__(D) paged_attn_join_kernel(const PagedAttnArgs a) {
  const int c = blockIdx.x + 1, g = blockIdx.y, G = a.G;
  const PaWs W = pa_carve(a.ws, G, D);
  const PaRec r = W.rec[c];
  if (r.n == 0 || r.off == 0 || r.off > r.per) return;
  // the part before the boundary is CTA c - 1's first unit if its stretch begins with the unit
  // (r.off == r.per) and otherwise its last
  const int first = 2 * (c - 1) + (r.off == r.per ? 0 : 1);
  const int parts = 1 + (int)((r.n - r.off + r.per - 1) / r.per);
  float M = -INFINITY;
  for (int k = 0; k < parts; ++k) {
    const int part = k == 0 ? first : 2 * (c - 1 + k);
    M = fmaxf(M, W.ml[(part * G + g) * 2]);
  }
  float L = 0.f, O = 0.f;
  if (M > -INFINITY) {
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const int part = k == 0 ? first : 2 * (c - 1 + k);
      const float f = exp2f(W.ml[(part * G + g) * 2] - M);
      L = fmaf(f, W.ml[(part * G + g) * 2 + 1], L);
      O = fmaf(f, W.o[((int64_t)part * G + g) * D + threadIdx.x], O);
    }
  }
  const int64_t h = (int64_t)r.row * a.Hq + r.head * G + g;
  store_out(static_cast<T*>(a.out) + h * D + threadIdx.x, L > 0.f ? O / L : 0.f);
  if (a.lse && threadIdx.x == 0) a.lse[h] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
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
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = sms < kPaCtas ? sms : kPaCtas;
  // (bf16: up to 8 heads are the columns of one product, so one bound serves them)
  if constexpr (sizeof(T) == 2)
    e = a.G <= 8 ? launch_one<T, D, 8>(a, grid, st) : launch_one<T, D, 16>(a, grid, st);
  else
    e = a.G <= 1   ? launch_one<T, D, 1>(a, grid, st)
        : a.G <= 4 ? launch_one<T, D, 4>(a, grid, st)
        : a.G <= 8 ? launch_one<T, D, 8>(a, grid, st)
                   : launch_one<T, D, 16>(a, grid, st);
  if (e != cudaSuccess || grid < 2) return e;
  paged_attn_join_kernel<T, D><<<dim3(grid - 1, a.G), D, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool paged_attn_supported(int64_t d, int64_t G) { return (d == 64 || d == 128) && G <= 16; }

size_t paged_attn_ws(int64_t d, int64_t G) {
  const PaWs w = pa_carve(nullptr, G, d);
  return reinterpret_cast<size_t>(w.o) +
         pa_align((size_t)kPaCtas * 2 * G * d * sizeof(float));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, bool bf16, cudaStream_t st) {
  if (bf16)
    return a.d == 64 ? launch_both<__nv_bfloat16, 64>(a, st) : launch_both<__nv_bfloat16, 128>(a, st);
  return a.d == 64 ? launch_both<float, 64>(a, st) : launch_both<float, 128>(a, st);
}

}  // namespace hils
