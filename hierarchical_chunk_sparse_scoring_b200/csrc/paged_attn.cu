// Attention of single tokens over a paged cache, split over the cache's length and joined.
//
//   out[t, h] = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale q.K_j - m),  lse = m + ln sum_j p_j
// over the tokens j the row sees, one pass with a running maximum m and sum (both fp32).
// Bound: HBM; every seen key and value row is read once for all G heads of its KV head, 4 G d
// flops for 2 d elements.
//
// Work split.  A unit is a (row, KV head); its tokens are cut into tiles of 16.  The tiles of
// all units in order (row, head, tile) form one list, and every CTA takes an equal stretch of it,
// whatever the rows' lengths, computed on the device: CTAs sum the rows' tile counts themselves.  A CTA
// writes units that lie within its stretch; the part of a unit that crosses a boundary goes to
// the workspace as (m, sum, unnormalised output), and the join kernel adds the parts in order.
#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace hils {
namespace {

constexpr int kPaTile = 16;       // tokens per tile
constexpr int kPaCtas = 296;      // CTAs at most (two per SM of 148)
constexpr int kPaMinTiles = 8;    // tiles a CTA takes at least
constexpr int kPaThreads = 256;
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
  __device__ __forceinline__ int tiles() const {
    return hi > lo ? (hi - 1) / kPaTile - lo / kPaTile + 1 : 0;
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

// Offset of token j's row in the pools, or -1 if its page is not in the pool.
__device__ __forceinline__ int64_t pa_offset(const PagedAttnArgs& a, int seq, int j, int head,
                                             bool& bad) {
  const int pi = j / a.page_size;
  const int page = a.table[seq * a.max_pages + pi];
  if (page < 0 || page >= a.n_pages) {
    bad = true;
    return -1;
  }
  return page * a.cs[0] + head * a.cs[1] + (int64_t)(j - pi * a.page_size) * a.cs[2];
}

// Where the CTA's stretch of the tile list begins.
struct PaStart {
  int64_t begin, end, per;   // tiles of the list
  int64_t off;               // of the first unit before `begin`
  int row, head;
};

template <int NT>
__device__ __forceinline__ PaStart pa_schedule(const PagedAttnArgs& a, bool& bad) {
  __shared__ int64_t sWarp[NT / 32];
  __shared__ int64_t sOff;
  __shared__ int sRow, sHead;
  const int chunk = (a.T + NT - 1) / NT;
  const int t0 = threadIdx.x * chunk;
  const int t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  int64_t mine = 0;
  for (int t = t0; t < t1; ++t) mine += pa_row(a, t, bad).tiles();
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
      const int64_t n = pa_row(a, t, bad).tiles();
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

// One warp per token of a tile in turn, lanes over the head dim.
template <typename T, int D, int GM>
__global__ void __launch_bounds__(kPaThreads) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int NW = kPaThreads / 32, EPL = D / 32;
  extern __shared__ float sm[];
  float* sO = sm;                  // [NW][G][D]
  float* sM = sm + NW * GM * D;    // [NW][G]
  float* sL = sM + NW * GM;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G;
  bool bad = false;
  const PaStart S = pa_schedule<kPaThreads>(a, bad);
  const PaWs W = pa_carve(a.ws, G, D);
  // rows that see nothing
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const PaRow r = pa_row(a, t, bad);
    if (r.seq < 0 || r.tiles() > 0) continue;
    for (int e = threadIdx.x; e < a.Hq * D; e += kPaThreads)
      store_out(static_cast<T*>(a.out) + (int64_t)t * a.Hq * D + e, 0.f);
    if (a.lse)
      for (int h = threadIdx.x; h < a.Hq; h += kPaThreads)
        a.lse[(int64_t)t * a.Hq + h] = -INFINITY;
  }
  if (threadIdx.x == 0) {
    PaRec rec;
    rec.off = 0;
    rec.n = 0;
    rec.per = S.per;
    rec.row = rec.head = 0;
    if (S.begin < S.end) {
      rec.off = S.off;
      rec.n = pa_row(a, S.row, bad).tiles();
      rec.row = S.row;
      rec.head = S.head;
    }
    W.rec[blockIdx.x] = rec;
  }
  int row = S.row, head = S.head;
  int64_t off = S.off, left = S.end - S.begin;
  bool first = true;
  const float sc = a.scale * kLog2e;
  while (left > 0) {
    const PaRow R = pa_row(a, row, bad);
    const int n = R.tiles();
    if (n == 0) { ++row; head = 0; continue; }
    const int take = (int)(left < n - off ? left : n - off);
    const T* q = static_cast<const T*>(a.q) + ((int64_t)row * a.Hq + head * G) * D;
    float qv[GM][EPL], o[GM][EPL], m[GM], l[GM];
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        qv[g][e] = g < G ? Elem<T>::to_f(q[g * D + lane + 32 * e]) * sc : 0.f;
        o[g][e] = 0.f;
      }
    }
    for (int i = warp; i < take; i += NW) {
      const int j0 = (R.lo / kPaTile + (int)off + i) * kPaTile;
      int64_t at = -1;
      const int j = j0 + (lane & 15);
      if (j >= R.lo && j < R.hi) at = pa_offset(a, R.seq, j, head, bad);
      for (int c = 0; c < kPaTile; ++c) {
        const int64_t ro = __shfl_sync(0xffffffffu, at, c);
        if (ro < 0) continue;
        float kv[EPL], vv[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          kv[e] = Elem<T>::to_f(static_cast<const T*>(a.K)[ro + lane + 32 * e]);
          vv[e] = Elem<T>::to_f(static_cast<const T*>(a.V)[ro + lane + 32 * e]);
        }
#pragma unroll
        for (int g = 0; g < GM; ++g) {
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) x = fmaf(qv[g][e], kv[e], x);
          x = warp_sum(x);
          if (x > m[g]) {
            const float f = exp2f(m[g] - x);
            m[g] = x;
            l[g] *= f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) o[g][e] *= f;
          }
          const float pj = x == -INFINITY ? 0.f : exp2f(x - m[g]);
          l[g] += pj;
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[g][e] = fmaf(pj, vv[e], o[g][e]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) sO[(warp * GM + g) * D + lane + 32 * e] = o[g][e];
      if (lane == 0) {
        sM[warp * GM + g] = m[g];
        sL[warp * GM + g] = l[g];
      }
    }
    __syncthreads();
    const bool whole = off == 0 && take == n;
    const int part = blockIdx.x * 2 + (first ? 0 : 1);
    for (int e = threadIdx.x; e < G * D; e += kPaThreads) {
      const int g = e / D, i = e - g * D;
      float M = -INFINITY;
      for (int w = 0; w < NW; ++w) M = fmaxf(M, sM[w * GM + g]);
      float L = 0.f, O = 0.f;
      if (M > -INFINITY)
        for (int w = 0; w < NW; ++w) {
          const float f = exp2f(sM[w * GM + g] - M);
          L = fmaf(f, sL[w * GM + g], L);
          O = fmaf(f, sO[(w * GM + g) * D + i], O);
        }
      if (whole) {
        const int64_t h = (int64_t)row * a.Hq + head * G + g;
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
    left -= take;
    off = 0;
    if (++head == a.Hkv) { head = 0; ++row; }
  }
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
  constexpr int NW = kPaThreads / 32;
  const int smem = NW * GM * (D + 2) * (int)sizeof(float);
  auto kern = paged_attn_kernel<T, D, GM>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kPaThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_both(const PagedAttnArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = 2 * sms < kPaCtas ? 2 * sms : kPaCtas;
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
