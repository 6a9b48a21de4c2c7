// Block tables, slot map and positions of one step of a paged cache, from the requests' lengths.
//
// Per sequence b: have = ceil(kv_len / page), need = ceil((kv_len + new) / page) - have pages;
// the exclusive sums of `new` and of `need` over the sequences number the step's tokens and the
// pages taken from the free stack.  A token finds its sequence by a binary search in the first
// sum, a new page its place in the table by one in the second.
// Bound: latency (a few KB of lengths, 12 bytes a token).  One launch; every CTA sums the lengths
// itself (8192 sequences at most, in shared memory), then takes its share of the tokens and pages.
// Where the new lengths overwrite the old ones the CTAs are one cluster of up to eight, whose
// barrier lies between reading and writing them (no second launch, no counter in the workspace);
// else there are as many as the tokens occupy, up to one per SM.  Threads take four tokens together
// once the tokens outnumber them: past 8192 in place, past 151552 otherwise.  (53 sequences, 131072
// tokens: 5.2 us, a token a thread; in place 17 us, with a token at a time 24.8 us.  256 decoding
// sequences: 4.2 us, in place 5.3 us.)
#include <cooperative_groups.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace hils {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;          // portable cluster size
constexpr int kPlanBatch = 4;            // tokens a thread works on together, if it has them
constexpr int kPlanCtas = 148;

// Last b with off[b] <= x (off ascending, off[0] = 0 <= x).
__device__ __forceinline__ int find(const int32_t* off, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* sLen = smem;             // kv_len
  int32_t* sHave = smem + a.B;      // its pages
  int32_t* sCu = smem + 2 * a.B;    // first token
  int32_t* sPg = smem + 3 * a.B;    // first new page
  __shared__ int64_t sWarp[kPlanThreads / 32];
  const uint32_t ps = (uint32_t)a.page_size;
  const int64_t cap = a.max_pages * ps < INT32_MAX ? a.max_pages * ps : INT32_MAX;
  bool bad = false;
  int free_n = a.n_free[0];
  if (free_n < 0 || free_n > a.n_pages) {
    bad = true;
    free_n = free_n < 0 ? 0 : a.n_pages;
  }
  // sums over the sequences, one of a thread's per round.  The tokens of the admitted ones are
  // numbered by a sum of their own once one is refused (one refused for pages leaves a gap).
  int64_t c_new = 0, c_need = 0, c_tok = 0, pages = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int32_t len = 0, add = 0;
    uint32_t have = 0, need = 0;
    if (b < a.B) {
      len = a.kv_len[b];
      add = a.new_len[b];
      if (len < 0 || add < 0 || (int64_t)len + add > cap) {
        bad = true;
        add = 0;
      }
      have = ((uint32_t)(len < 0 ? 0 : len) + ps - 1) / ps;
      if (add > 0) need = ((uint32_t)len + (uint32_t)add + ps - 1) / ps - have;
    }
    int64_t t_new, t_need, t_tok, t_pages;
    const int64_t e_new = c_new + block_scan<kPlanThreads>(add, sWarp, t_new);
    const int64_t e_need = c_need + block_scan<kPlanThreads>(need, sWarp, t_need);
    const bool admit = (add == 0 || e_new + add <= a.T) && (need == 0 || e_need + need <= free_n);
    if (!admit) bad = true;
    int64_t e_tok = c_tok + e_new - c_new;
    t_tok = t_new;
    t_pages = t_need;
    if (__syncthreads_or(!admit)) {
      e_tok = c_tok + block_scan<kPlanThreads>(admit ? add : 0, sWarp, t_tok);
      block_scan<kPlanThreads>(admit ? need : 0, sWarp, t_pages);
    }
    if (b < a.B) {
      sLen[b] = len;
      sHave[b] = (int32_t)have;
      sCu[b] = (int32_t)e_tok;
      // pages are admitted as a prefix, so the sum over all is exact wherever it is used; past
      // the stack it only has to stay above every page taken
      sPg[b] = (int32_t)(e_need < (int64_t)INT32_MAX ? e_need : (int64_t)INT32_MAX);
    }
    c_new += t_new;
    c_need += t_need;
    c_tok += t_tok;
    pages += t_pages;
  }
  const int n_tok = (int)c_tok, n_new = (int)pages;
  if constexpr (IN_PLACE)
    cg::this_cluster().sync();   // every CTA has read the lengths; sums visible to the block
  else
    __syncthreads();
  const int rank = blockIdx.x, stride = gridDim.x * kPlanThreads;
  const int me = rank * kPlanThreads + threadIdx.x;
  if (rank == 0) {
    for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
      const int32_t next = b + 1 < a.B ? sCu[b + 1] : n_tok;
      a.cu[b] = sCu[b];
      a.kv_len_out[b] = sLen[b] + (next - sCu[b]);
    }
    if (threadIdx.x == 0) {
      a.cu[a.B] = n_tok;
      a.n_free_out[0] = free_n - n_new;
    }
  }
  for (int64_t y = me; y < n_new; y += stride) {
    const int x = (int)y, b = find(sPg, a.B, x);
    a.table[b * a.max_pages + sHave[b] + (x - sPg[b])] = a.free_pages[free_n - 1 - x];
  }
  for (int64_t t0 = me; t0 < a.T; t0 += (int64_t)kPlanBatch * stride) {
    int32_t page[kPlanBatch], pos[kPlanBatch], seq[kPlanBatch], off[kPlanBatch];
#pragma unroll
    for (int k = 0; k < kPlanBatch; ++k) {
      const int64_t t = t0 + (int64_t)k * stride;
      page[k] = pos[k] = seq[k] = off[k] = -1;
      if (t < n_tok) {
        const int b = find(sCu, a.B, (int32_t)t);
        seq[k] = b;
        pos[k] = sLen[b] + ((int32_t)t - sCu[b]);
        const int32_t pi = (int32_t)((uint32_t)pos[k] / ps);
        off[k] = pos[k] - pi * (int32_t)ps;
        // (entries below `have` are not written here)
        page[k] = pi < sHave[b] ? a.table[b * a.max_pages + pi]
                                : a.free_pages[free_n - 1 - (sPg[b] + (pi - sHave[b]))];
      }
    }
#pragma unroll
    for (int k = 0; k < kPlanBatch; ++k) {
      const int64_t t = t0 + (int64_t)k * stride;
      if (t >= a.T) break;
      int32_t slot = -1;
      if (seq[k] >= 0) {
        if (page[k] >= 0 && page[k] < a.n_pages)
          slot = page[k] * (int32_t)ps + off[k];
        else
          bad = true;
      }
      a.slot[t] = slot;
      a.pos[t] = pos[k];
      a.seq[t] = seq[k];
    }
  }
  if (bad) record_status(a.status, kStatusDeviceCheck);
}

template <bool IN_PLACE>
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
  const int most = IN_PLACE ? kPlanCluster : kPlanCtas;
  const int64_t want = ((int64_t)a.T + kPlanThreads - 1) / kPlanThreads;
  int ctas = (int)(want < 1 ? 1 : want > most ? most : want);
  if (IN_PLACE)
    while (ctas & (ctas - 1)) ctas &= ctas - 1;   // a power of two
  auto kern = paged_plan_kernel<IN_PLACE>;
  constexpr int kWords = 4;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kPlanMaxB * kWords * (int)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)a.B * kWords * sizeof(int32_t);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = IN_PLACE ? ctas : 1;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = IN_PLACE ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  return a.kv_len_out == a.kv_len || a.n_free_out == a.n_free ? launch_plan<true>(a, st)
                                                              : launch_plan<false>(a, st);
}

}  // namespace hils
