// Block tables, slot map and positions of one step of a paged cache, from the requests' lengths.
//
// Per sequence b: have = ceil(kv_len / page), need = ceil((kv_len + new) / page) - have pages;
// the exclusive sums of `new` and of `need` over the sequences number the step's tokens and the
// pages taken from the free stack.  A token finds its sequence by a binary search in the first
// sum, a new page its place in the table by one in the second.
// Bound: latency (a few KB of lengths, 12 bytes a token).  One launch of one cluster of up to
// eight CTAs: every CTA sums the lengths itself (8192 sequences at most, in shared memory), then
// takes its share of the tokens and pages; the cluster barrier between reading the lengths and
// writing the new ones is what lets kv_len_out be kv_len without a second launch or a counter in
// the workspace.
#include <cooperative_groups.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace hils {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;          // portable cluster size
constexpr int kPlanTokensPerCta = 4096;  // below this a further CTA saves nothing

// Last b with off[b] <= x (off ascending, off[0] = 0 <= x).
__device__ __forceinline__ int find(const int32_t* off, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* sLen = smem;            // kv_len
  int32_t* sCu = smem + a.B;       // first token
  int32_t* sPg = smem + 2 * a.B;   // first new page
  __shared__ int64_t sWarp[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int ps = a.page_size;
  const int64_t cap = a.max_pages * ps < INT32_MAX ? a.max_pages * ps : INT32_MAX;
  bool bad = false;
  int free_n = a.n_free[0];
  if (free_n < 0 || free_n > a.n_pages) {
    bad = true;
    free_n = free_n < 0 ? 0 : a.n_pages;
  }
  // sums over the sequences, a thread's sequence per round; tokens of the admitted ones are
  // numbered by a third sum (a sequence refused for pages leaves a gap in the first)
  int64_t c_new = 0, c_need = 0, c_tok = 0, pages = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int32_t len = 0, add = 0;
    int64_t need = 0;
    if (b < a.B) {
      len = a.kv_len[b];
      add = a.new_len[b];
      if (len < 0 || add < 0 || (int64_t)len + add > cap) {
        bad = true;
        add = 0;
      }
      if (add > 0) need = ((int64_t)len + add + ps - 1) / ps - ((int64_t)len + ps - 1) / ps;
    }
    int64_t t_new, t_need, t_tok, t_pages;
    const int64_t e_new = c_new + block_scan<kPlanThreads>(add, sWarp, t_new);
    const int64_t e_need = c_need + block_scan<kPlanThreads>(need, sWarp, t_need);
    const bool admit = (add == 0 || e_new + add <= a.T) && (need == 0 || e_need + need <= free_n);
    if (!admit) bad = true;
    const int64_t e_tok = c_tok + block_scan<kPlanThreads>(admit ? add : 0, sWarp, t_tok);
    block_scan<kPlanThreads>(admit ? need : 0, sWarp, t_pages);
    if (b < a.B) {
      sLen[b] = len;
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
  cluster.sync();   // every CTA has read the lengths; sums visible to the block
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
  for (int x = me; x < n_new; x += stride) {
    const int b = find(sPg, a.B, x);
    const int64_t have = ((int64_t)sLen[b] + ps - 1) / ps;
    a.table[b * a.max_pages + have + (x - sPg[b])] = a.free_pages[free_n - 1 - x];
  }
  for (int t = me; t < a.T; t += stride) {
    int32_t slot = -1, pos = -1, seq = -1;
    if (t < n_tok) {
      const int b = find(sCu, a.B, t);
      const int32_t len = sLen[b];
      const int64_t have = ((int64_t)len + ps - 1) / ps;
      seq = b;
      pos = len + (t - sCu[b]);
      const int64_t pi = pos / ps;
      const int32_t page = pi < have ? a.table[b * a.max_pages + pi]
                                     : a.free_pages[free_n - 1 - (sPg[b] + (pi - have))];
      if (page >= 0 && page < a.n_pages)
        slot = page * ps + (pos - (int32_t)pi * ps);
      else
        bad = true;
    }
    a.slot[t] = slot;
    a.pos[t] = pos;
    a.seq[t] = seq;
  }
  if (bad) record_status(a.status, kStatusDeviceCheck);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  int ctas = 1;
  while (ctas < kPlanCluster && (int64_t)ctas * kPlanTokensPerCta < a.T) ctas *= 2;
  const size_t smem = (size_t)a.B * 3 * sizeof(int32_t);
  cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kPlanMaxB * 3 * (int)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
}

}  // namespace hils
