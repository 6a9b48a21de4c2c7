// Arguments of the paged-cache kernels (csrc/paged_plan.cu, csrc/paged_attn.cu), and their
// launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace hils {

struct PlanArgs {
  int32_t B, T, n_pages, page_size;
  int64_t max_pages;
  const int32_t *kv_len, *new_len, *free_pages, *n_free;
  int32_t *table, *kv_len_out, *n_free_out, *cu, *slot, *pos, *seq, *status;
};
constexpr int kPlanMaxB = 8192;
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st);

struct PagedAttnArgs {
  const void *q, *K, *V;
  const int32_t *table, *seq, *pos;
  void* out;
  float* lse;
  int64_t cs[3];      // cache strides: page, head, token
  int64_t max_pages, max_len;
  int32_t T, B, Hq, Hkv, G, d, n_pages, page_size, window;
  float scale;
  int32_t* status;
  char* ws;           // the region after the status word
  double inv_ctas;    // set by the launcher: 1 / CTAs, and the division by page_size
  uint64_t page_mul;
  int32_t page_shift;
};
bool paged_attn_supported(int64_t d, int64_t G);
// Bytes of the attention's share of the workspace (after the status word).
size_t paged_attn_ws(int64_t d, int64_t G);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, bool bf16, cudaStream_t st);

}  // namespace hils
