// Arguments of the query/key norm-and-rotation kernels (csrc/qk_norm.cu), and their launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace hils {

constexpr int kQkMaxD = 256;
constexpr int kQkMaxPairs = kQkMaxD / 2;
// Blocks of the backward kernel at most (four per SM of 148): each leaves one pair of partial
// weight gradients in the workspace.
constexpr int kQkBwdBlocks = 592;

struct RopeTable {
  int32_t rot, interleaved;
  float mscale;
  uint64_t turn[kQkMaxPairs];   // pair m's turns per position, freq / (2 pi) mod 1, times 2^64
};

// Row addressing: element (b, h, n, i) of a tensor at base + b st[0] + h st[1] + n st[2] + i.
struct QkArgs {
  const void *q, *k, *v, *wq, *wk;
  void *qo, *ko;               // forward outputs / backward: gradients of q and k
  const void *gq, *gk;         // backward: gradients of the outputs
  const int32_t *pos, *slot;   // slot: append only
  int64_t qs[3], ks[3], vs[3], qos[3], kos[3], gqs[3], gks[3];
  void *Kc, *Vc;               // append: the cache pools
  int64_t cs[3];
  int64_t N, tokens, pos0, n_slots;
  int32_t Hq, Hkv, d, page_size, norm;
  float eps;
  int32_t* status;
  double* dw_part;             // backward: [blocks][2][d]
  RopeTable rope;
};

cudaError_t launch_qk_norm_rope(const QkArgs& a, bool bf16, bool paged, cudaStream_t st);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, bool bf16, bool grad_bf16, float* dw_q,
                                    float* dw_k, cudaStream_t st);

}  // namespace hils
