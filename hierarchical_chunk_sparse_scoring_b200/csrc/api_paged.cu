// Host side of the C ABI for the query/key norms with rotary positions and for the paged cache:
// argument checks and kernel arguments.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "hils.h"
#include "host.h"
#include "paged.h"
#include "qk_norm.h"

namespace hils {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// Strides of a tensor with these sizes (those of a dimension of one entry are not used): 16-byte
// multiples, not negative; of an output, at least a row.
bool ok_strides(const int64_t (&st)[3], int64_t es, int64_t B, int64_t H, int64_t N, int64_t d,
                bool output) {
  const int64_t n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < 0 || st[i] % (16 / es) != 0) return false;
    if (st[i] > (INT64_MAX / 64) / n[i]) return false;   // offsets within 63 bits of bytes
    if (output && st[i] < d) return false;
  }
  return true;
}

hils_status check_rope(const hils_rope* r, int64_t d) {
  if (!r || r->rot_dim < 0 || (r->layout != HILS_ROPE_HALF && r->layout != HILS_ROPE_INTERLEAVED))
    return HILS_ERR_INVALID_ARG;
  if (r->rot_dim > d) return HILS_ERR_INVALID_ARG;
  if (r->rot_dim % 16 != 0 || r->rot_dim > kQkMaxD) return HILS_ERR_UNSUPPORTED;
  if (!std::isfinite(r->mscale)) return HILS_ERR_INVALID_ARG;
  for (int m = 0; m < r->rot_dim / 2; ++m)
    if (!std::isfinite(r->freq[m]) || std::fabs(r->freq[m]) > 1e6) return HILS_ERR_INVALID_ARG;
  return HILS_OK;
}

hils_status check_qk(const hils_qk_params* p, const hils_rope* rope) {
  if (!p) return HILS_ERR_INVALID_ARG;
  if (p->B < 0 || p->N < 0 || p->Hq < 0 || p->Hkv < 0 || p->d < 1 || p->pos0 < 0)
    return HILS_ERR_INVALID_ARG;
  if (p->dtype != HILS_F32 && p->dtype != HILS_BF16) return HILS_ERR_INVALID_ARG;
  if (p->norm != 0 && p->norm != 1) return HILS_ERR_INVALID_ARG;
  if (p->norm && (!std::isfinite(p->eps) || p->eps < 0.f)) return HILS_ERR_INVALID_ARG;
  if (p->d % 8 != 0 || p->d > kQkMaxD) return HILS_ERR_UNSUPPORTED;
  if (p->Hq > 65536 || p->Hkv > 65536) return HILS_ERR_UNSUPPORTED;
  if (p->N > 0 && p->B > INT32_MAX / p->N) return HILS_ERR_UNSUPPORTED;
  if (p->pos0 > INT32_MAX) return HILS_ERR_UNSUPPORTED;
  return check_rope(rope, p->d);
}

void copy3(int64_t (&to)[3], const int64_t (&from)[3]) {
  for (int i = 0; i < 3; ++i) to[i] = from[i];
}

// freq / (2 pi) mod 1 in units of 2^-64: positions are whole, so position times this, modulo 2^64, is
// the angle modulo one turn (within position 2^-65 turns and the rounding of the quotient to 64
// bits), and no floating-point reduction is needed on the device.
uint64_t turn_fraction(double freq) {
  const long double t = (long double)freq / 6.283185307179586476925286766559005768L;
  const long double f = t - floorl(t);                        // [0, 1]
  const long double u = floorl(f * 18446744073709551616.0L + 0.5L);
  return u >= 18446744073709551616.0L ? 0 : (uint64_t)u;      // (a whole turn is none)
}

QkArgs qk_args(const hils_qk_params* p, const hils_rope* rope) {
  QkArgs a = {};
  a.N = p->N;
  a.tokens = p->B * p->N;
  a.pos0 = p->pos0;
  a.Hq = (int32_t)p->Hq;
  a.Hkv = (int32_t)p->Hkv;
  a.d = (int32_t)p->d;
  a.norm = p->norm;
  a.eps = p->eps;
  copy3(a.qs, p->q_str);
  copy3(a.ks, p->k_str);
  copy3(a.vs, p->v_str);
  a.rope.rot = rope->rot_dim;
  a.rope.interleaved = rope->layout == HILS_ROPE_INTERLEAVED;
  a.rope.mscale = rope->mscale;
  for (int m = 0; m < rope->rot_dim / 2; ++m) a.rope.turn[m] = turn_fraction(rope->freq[m]);
  return a;
}

// An int32 array: read and written word by word, so any element of one may be its start.
bool ok_int(const int32_t* p, bool needed) {
  return !(reinterpret_cast<uintptr_t>(p) & 3u) && (p || !needed);
}

int64_t elem_size(int32_t dtype) { return dtype == HILS_BF16 ? 2 : 4; }

hils_status check_cache(const hils_paged_params* c) {
  if (!c) return HILS_ERR_INVALID_ARG;
  if (c->T < 0 || c->B < 0 || c->n_pages < 0 || c->max_pages < 0 || c->page_size < 1 ||
      c->window < 0)
    return HILS_ERR_INVALID_ARG;
  if (c->T > INT32_MAX - (1 << 16) || c->B > INT32_MAX - 1 ||
      c->n_pages > (int64_t)INT32_MAX / c->page_size || c->max_pages > INT32_MAX)
    return HILS_ERR_UNSUPPORTED;
  return HILS_OK;
}

bool attn_shape_ok(const hils_paged_params* c) {
  return c->Hq >= 1 && c->Hkv >= 1 && c->Hq % c->Hkv == 0 && c->Hq <= 65536 &&
         paged_attn_supported(c->d, c->Hq / c->Hkv);
}

// Whether two tensors share their first element, unless with the same strides (in the dimensions
// [B, H, N] of more than one entry) and element sizes, as an operator in place has them.
bool clash(const void* x, const int64_t (&xs)[3], int64_t ex, const void* y,
           const int64_t (&ys)[3], int64_t ey, int64_t B, int64_t H, int64_t N) {
  if (!x || x != y) return false;
  return ex != ey || (B > 1 && xs[0] != ys[0]) || (H > 1 && xs[1] != ys[1]) ||
         (N > 1 && xs[2] != ys[2]);
}

// A contiguous int32 array of a call.
struct Ints {
  const int32_t* p;
  int64_t n;
  bool overlaps(const Ints& o) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
    return n > 0 && o.n > 0 && a < b + 4 * (uint64_t)o.n && b < a + 4 * (uint64_t)n;
  }
};

hils_status done(cudaError_t e) { return e == cudaSuccess ? HILS_OK : HILS_ERR_CUDA; }

}  // namespace
}  // namespace hils

using namespace hils;

extern "C" hils_status hils_rope_init(hils_rope* rope, int32_t rot_dim, int32_t layout,
                                      int32_t scaling, double base, double factor,
                                      double train_len, double beta_fast, double beta_slow) {
  if (!rope || rot_dim < 0 || (layout != HILS_ROPE_HALF && layout != HILS_ROPE_INTERLEAVED) ||
      scaling < HILS_ROPE_PLAIN || scaling > HILS_ROPE_HOPE || !std::isfinite(base) ||
      !(base > 1.0))
    return HILS_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > kQkMaxD) return HILS_ERR_UNSUPPORTED;
  const bool stretch = scaling == HILS_ROPE_LINEAR || scaling == HILS_ROPE_NTK ||
                       scaling == HILS_ROPE_YARN;
  if (stretch && (!std::isfinite(factor) || !(factor >= 1.0))) return HILS_ERR_INVALID_ARG;
  if (scaling == HILS_ROPE_YARN &&
      (!std::isfinite(train_len) || !(train_len > 0.0) || !std::isfinite(beta_fast) ||
       !std::isfinite(beta_slow) || !(beta_fast > beta_slow)))
    return HILS_ERR_INVALID_ARG;
  if (scaling == HILS_ROPE_HOPE && std::isnan(train_len)) return HILS_ERR_INVALID_ARG;
  rope->rot_dim = rot_dim;
  rope->layout = layout;
  rope->mscale = scaling == HILS_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  rope->reserved = 0;
  if (scaling == HILS_ROPE_NTK && rot_dim > 2)
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int m = 0; m < 128; ++m) {
    double f = 0.0;
    if (m < rot_dim / 2) {
      const double th = std::pow(base, -2.0 * m / rot_dim);
      f = th;
      if (scaling == HILS_ROPE_LINEAR) f = th / factor;
      if (scaling == HILS_ROPE_YARN) {
        const double r = train_len * th / kTwoPi;
        double g = (r - beta_slow) / (beta_fast - beta_slow);
        g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
        f = g * th + (1.0 - g) * th / factor;
      }
      if (scaling == HILS_ROPE_HOPE && !(kTwoPi / th <= train_len)) f = 0.0;
    }
    rope->freq[m] = f;
  }
  return HILS_OK;
}

extern "C" hils_status hils_qk_norm_rope(const hils_qk_params* p, const hils_rope* rope,
                                         const void* q, const void* k, const void* w_q,
                                         const void* w_k, const int32_t* pos, void* q_out,
                                         void* k_out, hils_stream_t stream) {
  hils_status s = check_qk(p, rope);
  if (s != HILS_OK) return s;
  const bool any = p->B > 0 && p->N > 0;
  const bool anyq = any && p->Hq > 0, anyk = any && p->Hkv > 0;
  const int64_t es = elem_size(p->dtype);
  if (!ok_ptr(q, anyq) || !ok_ptr(q_out, anyq) || !ok_ptr(k, anyk) || !ok_ptr(k_out, anyk) ||
      !aligned16(w_q) || !aligned16(w_k) || (!p->norm && (w_q || w_k)) ||
      !ok_int(pos, false))
    return HILS_ERR_INVALID_ARG;
  if ((anyq && (!ok_strides(p->q_str, es, p->B, p->Hq, p->N, p->d, false) ||
                !ok_strides(p->qo_str, es, p->B, p->Hq, p->N, p->d, true))) ||
      (anyk && (!ok_strides(p->k_str, es, p->B, p->Hkv, p->N, p->d, false) ||
                !ok_strides(p->ko_str, es, p->B, p->Hkv, p->N, p->d, true))))
    return HILS_ERR_INVALID_ARG;
  if (!anyq && !anyk) return HILS_OK;
  if ((anyq && clash(q, p->q_str, es, q_out, p->qo_str, es, p->B, p->Hq, p->N)) ||
      (anyk && clash(k, p->k_str, es, k_out, p->ko_str, es, p->B, p->Hkv, p->N)) ||
      (anyq && anyk && (q_out == k || k_out == q || q_out == k_out)))
    return HILS_ERR_INVALID_ARG;
  if ((s = check_device()) != HILS_OK) return s;
  QkArgs a = qk_args(p, rope);
  a.q = q; a.k = k; a.wq = w_q; a.wk = w_k; a.pos = pos; a.qo = q_out; a.ko = k_out;
  copy3(a.qos, p->qo_str);
  copy3(a.kos, p->ko_str);
  return done(launch_qk_norm_rope(a, p->dtype == HILS_BF16, false,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t hils_qk_backward_workspace_size(const hils_qk_params* p) {
  if (!p || p->d < 1 || p->d > kQkMaxD || p->d % 8 != 0) return 0;
  return align_up((size_t)kQkBwdBlocks * 2 * (size_t)p->d * sizeof(double));
}

extern "C" hils_status hils_qk_norm_rope_backward(
    const hils_qk_params* p, const hils_rope* rope, const void* q, const void* k,
    const void* w_q, const void* w_k, const int32_t* pos, const void* dq_out, const void* dk_out,
    void* dq, void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
    hils_stream_t stream) {
  hils_status s = check_qk(p, rope);
  if (s != HILS_OK) return s;
  if (p->grad_dtype != HILS_F32 && p->grad_dtype != p->dtype) return HILS_ERR_INVALID_ARG;
  const bool any = p->B > 0 && p->N > 0;
  const bool anyq = any && p->Hq > 0, anyk = any && p->Hkv > 0;
  const bool dw = dw_q || dw_k;
  const int64_t es = elem_size(p->dtype), gs = elem_size(p->grad_dtype);
  if (!ok_ptr(q, anyq && p->norm) || !ok_ptr(k, anyk && p->norm) || !ok_ptr(dq_out, anyq) ||
      !ok_ptr(dq, anyq) || !ok_ptr(dk_out, anyk) || !ok_ptr(dk, anyk) || !aligned16(w_q) ||
      !aligned16(w_k) || !aligned16(dw_q) || !aligned16(dw_k) ||
      (!p->norm && (w_q || w_k || dw)) || !ok_int(pos, false))
    return HILS_ERR_INVALID_ARG;
  if ((anyq && (!ok_strides(p->q_str, es, p->B, p->Hq, p->N, p->d, false) ||
                !ok_strides(p->qo_str, gs, p->B, p->Hq, p->N, p->d, false) ||
                !ok_strides(p->dq_str, gs, p->B, p->Hq, p->N, p->d, true))) ||
      (anyk && (!ok_strides(p->k_str, es, p->B, p->Hkv, p->N, p->d, false) ||
                !ok_strides(p->ko_str, gs, p->B, p->Hkv, p->N, p->d, false) ||
                !ok_strides(p->dk_str, gs, p->B, p->Hkv, p->N, p->d, true))))
    return HILS_ERR_INVALID_ARG;
  if (dw && (!workspace || !aligned16(workspace) ||
             workspace_bytes < hils_qk_backward_workspace_size(p)))
    return HILS_ERR_WORKSPACE;
  if (!anyq && !anyk && !dw) return HILS_OK;
  // (without a norm q and k are not read)
  const void *xq = p->norm ? q : nullptr, *xk = p->norm ? k : nullptr;
  if ((anyq && (clash(dq_out, p->qo_str, gs, dq, p->dq_str, gs, p->B, p->Hq, p->N) ||
                clash(xq, p->q_str, es, dq, p->dq_str, gs, p->B, p->Hq, p->N))) ||
      (anyk && (clash(dk_out, p->ko_str, gs, dk, p->dk_str, gs, p->B, p->Hkv, p->N) ||
                clash(xk, p->k_str, es, dk, p->dk_str, gs, p->B, p->Hkv, p->N))) ||
      (anyq && anyk && (dq == dk || dq == dk_out || dk == dq_out || dq == xk || dk == xq)) ||
      (dw && dw_q == dw_k))
    return HILS_ERR_INVALID_ARG;
  if ((s = check_device()) != HILS_OK) return s;
  QkArgs a = qk_args(p, rope);
  if (!anyq) a.Hq = 0;
  if (!anyk) a.Hkv = 0;
  a.q = q; a.k = k; a.wq = w_q; a.wk = w_k; a.pos = pos;
  a.gq = dq_out; a.gk = dk_out; a.qo = dq; a.ko = dk;
  copy3(a.gqs, p->qo_str);
  copy3(a.gks, p->ko_str);
  copy3(a.qos, p->dq_str);
  copy3(a.kos, p->dk_str);
  a.dw_part = dw ? static_cast<double*>(workspace) : nullptr;
  return done(launch_qk_norm_rope_bwd(a, p->dtype == HILS_BF16, p->grad_dtype == HILS_BF16, dw_q,
                                      dw_k, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t hils_paged_workspace_size(const hils_paged_params* p) {
  if (check_cache(p) != HILS_OK) return 0;
  return kStatusBytes + (attn_shape_ok(p) ? paged_attn_ws(p->d, p->Hq / p->Hkv) : 0);
}

extern "C" hils_status hils_paged_plan(const hils_paged_params* p, const int32_t* kv_len,
                                       const int32_t* new_len, int32_t* block_table,
                                       const int32_t* free_pages, const int32_t* n_free,
                                       int32_t* kv_len_out, int32_t* n_free_out, int32_t* cu,
                                       int32_t* slot, int32_t* pos, int32_t* seq,
                                       void* workspace, size_t workspace_bytes,
                                       hils_stream_t stream) {
  hils_status s = check_cache(p);
  if (s != HILS_OK) return s;
  if (p->B > kPlanMaxB) return HILS_ERR_UNSUPPORTED;
  const bool rows = p->B > 0, tok = p->T > 0;
  // (free_pages is read only if pages are taken, which n_free[0] <= n_pages bounds)
  if (!ok_int(kv_len, rows) || !ok_int(new_len, rows) || !ok_int(kv_len_out, rows) ||
      !ok_int(block_table, rows && p->max_pages > 0) || !ok_int(free_pages, p->n_pages > 0) ||
      !ok_int(n_free, true) || !ok_int(n_free_out, true) || !ok_int(cu, true) ||
      !ok_int(slot, tok) || !ok_int(pos, tok) || !ok_int(seq, tok))
    return HILS_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < kStatusBytes)
    return HILS_ERR_WORKSPACE;
  const Ints in[] = {{kv_len, p->B}, {n_free, 1}, {new_len, p->B}, {free_pages, p->n_pages}};
  const Ints out[] = {{kv_len_out, p->B}, {n_free_out, 1}, {block_table, p->B * p->max_pages},
                      {cu, p->B + 1},     {slot, p->T},    {pos, p->T}, {seq, p->T}};
  for (int i = 0; i < 7; ++i) {
    for (int j = 0; j < 4; ++j)   // (lengths and the free count may be updated in place)
      if (out[i].overlaps(in[j]) && !(i == j && i < 2 && out[i].p == in[j].p))
        return HILS_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[i].overlaps(out[j])) return HILS_ERR_INVALID_ARG;
  }
  if ((s = check_device()) != HILS_OK) return s;
  PlanArgs a;
  a.B = (int32_t)p->B;
  a.T = (int32_t)p->T;
  a.n_pages = (int32_t)p->n_pages;
  a.page_size = p->page_size;
  a.max_pages = p->max_pages;
  a.kv_len = kv_len; a.new_len = new_len; a.free_pages = free_pages; a.n_free = n_free;
  a.table = block_table; a.kv_len_out = kv_len_out; a.n_free_out = n_free_out; a.cu = cu;
  a.slot = slot; a.pos = pos; a.seq = seq;
  a.status = static_cast<int32_t*>(workspace);
  return done(launch_paged_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" hils_status hils_paged_append(const hils_qk_params* p, const hils_rope* rope,
                                         const hils_paged_params* c, const void* q,
                                         const void* k, const void* v, const void* w_q,
                                         const void* w_k, const int32_t* pos,
                                         const int32_t* slot, void* q_out, void* K, void* V,
                                         void* workspace, size_t workspace_bytes,
                                         hils_stream_t stream) {
  hils_status s = check_qk(p, rope);
  if (s != HILS_OK) return s;
  if ((s = check_cache(c)) != HILS_OK) return s;
  if (p->B != 1 || p->N != c->T || p->Hq != c->Hq || p->Hkv != c->Hkv || p->d != c->d ||
      p->dtype != c->dtype)
    return HILS_ERR_INVALID_ARG;
  const bool any = p->N > 0;
  const bool anyq = any && p->Hq > 0, anyk = any && p->Hkv > 0, pool = anyk && c->n_pages > 0;
  const int64_t es = elem_size(p->dtype);
  if (!ok_ptr(q, anyq) || !ok_ptr(q_out, anyq) || !ok_ptr(k, anyk) || !ok_ptr(v, anyk) ||
      !ok_ptr(K, pool) || !ok_ptr(V, pool) || !aligned16(w_q) || !aligned16(w_k) ||
      (!p->norm && (w_q || w_k)) || !ok_int(pos, any) || !ok_int(slot, any))
    return HILS_ERR_INVALID_ARG;
  if ((anyq && (!ok_strides(p->q_str, es, p->B, p->Hq, p->N, p->d, false) ||
                !ok_strides(p->qo_str, es, p->B, p->Hq, p->N, p->d, true))) ||
      (anyk && (!ok_strides(p->k_str, es, p->B, p->Hkv, p->N, p->d, false) ||
                !ok_strides(p->v_str, es, p->B, p->Hkv, p->N, p->d, false))) ||
      (pool && !ok_strides(c->c_str, es, c->n_pages, c->Hkv, c->page_size, c->d, true)))
    return HILS_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < kStatusBytes)
    return HILS_ERR_WORKSPACE;
  if (!anyq && !anyk) return HILS_OK;
  if ((anyq && clash(q, p->q_str, es, q_out, p->qo_str, es, p->B, p->Hq, p->N)) ||
      (anyq && anyk && (q_out == k || q_out == v)) || (pool && K == V))
    return HILS_ERR_INVALID_ARG;
  if ((s = check_device()) != HILS_OK) return s;
  QkArgs a = qk_args(p, rope);
  a.q = q; a.k = k; a.v = v; a.wq = w_q; a.wk = w_k; a.pos = pos; a.slot = slot; a.qo = q_out;
  copy3(a.qos, p->qo_str);
  a.Kc = K; a.Vc = V;
  copy3(a.cs, c->c_str);
  a.page_size = c->page_size;
  a.n_slots = c->n_pages * c->page_size;
  a.status = static_cast<int32_t*>(workspace);
  return done(launch_qk_norm_rope(a, p->dtype == HILS_BF16, true,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" hils_status hils_paged_attn(const hils_paged_params* p, const void* q, const void* K,
                                       const void* V, const int32_t* block_table,
                                       const int32_t* seq, const int32_t* pos, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes,
                                       hils_stream_t stream) {
  hils_status s = check_cache(p);
  if (s != HILS_OK) return s;
  if (p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0 || p->d < 1 ||
      (p->dtype != HILS_F32 && p->dtype != HILS_BF16) || !std::isfinite(p->scale))
    return HILS_ERR_INVALID_ARG;
  if (!attn_shape_ok(p)) return HILS_ERR_UNSUPPORTED;
  if (!seq && p->T > p->B) return HILS_ERR_INVALID_ARG;
  const bool any = p->T > 0, pool = any && p->n_pages > 0;
  if (!ok_ptr(q, any) || !ok_ptr(out, any) || !ok_ptr(K, pool) || !ok_ptr(V, pool) ||
      !ok_int(block_table, any && p->B > 0 && p->max_pages > 0) || !ok_int(seq, false) ||
      !ok_int(pos, any) || !aligned16(lse))
    return HILS_ERR_INVALID_ARG;
  if (pool && !ok_strides(p->c_str, elem_size(p->dtype), p->n_pages, p->Hkv, p->page_size, p->d,
                          false))
    return HILS_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < hils_paged_workspace_size(p))
    return HILS_ERR_WORKSPACE;
  if (!any) return HILS_OK;
  if ((s = check_device()) != HILS_OK) return s;
  PagedAttnArgs a;
  // (an empty pool has no address; copies of nothing still name one)
  a.q = q; a.K = pool ? K : q; a.V = pool ? V : q; a.table = block_table; a.seq = seq; a.pos = pos;
  a.out = out; a.lse = lse;
  copy3(a.cs, p->c_str);
  a.max_pages = p->max_pages;
  const int64_t longest = p->max_pages * p->page_size;   // (below 2^62)
  a.max_len = longest < INT32_MAX - 64 ? longest : INT32_MAX - 64;
  a.T = (int32_t)p->T;
  a.B = (int32_t)p->B;
  a.Hq = (int32_t)p->Hq;
  a.Hkv = (int32_t)p->Hkv;
  a.G = (int32_t)(p->Hq / p->Hkv);
  a.d = (int32_t)p->d;
  a.n_pages = (int32_t)p->n_pages;
  a.page_size = p->page_size;
  a.window = p->window;
  a.scale = p->scale > 0.f ? p->scale : (float)(1.0 / std::sqrt((double)p->d));
  a.status = static_cast<int32_t*>(workspace);
  a.ws = static_cast<char*>(workspace) + kStatusBytes;
  return done(launch_paged_attn(a, p->dtype == HILS_BF16,
                                reinterpret_cast<cudaStream_t>(stream)));
}
