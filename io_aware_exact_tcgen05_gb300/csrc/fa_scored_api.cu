// fa_scored_api.cu -- the extern "C" boundary of the operators before the scores (declared in
// include/fa.h): head norms with rotation, row intervals and mask plans: argument validation
// and launch.  (The attention on capped and biased scores is beside the plain one, in fa_api.cu.)
#include <algorithm>
#include <cmath>

#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_kv.h"
#include "fa_prep.h"
#include "fa_scored.h"

namespace {

using fa::api_fail;

#define FA_TRY(expr)                 \
  do {                               \
    fa_status _s = (expr);           \
    if (_s != FA_OK) return _s;      \
  } while (0)

fa_status check_align(const void* p, const char* name, unsigned align, bool nullable) {
  if (!p && !nullable) return api_fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return api_fail(FA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align);
  return FA_OK;
}

fa_status check_rows(const char* who, int B, int Sq, int Sk) {
  if (B < 1 || Sq < 1 || Sk < 1)
    return api_fail(FA_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d Sq=%d Sk=%d)", who, B, Sq, Sk);
  if (B > 65535) return api_fail(FA_ERR_INVALID_ARG, "%s: B (%d) > 65535", who, B);
  if (1LL * B * Sq >= (1LL << 31) || 1LL * B * Sk >= (1LL << 31))
    return api_fail(FA_ERR_INVALID_ARG, "%s: too large for 32-bit row indices", who);
  return FA_OK;
}

// A strided view [B, S, H, d] with contiguous channels; `written`: no two elements may share an
// address.
fa_status check_view(const fa_heads* v, const char* name, int B, int S, int H, int d, bool written) {
  if (!v) return api_fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  FA_TRY(check_align(v->ptr, name, 16, false));
  const long long st[3] = {v->stride_b, v->stride_t, v->stride_h};
  const int n[3] = {B, S, H};
  struct Dim { long long st; int n; } dims[3];
  int k = 0;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;  // never stepped over
    if (st[i] < 0 || st[i] % 8 != 0)
      return api_fail(FA_ERR_INVALID_ARG, "%s: stride %lld (strides are >= 0 and multiples of 8)",
                      name, st[i]);
    if (st[i] > (1LL << 40))
      return api_fail(FA_ERR_INVALID_ARG, "%s: stride %lld is too large", name, st[i]);
    dims[k++] = {st[i], n[i]};
  }
  if (written) {
    std::sort(dims, dims + k, [](const Dim& a, const Dim& b) { return a.st < b.st; });
    long long extent = d;
    for (int i = 0; i < k; ++i) {
      if (dims[i].st < extent)
        return api_fail(FA_ERR_INVALID_ARG, "%s is written and overlaps itself", name);
      extent += dims[i].st * (dims[i].n - 1);
    }
  }
  return FA_OK;
}

// What the forward and the backward share: sizes, norm and rotation.
fa_status check_prep(const char* who, int B, int S, int Hq, int Hkv, int d, const void* q_weight,
                     const void* k_weight, float w_off, float eps, const int32_t* positions,
                     int n_axes, const float* inv_freq, const uint8_t* freq_axis, int rot_dim,
                     fa::PrepParams* p) {
  if (B < 1 || S < 1 || Hq < 1 || Hkv < 1)
    return api_fail(FA_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d S=%d Hq=%d Hkv=%d)", who, B, S,
                    Hq, Hkv);
  if (d != 64 && d != 128)
    return api_fail(FA_ERR_UNSUPPORTED, "head dimension %d (want 64 or 128)", d);
  if (1LL * B * S >= (1LL << 31))
    return api_fail(FA_ERR_INVALID_ARG, "%s: too many tokens for 32-bit indices", who);
  if (Hq > 65535 || Hkv > 65535)
    return api_fail(FA_ERR_INVALID_ARG, "%s: more than 65535 heads", who);
  FA_TRY(check_align(q_weight, "q_weight", 16, true));
  FA_TRY(check_align(k_weight, "k_weight", 16, true));
  if (!std::isfinite(w_off)) return api_fail(FA_ERR_INVALID_ARG, "weight_offset is not finite");
  if (!(std::isfinite(eps) && eps >= 0.f))
    return api_fail(FA_ERR_INVALID_ARG, "eps (%g) must be finite and >= 0", (double)eps);
  if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0)
    return api_fail(FA_ERR_INVALID_ARG, "rot_dim (%d) must be a multiple of 16 in [0, d = %d]",
                    rot_dim, d);
  if (rot_dim > 0) {
    FA_TRY(check_align(inv_freq, "inv_freq", 4, false));
    FA_TRY(check_align(positions, "positions", 4, true));
    if (n_axes < 1 || n_axes > 255)
      return api_fail(FA_ERR_INVALID_ARG, "n_axes (%d) must lie in [1, 255]", n_axes);
  }
  p->positions = positions;
  p->inv_freq = inv_freq;
  p->freq_axis = freq_axis;
  p->w_off = w_off;
  p->eps = eps;
  p->n_axes = n_axes;
  p->rot = rot_dim;
  p->B = B;
  p->S = S;
  p->d = d;
  return FA_OK;
}

fa_status sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return api_fail(FA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  return FA_OK;
}

void set_input(fa::PrepRole* r, const fa_heads* v) {
  r->x = v->ptr;
  r->xb = v->stride_b;
  r->xt = v->stride_t;
  r->xh = v->stride_h;
}

void set_grad(fa::PrepRole* r, const fa_heads* v) {
  r->dx = v->ptr;
  r->db = v->stride_b;
  r->dt = v->stride_t;
  r->dh = v->stride_h;
}

}  // namespace

extern "C" {

fa_status fa_row_bounds(const int32_t* cu_docs, const int32_t* prefix, int n_docs, int32_t* row_lo,
                        int32_t* row_hi, int B, int Sq, int Sk, int causal, int window,
                        cudaStream_t stream) {
  FA_TRY(check_rows("fa_row_bounds", B, Sq, Sk));
  FA_TRY(check_align(row_lo, "row_lo", 4, false));
  FA_TRY(check_align(row_hi, "row_hi", 4, false));
  FA_TRY(check_align(cu_docs, "cu_docs", 4, true));
  FA_TRY(check_align(prefix, "prefix", 4, true));
  if (cu_docs && (n_docs < 1 || n_docs > 1 << 30))
    return api_fail(FA_ERR_INVALID_ARG, "fa_row_bounds: n_docs (%d) must lie in [1, 2^30]", n_docs);
  if (window < 0)
    return api_fail(FA_ERR_INVALID_ARG, "window (%d) must be >= 0 (0: none)", window);
  FA_TRY(fa::api_check_device());
  const fa::RowBoundsParams p{cu_docs, prefix, row_lo, row_hi, n_docs, B, Sq, Sk, causal ? 1 : 0,
                              window};
  const cudaError_t e = fa::launch_row_bounds(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_row_bounds launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

size_t fa_mask_plan_size(int B, int Sq, int Sk) {
  if (B < 1 || Sq < 1 || Sk < 1) return 0;
  return 4 * fa::mask_plan_words(B, Sq, Sk);
}

fa_status fa_mask_plan(const int32_t* row_lo, const int32_t* row_hi, int B, int Sq, int Sk,
                       void* plan, size_t plan_bytes, cudaStream_t stream) {
  FA_TRY(check_rows("fa_mask_plan", B, Sq, Sk));
  FA_TRY(check_align(row_lo, "row_lo", 4, false));
  FA_TRY(check_align(row_hi, "row_hi", 4, false));
  if (Sq > 0x7fffffff - 256 || Sk > 0x7fffffff - 256)  // ends of tiles are 32-bit numbers
    return api_fail(FA_ERR_INVALID_ARG, "fa_mask_plan: Sq and Sk are at most 2^31 - 257");
  const size_t need = fa_mask_plan_size(B, Sq, Sk);
  if (!plan || plan_bytes < need)
    return api_fail(FA_ERR_WORKSPACE, "the mask plan of these sizes has %zu bytes, got %zu", need,
                    plan ? plan_bytes : size_t(0));
  FA_TRY(check_align(plan, "plan", 16, false));
  FA_TRY(fa::api_check_device());
  const cudaError_t e =
      fa::launch_mask_plan(row_lo, row_hi, B, Sq, Sk, fa::mask_plan_view(plan, B, Sq, Sk), stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_mask_plan launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

fa_status fa_qk_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* v, void* q_out,
                          void* k_out, void* v_out, const int32_t* row_start, int S_out,
                          const void* q_weight, const void* k_weight, float weight_offset,
                          float eps, const int32_t* positions, int n_axes, const float* inv_freq,
                          const uint8_t* freq_axis, int rot_dim, int interleaved, int B, int S,
                          int Hq, int Hkv, int d, cudaStream_t stream) {
  fa::PrepParams p{};
  FA_TRY(check_prep("fa_qk_norm_rope", B, S, Hq, Hkv, d, q_weight, k_weight, weight_offset, eps,
                    positions, n_axes, inv_freq, freq_axis, rot_dim, &p));
  if ((v == nullptr) != (v_out == nullptr))
    return api_fail(FA_ERR_INVALID_ARG, "v and v_out are given together or not at all");
  FA_TRY(check_view(q, "q", B, S, Hq, d, false));
  FA_TRY(check_view(k, "k", B, S, Hkv, d, false));
  if (v) FA_TRY(check_view(v, "v", B, S, Hkv, d, false));
  FA_TRY(check_align(q_out, "q_out", 16, false));
  FA_TRY(check_align(k_out, "k_out", 16, false));
  FA_TRY(check_align(v_out, "v_out", 16, true));
  FA_TRY(check_align(row_start, "row_start", 4, true));
  if (S_out < 1 || (!row_start && S_out < S))
    return api_fail(FA_ERR_INVALID_ARG, "S_out (%d): keys and values need %d rows", S_out,
                    row_start ? 1 : S);
  FA_TRY(fa::api_check_device());
  int n_sm = 0;
  FA_TRY(sm_count(&n_sm));
  p.interleaved = interleaved ? 1 : 0;
  p.row_start = row_start;
  set_input(&p.role[0], q);
  set_input(&p.role[1], k);
  if (v) set_input(&p.role[2], v);
  p.role[0].y = q_out;
  p.role[1].y = k_out;
  p.role[2].y = v_out;
  p.role[0].w = q_weight;
  p.role[1].w = k_weight;
  p.role[0].y_rows = S;
  p.role[1].y_rows = p.role[2].y_rows = S_out;
  p.role[0].heads = Hq;
  p.role[1].heads = Hkv;
  p.role[2].heads = v ? Hkv : 0;
  fa::prep_plan(&p, n_sm, false);
  const cudaError_t e = fa::launch_prep(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_qk_norm_rope launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d < 1 ? 0 : static_cast<size_t>(fa::prep_partial_rows()) * 2 * d * sizeof(float);
}

fa_status fa_qk_norm_rope_bwd(const fa_heads* q, const fa_heads* k, const void* dq_out,
                              const void* dk_out, const void* dv_out, const fa_heads* dq,
                              const fa_heads* dk, const fa_heads* dv, float* dq_weight,
                              float* dk_weight, const void* q_weight, const void* k_weight,
                              float weight_offset, float eps, const int32_t* positions,
                              int n_axes, const float* inv_freq, const uint8_t* freq_axis,
                              int rot_dim, int interleaved, int B, int S, int Hq, int Hkv, int d,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fa::PrepParams p{};
  FA_TRY(check_prep("fa_qk_norm_rope_bwd", B, S, Hq, Hkv, d, q_weight, k_weight, weight_offset, eps,
                    positions, n_axes, inv_freq, freq_axis, rot_dim, &p));
  if ((dv == nullptr) != (dv_out == nullptr))
    return api_fail(FA_ERR_INVALID_ARG, "dv and dv_out are given together or not at all");
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
    return api_fail(FA_ERR_INVALID_ARG, "a weight's gradient is asked for without the weight");
  if (q_weight) FA_TRY(check_view(q, "q", B, S, Hq, d, false));
  if (k_weight) FA_TRY(check_view(k, "k", B, S, Hkv, d, false));
  FA_TRY(check_view(dq, "dq", B, S, Hq, d, true));
  FA_TRY(check_view(dk, "dk", B, S, Hkv, d, true));
  if (dv) FA_TRY(check_view(dv, "dv", B, S, Hkv, d, true));
  FA_TRY(check_align(dq_out, "dq_out", 16, false));
  FA_TRY(check_align(dk_out, "dk_out", 16, false));
  FA_TRY(check_align(dv_out, "dv_out", 16, true));
  FA_TRY(check_align(dq_weight, "dq_weight", 4, true));
  FA_TRY(check_align(dk_weight, "dk_weight", 4, true));
  if (dq_weight || dk_weight) {
    const size_t need = fa_qk_norm_rope_bwd_workspace_size(d);
    if (!workspace || workspace_bytes < need)
      return api_fail(FA_ERR_WORKSPACE, "the weights' gradients need a workspace of %zu bytes, got %zu",
                      need, workspace ? workspace_bytes : size_t(0));
    FA_TRY(check_align(workspace, "workspace", 16, false));
  }
  FA_TRY(fa::api_check_device());
  int n_sm = 0;
  FA_TRY(sm_count(&n_sm));
  p.interleaved = interleaved ? 1 : 0;
  p.partial = static_cast<float*>(workspace);
  if (q_weight) set_input(&p.role[0], q);
  if (k_weight) set_input(&p.role[1], k);
  set_grad(&p.role[0], dq);
  set_grad(&p.role[1], dk);
  if (dv) set_grad(&p.role[2], dv);
  p.role[0].y = const_cast<void*>(dq_out);
  p.role[1].y = const_cast<void*>(dk_out);
  p.role[2].y = const_cast<void*>(dv_out);
  p.role[0].w = q_weight;
  p.role[1].w = k_weight;
  p.role[0].dw = dq_weight;
  p.role[1].dw = dk_weight;
  for (fa::PrepRole& r : p.role) r.y_rows = S;
  p.role[0].heads = Hq;
  p.role[1].heads = Hkv;
  p.role[2].heads = dv ? Hkv : 0;
  fa::prep_plan(&p, n_sm, true);
  const cudaError_t e = fa::launch_prep_bwd(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_qk_norm_rope_bwd launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

}  // extern "C"
