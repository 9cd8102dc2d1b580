// fa_kv_api.cu -- the extern "C" boundary of the paged 8-bit KV cache operators
// (declared in include/fa.h): argument validation and launch.
#include <cmath>

#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_kv.h"

namespace {

using fa::api_fail;

#define FA_TRY(expr)                 \
  do {                               \
    fa_status _s = (expr);           \
    if (_s != FA_OK) return _s;      \
  } while (0)

fa_status need_ptr(const void* p, const char* name, unsigned align) {
  if (!p) return api_fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return api_fail(FA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align);
  return FA_OK;
}

fa_status check_page_size(int ps) {
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128)
    return api_fail(FA_ERR_UNSUPPORTED, "page_size %d (want 16, 32, 64 or 128)", ps);
  return FA_OK;
}

fa_status check_shape(const fa::KvShape& s) {
  if (s.num_pages < 1 || s.Hkv < 1)
    return api_fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 (num_pages=%d Hkv=%d)", s.num_pages,
                    s.Hkv);
  FA_TRY(check_page_size(s.page_size));
  if (s.d != 64 && s.d != 128)
    return api_fail(FA_ERR_UNSUPPORTED, "head dimension %d (want 64 or 128)", s.d);
  if (s.Hkv > 65535) return api_fail(FA_ERR_INVALID_ARG, "Hkv (%d) > 65535", s.Hkv);
  return FA_OK;
}

// Most query rows of a call: row tiles are rounded up in 32 bits.
constexpr long long kMaxRows = 0x7fffffffLL - 64;

// Query rows of one KV head: heads of the group x Sq, and the limits of the grids.
fa_status check_rows(int B, int Hq, int Hkv, int Sq, int max_blocks, int page_size, int* rows) {
  if (B < 1 || Hq < 1 || Sq < 1 || max_blocks < 1)
    return api_fail(FA_ERR_INVALID_ARG, "sizes must be >= 1 (B=%d Hq=%d Sq=%d max_blocks=%d)", B,
                    Hq, Sq, max_blocks);
  if (Hq % Hkv != 0) return api_fail(FA_ERR_INVALID_ARG, "Hq (%d) %% Hkv (%d) != 0", Hq, Hkv);
  if (1LL * max_blocks * page_size > 0x7fffffffLL)
    return api_fail(FA_ERR_INVALID_ARG, "max_blocks x page_size exceeds 2^31 - 1 positions");
  if (1LL * B * Hkv > 65535)
    return api_fail(FA_ERR_INVALID_ARG, "B x Hkv (%lld) > 65535", 1LL * B * Hkv);
  const long long r = 1LL * (Hq / Hkv) * Sq;
  if (r * B * Hkv > kMaxRows)
    return api_fail(FA_ERR_INVALID_ARG, "tensor too large for 32-bit row indices");
  *rows = static_cast<int>(r);
  return FA_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

fa_status fa_kv_assign(const int32_t* seqlens, const int32_t* newlens, int B, int page_size,
                       int32_t* block_table, int max_blocks, const int32_t* free_pages, int n_free,
                       int64_t* slot_map, int total_new, int32_t* cu_new, int32_t* seqlens_out,
                       int32_t* cu_seqlens_k, int32_t* n_used, cudaStream_t stream) {
  if (B < 1 || max_blocks < 1 || n_free < 0 || total_new < 0 || total_new > 1 << 30)
    return api_fail(FA_ERR_INVALID_ARG,
                    "fa_kv_assign: B=%d max_blocks=%d must be >= 1, n_free=%d >= 0, total_new=%d in "
                    "[0, 2^30]", B, max_blocks, n_free, total_new);
  FA_TRY(check_page_size(page_size));
  if (1LL * max_blocks * page_size > 0x7fffffffLL)
    return api_fail(FA_ERR_INVALID_ARG, "max_blocks x page_size exceeds 2^31 - 1 positions");
  FA_TRY(need_ptr(seqlens, "seqlens", 4));
  FA_TRY(need_ptr(newlens, "newlens", 4));
  FA_TRY(need_ptr(block_table, "block_table", 4));
  if (n_free > 0) FA_TRY(need_ptr(free_pages, "free_pages", 4));
  if (total_new > 0) FA_TRY(need_ptr(slot_map, "slot_map", 8));
  FA_TRY(need_ptr(cu_new, "cu_new", 4));
  FA_TRY(need_ptr(seqlens_out, "seqlens_out", 4));
  FA_TRY(need_ptr(cu_seqlens_k, "cu_seqlens_k", 4));
  FA_TRY(need_ptr(n_used, "n_used", 4));
  // every CTA reads the lengths and the free list while another writes the results
  const size_t nb = 4 * static_cast<size_t>(B);
  const struct { const void* p; size_t n; const char* name; } in[3] = {
      {seqlens, nb, "seqlens"}, {newlens, nb, "newlens"}, {free_pages, 4 * static_cast<size_t>(n_free),
                                                           "free_pages"}};
  const struct { const void* p; size_t n; const char* name; } out[6] = {
      {block_table, nb * max_blocks, "block_table"}, {slot_map, 8 * static_cast<size_t>(total_new),
                                                      "slot_map"},
      {cu_new, nb + 4, "cu_new"}, {seqlens_out, nb, "seqlens_out"}, {cu_seqlens_k, nb + 4,
                                                                     "cu_seqlens_k"},
      {n_used, 4, "n_used"}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(i.p, i.n, o.p, o.n))
        return api_fail(FA_ERR_INVALID_ARG, "fa_kv_assign: %s overlaps %s", o.name, i.name);
  FA_TRY(fa::api_check_device());
  fa::KvAssignParams p{};
  p.seqlens = seqlens;
  p.newlens = newlens;
  p.block_table = block_table;
  p.free_pages = free_pages;
  p.slot_map = slot_map;
  p.cu_new = cu_new;
  p.seqlens_out = seqlens_out;
  p.cu_k = cu_seqlens_k;
  p.n_used = n_used;
  p.B = B;
  p.page_size = page_size;
  p.max_blocks = max_blocks;
  p.n_free = n_free;
  p.total_new = total_new;
  const cudaError_t e = fa::launch_kv_assign(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_kv_assign launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

fa_status fa_kv_write_fp8(const void* k, const void* v, long long k_stride_h, long long k_stride_t,
                          long long v_stride_h, long long v_stride_t, const int64_t* slot_map,
                          int n_tokens, void* k_cache, void* v_cache, float* k_scale,
                          float* v_scale, int8_t* k_bounds, int num_pages, int Hkv, int page_size,
                          int d, cudaStream_t stream) {
  fa::KvWriteParams p{};
  p.s = {num_pages, Hkv, page_size, d};
  FA_TRY(check_shape(p.s));
  if (n_tokens < 0 || n_tokens > 1 << 30)
    return api_fail(FA_ERR_INVALID_ARG, "n_tokens (%d) must lie in [0, 2^30]", n_tokens);
  FA_TRY(need_ptr(k_cache, "k_cache", 16));
  FA_TRY(need_ptr(v_cache, "v_cache", 16));
  FA_TRY(need_ptr(k_scale, "k_scale", 4));
  FA_TRY(need_ptr(v_scale, "v_scale", 4));
  if (k_bounds) FA_TRY(need_ptr(k_bounds, "k_bounds", 16));
  if (n_tokens == 0) return fa::api_ok();
  if (2LL * Hkv * ((n_tokens + 15) / 16) >= 1LL << 31)
    return api_fail(FA_ERR_INVALID_ARG, "n_tokens (%d) x Hkv (%d) is too large for one call",
                    n_tokens, Hkv);
  FA_TRY(need_ptr(k, "k", 16));
  FA_TRY(need_ptr(v, "v", 16));
  FA_TRY(need_ptr(slot_map, "slot_map", 8));
  for (long long st : {k_stride_h, k_stride_t, v_stride_h, v_stride_t})
    if (st < 0 || st % 8 != 0)
      return api_fail(FA_ERR_INVALID_ARG,
                      "strides of k and v (%lld) must be >= 0 and multiples of 8 elements", st);
  FA_TRY(fa::api_check_device());
  p.k = k;
  p.v = v;
  p.k_stride_h = k_stride_h;
  p.k_stride_t = k_stride_t;
  p.v_stride_h = v_stride_h;
  p.v_stride_t = v_stride_t;
  p.slot_map = slot_map;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_bounds = k_bounds;
  p.n_tokens = n_tokens;
  const cudaError_t e = fa::launch_kv_write(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_kv_write_fp8 launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

fa_status fa_kv_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, const int32_t* block_table,
                         const int32_t* cu_seqlens_k, void* k, void* v, int nseq, int max_blocks,
                         int num_pages, int total_k, int Hkv, int page_size, int d,
                         cudaStream_t stream) {
  fa::KvReadParams p{};
  p.s = {num_pages, Hkv, page_size, d};
  FA_TRY(check_shape(p.s));
  if (nseq < 1 || max_blocks < 1 || total_k < 0 || total_k > 1 << 30)
    return api_fail(FA_ERR_INVALID_ARG,
                    "nseq=%d max_blocks=%d must be >= 1, total_k=%d in [0, 2^30]", nseq, max_blocks,
                    total_k);
  FA_TRY(need_ptr(k_cache, "k_cache", 16));
  FA_TRY(need_ptr(v_cache, "v_cache", 16));
  FA_TRY(need_ptr(k_scale, "k_scale", 4));
  FA_TRY(need_ptr(v_scale, "v_scale", 4));
  FA_TRY(need_ptr(block_table, "block_table", 4));
  FA_TRY(need_ptr(cu_seqlens_k, "cu_seqlens_k", 4));
  if (total_k == 0) return fa::api_ok();
  FA_TRY(need_ptr(k, "k", 16));
  FA_TRY(need_ptr(v, "v", 16));
  FA_TRY(fa::api_check_device());
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.cu_k = cu_seqlens_k;
  p.k = k;
  p.v = v;
  p.nseq = nseq;
  p.max_blocks = max_blocks;
  p.total_k = total_k;
  const cudaError_t e = fa::launch_kv_read(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_kv_read_fp8 launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

size_t fa_select_blocks_workspace_size(int B, int Hkv, int max_blocks) {
  if (B < 1 || Hkv < 1 || max_blocks < 1) return 0;
  return static_cast<size_t>(B) * Hkv * max_blocks * sizeof(uint32_t);
}

fa_status fa_select_blocks(const void* q, const int8_t* k_bounds, const float* k_scale,
                           const int32_t* block_table, const int32_t* seqlens_k, int32_t* sel,
                           int32_t* n_sel, int B, int Hq, int Hkv, int Sq, int num_pages,
                           int max_blocks, int page_size, int d, int k_blocks, int n_first,
                           int n_last, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  fa::SelectParams p{};
  p.s = {num_pages, Hkv, page_size, d};
  FA_TRY(check_shape(p.s));
  FA_TRY(check_rows(B, Hq, Hkv, Sq, max_blocks, page_size, &p.rows));
  if (k_blocks < 1 || n_first < 0 || n_last < 0 || 1LL * n_first + n_last > k_blocks)
    return api_fail(FA_ERR_INVALID_ARG,
                    "k_blocks=%d must be >= 1 and >= n_first=%d + n_last=%d (both >= 0)", k_blocks,
                    n_first, n_last);
  FA_TRY(need_ptr(q, "q", 16));
  FA_TRY(need_ptr(k_bounds, "k_bounds", 16));
  FA_TRY(need_ptr(k_scale, "k_scale", 4));
  FA_TRY(need_ptr(block_table, "block_table", 4));
  FA_TRY(need_ptr(seqlens_k, "seqlens_k", 4));
  FA_TRY(need_ptr(sel, "sel", 4));
  FA_TRY(need_ptr(n_sel, "n_sel", 4));
  const size_t need = fa_select_blocks_workspace_size(B, Hkv, max_blocks);
  if (!workspace || workspace_bytes < need)
    return api_fail(FA_ERR_WORKSPACE, "block selection workspace needs %zu bytes, got %zu", need,
                    workspace ? workspace_bytes : size_t(0));
  FA_TRY(need_ptr(workspace, "workspace", 16));
  FA_TRY(fa::api_check_device());
  p.q = q;
  p.k_bounds = k_bounds;
  p.k_scale = k_scale;
  p.block_table = block_table;
  p.seqlens = seqlens_k;
  p.sel = sel;
  p.n_sel = n_sel;
  p.keys = static_cast<uint32_t*>(workspace);
  p.B = B;
  p.Hq = Hq;
  p.Sq = Sq;
  p.max_blocks = max_blocks;
  p.k_blocks = k_blocks;
  p.n_first = n_first;
  p.n_last = n_last;
  const cudaError_t e = fa::launch_select(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_select_blocks launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

size_t fa_decode_paged_fp8_workspace_size(int B, int Hq, int Hkv, int Sq, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || d < 1 || Hq % Hkv != 0) return 0;
  const long long rows = 1LL * (Hq / Hkv) * Sq;
  if (rows > kMaxRows) return 0;  // the call refuses it
  return fa::decode_paged_workspace(B, Hkv, static_cast<int>(rows), d);
}

fa_status fa_decode_paged_fp8(const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale,
                              const int32_t* block_table, const int32_t* seqlens_k,
                              const int32_t* sel, const int32_t* n_sel, void* o, float* lse, int B,
                              int Hq, int Hkv, int Sq, int num_pages, int max_blocks, int max_sel,
                              int page_size, int d, float scale, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  fa::PagedDecodeParams p{};
  p.s = {num_pages, Hkv, page_size, d};
  FA_TRY(check_shape(p.s));
  FA_TRY(check_rows(B, Hq, Hkv, Sq, max_blocks, page_size, &p.rows));
  FA_TRY(need_ptr(q, "q", 16));
  FA_TRY(need_ptr(k_cache, "k_cache", 16));
  FA_TRY(need_ptr(v_cache, "v_cache", 16));
  FA_TRY(need_ptr(k_scale, "k_scale", 4));
  FA_TRY(need_ptr(v_scale, "v_scale", 4));
  FA_TRY(need_ptr(block_table, "block_table", 4));
  FA_TRY(need_ptr(seqlens_k, "seqlens_k", 4));
  FA_TRY(need_ptr(o, "o", 16));
  if (lse) FA_TRY(need_ptr(lse, "lse", 16));
  if ((sel == nullptr) != (n_sel == nullptr))
    return api_fail(FA_ERR_INVALID_ARG, "sel and n_sel are given together or not at all");
  if (sel) {
    FA_TRY(need_ptr(sel, "sel", 4));
    FA_TRY(need_ptr(n_sel, "n_sel", 4));
    if (max_sel < 1) return api_fail(FA_ERR_INVALID_ARG, "max_sel (%d) must be >= 1", max_sel);
    if (1LL * max_sel * page_size > 0x7fffffffLL)
      return api_fail(FA_ERR_INVALID_ARG, "max_sel x page_size exceeds 2^31 - 1 positions");
  }
  if (!std::isfinite(scale) || scale < 0.f)
    return api_fail(FA_ERR_INVALID_ARG, "scale (%g) must be finite and >= 0", (double)scale);
  const size_t need = fa::decode_paged_workspace(B, Hkv, p.rows, d);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return api_fail(FA_ERR_WORKSPACE, "paged decode workspace needs %zu bytes, got %zu", need,
                      workspace ? workspace_bytes : size_t(0));
    FA_TRY(need_ptr(workspace, "workspace", 16));
  }
  FA_TRY(fa::api_check_device());
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seqlens = seqlens_k;
  p.sel = sel;
  p.n_sel = n_sel;
  p.o = o;
  p.lse = lse;
  p.workspace = workspace;
  p.B = B;
  p.Hq = Hq;
  p.Sq = Sq;
  p.max_blocks = max_blocks;
  p.max_sel = sel ? max_sel : 0;
  p.block_shift = page_size == 16 ? 0 : page_size == 32 ? 1 : page_size == 64 ? 2 : 3;
  p.scale_log2 = fa::api_scale_log2(scale);
  const cudaError_t e = fa::launch_decode_paged(p, stream);
  if (e != cudaSuccess)
    return api_fail(FA_ERR_CUDA, "fa_decode_paged_fp8 launch: %s", cudaGetErrorString(e));
  return fa::api_ok();
}

}  // extern "C"
