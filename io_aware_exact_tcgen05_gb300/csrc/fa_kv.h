// fa_kv.h -- parameter blocks and launch entry points of the paged 8-bit KV
// cache operators (fa_kv_api.cu and the kernel translation units).  Host-side
// declarations and plain structs only.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "../../include/fa.h"

namespace fa {

// Status helpers of fa_api.cu for other translation units: record the detail
// text and return the status; check that the current device is an sm_103a one.
fa_status api_fail(fa_status s, const char* fmt, ...);
fa_status api_ok();
fa_status api_check_device();
float api_scale_log2(float scale);

// Sizes every operator on the cache shares.  A cache tensor holds e4m3 codes
// [num_pages, Hkv, page_size, d]; its scales are fp32 [num_pages, Hkv].
struct KvShape {
  int num_pages, Hkv, page_size, d;
};

struct KvAssignParams {
  const int32_t* seqlens;
  const int32_t* newlens;
  int32_t* block_table;
  const int32_t* free_pages;
  int64_t* slot_map;
  int32_t* cu_new;
  int32_t* seqlens_out;
  int32_t* cu_k;
  int32_t* n_used;
  int B, page_size, max_blocks, n_free, total_new;
};
cudaError_t launch_kv_assign(const KvAssignParams& p, cudaStream_t stream);

struct KvWriteParams {
  const void* k;  // bf16, element (h, t, c) at h * stride_h + t * stride_t + c
  const void* v;
  long long k_stride_h, k_stride_t, v_stride_h, v_stride_t;
  const int64_t* slot_map;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  int8_t* k_bounds;  // [num_pages, Hkv, 2, d] or nullptr
  int n_tokens;
  KvShape s;
};
cudaError_t launch_kv_write(const KvWriteParams& p, cudaStream_t stream);

struct KvReadParams {
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* cu_k;
  void* k;  // bf16 [Hkv, total_k, d]
  void* v;
  int nseq, max_blocks, total_k;
  KvShape s;
};
cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream);

struct SelectParams {
  const void* q;  // bf16 [B, Hq, Sq, d]
  const int8_t* k_bounds;
  const float* k_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  int32_t* sel;
  int32_t* n_sel;
  uint32_t* keys;  // workspace [B, Hkv, max_blocks]
  int B, Hq, Sq, rows, max_blocks, k_blocks, n_first, n_last;
  KvShape s;
};
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream);

struct PagedDecodeParams {
  const void* q;  // bf16 [B, Hq, Sq, d]
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* sel;    // [B, Hkv, max_sel] or nullptr: every block
  const int32_t* n_sel;  // [B, Hkv]
  void* o;
  float* lse;
  void* workspace;
  int B, Hq, Sq, rows, max_blocks, max_sel;
  int block_shift;       // log2(page_size / 16)
  float scale_log2;
  KvShape s;
};
cudaError_t launch_decode_paged(const PagedDecodeParams& p, cudaStream_t stream);
size_t decode_paged_workspace(int B, int Hkv, int rows, int d);

}  // namespace fa
