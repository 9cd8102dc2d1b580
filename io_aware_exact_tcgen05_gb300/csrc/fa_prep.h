// fa_prep.h -- parameter blocks of the pass between a projection and the scores (fa_prep.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace fa {

// Queries, keys or values of a pass, as one role of the kernels sees them: strided rows
// [B][S][heads][d] on the projection's side, head-major rows on the attention's.
struct PrepRole {
  const void* x;        // projection (forward input; backward: input of the norm, may be nullptr)
  long long xb, xt, xh; // strides in elements (channels are contiguous)
  void* dx;             // backward: gradient of the projection
  long long db, dt, dh;
  void* y;              // head-major [B][heads][y_rows][d]: forward output, backward input
  const void* w;        // bf16 [d] or nullptr: no norm
  float* dw;            // backward: fp32 [d] or nullptr
  int y_rows;           // rows of a head in y
  int heads;
};

struct PrepParams {
  PrepRole role[3];           // queries, keys, values
  const int32_t* positions;   // [n_axes][B][S] or nullptr: the row
  const float* inv_freq;      // [rot / 2]
  const uint8_t* freq_axis;   // [rot / 2] or nullptr: axis 0
  const int32_t* row_start;   // [B] or nullptr: first row of keys and values
  float* partial;             // backward: [blocks][queries, keys][d]
  float w_off, eps;
  int n_axes, rot, interleaved;
  int B, S, d;
  int blocks;
};

// Sets the CTAs for a device of n_sm SMs.
void prep_plan(PrepParams* p, int n_sm, bool back);
// Most rows of `partial` that a backward pass uses.
int prep_partial_rows();
cudaError_t launch_prep(const PrepParams& p, cudaStream_t stream);
cudaError_t launch_prep_bwd(const PrepParams& p, cudaStream_t stream);

}  // namespace fa
