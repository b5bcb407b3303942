// prologue.cuh -- what a training call does before its first product, in one
// kernel (prologue.cu): the rescaled activations, a gradient's rows or scales,
// and the weight rows that TMA cannot read in place.
#pragma once

#include <cuda_fp16.h>

#include "gemm_common.cuh"

namespace nvfp4 {

// Parts whose count of rows is 0 are left out.
struct Prologue {
  // x bf16 [M, K] -> fp16 [m_rows, K] times an exact power of two per token
  // (rows M .. m_rows - 1 zeros), tok_scale[m] = *global over that power; and,
  // where given, the token's line of keys cleared.
  const uint16_t* x;
  int64_t M, K, m_rows;
  __half* x16;
  float* tok_scale;
  unsigned long long* keys;
  // dy [n_dy, N] -> fp16 [n_dy, dy_stride] the same way, factor[m] = *global
  // over the power.
  const void* dy;
  int64_t n_dy, N, dy_stride;
  __half* d16;
  // dh [n_dh, I] and x: the power of two of a gated block's gradients (glu.cu).
  const void* dh;
  int64_t n_dh, I;
  float* up2;
  float* factor;  // (dy's or dh's)
  int grad_bf16;  // dy's or dh's type
  // weight rows
  const uint8_t *packed, *scales;
  int64_t w_rows;
  uint8_t *packed_to, *scales_to;  // null: read in place
  int64_t packed_bytes, packed_stride, scales_bytes, scales_stride;  // of a row
  const float* global;
  int32_t* status;  // null: keep it
  uint32_t* flags;
  int n_flags;
};

// Launched as a programmatic dependent; lets the next kernel start at once.  A
// kernel that follows it directly must wait for it (griddepcontrol.wait)
// before it reads staged weight rows, too.
cudaError_t prologue_launch(const Prologue& p, cudaStream_t stream);

// The staging of a call's weight [rows, K] (WeightStage), for its first chunk.
static inline void prologue_weights(Prologue& p, const WeightStage& w, const uint8_t* packed,
                                    const uint8_t* scales, int64_t rows, int64_t K, uint8_t* ws) {
  p.packed = packed;
  p.scales = scales;
  p.w_rows = rows;
  p.packed_to = w.packed ? ws + w.packed_off : nullptr;
  p.scales_to = w.scales ? ws + w.scales_off : nullptr;
  p.packed_bytes = K / 2;
  p.packed_stride = (int64_t)w.packed_stride;
  p.scales_bytes = K / 16;
  p.scales_stride = (int64_t)w.scales_stride;
}

}  // namespace nvfp4
