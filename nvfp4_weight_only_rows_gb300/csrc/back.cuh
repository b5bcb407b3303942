// back.cuh -- the product back through a packed weight (back.cu) as the
// gradients use it: out[m, k] = factor[m] sum_n d[m, n] W[n, k].
#pragma once

#include <cuda_fp16.h>

#include "gemm_common.cuh"

namespace nvfp4 {

// The product's cut into tiles of 128 columns x BN tokens, or, for a pair of
// CTAs, 256 columns x 2 BN tokens: n_whole of them whole, n_rest in n_splits
// parts along the weight's rows; and its workspace after `off`: the sums of
// those parts.
struct BackLayout {
  size_t part, total;
  int64_t n_whole, n_rest;
  int grid, BN, n_ttiles, n_splits, n_kb;
  bool pair, fine;  // pairs of CTAs; stages of 128 rows
};
BackLayout back_layout(int64_t M, int64_t N, int64_t K, int sms, size_t off);

// The token tile of a call: as many tiles as 128-token ones would be, of equal
// size (203 tokens: two of 112, not 128).
static inline int train_token_tile(int64_t M) {
  const int64_t tiles = std::max<int64_t>(1, (M + kMaxBN - 1) / kMaxBN);
  return lm_head_token_tile((M + tiles - 1) / tiles);
}

struct BackCall {
  int64_t M, N, K;
  const __half* d;      // [M, stride]
  int64_t d_stride;     // elements, a multiple of 8, >= N
  const uint8_t *packed, *scales;  // as in the call; `stage` says where TMA reads them
  const WeightStage* stage;
  const float* factor;  // [M]
  void* out;            // [M, K]
  int out_dtype;
  bool fresh;           // the kernel before may have staged the weight
};
// Two kernels at most, programmatic dependents of the kernel before.
cudaError_t back_launch(const BackCall& c, const BackLayout& L, uint8_t* ws, cudaStream_t stream);

// Tokens of a call that are worked on at a time, so that a fp16 row of
// `row_bytes` for each fits `kChunkBytes`: whole tiles of 128.
constexpr int64_t kChunkBytes = (int64_t)512 << 20;
static inline int64_t chunk_tokens(int64_t M, int64_t row_bytes) {
  const int64_t fit = kChunkBytes / row_bytes / kMaxBN * kMaxBN;
  return M < kMaxBN ? M : std::min(M, std::max<int64_t>(fit, kMaxBN));
}

}  // namespace nvfp4
