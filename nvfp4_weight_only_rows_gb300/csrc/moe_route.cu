// moe_route.cu -- the router's choice of a mixture-of-experts layer: per
// token the k experts with the largest scores and their weights.
//
// One warp per token.  The E router logits sit in registers (expert 32 r +
// lane in register r of the lane) as 32-bit order keys; k rounds each take
// the largest key of the warp (one integer reduction) and, of the experts
// that hold it, the lowest (a second one).  Softmax and sigmoid both rise
// with the logit, so without a bias the choice is made on the logits
// themselves, exactly, and scores are computed for what was chosen.  All sums
// are fp32.
//
// A call reads M E logits once and writes 8 M k bytes; a prompt of 16384
// tokens and 256 experts is 18 MB (2.7 us at the copy rate), a decode batch
// is one launch.
#include "gemm_common.cuh"

namespace nvfp4 {

constexpr int kRouteWarps = 4;    // tokens of one CTA
constexpr uint32_t kTaken = 0u;   // below every order key

// Order key of a score or logit: value order, -0 with +0, any NaN on top.
__device__ __forceinline__ uint32_t route_key(float v) {
  return v != v ? 0xFFFFFFFFu : logit_order(v);
}

__device__ __forceinline__ float route_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float route_logit(const uint16_t* p) {
  return __uint_as_float((uint32_t)__ldg(p) << 16);
}

// kR: logits per lane (E <= 32 kR).  T: float, or uint16_t for bf16 bits.
template <int kR, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(
    const T* __restrict__ logits, int64_t M, int E, int k, int scoring, int renorm,
    const float* __restrict__ bias, float scale, int32_t* __restrict__ ids,
    float* __restrict__ weights) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t m = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (m >= M) return;
  const bool softmax = scoring == NVFP4_ROUTE_SOFTMAX;
  const T* row = logits + m * E;
  float x[kR];
  uint32_t key[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int e = 32 * r + lane;
    x[r] = e < E ? route_logit(row + e) : __int_as_float(0xFF800000);
  }
  // the softmax's maximum and sum: needed where a score itself is (a bias
  // is added to it, or it is returned as it is)
  float top = 0.0f, total = 1.0f;
  if (softmax) {
    top = x[0];
#pragma unroll
    for (int r = 1; r < kR; ++r) top = fmaxf(top, x[r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (bias != nullptr || !renorm) {
      total = 0.0f;
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (32 * r + lane < E) total += expf(x[r] - top);
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
  }
  auto score = [&](float v) {
    // a token whose logits are all -inf has no expert: every score is zero
    if (softmax)
      return top == __int_as_float(0xFF800000) && v == v ? 0.0f : expf(v - top) / total;
    return 1.0f / (1.0f + expf(-v));
  };
  uint32_t best = kTaken;
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int e = 32 * r + lane;
    key[r] = e < E ? route_key(bias != nullptr ? score(x[r]) + __ldg(bias + e) : x[r]) : kTaken;
    best = max(best, key[r]);
  }
  int my_id = 0;
  float my_x = 0.0f;
  for (int j = 0; j < k; ++j) {
    const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int r = kR - 1; r >= 0; --r)
      if (key[r] == mx) e = 32 * r + lane;
    e = __reduce_min_sync(0xFFFFFFFFu, e);
    float v = 0.0f;
    best = kTaken;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if ((e >> 5) == (uint32_t)r) {  // warp-uniform
        v = x[r];
        if ((e & 31) == (uint32_t)lane) key[r] = kTaken;
      }
      best = max(best, key[r]);
    }
    v = __shfl_sync(0xFFFFFFFFu, v, e & 31);
    if (lane == j) {
      my_id = (int)e;
      my_x = v;
    }
  }
  float w = lane < k ? score(my_x) : 0.0f;
  if (renorm) {
    float sum = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    w = sum == 0.0f ? 0.0f : w / sum;
  }
  if (lane < k) {
    ids[m * k + lane] = my_id;
    weights[m * k + lane] = w * scale;
  }
}

template <typename T>
static cudaError_t route_dispatch(const T* logits, int64_t M, int E, int k, int scoring,
                                  int renorm, const float* bias, float scale, int32_t* ids,
                                  float* weights, cudaStream_t stream) {
  PdlLaunch l(dim3((unsigned)((M + kRouteWarps - 1) / kRouteWarps)), dim3(32 * kRouteWarps), 0,
              stream);
  auto kern = E <= 64    ? moe_route_kernel<2, T>
              : E <= 128 ? moe_route_kernel<4, T>
              : E <= 256 ? moe_route_kernel<8, T>
                         : moe_route_kernel<16, T>;
  return cudaLaunchKernelEx(&l.cfg, kern, logits, M, E, k, scoring, renorm, bias, scale, ids,
                            weights);
}

nvfp4_status moe_route_launch(const void* logits, int dtype, int64_t M, int E, int k, int scoring,
                              int renorm, const float* bias, float scale, int32_t* ids,
                              float* weights, cudaStream_t stream) {
  const cudaError_t err =
      dtype == NVFP4_OUT_BF16
          ? route_dispatch(static_cast<const uint16_t*>(logits), M, E, k, scoring, renorm, bias,
                           scale, ids, weights, stream)
          : route_dispatch(static_cast<const float*>(logits), M, E, k, scoring, renorm, bias,
                           scale, ids, weights, stream);
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
