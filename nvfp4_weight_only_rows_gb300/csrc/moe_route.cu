// moe_route.cu -- the router's choice of a mixture-of-experts layer: per
// token the k experts with the largest scores and their weights.
//
// One warp per token, kR consecutive experts per lane.  Softmax and sigmoid
// both rise with the logit, so without a bias the choice is made on the
// logits themselves, exactly, and scores are computed for what was chosen.
// A candidate is one word: the upper bits of its 32-bit order key above the
// complement of its expert, so that one integer maximum over the warp picks
// the largest key and, of equal ones, the lowest expert.  Each lane sorts its
// words once; a round then is that maximum and a shift in the lane that held
// it.  bf16 logits fit their words whole.  For fp32 keys k + 1 rounds show
// whether two neighbours of the order share all the bits kept (values within
// 2^-14 of each other): only then the token is done again by whole keys, two
// reductions a round.  All sums are fp32.
//
// A call reads M E logits once and writes 8 M k bytes: a prompt of 16384
// tokens and 256 experts is 18 MB (2.7 us at the copy rate), and bound by
// instruction issue (about 250 a token).
#include "gemm_common.cuh"

namespace nvfp4 {

constexpr int kRouteWarps = 4;    // tokens of one CTA
constexpr uint32_t kTaken = 0u;   // below every order key

// Order key of a score or logit: value order, -0 with +0, any NaN on top (the
// sum turns -0 into +0 and every NaN into the positive 0x7FFFFFFF).
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Batcher's odd-even merge sort of kN words, largest first.
template <int kN>
__device__ __forceinline__ void sort_desc(uint32_t (&a)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j <= kN - 1 - q; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = a[i + j], y = a[i + j + q];
            a[i + j] = max(x, y);
            a[i + j + q] = min(x, y);
          }
        }
      }
    }
  }
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
  constexpr uint32_t kIdMask = 32 * kR - 1;
  constexpr float kNegInf = -__builtin_huge_valf();
  const int lane = threadIdx.x & 31;
  const int64_t m = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (m >= M) return;
  const bool softmax = scoring == NVFP4_ROUTE_SOFTMAX;
  const T* row = logits + m * E;
  const int e0 = lane * kR;  // this lane's experts e0 .. e0 + kR - 1
  float x[kR];
  constexpr int kVec = 16 / sizeof(T);
  bool vec = false;
  if constexpr (kR % kVec == 0)
    vec = E % kVec == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  if constexpr (kR % kVec == 0) {
    if (vec) {  // whole vectors inside the row
#pragma unroll
      for (int r = 0; r < kR; r += kVec) {
        if (e0 + r < E) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0 + r));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
              x[r + i] = __uint_as_float(w[i]);
            } else {
              x[r + 2 * i] = __uint_as_float(w[i] << 16);
              x[r + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) x[r + i] = kNegInf;
        }
      }
    }
  }
  if (!vec) {
#pragma unroll
    for (int r = 0; r < kR; ++r) x[r] = e0 + r < E ? route_logit(row + e0 + r) : kNegInf;
  }
  // the softmax's maximum and sum: needed where a score itself is (a bias
  // is added to it, or it is returned as it is)
  float top = 0.0f, total = 1.0f;
  if (softmax) {
    top = x[0];
#pragma unroll
    for (int r = 1; r < kR; ++r) top = fmaxf(top, x[r]);
    // (a NaN is not in this maximum; it reaches every score through the sum,
    // or through its own)
    const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, route_key(top));
    top = key_value(t);
    if (bias != nullptr || !renorm) {
      total = 0.0f;
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (e0 + r < E) total += expf(x[r] - top);
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
  }
  auto score = [&](float v) {
    // a token whose logits are all -inf has no expert: every score is zero
    if (softmax) return top == kNegInf && v == v ? 0.0f : expf(v - top) / total;
    return 1.0f / (1.0f + expf(-v));
  };
  uint32_t key[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r)
    key[r] = e0 + r >= E ? kTaken
                         : route_key(bias != nullptr ? score(x[r]) + __ldg(bias + e0 + r) : x[r]);

  int my_id = 0;
  bool near = false;
  {
    uint32_t word[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r)
      word[r] = key[r] == kTaken ? kTaken : (key[r] & ~kIdMask) | (~(uint32_t)(e0 + r) & kIdMask);
    sort_desc(word);
    const bool whole = sizeof(T) == 2 && bias == nullptr;  // the words hold the keys
    uint32_t mine = kTaken;  // lane j: the word of round j
    const int rounds = k + (whole ? 0 : 1);
#pragma unroll 2
    for (int j = 0; j < rounds; ++j) {
      const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, word[0]);
      const bool pop = word[0] == mx;
#pragma unroll
      for (int r = 0; r + 1 < kR; ++r) word[r] = pop ? word[r + 1] : word[r];
      word[kR - 1] = pop ? kTaken : word[kR - 1];
      mine = lane == j ? mx : mine;
    }
    my_id = (int)(~mine & kIdMask);
    if (!whole) {
      // round 32 (k of 32) is in no lane: such tokens go by whole keys
      const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
      near = rounds > 32 || __any_sync(0xFFFFFFFFu, lane > 0 && lane < rounds &&
                                                        ((mine ^ before) & ~kIdMask) == 0u);
    }
  }
  if (near) {  // warp-uniform
    uint32_t best = kTaken;
#pragma unroll
    for (int r = 0; r < kR; ++r) best = max(best, key[r]);
    for (int j = 0; j < k; ++j) {
      const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, best);
      uint32_t e = 0xFFFFFFFFu;
#pragma unroll
      for (int r = kR - 1; r >= 0; --r)
        if (key[r] == mx) e = e0 + r;
      e = __reduce_min_sync(0xFFFFFFFFu, e);
      best = kTaken;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if ((uint32_t)(e0 + r) == e) key[r] = kTaken;
        best = max(best, key[r]);
      }
      if (lane == j) my_id = (int)e;
    }
  }
  float w = lane < k ? score(route_logit(row + min(my_id, E - 1))) : 0.0f;
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
