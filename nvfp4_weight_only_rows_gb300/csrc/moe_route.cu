// moe_route.cu -- the router's choice of a mixture-of-experts layer: per
// token the k experts with the largest scores and their weights.
//
// One warp per token, kR consecutive experts per lane.  Softmax and sigmoid
// both rise with the logit, so without a bias the choice is made on the
// logits themselves, exactly, and scores are computed for what was chosen.
// A candidate is one word: the upper bits of its 32-bit order key above the
// complement of its expert, so that one integer maximum over the warp picks
// the largest key and, of equal ones, the lowest expert.  Each lane sorts its
// words once and leaves them in shared memory; a round then is that maximum
// and a step of the lane that held it (shifting them in registers: 16384 x 256
// fp32 10.3 against 8.2 us).  bf16 logits fit their words whole.  For fp32
// keys k + 1 rounds show whether two neighbours of the order share all the
// bits kept (values within 2^-14 of each other): only then the token is done
// again by whole keys, two reductions a round.  All sums are fp32.
//
// A call reads M E logits once and writes 8 M k bytes: 16384 x 256 fp32 is 18
// MB, 2.7 us at the copy rate, and takes 8.2 us; 65536 x 256 28.7 us, 262144 x
// 256 106 us.  bf16 logits take 2% less, a bias 12.5 us (sigmoid, 16384 x 256;
// 384 experts 29.7 us: 16 words a lane).  One token 2.0 us.  Bound by
// instruction issue: 415 warp instructions a token, 240 ns of an SM quarter in
// the long runs, which is 6.5 of the 8.2 us; the rest is the launch and the
// first loads.  Four tokens a warp with their rounds side by side took 8.2 us
// too; CTAs of 8 or 16 tokens 8.4; a grid of resident CTAs that loop 10.7 or
// more.
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

struct RouteArgs {
  const void* logits;
  int64_t M;
  int E, k, scoring, renorm;
  const float* bias;
  float scale;
  int32_t* ids;
  float* weights;
  bool vec;  // rows are whole aligned 16-byte vectors
};

constexpr float kNegInf = -__builtin_huge_valf();

// The row's logits e0 .. e0 + kR - 1, -inf past its end.
template <int kR, typename T>
__device__ __forceinline__ void route_load(const T* row, int e0, int E, bool vec, float (&x)[kR]) {
  constexpr int kVec = 16 / sizeof(T);
  if constexpr (kR % kVec == 0) {
    if (vec) {
#pragma unroll
      for (int r = 0; r < kR; r += kVec) {
        uint4 v;
        const bool in = e0 + r < E;
        if (in) v = __ldg(reinterpret_cast<const uint4*>(row + e0 + r));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4) {
            x[r + i] = in ? __uint_as_float(w[i]) : kNegInf;
          } else {
            x[r + 2 * i] = in ? __uint_as_float(w[i] << 16) : kNegInf;
            x[r + 2 * i + 1] = in ? __uint_as_float(w[i] & 0xFFFF0000u) : kNegInf;
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r) x[r] = e0 + r < E ? route_logit(row + e0 + r) : kNegInf;
}

// A token's maximum and sum where scores themselves are needed: a bias is
// added to them, or they are returned as they are.
struct RouteSoftmax {
  float top, total;
};

template <int kR>
__device__ __forceinline__ RouteSoftmax route_softmax(const float (&x)[kR], int e0, int E) {
  float top = x[0], total = 0.0f;
#pragma unroll
  for (int r = 1; r < kR; ++r) top = fmaxf(top, x[r]);
  // (a NaN is not in this maximum; it reaches every score through the sum,
  // or through its own)
  top = key_value(__reduce_max_sync(0xFFFFFFFFu, route_key(top)));
#pragma unroll
  for (int r = 0; r < kR; ++r)
    if (e0 + r < E) total += expf(x[r] - top);
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  return {top, total};
}

__device__ __forceinline__ float route_score(float v, bool softmax, RouteSoftmax s) {
  // a token whose logits are all -inf has no expert: every score is zero
  if (softmax) return s.top == kNegInf && v == v ? 0.0f : expf(v - s.top) / s.total;
  return 1.0f / (1.0f + expf(-v));
}

// Selection keys, kTaken past the row's end.
template <int kR>
__device__ __forceinline__ void route_keys(const float (&x)[kR], int e0, const RouteArgs& p,
                                           RouteSoftmax s, uint32_t (&key)[kR]) {
  float v[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) v[r] = x[r];
  if (p.bias != nullptr) {
    const bool softmax = p.scoring == NVFP4_ROUTE_SOFTMAX;
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if (e0 + r < p.E) v[r] = route_score(x[r], softmax, s) + __ldg(p.bias + e0 + r);
  }
  if (e0 + kR <= p.E) {
#pragma unroll
    for (int r = 0; r < kR; ++r) key[r] = route_key(v[r]);
  } else {
#pragma unroll
    for (int r = 0; r < kR; ++r) key[r] = e0 + r < p.E ? route_key(v[r]) : kTaken;
  }
}

// kR: logits per lane (E <= 32 kR).  T: float, or uint16_t for bf16 bits.
template <int kR, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const RouteArgs p) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr uint32_t kIdMask = 32 * kR - 1;
  __shared__ uint32_t s_word[kRouteWarps][kR + 2][32];  // a lane's words in order
  __shared__ uint32_t s_best[kRouteWarps][33];  // the words picked, in order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (m >= p.M) return;
  const bool softmax = p.scoring == NVFP4_ROUTE_SOFTMAX;
  const bool sums = softmax && (p.bias != nullptr || !p.renorm);
  const bool whole = sizeof(T) == 2 && p.bias == nullptr;  // the words hold the keys
  const int rounds = p.k + (whole ? 0 : 1);
  const T* row = static_cast<const T*>(p.logits) + m * p.E;
  const int e0 = lane * kR;  // this lane's experts e0 .. e0 + kR - 1

  float x[kR];
  route_load(row, e0, p.E, p.vec, x);
  RouteSoftmax soft = {0.0f, 1.0f};
  if (sums) soft = route_softmax(x, e0, p.E);
  uint32_t key[kR];
  route_keys(x, e0, p, soft, key);
  {
    uint32_t word[kR];
    if (e0 + kR <= p.E) {
#pragma unroll
      for (int r = 0; r < kR; ++r) word[r] = (key[r] | kIdMask) - (uint32_t)(e0 + r);
    } else {
#pragma unroll
      for (int r = 0; r < kR; ++r)
        word[r] = e0 + r < p.E ? (key[r] | kIdMask) - (uint32_t)(e0 + r) : kTaken;
    }
    sort_desc(word);
    // the last round may find every expert taken: one more row to read
#pragma unroll
    for (int r = 1; r < kR; ++r) s_word[warp][r][lane] = word[r];
    s_word[warp][kR][lane] = s_word[warp][kR + 1][lane] = kTaken;
    uint32_t head = word[0];
    const uint32_t* at = &s_word[warp][0][lane];
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
      const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, head);
      if (head == mx) {
        s_best[warp][j] = mx;
        at += 32;
        head = *at;
      }
    }
  }
  __syncwarp();

  const bool on = lane < p.k;
  const uint32_t mine = on ? s_best[warp][lane] : kTaken;
  int id = on ? (int)(~mine & kIdMask) : 0;
  if (__any_sync(0xFFFFFFFFu,
                 !whole && on && ((mine ^ s_best[warp][lane + 1]) & ~kIdMask) == 0u)) {
    uint32_t most = kTaken;
#pragma unroll
    for (int r = 0; r < kR; ++r) most = max(most, key[r]);
    for (int j = 0; j < p.k; ++j) {
      const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, most);
      uint32_t e = 0xFFFFFFFFu;
#pragma unroll
      for (int r = kR - 1; r >= 0; --r)
        if (key[r] == mx) e = e0 + r;
      e = __reduce_min_sync(0xFFFFFFFFu, e);
      most = kTaken;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if ((uint32_t)(e0 + r) == e) key[r] = kTaken;
        most = max(most, key[r]);
      }
      if (lane == j) id = (int)e;
    }
  }
  const float v = on ? route_logit(row + min(id, p.E - 1)) : 0.0f;
  // without sums the choice is by logits, and the first is their maximum
  if (!sums) soft.top = __shfl_sync(0xFFFFFFFFu, v, 0);
  float w = on ? route_score(v, softmax, soft) : 0.0f;
  if (p.renorm) {
    float sum = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    w = sum == 0.0f ? 0.0f : w / sum;
  }
  if (on) {
    p.ids[m * p.k + lane] = id;
    p.weights[m * p.k + lane] = w * p.scale;
  }
}

template <typename T>
static cudaError_t route_dispatch(const RouteArgs& p, cudaStream_t stream) {
  PdlLaunch l(dim3((unsigned)((p.M + kRouteWarps - 1) / kRouteWarps)), dim3(32 * kRouteWarps), 0,
              stream);
  auto kern = p.E <= 64    ? moe_route_kernel<2, T>
              : p.E <= 128 ? moe_route_kernel<4, T>
              : p.E <= 256 ? moe_route_kernel<8, T>
                           : moe_route_kernel<16, T>;
  return cudaLaunchKernelEx(&l.cfg, kern, p);
}

nvfp4_status moe_route_launch(const void* logits, int dtype, int64_t M, int E, int k, int scoring,
                              int renorm, const float* bias, float scale, int32_t* ids,
                              float* weights, cudaStream_t stream) {
  const int per = dtype == NVFP4_OUT_BF16 ? 8 : 4;
  const RouteArgs p{logits, M, E, k, scoring, renorm, bias, scale, ids, weights,
                    E % per == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0};
  const cudaError_t err = dtype == NVFP4_OUT_BF16 ? route_dispatch<uint16_t>(p, stream)
                                                  : route_dispatch<float>(p, stream);
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
