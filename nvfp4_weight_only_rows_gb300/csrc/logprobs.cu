// logprobs.cu -- log probabilities of given tokens from a matrix of logits,
// with entropy, rank and the top alternatives, and their gradient.
//
// With z = s l (s the inverse temperature) and, over the rows's N logits,
//   S = sum exp(z - m),  T = sum (z - m) exp(z - m),   m the row maximum:
//   lse = m + log S,  log p(t) = z_t - lse,  entropy = log S - T / S.
// S and T merge under a new maximum m' as S' = S e, T' = e (T + (m - m') S),
// e = exp(m - m'), so one pass over the logits keeps them per thread (fp32)
// and a row is joined over threads, warps and the CTAs of a cluster.
//
// The top k come out of the same pass: each thread also keeps the largest
// logit it saw.  The k-th largest of those maxima bounds the row's k-th
// largest logit from below, and only threads whose maximum reaches the bound
// can hold a logit that does, so a second look (from L2) covers about k
// threads' shares of the row and yields a few more than k keys
// (order key << 32 | ~index: distinct, lower index first on ties).
#include <cooperative_groups.h>

#include "gemm_common.cuh"

namespace cg = cooperative_groups;

namespace nvfp4 {

constexpr int kLpThreads = 512;
constexpr int kLpCand = 1024;      // keys a CTA ranks in shared memory
constexpr int kLpMaxCluster = 8;   // CTAs that share a row
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// exp(d) for d <= 0; a result below 2^-126 is zero
__device__ __forceinline__ float exp_neg(float d) { return ex2(d * kLog2e); }

// Order key of a logit: value order, -0 with +0, any NaN on top; never 0.
__device__ __forceinline__ uint32_t lp_key(float v) {
  return v != v ? 0xFFFFFFFFu : logit_order(v);
}

// 16 bytes of logits as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ static __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  __device__ static __forceinline__ float load(const float* p) { return *p; }
  __device__ static __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  __device__ static __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  __device__ static __forceinline__ float load(const uint16_t* p) {
    return __uint_as_float((uint32_t)*p << 16);
  }
  __device__ static __forceinline__ void store(uint16_t* p, float v) {
    *p = (uint16_t)pack2(v, 0.0f);
  }
};

// A row's elements as `head` single ones up to a 16-byte boundary, `nv`
// vectors, and the rest single again.
struct RowSplit {
  int64_t head, nv;
};
template <typename T>
__device__ __forceinline__ RowSplit split_row(const T* row, int64_t N) {
  const int64_t head =
      min((int64_t)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)), N);
  return {head, (N - head) / Vec<T>::kN};
}

// The softmax state of a part of a row (of the scaled logits).
struct LpStats {
  float m, S, T;
};
__device__ __forceinline__ LpStats lp_merge(const LpStats& a, const LpStats& b) {
  const float m = max_nan(a.m, b.m);
  const float da = a.m - m, db = b.m - m;  // both finite or NaN: m starts at the lowest finite
  const float ea = exp_neg(da), eb = exp_neg(db);
  // a part that vanished adds nothing (da S may have overflowed)
  const float ta = ea == 0.0f ? 0.0f : ea * (a.T + da * a.S);
  const float tb = eb == 0.0f ? 0.0f : eb * (b.T + db * b.S);
  return {m, a.S * ea + b.S * eb, ta + tb};
}

struct LpArgs {
  const void* logits;
  int64_t N, ld;
  const int64_t* tokens;
  float s;
  int k;
  float *logprob, *entropy, *lse, *top_lp;
  int64_t *rank, *top_ids;
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LpArgs p) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kV = Vec<T>::kN;
  constexpr int kU = 32 / kV;  // vectors of a batch: their loads are in flight together
  __shared__ unsigned long long s_cand[kLpCand];
  __shared__ unsigned long long s_top[NVFP4_TOPK_MAX];
  __shared__ uint32_t s_hist[256];
  __shared__ uint16_t s_hot[kLpThreads];
  __shared__ LpStats s_stats[kLpThreads / 32];
  __shared__ uint32_t s_cnt[kLpThreads / 32], s_hi[kLpThreads / 32], s_lo[kLpThreads / 32];
  __shared__ LpStats s_row;
  __shared__ uint32_t s_row_cnt, s_n, s_nhot;
  __shared__ unsigned long long s_prefix;
  __shared__ uint32_t s_need;

  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t m_row = blockIdx.x / C;
  const T* row = static_cast<const T*>(p.logits) + m_row * p.ld;
  const int64_t tok = p.tokens[m_row];
  const bool has = tok >= 0 && tok < p.N;
  const float x_tok = has ? Vec<T>::load(row + tok) : __int_as_float(0x7F800000);
  const RowSplit rs = split_row(row, p.N);
  const int64_t v0 = rs.nv * rank / C, v1 = rs.nv * (rank + 1) / C;
  const uint4* vec = reinterpret_cast<const uint4*>(row + rs.head);
  // the single elements go to the first CTA, one per thread
  const int64_t singles = rank == 0 ? p.N - rs.nv * kV : 0;
  auto single_at = [&](int64_t i) { return i < rs.head ? i : i + rs.nv * kV; };

  // ---- one pass: softmax state, the largest logit, logits above the token's
  float xmax = __int_as_float(0xFF800000);
  LpStats st{kLowest, 0.0f, 0.0f};
  uint32_t above = 0;
  auto take = [&](const auto& x) {
    constexpr int n = sizeof(x) / sizeof(float);
    float bm = x[0];
#pragma unroll
    for (int i = 1; i < n; ++i) bm = max_nan(bm, x[i]);
    if (!(bm <= x_tok)) {
#pragma unroll
      for (int i = 0; i < n; ++i) above += x[i] > x_tok ? 1u : 0u;
    }
    if (!(bm <= xmax)) {
      xmax = max_nan(xmax, bm);
      const float m = max_nan(p.s * xmax, kLowest);
      const float d = st.m - m, e = exp_neg(d);
      st.T = e == 0.0f ? 0.0f : e * (st.T + d * st.S);
      st.S *= e;
      st.m = m;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      // a logit of -inf adds nothing: its d is held finite so that 0 d = 0
      const float d = max_nan(__fmaf_rn(x[i], p.s, -st.m), -1e30f);
      const float e = exp_neg(d);
      st.S += e;
      st.T = __fmaf_rn(d, e, st.T);
    }
  };
  int64_t v = v0 + tid;
  for (; v + (kU - 1) * kLpThreads < v1; v += kU * kLpThreads) {
    uint4 raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) raw[u] = __ldg(vec + v + u * kLpThreads);
    float x[kU * kV];
#pragma unroll
    for (int u = 0; u < kU; ++u) Vec<T>::unpack(raw[u], x + u * kV);
    take(x);
  }
  for (; v < v1; v += kLpThreads) {
    float x[kV];
    Vec<T>::unpack(__ldg(vec + v), x);
    take(x);
  }
  if (tid < singles) {
    const float x[1] = {Vec<T>::load(row + single_at(tid))};
    take(x);
  }

  // ---- over the block
  const bool any = v0 + tid < v1 || tid < singles;
  const uint32_t key = any ? lp_key(xmax) : 0u;
  LpStats w = st;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const LpStats other{__shfl_xor_sync(0xFFFFFFFFu, w.m, o), __shfl_xor_sync(0xFFFFFFFFu, w.S, o),
                        __shfl_xor_sync(0xFFFFFFFFu, w.T, o)};
    // the same order of operands on both sides, so that all lanes agree
    w = (lane & o) ? lp_merge(other, w) : lp_merge(w, other);
  }
  const uint32_t wc = __reduce_add_sync(0xFFFFFFFFu, above);
  const uint32_t whi = __reduce_max_sync(0xFFFFFFFFu, key);
  const uint32_t wlo = __reduce_min_sync(0xFFFFFFFFu, any ? key : 0xFFFFFFFFu);
  if (lane == 0) {
    s_stats[warp] = w;
    s_cnt[warp] = wc;
    s_hi[warp] = whi;
    s_lo[warp] = wlo;
  }
  if (tid == 0) {
    s_n = 0;
    s_nhot = 0;
  }
  __syncthreads();
  if (tid == 0) {
    LpStats a = s_stats[0];
    uint32_t c = s_cnt[0];
    for (int i = 1; i < kLpThreads / 32; ++i) {
      a = lp_merge(a, s_stats[i]);
      c += s_cnt[i];
    }
    s_row = a;
    s_row_cnt = c;
  }

  // ---- the CTA's k largest keys, sorted, zeros where its share has fewer
  if (p.k > 0) {
    uint32_t hi = 0u, lo = 0xFFFFFFFFu;
    for (int i = 0; i < kLpThreads / 32; ++i) {
      hi = max(hi, s_hi[i]);
      lo = min(lo, s_lo[i]);
    }
    // a bound that at least k threads' maxima reach, and few more than k:
    // bisection between the smallest and the largest of them
    uint32_t bound = 1u;
    if (__syncthreads_count(any) >= p.k) {
      bound = lo;
      uint64_t up = (uint64_t)hi + 1;  // no maximum reaches `up`
      while (up - bound > 1) {
        const uint32_t mid = (uint32_t)((bound + up) >> 1);
        const int c = __syncthreads_count(key >= mid);
        if (c >= p.k) {
          bound = mid;
          if (c <= p.k + p.k / 4 + 4) break;
        } else {
          up = mid;
        }
      }
    }
    const bool hot = any && key >= bound;
    const uint32_t bal = __ballot_sync(0xFFFFFFFFu, hot);
    if (bal) {
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&s_nhot, (uint32_t)__popc(bal));
      at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(bal & ((1u << lane) - 1u));
      if (hot) s_hot[at] = (uint16_t)tid;
    }
    __syncthreads();
    // the hot threads' shares again, spread over the block
    auto see = [&](float x, int64_t n) {
      const uint32_t kx = lp_key(x);
      if (kx >= bound) {
        const uint32_t at = atomicAdd(&s_n, 1u);
        if (at < (uint32_t)kLpCand)
          s_cand[at] = ((unsigned long long)kx << 32) | (uint32_t)~(uint32_t)n;
      }
    };
    const uint32_t per = (uint32_t)((v1 - v0 + kLpThreads - 1) / kLpThreads) + 1;  // vectors, a single
    const uint32_t todo = per * s_nhot;  // about N / kV at most
    for (uint32_t i = tid; i < todo; i += kLpThreads) {
      const int h = s_hot[i / per];
      const uint32_t j = i % per;
      if (j == per - 1) {
        if (h < singles) see(Vec<T>::load(row + single_at(h)), single_at(h));
        continue;
      }
      const int64_t vv = v0 + h + (int64_t)j * kLpThreads;
      if (vv >= v1) continue;
      float x[kV];
      Vec<T>::unpack(__ldg(vec + vv), x);
#pragma unroll
      for (int q = 0; q < kV; ++q) see(x[q], rs.head + vv * kV + q);
    }
    for (int i = tid; i < p.k; i += kLpThreads) s_top[i] = 0ull;
    __syncthreads();
    int n = (int)s_n;
    if (n > kLpCand) {
      // heavily tied logits: the k-th largest key by 8-bit digits from the
      // top, over the whole share, then exactly the keys that reach it
      const int64_t mine = (v1 - v0) * kV + singles;
      auto key_at = [&](int64_t i) {
        const int64_t at = i < (v1 - v0) * kV ? rs.head + v0 * kV + i : single_at(i - (v1 - v0) * kV);
        return ((unsigned long long)lp_key(Vec<T>::load(row + at)) << 32) | (uint32_t)~(uint32_t)at;
      };
      unsigned long long prefix = 0ull, mask = 0ull;
      uint32_t need = (uint32_t)p.k;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kLpThreads) s_hist[i] = 0;
        __syncthreads();
        for (int64_t i = tid; i < mine; i += kLpThreads) {
          const unsigned long long kk = key_at(i);
          if ((kk & mask) == prefix) atomicAdd(&s_hist[(uint32_t)(kk >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
          int b = 255;
          while (s_hist[b] < need) need -= s_hist[b--];
          s_prefix = prefix | ((unsigned long long)b << shift);
          s_need = need;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        mask |= 0xFFull << shift;
      }
      if (tid == 0) s_n = 0;
      __syncthreads();
      for (int64_t i = tid; i < mine; i += kLpThreads) {
        const unsigned long long kk = key_at(i);
        if (kk >= prefix) s_cand[atomicAdd(&s_n, 1u)] = kk;  // exactly k of them
      }
      __syncthreads();
      n = (int)s_n;
    }
    for (int i = tid; i < n; i += kLpThreads) {
      const unsigned long long kk = s_cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += s_cand[j] > kk ? 1 : 0;
      if (r < p.k) s_top[r] = kk;
    }
  }
  __syncthreads();

  // ---- over the cluster, in the first CTA
  if (C > 1) cl.sync();
  if (rank == 0) {
    const unsigned long long* keys = s_top;
    if (C > 1) {
      if (tid == 0) {
        LpStats a = s_row;
        uint32_t c = s_row_cnt;
        for (int i = 1; i < C; ++i) {
          a = lp_merge(a, *cl.map_shared_rank(&s_row, i));
          c += *cl.map_shared_rank(&s_row_cnt, i);
        }
        s_row = a;
        s_row_cnt = c;
      }
      if (p.k > 0) {
        for (int i = tid; i < C * p.k; i += kLpThreads)
          s_cand[i] = cl.map_shared_rank(s_top, i / p.k)[i % p.k];
        __syncthreads();
        const int n = C * p.k;
        for (int i = tid; i < n; i += kLpThreads) {
          const unsigned long long kk = s_cand[i];
          int r = 0;
          for (int j = 0; j < n; ++j) r += s_cand[j] > kk ? 1 : 0;
          if (kk != 0ull && r < p.k) s_top[r] = kk;  // k <= N keys are not zero
        }
      }
      __syncthreads();
    }
    const LpStats a = s_row;
    const bool empty = a.S == 0.0f;  // every logit is -inf
    const float logS = empty ? __int_as_float(0xFF800000) : logf(a.S);
    auto logp = [&](float x) { return empty ? logS : __fmaf_rn(x, p.s, -a.m) - logS; };
    if (tid == 0) {
      p.logprob[m_row] = has ? logp(x_tok) : 0.0f;
      p.entropy[m_row] = empty ? 0.0f : logS - a.T / a.S;
      p.lse[m_row] = empty ? logS : a.m + logS;
      p.rank[m_row] = has ? (int64_t)s_row_cnt + 1 : 0;
    }
    for (int j = tid; j < p.k; j += kLpThreads) {
      const unsigned long long kk = keys[j];
      p.top_ids[m_row * p.k + j] = (int64_t)(uint32_t)~(uint32_t)kk;
      p.top_lp[m_row * p.k + j] = logp(key_value((uint32_t)(kk >> 32)));
    }
  }
  if (C > 1) cl.sync();  // no CTA leaves while the first one reads its shared memory
}

// dl_n = s (a (1[n = t] - p_n) - b p_n (log p_n + H)): one read and one write
// of the row, p from the forward's log-sum-exp.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;  // vectors per thread

struct LpGradArgs {
  const void* logits;
  int64_t N, ld, ld_out;
  const int64_t* tokens;
  float s;
  const float *lse, *entropy, *g_lp, *g_ent;
  void* out;
};

template <typename T>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const LpGradArgs p) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kV = Vec<T>::kN;
  const int64_t m = blockIdx.y;
  const T* row = static_cast<const T*>(p.logits) + m * p.ld;
  T* out = static_cast<T*>(p.out) + m * p.ld_out;
  const int64_t tok = p.tokens[m];
  const bool has = tok >= 0 && tok < p.N;
  const float lse = p.lse[m];
  const float a = has ? p.s * p.g_lp[m] : 0.0f;
  const float b = p.g_ent ? p.s * p.g_ent[m] : 0.0f;
  const float c0 = b != 0.0f ? -(a + b * p.entropy[m]) : -a, c1 = -b;
  const bool empty = lse == __int_as_float(0xFF800000);  // no logit of the row is finite
  auto grad = [&](float x) {
    // p log p = 0 at a logit of -inf: log p is held finite
    const float lp = max_nan(__fmaf_rn(x, p.s, -lse), -1e30f);
    return empty ? 0.0f : exp_neg(lp) * __fmaf_rn(c1, lp, c0);
  };
  const RowSplit rs = split_row(row, p.N);
  // the output's rows may start elsewhere against a 16-byte boundary
  const bool vec_out = ((reinterpret_cast<uintptr_t>(out + rs.head)) & 15) == 0;
  const uint4* src = reinterpret_cast<const uint4*>(row + rs.head);
  const int64_t v0 = (int64_t)blockIdx.x * kGradThreads * kGradVecs + threadIdx.x;
  uint4 raw[kGradVecs];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int64_t v = v0 + u * kGradThreads;
    if (v < rs.nv) raw[u] = src[v];
  }
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int64_t v = v0 + u * kGradThreads;
    if (v >= rs.nv) continue;
    float x[kV];
    Vec<T>::unpack(raw[u], x);
    const int64_t n0 = rs.head + v * kV;
#pragma unroll
    for (int i = 0; i < kV; ++i) x[i] = grad(x[i]);
    if (has && !empty && tok >= n0 && tok < n0 + kV) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (n0 + i == tok) x[i] += a;
    }
    if (vec_out) {
      *reinterpret_cast<uint4*>(out + n0) = Vec<T>::pack(x);
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) Vec<T>::store(out + n0 + i, x[i]);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < p.N - rs.nv * kV) {
    const int64_t n = (int64_t)threadIdx.x < rs.head ? threadIdx.x : threadIdx.x + rs.nv * kV;
    float g = grad(Vec<T>::load(row + n));
    if (has && !empty && n == tok) g += a;
    Vec<T>::store(out + n, g);
  }
}

// ------------------------------------------------------------ host side
// CTAs per row: enough that few rows still fill the GPU, while a CTA keeps
// at least 4096 logits.
static int lp_cluster(int64_t M, int64_t N, int sms) {
  int c = 1;
  while (c < kLpMaxCluster && M * c < 2 * sms && N / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename T>
static cudaError_t lp_launch(const LpArgs& a, int64_t M, int c, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * c));
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a);
}

nvfp4_status logprobs_launch(const void* logits, int dtype, int64_t M, int64_t N, int64_t ld,
                             const int64_t* tokens, float s, int k, float* logprob, float* entropy,
                             float* lse, int64_t* rank, int64_t* top_ids, float* top_lp,
                             cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const LpArgs a{logits, N, ld, tokens, s, k, logprob, entropy, lse, top_lp, rank, top_ids};
  const int c = lp_cluster(M, N, sms);
  const cudaError_t err = dtype == NVFP4_OUT_BF16 ? lp_launch<uint16_t>(a, M, c, stream)
                                                  : lp_launch<float>(a, M, c, stream);
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status logprobs_grad_launch(const void* logits, int dtype, int64_t M, int64_t N, int64_t ld,
                                  const int64_t* tokens, float s, const float* lse,
                                  const float* entropy, const float* g_lp, const float* g_ent,
                                  void* out, int64_t ld_out, cudaStream_t stream) {
  const int64_t per = kGradThreads * kGradVecs * (dtype == NVFP4_OUT_BF16 ? 8 : 4);
  // rows beyond the grid's y limit go to further launches
  for (int64_t m0 = 0; m0 < M; m0 += 65535) {
    const int64_t rows = M - m0 < 65535 ? M - m0 : 65535;
    const size_t es = dtype == NVFP4_OUT_BF16 ? 2 : 4;
    const LpGradArgs a{static_cast<const uint8_t*>(logits) + m0 * ld * es,
                       N,
                       ld,
                       ld_out,
                       tokens + m0,
                       s,
                       lse + m0,
                       entropy ? entropy + m0 : nullptr,
                       g_lp + m0,
                       g_ent ? g_ent + m0 : nullptr,
                       static_cast<uint8_t*>(out) + m0 * ld_out * es};
    PdlLaunch l(dim3((unsigned)((N + per - 1) / per), (unsigned)rows), dim3(kGradThreads), 0,
                stream);
    const cudaError_t err =
        dtype == NVFP4_OUT_BF16
            ? cudaLaunchKernelEx(&l.cfg, logprobs_grad_kernel<uint16_t>, a)
            : cudaLaunchKernelEx(&l.cfg, logprobs_grad_kernel<float>, a);
    if (err != cudaSuccess) return NVFP4_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
