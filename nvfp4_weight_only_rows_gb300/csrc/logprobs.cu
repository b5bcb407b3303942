// logprobs.cu -- log probabilities of given tokens from a matrix of logits,
// with entropy, rank and the top alternatives, and their gradient.
//
// With s the inverse temperature, c = s log2 e, m the largest of the row's
// logits l and z = c (l - m), a power of two,
//   S = sum 2^z,  T = sum z 2^z:   lse = s m + ln2 log2 S,
//   log p(t) = s (l_t - m) - ln2 log2 S,  entropy = ln2 (log2 S - T / S).
// S and T merge under a new maximum m' as S' = S e, T' = e (T + d S), d =
// c (m - m'), e = 2^d, so one pass over the logits keeps them per thread (fp32)
// and a row is joined over threads, warps and the CTAs of a cluster.  The
// pass is bound by instruction issue before HBM where the logits are bf16
// (11 instructions an element fit the copy rate): maxima and comparisons on
// bf16 pairs, sums on fp32 pairs.
//
// The top k come out of the same pass: each thread also keeps the largest
// logit it saw.  The k-th largest of those maxima bounds the row's k-th
// largest logit from below, and only threads whose maximum reaches the bound
// can hold a logit that does, so a second look (from L2) covers about k
// threads' shares of the row and yields a few more than k keys
// (order key << 32 | ~index: distinct, lower index first on ties).
#include <cuda_bf16.h>

#include "gemm_common.cuh"

namespace nvfp4 {

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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// fma, mul and add on two fp32 at once.
__device__ __forceinline__ uint64_t pack2f(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2f(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
// Two logits (bits) into the sums: z = c (x - m), S += 2^z, T += z 2^z, for
// both at once.  m2: -m.
__device__ __forceinline__ void lp_pair(uint32_t x0, uint32_t x1, uint64_t c2, uint64_t m2,
                                        uint64_t& S, uint64_t& T) {
  asm("{\n\t.reg .b64 x, d, e;\n\t.reg .f32 a, b;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "add.rn.f32x2 d, x, %5;\n\t"
      "mul.rn.f32x2 d, d, %4;\n\t"
      "mov.b64 {a, b}, d;\n\t"
      "ex2.approx.ftz.f32 a, a;\n\t"
      "ex2.approx.ftz.f32 b, b;\n\t"
      "mov.b64 e, {a, b};\n\t"
      "add.rn.f32x2 %0, %0, e;\n\t"
      "fma.rn.f32x2 %1, d, e, %1;\n\t}"
      : "+l"(S), "+l"(T)
      : "r"(x0), "r"(x1), "l"(c2), "l"(m2));
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct LpArgs {
  const void* logits;
  int64_t N, ld;
  const int64_t* tokens;
  float s, c;  // the inverse temperature, and times log2 e
  int k;
  float *logprob, *entropy, *lse, *top_lp;
  int64_t *rank, *top_ids;
};

constexpr float kMaxScale = 1e12f;  // c in the main pass: times the floor below it is finite

// c times a difference of logits; c itself is beyond fp32 for the largest
// inverse temperatures.
__device__ __forceinline__ float lp_scaled(const LpArgs& p, float d) {
  return p.c <= kMaxScale ? p.c * d : kLog2e * (p.s * d);
}

// Softmax state of a part of a row relative to its largest logit m.
struct LpStats {
  float m, S, T;
};
// ... seen from a maximum m >= a.m.  A part that vanishes adds nothing (the
// product d S may have overflowed).
__device__ __forceinline__ LpStats lp_shift(const LpStats& a, float m, const LpArgs& p) {
  const float d = lp_scaled(p, a.m - m), e = ex2(d);
  return {m, a.S * e, e == 0.0f ? 0.0f : e * __fmaf_rn(d, a.S, a.T)};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable p in the cluster's first CTA.
__device__ __forceinline__ uint32_t first_cta_addr(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Logits are held at or above this in the main pass, so that a masked one
// (-inf) has a finite d and 0 d = 0.  What is held there has to vanish against
// the largest logit, and its d to stay finite; where it does not (a share with
// nothing else left, an extreme temperature, a largest logit near fp32's own)
// the share is looked at again without the floor, with d held at -1e30.
constexpr float kFloor = -0x1p83f;  // also a bf16
constexpr float kMinDrop = 1500.0f, kMaxDrop = 1e38f;  // -d of what is held there

// T: float, or uint16_t for bf16 bits; kT threads; kU vectors of a batch, whose
// loads are in flight together (4 let 1024 threads share an SM).
template <typename T, int kT, int kU>
__global__ void __launch_bounds__(kT, kU == 4 ? 1024 / kT : 1) logprobs_kernel(const LpArgs p) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kV = Vec<T>::kN;
  constexpr int kW = kT / 32;
  __shared__ unsigned long long s_cand[kLpCand];
  __shared__ unsigned long long s_top[NVFP4_TOPK_MAX];
  __shared__ unsigned long long s_merge[kLpMaxCluster * NVFP4_TOPK_MAX];
  __shared__ float4 s_part[kLpMaxCluster];  // per CTA: m, S, T, count
  __shared__ uint32_t s_hist[256];
  __shared__ uint16_t s_hot[kT];
  __shared__ float s_S[kW], s_T[kW];
  __shared__ uint32_t s_cnt[kW], s_hi[kW], s_lo[kW];
  __shared__ uint32_t s_n, s_nhot, s_prefix, s_need, s_eq[kW];

  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  if (C > 1) cluster_arrive();  // every CTA of the cluster runs before one writes to another
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t m_row = blockIdx.x / C;
  const T* row = static_cast<const T*>(p.logits) + m_row * p.ld;
  const RowSplit rs = split_row(row, p.N);
  const int64_t v0 = rs.nv * rank / C, v1 = rs.nv * (rank + 1) / C;
  const uint4* vec = reinterpret_cast<const uint4*>(row + rs.head);
  // the single elements go to the first CTA, one per thread
  const int singles = rank == 0 ? (int)(p.N - rs.nv * kV) : 0;
  auto single_at = [&](int64_t i) { return i < rs.head ? i : i + rs.nv * kV; };

  uint4 raw[kU];
  int64_t v = v0 + tid;
  // past the end: -inf, which adds nothing
  const uint32_t pad = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = at + u * kT;
      raw[u] = i < v1 ? __ldg(vec + i) : make_uint4(pad, pad, pad, pad);
    }
  };
  fetch(v);
  const int64_t tok = p.tokens[m_row];
  const bool has = tok >= 0 && tok < p.N;
  const float x_tok = has ? Vec<T>::load(row + tok) : __int_as_float(0x7F800000);

  // ---- one pass: softmax state, the largest logit, logits above the token's
  float largest = __int_as_float(0xFF800000);  // without the floor
  LpStats st{kFloor, 0.0f, 0.0f};
  uint64_t S2 = 0ull, T2 = 0ull;
  const uint64_t c2 = pack2f(p.c, p.c);
  uint32_t above = 0;
  auto raise = [&](float bm) {  // a new largest logit
    const float m = max_nan(st.m, bm);
    const float d = p.c * (st.m - m), e = ex2(d);
    const float2 S = unpack2f(S2), t = unpack2f(T2);
    T2 = e == 0.0f ? 0ull : pack2f(e * __fmaf_rn(d, S.x, t.x), e * __fmaf_rn(d, S.y, t.y));
    S2 = pack2f(S.x * e, S.y * e);
    st.m = m;
  };
  while (v < v1) {
    constexpr int kWords = 4 * kU;
    uint32_t x[kWords];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      x[4 * u] = raw[u].x;
      x[4 * u + 1] = raw[u].y;
      x[4 * u + 2] = raw[u].z;
      x[4 * u + 3] = raw[u].w;
    }
    v += kU * kT;
    if (v < v1) fetch(v);
    float bm;
    if constexpr (sizeof(T) == 2) {
      uint32_t b2 = x[0];
#pragma unroll
      for (int i = 1; i < kWords; ++i) b2 = max2_nan(b2, x[i]);
      bm = max_nan(__uint_as_float(b2 << 16), __uint_as_float(b2 & 0xFFFF0000u));
      if (!(bm <= x_tok)) {
        const __nv_bfloat162 t2 = __float2bfloat162_rn(x_tok);  // a bf16 (or +inf) as it is
        __nv_bfloat162 n2 = __float2bfloat162_rn(0.0f);  // counts of at most 4 kU: exact
#pragma unroll
        for (int i = 0; i < kWords; ++i)
          n2 = __hadd2(n2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), t2));
        above += (uint32_t)(__low2float(n2) + __high2float(n2));
      }
      const uint32_t f2 = __float_as_uint(kFloor) >> 16 | (__float_as_uint(kFloor) & 0xFFFF0000u);
#pragma unroll
      for (int i = 0; i < kWords; ++i) x[i] = max2_nan(x[i], f2);
    } else {
      bm = __uint_as_float(x[0]);
#pragma unroll
      for (int i = 1; i < kWords; ++i) bm = max_nan(bm, __uint_as_float(x[i]));
      if (!(bm <= x_tok)) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) above += __uint_as_float(x[i]) > x_tok ? 1u : 0u;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        x[i] = __float_as_uint(max_nan(__uint_as_float(x[i]), kFloor));
    }
    largest = max_nan(largest, bm);
    if (!(bm <= st.m)) raise(bm);
    const uint64_t m2 = pack2f(-st.m, -st.m);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) lp_pair(x[i] << 16, x[i] & 0xFFFF0000u, c2, m2, S2, T2);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 2) lp_pair(x[i], x[i + 1], c2, m2, S2, T2);
    }
  }
  float single = __int_as_float(0xFF800000);
  if (tid < singles) {
    single = Vec<T>::load(row + single_at(tid));
    above += single > x_tok ? 1u : 0u;
    largest = max_nan(largest, single);
    const float x = max_nan(single, kFloor);
    if (!(x <= st.m)) raise(x);
    const float d = p.c * (x - st.m), e = ex2(d);
    st.S = e;
    st.T = d * e;
  }
  {
    const float2 S = unpack2f(S2), t = unpack2f(T2);
    st.S += S.x + S.y;
    st.T += t.x + t.y;
  }

  // ---- over the block: the largest logit first, then plain sums
  const bool any = v0 + tid < v1 || tid < singles;
  const uint32_t key = any ? lp_key(st.m) : 0u;
  {
    const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, above);
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, key);
    const uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, any ? key : 0xFFFFFFFFu);
    if (lane == 0) {
      s_cnt[warp] = c;
      s_hi[warp] = hi;
      s_lo[warp] = lo;
    }
  }
  if (tid == 0) {
    s_n = 0;
    s_nhot = 0;
  }
  const int n_any = __syncthreads_count(any);
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, lane < kW ? s_hi[lane] : 0u);
  const uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, lane < kW ? s_lo[lane] : 0xFFFFFFFFu);
  float m_blk = key_value(hi);
  // the share's vectors, four at a time per thread, and its singles: f of each
  // logit
  auto for_each = [&](auto f) {
    constexpr int kB = 4;
    for (int64_t i0 = v0 + tid; i0 < v1; i0 += kB * kT) {
      uint4 r[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) r[u] = i0 + u * kT < v1 ? __ldg(vec + i0 + u * kT) : make_uint4(pad, pad, pad, pad);
#pragma unroll 1
      for (int u = 0; u < kB; ++u) {
        float x[kV];
        Vec<T>::unpack(r[u], x);
        if (i0 + u * kT < v1)
#pragma unroll
          for (int q = 0; q < kV; ++q) f(x[q]);
      }
    }
    if (tid < singles) f(single);
  };
  // (block-uniform)
  const float drop = p.c * (m_blk - kFloor);
  const bool plain = !(drop >= kMinDrop && drop <= kMaxDrop) || p.c > kMaxScale;
  if (!plain) {
    st = lp_shift(st, m_blk, p);
  } else {
    const uint32_t wk = __reduce_max_sync(0xFFFFFFFFu, lp_key(largest));
    __syncthreads();
    if (lane == 0) s_hi[warp] = wk;
    __syncthreads();
    const float top = key_value(__reduce_max_sync(0xFFFFFFFFu, lane < kW ? s_hi[lane] : 0u));
    m_blk = max_nan(top, kLowest);
    st = {m_blk, 0.0f, 0.0f};
    if (!(top < kLowest))  // (all -inf: nothing)
      for_each([&](float x) {
        const float d = max_nan(lp_scaled(p, x - m_blk), -1e30f), e = ex2(d);
        st.S += e;
        st.T = __fmaf_rn(d, e, st.T);
      });
  }
  {
    const float S = warp_sum(st.S), t = warp_sum(st.T);
    if (lane == 0) {
      s_S[warp] = S;
      s_T[warp] = t;
    }
  }

  // ---- the CTA's k largest keys, sorted, zeros where its share has fewer
  if (p.k > 0) {
    // a bound that at least k threads' maxima reach, and few more than k:
    // bisection between the smallest and the largest of them
    // The maxima say nothing at or below the floor: the bound stays above it.
    const uint32_t floor_key = lp_key(kFloor);
    uint32_t bound = floor_key + 1u;
    if (n_any >= p.k && lo >= bound) bound = lo;
    if (hi >= bound && n_any >= p.k) {
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
    auto see = [&](float x, int64_t at_n) {
      const uint32_t kx = lp_key(x);
      if (kx >= bound) {
        const uint32_t at = atomicAdd(&s_n, 1u);
        if (at < (uint32_t)kLpCand)
          s_cand[at] = ((unsigned long long)kx << 32) | (uint32_t)~(uint32_t)at_n;
      }
    };
    if (hot && tid < singles) see(single, single_at(tid));
    __syncthreads();
    // the hot threads' vectors again, spread over the block
    const uint32_t per = (uint32_t)((v1 - v0 + kT - 1) / kT);
    const uint32_t todo = per * s_nhot;  // about N / kV at most
    for (uint32_t i = tid; i < todo; i += kT) {
      const int64_t vv = v0 + s_hot[i / per] + (int64_t)(i % per) * kT;
      if (vv >= v1) continue;
      float x[kV];
      Vec<T>::unpack(__ldg(vec + vv), x);
#pragma unroll
      for (int q = 0; q < kV; ++q) see(x[q], rs.head + vv * kV + q);
    }
    for (int i = tid; i < p.k; i += kT) s_top[i] = 0ull;
    __syncthreads();
    int n = (int)s_n;

    // the share's elements in increasing order of the column: the head, the
    // vectors, the tail
    const int64_t n_el = (v1 - v0) * kV, mine = n_el + singles;
    const int64_t h0 = singles ? rs.head : 0;
    auto index_at = [&](int64_t i) {
      return i < h0 ? i : i - h0 < n_el ? rs.head + v0 * kV + i - h0 : rs.nv * kV + i - n_el;
    };
    auto key_at = [&](int64_t i) { return lp_key(Vec<T>::load(row + index_at(i))); };
    auto full_key = [&](uint32_t kx, int64_t i) {
      return ((unsigned long long)kx << 32) | (uint32_t)~(uint32_t)index_at(i);
    };
    // the first `left` elements of key `kx`, in order, appended to s_cand;
    // returns how many are missing
    auto take_first = [&](uint32_t kx, int64_t left) {
      constexpr int kE = 4;  // consecutive elements of a thread
      for (int64_t i0 = 0; i0 < mine && left > 0; i0 += kT * kE) {
        uint32_t eq = 0;
        const int64_t i = i0 + tid * kE;
#pragma unroll
        for (int q = 0; q < kE; ++q)
          if (i + q < mine && key_at(i + q) == kx) eq |= 1u << q;
        int incl = __popc(eq);
        const int own = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) s_eq[warp] = incl;
        __syncthreads();
        int at = incl - own, total = 0;
        for (int w = 0; w < kW; ++w) {
          const int c = s_eq[w];
          if (w < warp) at += c;
          total += c;
        }
#pragma unroll
        for (int q = 0; q < kE; ++q)
          if ((eq >> q) & 1u) {
            if (at < left) s_cand[atomicAdd(&s_n, 1u)] = full_key(kx, i + q);
            ++at;
          }
        left -= total;
        __syncthreads();
      }
      return left;
    };
    if (n > kLpCand) {
      // heavily tied logits: the value of the k-th largest by 8-bit digits
      // from the top, then the keys above it and the first of those equal
      uint32_t prefix = 0u, mask = 0u, need = (uint32_t)p.k;
      for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int i = tid; i < 256; i += kT) s_hist[i] = 0;
        __syncthreads();
        for (int64_t i0 = 0; i0 < mine; i0 += kT) {
          const int64_t i = i0 + tid;
          const uint32_t kk = i < mine ? key_at(i) : 0u;
          const bool in = i < mine && (kk & mask) == prefix;
          const uint32_t bin = (kk >> shift) & 255u;
          // lanes of one bin count at once
          const uint32_t same = __match_any_sync(0xFFFFFFFFu, in ? bin : 256u);
          if (in && (same & ((1u << lane) - 1u)) == 0u)
            atomicAdd(&s_hist[bin], (uint32_t)__popc(same));
        }
        __syncthreads();
        if (tid == 0) {
          int b = 255;
          while (s_hist[b] < need) need -= s_hist[b--];
          s_prefix = prefix | ((uint32_t)b << shift);
          s_need = need;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        mask |= 0xFFu << shift;
      }
      __syncthreads();
      if (tid == 0) s_n = 0;
      __syncthreads();
      for (int64_t i = tid; i < mine; i += kT) {
        const uint32_t kk = key_at(i);
        if (kk > prefix) s_cand[atomicAdd(&s_n, 1u)] = full_key(kk, i);  // fewer than k
      }
      take_first(prefix, need);
      __syncthreads();
      n = (int)s_n;
    } else if (n < p.k && n < mine) {
      // fewer than k logits above the floor: from the values below it, the
      // largest first (a mask has one: one round)
      int64_t left = min((int64_t)p.k, mine) - n;
      uint32_t below = bound;
      while (left > 0) {
        uint32_t mx = 0u;
        for_each([&](float x) {
          const uint32_t kk = lp_key(x);
          if (kk < below) mx = max(mx, kk);
        });
        mx = __reduce_max_sync(0xFFFFFFFFu, mx);
        __syncthreads();
        if (lane == 0) s_eq[warp] = mx;
        __syncthreads();
        below = __reduce_max_sync(0xFFFFFFFFu, lane < kW ? s_eq[lane] : 0u);
        __syncthreads();
        left = take_first(below, left);
      }
      __syncthreads();
      n = (int)s_n;
    }
    for (int i = tid; i < n; i += kT) {
      const unsigned long long kk = s_cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += s_cand[j] > kk ? 1 : 0;
      if (r < p.k) s_top[r] = kk;
    }
  }
  __syncthreads();

  // ---- over the cluster, in its first CTA
  if (C > 1) cluster_wait();
  if (warp == 0) {
    const float S = warp_sum(lane < kW ? s_S[lane] : 0.0f);
    const float t = warp_sum(lane < kW ? s_T[lane] : 0.0f);
    const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, lane < kW ? s_cnt[lane] : 0u);
    if (lane == 0) {
      const uint32_t to = first_cta_addr(&s_part[rank]);
      st_cluster(to, __float_as_uint(m_blk));
      st_cluster(to + 4, __float_as_uint(S));
      st_cluster(to + 8, __float_as_uint(t));
      st_cluster(to + 12, c);
    }
  }
  if (C > 1) {
    for (int i = tid; i < p.k; i += kT)
      st_cluster(first_cta_addr(&s_merge[rank * p.k + i]), s_top[i]);
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    // A key's place is the number of larger keys in all lists, its own among
    // them; k <= N keys of the row are not zero, so every place gets one.  The
    // lists are searched side by side: one row with k = 20 in 8.4 against 9.3 us
    // with one list after another.
    int top = 1;
    while (2 * top <= p.k) top *= 2;
    for (int i = tid; i < C * p.k; i += kT) {
      const unsigned long long kk = s_merge[i];
      if (kk == 0ull) continue;
      int at[kLpMaxCluster] = {};
      for (int step = top; step; step >>= 1) {
#pragma unroll
        for (int c = 0; c < kLpMaxCluster; ++c)
          if (c < C && at[c] + step <= p.k && s_merge[c * p.k + at[c] + step - 1] > kk)
            at[c] += step;
      }
      int r = 0;
#pragma unroll
      for (int c = 0; c < kLpMaxCluster; ++c) r += at[c];
      if (r < p.k) s_top[r] = kk;
    }
  }
  __syncthreads();
  float4 part = lane < C ? s_part[lane] : make_float4(kLowest, 0.0f, 0.0f, 0.0f);
  float m = part.x;
#pragma unroll
  for (int o = kLpMaxCluster / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  m = __shfl_sync(0xFFFFFFFFu, m, 0);
  const LpStats a = lp_shift({part.x, part.y, part.z}, m, p);
  const float S = warp_sum(a.S), t = warp_sum(a.T);
  const bool empty = S == 0.0f;  // every logit is -inf
  const float logS = empty ? __int_as_float(0xFF800000) : kLn2 * log2f(S);
  auto logp = [&](float x) { return empty ? logS : __fmaf_rn(p.s, x - m, -logS); };
  if (warp == 0) {
    const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, lane < C ? __float_as_uint(part.w) : 0u);
    if (lane == 0) {
      p.logprob[m_row] = has ? logp(x_tok) : 0.0f;
      p.entropy[m_row] = empty ? 0.0f : logS - kLn2 * (t / S);
      p.lse[m_row] = empty ? logS : __fmaf_rn(p.s, m, logS);
      p.rank[m_row] = has ? (int64_t)c + 1 : 0;
    }
  }
  for (int j = tid; j < p.k; j += kT) {
    const unsigned long long kk = s_top[j];
    p.top_ids[m_row * p.k + j] = (int64_t)(uint32_t)~(uint32_t)kk;
    p.top_lp[m_row * p.k + j] = logp(key_value((uint32_t)(kk >> 32)));
  }
}

// dl_n = s (a (1[n = t] - p_n) - b p_n (log p_n + H)): one read and one write
// of the row, p from the forward's log-sum-exp.
//
// Bound by HBM.  kStream reads and writes past the caches' reuse (evict
// first, both: neither alone helps), in CTAs of 512 threads: 2048 x 128256
// bf16 177 -> 152 us (1.03 of the copy rate, which caches its writes), 64 x
// 128256 bf16 8.0 -> 7.5 us.  Below 32 MB a gradient stays for its reader, in
// CTAs of 256: 19 x 50257 fp32 2.9 against 3.2 us.
constexpr int kGradVecs = 4;  // vectors per thread

struct LpGradArgs {
  const void* logits;
  int64_t N, ld, ld_out;
  const int64_t* tokens;
  float s;
  const float *lse, *entropy, *g_lp, *g_ent;
  void* out;
};

template <typename T, int kT, bool kStream>
__global__ void __launch_bounds__(kT) logprobs_grad_kernel(const LpGradArgs p) {
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
    // p log p = 0 at a logit of -inf: log p is held where p is zero already, and
    // low enough that no gradient b of the entropy takes b log p to infinity
    const float lp = max_nan(__fmaf_rn(x, p.s, -lse), -100.0f);
    return empty ? 0.0f : exp_neg(lp) * __fmaf_rn(c1, lp, c0);
  };
  const RowSplit rs = split_row(row, p.N);
  // the output's rows may start elsewhere against a 16-byte boundary
  const bool vec_out = ((reinterpret_cast<uintptr_t>(out + rs.head)) & 15) == 0;
  const uint4* src = reinterpret_cast<const uint4*>(row + rs.head);
  const int64_t v0 = (int64_t)blockIdx.x * kT * kGradVecs + threadIdx.x;
  uint4 raw[kGradVecs];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int64_t v = v0 + u * kT;
    if (v < rs.nv) raw[u] = kStream ? __ldcs(src + v) : src[v];
  }
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int64_t v = v0 + u * kT;
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
      if constexpr (kStream) __stcs(reinterpret_cast<uint4*>(out + n0), Vec<T>::pack(x));
      else *reinterpret_cast<uint4*>(out + n0) = Vec<T>::pack(x);
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
// CTAs per row: as many as keep the grid within one and a half CTAs per SM
// and a share at 8192 logits.  Measured (k = 0 / 5): 1 row of 128256 fp32
// 9.5 / 11.4 us with one CTA, 4.3 / 8.0 with eight; 64 rows of 151936 fp32
// 11.1 / 13.4, 8.0 / 10.6, 8.4 / 12.0 and 11.9 / 20.0 with 1, 2, 4 and 8.
static int lp_cluster(int64_t M, int64_t N, int sms) {
  int c = 1;
  while (c < kLpMaxCluster && M * 2 * c <= sms + sms / 2 && N / (2 * c) >= 8192) c *= 2;
  return c;
}

// Shares above this take 512 threads while the grid is at most two CTAs an SM
// or many alternatives are asked for, others 256: 256 rows of 128256 fp32 23.5
// against 29.1 us, 512 rows of 32000 bf16 11.2 against 9.2 us, 2048 rows of
// 128256 bf16 94.3 against 87.1 us (k = 20: 114 against 125).  A grid of one
// CTA an SM loads twice as far ahead: 64 rows of 151936 fp32 15.0 -> 13.6 us.
constexpr int64_t kLpWideShare = 32768;

template <typename T, int kT, int kU>
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
  cfg.blockDim = dim3(kT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kT, kU>, a);
}

nvfp4_status logprobs_launch(const void* logits, int dtype, int64_t M, int64_t N, int64_t ld,
                             const int64_t* tokens, float s, int k, float* logprob, float* entropy,
                             float* lse, int64_t* rank, int64_t* top_ids, float* top_lp,
                             cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const LpArgs a{logits, N, ld, tokens, s, (float)(s * 1.4426950408889634), k, logprob, entropy, lse, top_lp, rank, top_ids};
  const int c = lp_cluster(M, N, sms);
  const bool wide = N / c > kLpWideShare && (M * c <= 2 * sms || k >= 16);
  auto launch = [&](auto type) {
    using T = decltype(type);
    if (!wide) return lp_launch<T, 256, 4>(a, M, c, stream);
    return M * c <= sms ? lp_launch<T, 512, 8>(a, M, c, stream) : lp_launch<T, 512, 4>(a, M, c, stream);
  };
  const cudaError_t err = dtype == NVFP4_OUT_BF16 ? launch(uint16_t{}) : launch(float{});
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4_status logprobs_grad_launch(const void* logits, int dtype, int64_t M, int64_t N, int64_t ld,
                                  const int64_t* tokens, float s, const float* lse,
                                  const float* entropy, const float* g_lp, const float* g_ent,
                                  void* out, int64_t ld_out, cudaStream_t stream) {
  const size_t es = dtype == NVFP4_OUT_BF16 ? 2 : 4;
  const bool stream_it = 2 * (double)M * (double)N * (double)es >= (double)(32 << 20);
  const int threads = stream_it ? 512 : 256;
  const int64_t per = threads * kGradVecs * (16 / (int64_t)es);
  // rows beyond the grid's y limit go to further launches
  for (int64_t m0 = 0; m0 < M; m0 += 65535) {
    const int64_t rows = M - m0 < 65535 ? M - m0 : 65535;
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
    PdlLaunch l(dim3((unsigned)((N + per - 1) / per), (unsigned)rows), dim3((unsigned)threads), 0,
                stream);
    auto kern = dtype == NVFP4_OUT_BF16
                    ? (stream_it ? logprobs_grad_kernel<uint16_t, 512, true>
                                 : logprobs_grad_kernel<uint16_t, 256, false>)
                    : (stream_it ? logprobs_grad_kernel<float, 512, true>
                                 : logprobs_grad_kernel<float, 256, false>);
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, kern, a);
    if (err != cudaSuccess) return NVFP4_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
