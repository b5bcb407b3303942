// moe.cu -- the expert layer of a mixture-of-experts model for a few tokens:
// for every (token m, slot j) pair p with expert e = ids[m, j],
//   g | u = G13[e] (W13[e] x_m),  h = g / (1 + exp(-g)) u,
//   out_m = sum_j w[m, j] G2[e] (W2[e] h),
// W13, W2 in NVFP4 (e2m1 code times E4M3 block scale; G the expert's global
// scale).
//
// With few tokens the weights of the chosen experts are read once and
// everything else is small, so the layer is bound by HBM: 9/16 byte a
// weight.  Two products and a combine:
//   moe_gemm_kernel<1>  gu[p, 0:2I] = W13[e] x     (fp32, no global scale)
//   moe_gemm_kernel<2>  y[p, 0:H]   = W2[e] h      (h from gu as it is read)
//   moe_combine_kernel  out = sum over a token's slots, in slot order
// Every sum has a fixed order: the result does not depend on the schedule.
//
// The products run on mma.sync m16n8k16 (fp16 in, fp32 sums): 16 weight rows
// by 8 pairs of one expert.  Codes go from global memory straight into the
// registers that feed the MMA (a warp's lane (g, t) reads 32 bytes of rows g
// and g + 8: the 64 weights k = 256 s + 64 t ..), are converted with the
// hardware e2m1 conversion and multiplied by their block scale, which is
// exact in fp16.  Which k sit in which MMA does not matter as long as the
// activations agree: MMA j of a stage takes 4 weights of each t.  A tile of
// 8 pairs is far too narrow for a tcgen05 MMA's 128 rows to be cut into the
// 16-row pieces that spread one token's 21 MB of weights over 152 SMs.
//
// Activations: a stage (256 k of a pair) is carried as fp16 after a
// power-of-two rescale by the stage's largest magnitude (exact for bf16 x
// within 2^28 of that maximum), built by each CTA in shared memory.  h, an
// fp32 value, is carried as two fp16, 22 bits, at twice the MMAs of the second
// product.  (One fp16 moved a bf16 result by 9e-4 of it, half of that result's
// own rounding, and saved 0.7 us at one token.)
//
// Work: the items (expert segment, 16-row tile) are split evenly over the
// CTAs, and inside a CTA the (tile, stage) steps of a segment evenly over its
// warps; a tile cut between warps is joined in shared memory in warp order.
//
// Measured: 1 token of H 2048, I 768, top 8 of 128 (21 MB, 3.2 us at the copy
// rate) 14.9 us, most of it the latency of three dependent kernels' first
// loads and of the boundaries between them.
#include <cuda_fp16.h>

#include <type_traits>

#include "gemm_common.cuh"

namespace nvfp4 {

constexpr int kMoeWarps = 8;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeTileN = 4;              // 8-pair tiles of a segment at most
constexpr int kMoeMulStride = 8 * kMoeTileN;
constexpr int kMoeDepth = 2;              // stages of weights in flight per warp
constexpr int kMoeMaxExperts = NVFP4_MOE_MAX_EXPERTS;
constexpr size_t kMoeActBytes = 64 << 10;  // activations a CTA holds at most

struct MoeArgs {
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  const uint8_t *p13, *s13, *p2, *s2;
  const float *g13, *g2;
  void* out;
  float *gu, *y;
  int32_t *status, *bad_flags;  // bad_flags: one word per CTA of each product
  int M, k, H, I, E;
  int seg1, seg2;  // pairs of a segment in either product
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One lane's weights of a stage: 64 codes and 4 block scales of two rows.
struct MoeFrag {
  uint32_t w[2][8];
  uint32_t s[2];
};

// kWide: rows are 32-byte multiples (K % 64 == 0) and so are the bases.
// k0: the lane's first k; codes / scales point at it.
template <bool kWide>
__device__ __forceinline__ void moe_load_row(const uint8_t* codes, const uint8_t* scales,
                                             int left, uint32_t (&w)[8], uint32_t& s) {
  if constexpr (kWide) {
    if (left > 0) {
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7])
                   : "l"(codes));
      s = __ldg(reinterpret_cast<const uint32_t*>(scales));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0u;
      s = 0u;
    }
  } else {
    s = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (left > 16 * b) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes) + b);
        w[2 * b] = v.x;
        w[2 * b + 1] = v.y;
        s |= (uint32_t)__ldg(scales + b) << (8 * b);
      } else {
        w[2 * b] = 0u;
        w[2 * b + 1] = 0u;
      }
    }
  }
}

// Byte offset of chunk (i, t) of pair c in a stage: the 8 values k = 64 t +
// 8 i ..; neighbouring pairs start in the other half of the 128-byte line, so
// a warp's 16-byte reads have no bank conflicts.
__device__ __forceinline__ uint32_t moe_chunk(int c, int i, int t) {
  return (uint32_t)(c * 32 + ((i * 4 + t) ^ ((c & 1) << 2))) * 16u;
}

// Fill the activations of pairs list[0, T): for stage s and pair c, 256 fp16
// values at s_act + (s T + c) 512 and the multiplier that undoes their
// rescale at s_mul[s * kMoeMulStride + c].  kSplit: what the rounding to fp16
// left, as fp16 of the same scale, lo_off bytes further.
template <int kStep, bool kSplit>
__device__ __forceinline__ void moe_build(const MoeArgs& p, const int* list, int T, int n_stages,
                                          float g13, uint8_t* s_act, size_t lo_off,
                                          float* s_mul) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = kStep == 1 ? p.H : p.I;
  const int i = lane >> 2, t = lane & 3;
  for (int w = warp; w < T * n_stages; w += kMoeWarps) {
    const int s = w / T, c = w % T;
    const int pair = list[c];
    const int k0 = 256 * s + 64 * t + 8 * i;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.0f;
    if (k0 < K) {
      if constexpr (kStep == 1) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(pair / p.k) * K + k0));
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[2 * q] = __uint_as_float(u[q] << 16);
          v[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
        }
      } else {
        const float4* ga = reinterpret_cast<const float4*>(p.gu + (int64_t)pair * 2 * K + k0);
        const float4* up = reinterpret_cast<const float4*>(p.gu + (int64_t)pair * 2 * K + K + k0);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 a = __ldcg(ga + q), b = __ldcg(up + q);
          const float gv[4] = {a.x, a.y, a.z, a.w}, uv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float g = gv[r] * g13;
            v[4 * q + r] = g / (1.0f + __expf(-g)) * (uv[r] * g13);
          }
        }
      }
    }
    uint32_t mx = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) mx = max(mx, __float_as_uint(v[q]) & 0x7FFFFFFFu);
    mx = __reduce_max_sync(0xFFFFFFFFu, mx);
    // scale 2^(141 - e) takes the maximum, 2^(e - 127) .., to 2^14 ..
    const int e = max((int)(mx >> 23), 21);
    const float up = __uint_as_float((uint32_t)(268 - e) << 23);    // 2^(141 - e)
    const float down = __uint_as_float((uint32_t)(e - 14) << 23);   // 2^(e - 141)
    uint32_t h[4], l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float a = v[2 * q] * up, b = v[2 * q + 1] * up;
      const __half2 hv = __floats2half2_rn(a, b);
      h[q] = *reinterpret_cast<const uint32_t*>(&hv);
      if constexpr (kSplit) {
        const float2 r = __half22float2(hv);
        const __half2 lv = __floats2half2_rn(a - r.x, b - r.y);
        l[q] = *reinterpret_cast<const uint32_t*>(&lv);
      }
    }
    uint8_t* at = s_act + (size_t)s * T * 512 + moe_chunk(c, i, t);
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    if constexpr (kSplit) *reinterpret_cast<uint4*>(at + lo_off) = make_uint4(l[0], l[1], l[2], l[3]);
    if (lane == 0) s_mul[s * kMoeMulStride + c] = down;
  }
}

// A warp's loads of its steps [f0, f1) of a segment: step f is stage f %
// n_stages of the 16-row tile q0 + f / n_stages.  kMoeDepth of them are in
// flight, the first ones before the activations are built.
template <bool kWide>
struct MoeStream {
  const uint8_t *codes, *scales;
  int K, n_stages, tile, stage, left;
  MoeFrag ring[kMoeDepth];

  __device__ __forceinline__ void fetch(MoeFrag& a) {
    if (left > 0) {
      const int lane = threadIdx.x & 31, k0 = 256 * stage + 64 * (lane & 3);
      const int64_t r = (int64_t)tile * 16 + (lane >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        moe_load_row<kWide>(codes + (r + 8 * h) * (K / 2) + k0 / 2,
                            scales + (r + 8 * h) * (K / 16) + k0 / 16, K - k0, a.w[h], a.s[h]);
      --left;
      if (++stage == n_stages) {
        stage = 0;
        ++tile;
      }
    }
  }
  __device__ __forceinline__ void begin(const uint8_t* c, const uint8_t* s, int k, int ns, int q0,
                                        int f0, int f1) {
    codes = c;
    scales = s;
    K = k;
    n_stages = ns;
    tile = q0 + f0 / ns;
    stage = f0 % ns;
    left = f1 - f0;
#pragma unroll
    for (int d = 0; d < kMoeDepth; ++d) fetch(ring[d]);
  }
};

// The products of those steps.  Tiles the warp has from first to last stage
// go to dst; a first or last tile it shares goes to part[0] (begun by an
// earlier warp) or part[1] (begun here).
template <int kNT, bool kWide, bool kSplit>
__device__ __forceinline__ void moe_steps(MoeStream<kWide>& in, int N, int n_stages, int q0, int f0,
                                          int f1, int T, const int* list, const uint8_t* s_act,
                                          size_t lo_off, const float* s_mul, float* dst,
                                          float4* part, uint32_t& bad_scales) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float acc[kNT][4];
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
  int col[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n) col[n] = min(8 * n + g, T - 1);  // unused columns repeat the last
  int q = q0 + f0 / n_stages, s = f0 % n_stages;
  bool opened = s == 0;  // this warp has the current tile from its first stage

  auto flush = [&](bool closed) {
    if (opened && closed) {
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 8 * n + 2 * t + j;
          if (c < T) {
            float* o = dst + (int64_t)list[c] * N + q * 16 + g;
            o[0] = acc[n][j];
            o[8] = acc[n][2 + j];
          }
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
        part[((opened ? 1 : 0) * kMoeTileN + n) * 32 + lane] =
            make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
  };

  auto step = [&](const MoeFrag& a) {
    float c[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[n][j] = 0.0f;
    uint32_t sf[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bad_scales |= bad_scales4(a.s[h]);
      scales4_to_f16(a.s[h], sf[h][0], sf[h][1]);
    }
    const uint8_t* act = s_act + (size_t)s * T * 512;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t lo[4], hi[4];
      const int b = i >> 1;  // the lane's 16-weight block
      dequant8(a.w[0][i], b & 1 ? dup_hi(sf[0][b >> 1]) : dup_lo(sf[0][b >> 1]), lo);
      dequant8(a.w[1][i], b & 1 ? dup_hi(sf[1][b >> 1]) : dup_lo(sf[1][b >> 1]), hi);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const uint4 x = *reinterpret_cast<const uint4*>(act + moe_chunk(col[n], i, t));
        mma16816(c[n], lo[0], hi[0], lo[1], hi[1], x.x, x.y);
        mma16816(c[n], lo[2], hi[2], lo[3], hi[3], x.z, x.w);
        if constexpr (kSplit) {
          const uint4 y = *reinterpret_cast<const uint4*>(act + lo_off + moe_chunk(col[n], i, t));
          mma16816(c[n], lo[0], hi[0], lo[1], hi[1], y.x, y.y);
          mma16816(c[n], lo[2], hi[2], lo[3], hi[3], y.z, y.w);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const float2 m = *reinterpret_cast<const float2*>(s_mul + s * kMoeMulStride + 8 * n + 2 * t);
      acc[n][0] = __fmaf_rn(c[n][0], m.x, acc[n][0]);
      acc[n][1] = __fmaf_rn(c[n][1], m.y, acc[n][1]);
      acc[n][2] = __fmaf_rn(c[n][2], m.x, acc[n][2]);
      acc[n][3] = __fmaf_rn(c[n][3], m.y, acc[n][3]);
    }
    if (++s == n_stages) {
      flush(true);
      s = 0;
      ++q;
      opened = true;
    }
  };

  for (int f = f0; f < f1; f += kMoeDepth) {
#pragma unroll
    for (int d = 0; d < kMoeDepth; ++d) {
      if (f + d < f1) {
        step(in.ring[d]);
        in.fetch(in.ring[d]);
      }
    }
  }
  if (s != 0) flush(false);
}

template <int kStep, bool kWide>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_gemm_kernel(const MoeArgs p) {
  constexpr bool kSplit = kStep == 2;  // h; x is exact
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_cnt[kMoeMaxExperts];
  __shared__ int s_exp[kMoeMaxExperts];   // active experts
  __shared__ int s_seg[kMoeMaxExperts + 1];  // segments before each of them
  __shared__ int s_list[8 * kMoeTileN];
  __shared__ int s_active;
  __shared__ float4 s_part[kMoeWarps][2 * kMoeTileN * 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.M * p.k;
  const int N = kStep == 1 ? 2 * p.I : p.H, K = kStep == 1 ? p.H : p.I;
  const int n_stages = (K + 255) / 256, RT = N / 16;
  const int seg = kStep == 1 ? p.seg1 : p.seg2;
  float* s_mul = reinterpret_cast<float*>(smem);                             // [n_stages][kMoeMulStride]
  uint8_t* s_act = smem + (size_t)n_stages * kMoeMulStride * sizeof(float);
  const size_t lo_off = (size_t)n_stages * seg * 512;
  float* dst = kStep == 1 ? p.gu : p.y;

  // Step 1 waits for what the caller enqueued before; step 2's inputs other
  // than gu were complete before step 1 let it start.
  if constexpr (kStep == 1) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

  // ---- the experts that have pairs, and their segments
  if (P <= 32) {
    // a pair a lane, the experts in order of their first pair
    if (warp == 0) {
      const int e = lane < P ? __ldg(p.ids + lane) : -1;
      const bool valid = e >= 0 && e < p.E;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, valid ? e : -1);
      const bool leads = valid && (same & ((1u << lane) - 1u)) == 0u;
      const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
      const int n = leads ? (__popc(same) + seg - 1) / seg : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      if (leads) {
        const int at = __popc(leaders & ((1u << lane) - 1u));
        s_exp[at] = e;
        s_cnt[e] = __popc(same);
        s_seg[at] = incl - n;
      }
      if (lane == 31) {
        s_active = __popc(leaders);
        s_seg[__popc(leaders)] = incl;
      }
    }
    __syncthreads();
  } else {
    for (int e = tid; e < p.E; e += kMoeThreads) s_cnt[e] = 0;
    __syncthreads();
    for (int i = tid; i < P; i += kMoeThreads) {
      const int e = __ldg(p.ids + i);
      if (e >= 0 && e < p.E) atomicAdd(&s_cnt[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int a = 0, before = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < p.E ? (s_cnt[e] + seg - 1) / seg : 0;
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, n > 0);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += y;
        }
        if (n > 0) {
          const int at = a + __popc(bal & ((1u << lane) - 1u));
          s_exp[at] = e;
          s_seg[at] = before + incl - n;
        }
        a += __popc(bal);
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) {
        s_seg[a] = before;
        s_active = a;
      }
    }
    __syncthreads();
  }
  const int n_act = s_active;
  const int64_t total = (int64_t)s_seg[n_act] * RT;
  int64_t it = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  bool waited = kStep == 1;  // step 2 waits for gu with its first weights under way
  uint32_t bad_scales = 0;
  while (it < end) {
    const int sg = (int)(it / RT), q0 = (int)(it % RT);
    const int nq = (int)min((int64_t)(RT - q0), end - it);
    it += nq;
    // the segment's expert: the last whose segments begin at or before sg
    int lo = 0, hi = n_act - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_seg[mid] <= sg) lo = mid;
      else hi = mid - 1;
    }
    const int e = s_exp[lo];
    const int skip = (sg - s_seg[lo]) * seg;
    const int T = min(seg, s_cnt[e] - skip);
    // its pairs, in order
    if (warp == 0) {
      int seen = 0;
      for (int i0 = 0; i0 < P && seen < skip + T; i0 += 32) {
        const bool mine = i0 + lane < P && __ldg(p.ids + i0 + lane) == e;
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, mine);
        const int at = seen + __popc(bal & ((1u << lane) - 1u)) - skip;
        if (mine && at >= 0 && at < T) s_list[at] = i0 + lane;
        seen += __popc(bal);
      }
    }
    const int steps = nq * n_stages;
    auto first = [&](int w) { return (int)((int64_t)steps * w / kMoeWarps); };
    const int f0 = first(warp), f1 = first(warp + 1);
    MoeStream<kWide> in;
    in.begin((kStep == 1 ? p.p13 : p.p2) + (int64_t)e * N * (K / 2),
             (kStep == 1 ? p.s13 : p.s2) + (int64_t)e * N * (K / 16), K, n_stages, q0, f0, f1);
    if (!waited) {
      grid_dependency_wait();
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      waited = true;
    }
    __syncthreads();
    moe_build<kStep, kSplit>(p, s_list, T, n_stages, __ldg(p.g13 + e), s_act, lo_off, s_mul);
    __syncthreads();
    if (f0 < f1) {
      auto go = [&](auto nt) {
        moe_steps<decltype(nt)::value, kWide, kSplit>(in, N, n_stages, q0, f0, f1, T, s_list, s_act,
                                                      lo_off, s_mul, dst, s_part[warp], bad_scales);
      };
      if (T <= 8) go(std::integral_constant<int, 1>{});
      else if (T <= 16) go(std::integral_constant<int, 2>{});
      else go(std::integral_constant<int, 4>{});
    }
    __syncthreads();
    // tiles cut between warps: the warp that opened one adds the others'
    // parts in warp order
    if (f1 > f0 && f1 < steps && f1 % n_stages != 0 && f1 / n_stages * n_stages >= f0) {
      const int q = f1 / n_stages, close = (q + 1) * n_stages;
      const int g = lane >> 2, t = lane & 3;
      for (int n = 0; n * 8 < T; ++n) {
        float4 sum = s_part[warp][(kMoeTileN + n) * 32 + lane];
        for (int w = warp + 1; w < kMoeWarps && first(w) < close; ++w) {
          if (first(w) == first(w + 1)) continue;
          const float4 v = s_part[w][n * 32 + lane];
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        const int c = 8 * n + 2 * t;
        float* o = dst + (q0 + q) * 16 + g;
        if (c < T) {
          o[(int64_t)s_list[c] * N] = sum.x;
          o[(int64_t)s_list[c] * N + 8] = sum.z;
        }
        if (c + 1 < T) {
          o[(int64_t)s_list[c + 1] * N] = sum.y;
          o[(int64_t)s_list[c + 1] * N + 8] = sum.w;
        }
      }
    }
    if (it < end) __syncthreads();
  }
  if (!waited) {  // no work here: the flags below are read after this kernel all the same
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const int bad = __syncthreads_or(bad_scales != 0u);
  if (tid == 0) p.bad_flags[(kStep - 1) * gridDim.x + blockIdx.x] = bad;
}

// out[m, :] = sum over the slots j of w[m, j] G2[e] y[m k + j, :], four
// columns a thread; the row of CTAs past the tokens reads the flags.
template <bool kBf16>
__global__ void __launch_bounds__(256) moe_combine_kernel(const MoeArgs p, int n_flags) {
  const int m = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  if (m == p.M) {
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x != 0) return;
    int bad = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n_flags; i += blockDim.x) bad |= __ldcg(p.bad_flags + i);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? NVFP4_ERR_NONFINITE : NVFP4_OK;
    return;
  }
  constexpr int kAt = 8;  // slots whose loads are in flight together
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  bool waited = false;
  for (int j0 = 0; j0 < p.k; j0 += kAt) {
    float w[kAt];
    bool live[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int64_t pair = (int64_t)m * p.k + j0 + j;
      const int e = j0 + j < p.k ? __ldg(p.ids + pair) : -1;
      live[j] = e >= 0 && e < p.E;
      w[j] = live[j] ? __ldg(p.weights + pair) * __ldg(p.g2 + e) : 0.0f;
    }
    if (!waited) {
      grid_dependency_wait();
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      waited = true;
    }
    float4 v[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j)
      if (live[j] && 4 * c < p.H)
        v[j] = __ldcg(reinterpret_cast<const float4*>(p.y + ((int64_t)m * p.k + j0 + j) * p.H) + c);
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (live[j]) {
        sum.x = __fmaf_rn(w[j], v[j].x, sum.x);
        sum.y = __fmaf_rn(w[j], v[j].y, sum.y);
        sum.z = __fmaf_rn(w[j], v[j].z, sum.z);
        sum.w = __fmaf_rn(w[j], v[j].w, sum.w);
      }
    }
  }
  if (4 * c < p.H) {
    const int64_t at = ((int64_t)m * p.H >> 2) + c;
    if constexpr (kBf16) {
      uint2 o;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(sum.y), "f"(sum.x));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(sum.w), "f"(sum.z));
      reinterpret_cast<uint2*>(p.out)[at] = o;
    } else {
      reinterpret_cast<float4*>(p.out)[at] = sum;
    }
  }
}

// ------------------------------------------------------------ host side
struct MoeLayout {
  size_t flags, gu, y, total;
};

static MoeLayout moe_layout(int64_t pairs, int64_t H, int64_t I, int sms) {
  MoeLayout L;
  L.flags = kWsHeader;
  L.gu = align_up(L.flags + (size_t)4 * sms * sizeof(int32_t), 256);
  L.y = align_up(L.gu + (size_t)pairs * 2 * I * sizeof(float), 256);
  L.total = align_up(L.y + (size_t)pairs * H * sizeof(float), 256);
  return L;
}

size_t moe_tc_workspace_bytes(int64_t M, int64_t k, int64_t H, int64_t I);
bool moe_tc_takes(int64_t k, int64_t H, int64_t I);
nvfp4_status moe_tc_launch(const void* x, int64_t M, int64_t k, int64_t H, int64_t I, int64_t E,
                           const int32_t* ids, const float* weights, const uint8_t* p13,
                           const uint8_t* s13, const float* g13, const uint8_t* p2,
                           const uint8_t* s2, const float* g2, void* out, int out_dtype,
                           void* workspace, cudaStream_t stream);

// The FP4 tensor-core route (moe_tc.cu: five kernels instead of three, but 7
// TB/s between them) is taken for more weight than about 85 MB counted once
// per pair (27/16 byte per element of an H x I matrix), or for 6 pairs an
// expert, where the products here turn from bandwidth to issue bound.
// Measured (here / there): H 2048, I 768, top 8 of 128: 1 token 14.9 / 23.7 us,
// 3 tokens 30.4 / 30.0, 4 tokens 34.7 / 33.0, 6 tokens 43.0 / 37.2; H = I = 2880,
// top 4 of 32: 1 token 29.4 / 30.6, 2 tokens 46.5 / 37.6; H 1024, I 512, top 2 of
// 64: 16 tokens 18.3 / 20.8, 32 tokens 24.3 / 23.3, 48 tokens 29.8 / 25.4; H 512,
// I 256, top 2 of 16: 32 tokens 16.6 / 17.1, 48 tokens 17.6 / 17.7, 128 tokens
// 33.7 / 21.0.  With P H I from 32M to the threshold the routes are within 5%.
constexpr int64_t kMoeFewWork = 48 << 20;
constexpr int64_t kMoeFewPairs = 6;
static bool moe_use_tc(int64_t M, int64_t k, int64_t H, int64_t I, int64_t E) {
  const int64_t P = M * k;
  return (P * H * I >= kMoeFewWork || P >= kMoeFewPairs * E) && moe_tc_takes(k, H, I);
}

// Enough for either route: which one is taken depends on E too.
size_t moe_workspace_bytes(int64_t M, int64_t k, int64_t H, int64_t I) {
  const size_t few = moe_layout(M * k, H, I, std::max(sm_count(), 1)).total;
  return moe_tc_takes(k, H, I) ? std::max(few, moe_tc_workspace_bytes(M, k, H, I)) : few;
}

// Bytes of a pair's activations in a stage: x as one fp16, h as two.
static int64_t moe_stage_bytes(int step) { return step == 1 ? 512 : 1024; }

// Pairs of a segment: what fits the activation budget, in whole tiles of 8
// where more than one does, but never more than an expert can have.
static int moe_segment(int64_t K, int64_t pairs, int step) {
  const int64_t row = (K + 255) / 256 * moe_stage_bytes(step);
  int64_t n = (int64_t)kMoeActBytes / row;
  n = n >= 8 ? std::min<int64_t>(n / 8 * 8, 8 * kMoeTileN) : std::max<int64_t>(n, 1);
  return (int)(n >= 8 ? n : std::min(n, pairs));
}

static size_t moe_smem(int64_t K, int seg, int step) {
  const int64_t stages = (K + 255) / 256;
  return (size_t)stages * (kMoeMulStride * sizeof(float) + (size_t)seg * moe_stage_bytes(step));
}

template <int kStep>
static cudaError_t moe_gemm_launch(const MoeArgs& a, bool wide, int grid, cudaStream_t stream) {
  const size_t smem = moe_smem(kStep == 1 ? a.H : a.I, kStep == 1 ? a.seg1 : a.seg2, kStep);
  auto kern = wide ? moe_gemm_kernel<kStep, true> : moe_gemm_kernel<kStep, false>;
  static std::atomic<uint64_t> limit_set[2];
  const cudaError_t err = smem_limit_once(limit_set[wide], reinterpret_cast<const void*>(kern),
                                          moe_smem(NVFP4_MOE_MAX_DIM, 1, 2));
  if (err != cudaSuccess) return err;
  PdlLaunch l(dim3((unsigned)grid), dim3(kMoeThreads), smem, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a);
}

nvfp4_status moe_launch(const void* x, int64_t M, int64_t k, int64_t H, int64_t I, int64_t E,
                        const int32_t* ids, const float* weights, const uint8_t* p13,
                        const uint8_t* s13, const float* g13, const uint8_t* p2,
                        const uint8_t* s2, const float* g2, void* out, int out_dtype,
                        void* workspace, cudaStream_t stream) {
  if (moe_use_tc(M, k, H, I, E))
    return moe_tc_launch(x, M, k, H, I, E, ids, weights, p13, s13, g13, p2, s2, g2, out, out_dtype,
                         workspace, stream);
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const MoeLayout L = moe_layout(M * k, H, I, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.ids = ids;
  a.weights = weights;
  a.p13 = p13;
  a.s13 = s13;
  a.g13 = g13;
  a.p2 = p2;
  a.s2 = s2;
  a.g2 = g2;
  a.out = out;
  a.gu = reinterpret_cast<float*>(ws + L.gu);
  a.y = reinterpret_cast<float*>(ws + L.y);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.bad_flags = reinterpret_cast<int32_t*>(ws + L.flags);
  a.M = (int)M;
  a.k = (int)k;
  a.H = (int)H;
  a.I = (int)I;
  a.E = (int)E;
  a.seg1 = moe_segment(H, M * k, 1);
  a.seg2 = moe_segment(I, M * k, 2);
  // whole 32-byte pieces of every row
  auto wide = [](const uint8_t* codes, const uint8_t* scales, int64_t K) {
    return K % 64 == 0 && reinterpret_cast<uintptr_t>(codes) % 32 == 0 &&
           reinterpret_cast<uintptr_t>(scales) % 4 == 0;
  };
  const int grid = 2 * sms;
  cudaError_t err = moe_gemm_launch<1>(a, wide(p13, s13, H), grid, stream);
  if (err == cudaSuccess) err = moe_gemm_launch<2>(a, wide(p2, s2, I), grid, stream);
  if (err == cudaSuccess) {
    PdlLaunch l(dim3((unsigned)((H / 4 + 255) / 256), (unsigned)M + 1), dim3(256), 0, stream);
    err = out_dtype == NVFP4_OUT_BF16
              ? cudaLaunchKernelEx(&l.cfg, moe_combine_kernel<true>, a, 2 * grid)
              : cudaLaunchKernelEx(&l.cfg, moe_combine_kernel<false>, a, 2 * grid);
  }
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
