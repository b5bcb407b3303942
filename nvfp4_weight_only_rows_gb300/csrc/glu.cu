// glu.cu -- the gated half of a feed-forward block on an NVFP4 weight, and its
// gradient: with W13 = [gate rows; up rows],
//   g = W13[0:I] x,  u = W13[I:2I] x,  h = act(g) u,
//   dg = dh u act'(g),  du = dh act(g),  dx = [dg | du] W13.
//
// Forward: one product kernel (w4a16_tc_kernel) whose 128-row units are 64 gate
// rows and the 64 up rows of the same places, 16 of each in a warp's 32 TMEM
// lanes.  A pair meets by one shuffle a value: of 16 tokens the gate's lane
// finishes the first eight, the up's lane the others.  g and u never leave the
// chip, and W13 is read once.
//
// Backward: the same product again (g and u are not kept: they would be
// 4 I bytes a token), which writes dg and du as fp16 to the workspace, then
// the product back through W13 (back.cu).  fp16 needs a power of two per token
// that no value overflows: |g|, |u| <= |x|_1 max|W13| and max|W13| <= 2688
// global, |act(v)| <= |v|, |act'| < 1.13, so |dg|, |du| < 1.13 max|dh| |x|_1
// 2688 |global|.  The bound is loose by about 2^10 for normal activations and
// weights, and taking it by exponents costs up to 2^4 more; fp16's 40 binades
// from 2^15 down to its last subnormal leave 2^-25 of it at full precision, 11
// bits, and an error of 2^-36 of it below.
#include "back.cuh"
#include "prologue.cuh"
#include "w4a16_tc.cuh"

namespace nvfp4 {

// act(g) and, for the gradient, act'(g).
template <int kAct, bool kGrad>
__device__ __forceinline__ float activation(float g, float* slope) {
  if constexpr (kAct == NVFP4_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + expf(-g));
    if (kGrad) *slope = s * (1.0f + g * (1.0f - s));
    return g * s;
  } else {
    constexpr float c2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    constexpr float cube = 0.044715f;
    const float s = __fdividef(1.0f, 1.0f + expf(-c2 * (g + cube * g * g * g)));
    if (kGrad) {
      // beyond 30 the second term is 0; its factors would overflow
      const float b = fminf(fmaxf(g, -30.0f), 30.0f);
      *slope = s + b * s * (1.0f - s) * c2 * (1.0f + 3.0f * cube * b * b);
    }
    return g * s;
  }
}

struct GluArgs {
  int64_t I;
  void* out;            // [M, I]
  // the gradient
  const void* dh;       // [M, I]
  const float* up2;     // [M] the power of two that dg and du are stored times
  __half* d16;          // [tokens, stride]: dg then du
  int64_t stride;
};

// kGrad: dg and du to d16 from dh; else h to out.  kBf16: dh's or h's type.
template <int kAct, bool kGrad, bool kBf16, int kWarps>
struct GluEpilogue {
  static constexpr int kWideWarps = kWarps;
  static constexpr bool kOwn = true, kPaired = true;
  static constexpr int kFirstPart = 0, kNextPart = 0;
  static constexpr int kInfoBytes = (kGrad ? 2 : 1) * kMaxBN * 4;
  int64_t half;  // rows from a gate to its up
  int staged;    // the weight is read from a copy in the workspace
  GluArgs a;
  struct Unit {
    int64_t i;     // column of h
    int64_t t;     // this lane's first token of a chunk
    bool valid;
    float dh[kGrad ? 8 : 1];  // of the next chunk
  };

  // dh of this lane's eight tokens of a chunk
  __device__ void load(const GemmArgs& p, Unit& u, int c) const {
    const int64_t t0 = u.t + c, live = u.valid && c < p.BN ? p.M - t0 : 0;
    const int64_t at = t0 * a.I + u.i;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u.dh[j] = 0.0f;
      if (j >= live) continue;
      if constexpr (kBf16)
        u.dh[j] = __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(a.dh) + at + j * a.I));
      else
        u.dh[j] = __ldg(static_cast<const float*>(a.dh) + at + j * a.I);
    }
  }

  __device__ Unit unit(const GemmArgs& p, uint32_t u, int q, int lane, int c0) const {
    const uint32_t tile = u / (uint32_t)p.n_ttiles;
    const int64_t t0 = (int64_t)(u - tile * (uint32_t)p.n_ttiles) * p.BN;
    const int64_t i = (int64_t)tile * 64 + q * 16 + (lane & 15);
    Unit r = {i, t0 + (lane & 16) / 2, i < a.I};
    if constexpr (kGrad) load(p, r, c0);
    return r;
  }

  __device__ void info(const GemmArgs& p, uint32_t u, int lane, uint8_t* s) const {
    float* mul = reinterpret_cast<float*>(s);
    const int64_t t0 = (int64_t)(u % (uint32_t)p.n_ttiles) * p.BN;
    float scale[kMaxBN / 32], up2[kMaxBN / 32];
#pragma unroll
    for (int i = 0; i < kMaxBN / 32; ++i) {  // all loads in flight together
      const int t = lane + 32 * i;
      const bool live = t < p.BN && t0 + t < p.M;
      scale[i] = live ? __ldcg(p.tok_scale + t0 + t) : 0.0f;
      up2[i] = kGrad && live ? __ldcg(a.up2 + t0 + t) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kMaxBN / 32; ++i) {
      mul[lane + 32 * i] = scale[i];
      if (kGrad) mul[kMaxBN + lane + 32 * i] = up2[i];
    }
  }

  __device__ void chunk(const GemmArgs& p, Unit& u, int c, int c_next, const float (&v)[16],
                        int lane, const uint8_t* s) const {
    const bool up = (lane & 16) != 0;
    const int64_t t0 = u.t + c;
    const int64_t live = u.valid ? p.M - t0 : 0;
    float dh[kGrad ? 8 : 1];
    if constexpr (kGrad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dh[j] = u.dh[j];
      load(p, u, c_next);
    }
    float mul[16];
    lds_f32x16(reinterpret_cast<const float*>(s) + c, mul);
    float mine[8], other[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float lo = v[j] * mul[j], hi = v[j + 8] * mul[j + 8];
      mine[j] = up ? hi : lo;
      other[j] = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, 16);
    }
    const float* p2 = reinterpret_cast<const float*>(s) + kMaxBN + c + (up ? 8 : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g = up ? other[j] : mine[j], w = up ? mine[j] : other[j];
      float slope = 0.0f;
      const float act = activation<kAct, kGrad>(g, &slope);
      if (j >= live) continue;
      if constexpr (kGrad) {
        const float d = dh[j] * p2[j];
        __half* o = a.d16 + (t0 + j) * a.stride + u.i;
        o[0] = __float2half_rn(d * w * slope);
        o[a.I] = __float2half_rn(d * act);
      } else if constexpr (kBf16) {
        static_cast<__nv_bfloat16*>(a.out)[(t0 + j) * a.I + u.i] = __float2bfloat16_rn(act * w);
      } else {
        static_cast<float*>(a.out)[(t0 + j) * a.I + u.i] = act * w;
      }
    }
  }
};

// ------------------------------------------------------------ host side
// Workspace: [status header][fp16 x][token multipliers][partials of cut
// units][their counters and flags][staged weight rows]; for the gradient also
// [powers of two][factors][dg and du] before the partials, and the product
// back's sums after the flags.
struct GluLayout {
  size_t x16, tok, up2, factor, d16, split_part, cnt, ready, end;
  int64_t stride;
  int BN, grid, n_flags;
  BackLayout back;
};

static GluLayout glu_layout(int64_t M, int64_t I, int64_t K, bool grad, int sms) {
  GluLayout l;
  l.BN = train_token_tile(M);
  const int64_t m_pad = (M + l.BN - 1) / l.BN * l.BN;
  l.grid = (int)std::min<int64_t>(sms, ((I + 63) / 64) * (m_pad / l.BN));
  l.stride = (2 * I + 7) / 8 * 8;
  l.x16 = kWsHeader;
  l.tok = l.x16 + align_up((size_t)m_pad * K * 2, 1024);
  l.up2 = l.tok + align_up((size_t)m_pad * 4, 256);
  l.factor = l.up2 + (grad ? align_up((size_t)M * 4, 256) : 0);
  l.d16 = l.factor + (grad ? align_up((size_t)M * 4, 256) : 0);
  l.split_part = l.d16 + (grad ? align_up((size_t)m_pad * l.stride * 2, 256) : 0);
  l.cnt = l.split_part + align_up((size_t)l.grid * 4 * l.BN * 32 * 4, 256);
  l.ready = l.cnt + align_up((size_t)l.grid * 16 * 4, 256);
  l.end = l.ready + align_up((size_t)l.grid * 16 * 4, 256);
  l.n_flags = (int)((l.end - l.cnt) / 4);
  l.back = {};
  if (grad) {
    l.back = back_layout(M, 2 * I, K, sms, l.end);
    l.end = l.back.total;
  }
  return l;
}

static int64_t glu_chunk(int64_t M, int64_t I, int64_t K, bool grad) {
  return chunk_tokens(M, std::max(K * 2, grad ? (2 * I + 7) / 8 * 16 : (int64_t)0));
}

static WeightStage glu_stage(int64_t M, int64_t I, int64_t K, bool grad, int sms) {
  const int64_t chunk = glu_chunk(M, I, K, grad);
  size_t end = glu_layout(chunk, I, K, grad, sms).end;
  if (M % chunk) end = std::max(end, glu_layout(M % chunk, I, K, grad, sms).end);
  return weight_stage(2 * I, K, end, true);
}

size_t glu_workspace_bytes(int64_t M, int64_t I, int64_t K, bool grad) {
  return glu_stage(M, I, K, grad, std::max(sm_count(), 1)).total;
}

template <int kAct, bool kGrad, bool kBf16>
static cudaError_t glu_gemm(const GluArgs& ga, bool staged, const CUtensorMap& tm_packed,
                            const CUtensorMap& tm_scales, const CUtensorMap& tm_x,
                            const GemmArgs& a, int grid, cudaStream_t stream) {
  GluEpilogue<kAct, kGrad, kBf16, 8> few;
  few.half = ga.I;
  few.staged = staged;
  few.a = ga;
  if (a.BN <= kDeepTokens)
    return launch_gemm_with<3, 6, 3>(few, tm_packed, tm_scales, tm_x, a, grid, stream);
  if constexpr (kGrad) {  // (forward, 8 warps are level with 16 for short sums, too)
    if (a.n_kb <= kManyWarpStages) {
      const GluEpilogue<kAct, kGrad, kBf16, 16> many{ga.I, staged, ga};
      return launch_gemm_with<2, 4, 2>(many, tm_packed, tm_scales, tm_x, a, grid, stream);
    }
  }
  return launch_gemm_with<2, 4, 2>(few, tm_packed, tm_scales, tm_x, a, grid, stream);
}

template <int kAct, bool kGrad>
static cudaError_t glu_gemm_typed(bool bf16, const GluArgs& ga, bool staged, const CUtensorMap& tm_packed,
                                  const CUtensorMap& tm_scales, const CUtensorMap& tm_x,
                                  const GemmArgs& a, int grid, cudaStream_t stream) {
  return bf16 ? glu_gemm<kAct, kGrad, true>(ga, staged, tm_packed, tm_scales, tm_x, a, grid, stream)
              : glu_gemm<kAct, kGrad, false>(ga, staged, tm_packed, tm_scales, tm_x, a, grid, stream);
}

// dh null: h to out.  dtype: h's or dh's; out_dtype: dx's.
nvfp4_status glu_launch(const void* x, int64_t M, int64_t K, const uint8_t* packed,
                        const uint8_t* scales, const float* global, int64_t I, int act,
                        const void* dh, int dtype, void* out, int out_dtype, void* workspace,
                        cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const bool grad = dh != nullptr;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const WeightStage wst = glu_stage(M, I, K, grad, sms);
  const bool staged = wst.packed || wst.scales;
  CUtensorMap tm_packed, tm_scales, tm_x;
  if (!encode_weight_maps(&tm_packed, &tm_scales, wst, packed, scales, 2 * I, K, ws, kRows / 2))
    return NVFP4_ERR_CUDA;
  const int64_t chunk = glu_chunk(M, I, K, grad);
  const bool bf16 = dtype == NVFP4_OUT_BF16;
  const size_t size = bf16 ? 2 : 4, out_size = out_dtype == NVFP4_OUT_BF16 ? 2 : 4;
  for (int64_t m0 = 0; m0 < M; m0 += chunk) {
    const int64_t rows = std::min(chunk, M - m0);
    const GluLayout L = glu_layout(rows, I, K, grad, sms);
    const int64_t n_tt = (rows + L.BN - 1) / L.BN;
    const uint8_t* xs = static_cast<const uint8_t*>(x) + (size_t)m0 * K * 2;
    const uint8_t* dhs = grad ? static_cast<const uint8_t*>(dh) + (size_t)m0 * I * size : nullptr;
    __half* x16 = reinterpret_cast<__half*>(ws + L.x16);
    float* tok = reinterpret_cast<float*>(ws + L.tok);
    float* up2 = reinterpret_cast<float*>(ws + L.up2);
    float* factor = reinterpret_cast<float*>(ws + L.factor);
    Prologue pro = {};
    pro.x = reinterpret_cast<const uint16_t*>(xs);
    pro.M = rows;
    pro.K = K;
    pro.m_rows = n_tt * L.BN;
    pro.x16 = x16;
    pro.tok_scale = tok;
    pro.dh = dhs;
    pro.n_dh = grad ? rows : 0;
    pro.I = I;
    pro.up2 = up2;
    pro.factor = factor;
    pro.grad_bf16 = bf16;
    pro.global = global;
    pro.flags = reinterpret_cast<uint32_t*>(ws + L.cnt);
    pro.n_flags = L.n_flags;
    if (m0 == 0) {
      pro.status = reinterpret_cast<int32_t*>(ws);
      prologue_weights(pro, wst, packed, scales, 2 * I, K, ws);
    }
    cudaError_t e = prologue_launch(pro, stream);
    if (e != cudaSuccess) return NVFP4_ERR_CUDA;
    if (!encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x16, (uint64_t)K,
                   (uint64_t)(n_tt * L.BN), (uint64_t)K * 2, 64, (uint32_t)L.BN,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return NVFP4_ERR_CUDA;
    GemmArgs a = {};
    a.M = rows;
    a.N = 2 * I;
    a.K = K;
    a.BN = L.BN;
    a.n_ttiles = (int)n_tt;
    a.n_units = ((I + 63) / 64) * n_tt;
    a.n_kb = (int)((K + kKB - 1) / kKB);
    schedule_units(a, L.grid);
    a.tok_scale = tok;
    a.status = reinterpret_cast<int32_t*>(ws);
    a.split_cnt = reinterpret_cast<uint32_t*>(ws + L.cnt);
    a.split_ready = reinterpret_cast<uint32_t*>(ws + L.ready);
    a.split_part = reinterpret_cast<float*>(ws + L.split_part);
    const int stages = L.BN <= kDeepTokens ? 3 : 2;
    a.dbuf_log2 = (4 * L.BN + stages * (kKB / 2) <= 512) ? 2u : 1u;
    a.tmem_cols = ((L.BN << a.dbuf_log2) + stages * (kKB / 2) <= 256) ? 256u : 512u;
    GluArgs ga = {};
    ga.I = I;
    ga.out = grad ? nullptr : static_cast<uint8_t*>(out) + (size_t)m0 * I * size;
    ga.dh = dhs;
    ga.up2 = up2;
    ga.d16 = reinterpret_cast<__half*>(ws + L.d16);
    ga.stride = L.stride;
    if (act == NVFP4_ACT_SILU)
      e = grad ? glu_gemm_typed<NVFP4_ACT_SILU, true>(bf16, ga, staged, tm_packed, tm_scales, tm_x, a,
                                                      L.grid, stream)
               : glu_gemm_typed<NVFP4_ACT_SILU, false>(bf16, ga, staged, tm_packed, tm_scales, tm_x, a,
                                                       L.grid, stream);
    else
      e = grad ? glu_gemm_typed<NVFP4_ACT_GELU_TANH, true>(bf16, ga, staged, tm_packed, tm_scales, tm_x, a,
                                                           L.grid, stream)
               : glu_gemm_typed<NVFP4_ACT_GELU_TANH, false>(bf16, ga, staged, tm_packed, tm_scales, tm_x,
                                                            a, L.grid, stream);
    if (e == cudaSuccess && grad) {
      const BackCall c{rows, 2 * I, K, ga.d16, L.stride, packed, scales, &wst, factor,
                       static_cast<uint8_t*>(out) + (size_t)m0 * K * out_size, out_dtype, false};
      e = back_launch(c, L.back, ws, stream);
    }
    if (e != cudaSuccess) return NVFP4_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
