// lm_head.cu -- the weight-only W4A16 lm_head product on sm_103a tensor cores.
//
// logits[m, n] = global * sum_k x[m, k] * e2m1(code[n, k]) * f32(scale[n, k/16])
// (`CompressedTensorsW4A16Fp4.apply_weights` on the page
// "vllm.model_executor.layers.quantization.compressed_tensors.schemes", with
// the checkpoint layout `_quantize_nvfp4` writes on the page
// "vllm.model_executor.layers.quantization.online.lm_head").
//
// Two kernels per call (the second launched as a programmatic dependent of
// the first, so it streams weights while the first finishes):
//  1. w4a16_prep_x_kernel: each token row of x (bf16) is rescaled by an
//     exact power of two 2^e so that its largest magnitude lands in
//     [2^14, 2^15), and stored as fp16 in the workspace; the token's output
//     multiplier global * 2^-e is stored beside it.  fp16 holds every bf16
//     value of that row exactly down to 2^-28 of the row maximum.
//  2. w4a16_tc_kernel: a persistent, warp-specialized tcgen05 GEMM in the
//     swapped orientation D[vocab row, token] = A . B^T:
//       A = dequantized weights, 128 vocabulary rows x 256 k per stage, held
//           in TENSOR MEMORY (the "ts" MMA form), written by eight dequant
//           warps with one thread per row and half a stage per warp: e2m1
//           pairs -> fp16 pairs with the hardware cvt, times the E4M3 block
//           scale (fp16, exact);
//       B = the fp16 activations, four TMA boxes [BN tokens x 64 k] per
//           stage in shared memory with the 128-byte swizzle;
//       D = fp32 accumulators in tensor memory, double buffered, drained by
//           four epilogue warps (tcgen05.ld, x token multiplier, store).
//     Packed codes and scales arrive by TMA in 256-k stages; every product
//     x * w is exact in fp32, so the only rounding is the fp32 summation.
//
// Warp roles (480 threads): 0 packed/scale TMA producer, 1 activation TMA
// producer, 2 MMA issuer (and TMEM owner), 3-10 dequant (two warps per TMEM
// lane quadrant taking 256-k stages in turn), 11-14 epilogue.  The producer
// and MMA warps run warp-uniform loops and issue from one elected lane.
// Every pipeline wait is bounded in time; on expiry the CTA raises
// NVFP4_ERR_TIMEOUT in the workspace status word, drains what it issued and
// returns.
#include "w4a16_tc.cuh"

namespace nvfp4 {

// The plain product's stream-K tail gives the CTAs of higher index (which
// enter later: the first MMA of a decode call comes 2.8 to 5.6 us after the
// first CTA's entry, correlated 0.8 with the index at M = 64) fewer stages,
// up to 4/64 of the mean less (the skew bound passed to schedule_units).
// Same box, the four decode calls M = 1, 8, 32, 64: 224.4 -> 223.5 us; M = 8
// alone 52.8 -> 51.7 us; a skew of 8 gave 224.6 us, of 12 227.1 us.
constexpr uint32_t kDecodeTailSkew = 4;

// ------------------------------------------------------------ activations
// kWarpsPerRow warps per token row (4, with a 128-thread CTA per row, for
// few rows, where the latency of one row is what counts and the CTA must
// fit beside a GEMM CTA on its SM; 1: a warp per row, 8 rows per 256-thread
// CTA, for many rows); rows m_rows and beyond do not exist, rows
// M .. m_rows-1 are zero padding.
template <int kWarpsPerRow>
__global__ void __launch_bounds__(256) w4a16_prep_x_kernel(const uint16_t* __restrict__ x,
                                                           int64_t M, int64_t K, int64_t m_rows,
                                                           const float* __restrict__ global,
                                                           __half* __restrict__ x16,
                                                           float* __restrict__ tok_scale,
                                                           int32_t* __restrict__ status,
                                                           uint32_t* __restrict__ split_flags,
                                                           int n_split_flags,
                                                           unsigned long long* __restrict__ am_keys,
                                                           uint32_t* __restrict__ tk_hist,
                                                           int tk_hstride,
                                                           const int32_t* __restrict__ grp_off,
                                                           const float* __restrict__ grp_global,
                                                           int n_groups) {
  // launched as a programmatic dependent of whatever ran before it: wait for
  // that kernel's results before touching memory (the previous call's GEMM
  // may still be reading this workspace)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the GEMM may launch now: it waits for this grid's results (griddepcontrol.wait)
  // only where it reads them, and streams the weights meanwhile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {  // a fresh call: clear the status word and the split-K flags
    if (threadIdx.x == 0) *status = NVFP4_OK;
    for (int i = threadIdx.x; i < n_split_flags; i += blockDim.x) split_flags[i] = 0;
  }
  __shared__ int32_t s_grp[kMaxGroups + 1];
  if (grp_off) {  // grouped: the group offsets, loaded by the whole block
    for (int e = threadIdx.x; e <= n_groups; e += blockDim.x) s_grp[e] = grp_off[e];
    __syncthreads();
  }
  constexpr int kT = 32 * kWarpsPerRow;  // threads of one row
  const int lane = threadIdx.x % kT;
  const int64_t m = (int64_t)blockIdx.x * (blockDim.x / kT) + threadIdx.x / kT;
  if (m >= m_rows) return;  // uniform over the row's threads
  token_state_clear(am_keys, tk_hist, tk_hstride, m, lane, kT);  // argmax / top-k: nothing seen yet
  uint4* d4 = reinterpret_cast<uint4*>(x16 + m * K);
  const int64_t nv = K / 8;
  if (m >= M) {  // padding rows of the last token tile
    for (int64_t i = lane; i < nv; i += kT) d4[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(x + m * K);
  uint32_t mx = 0;
  for (int64_t i = lane; i < nv; i += kT) {
    const uint4 v = src[i];
    const uint32_t k = 0x7FFF7FFFu;
    mx = __vmaxu2(mx, v.x & k);
    mx = __vmaxu2(mx, v.y & k);
    mx = __vmaxu2(mx, v.z & k);
    mx = __vmaxu2(mx, v.w & k);
  }
  mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if constexpr (kWarpsPerRow > 1) {  // the CTA is one row: combine its warps
    __shared__ uint32_t red[kWarpsPerRow];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = 0;
    for (int w = 0; w < kWarpsPerRow; ++w) mx = max(mx, red[w]);
  }
  int e = 0;
  if (mx != 0 && mx < 0x7F80u) {
    const int E = ilogbf(__uint_as_float(mx << 16));  // floor(log2(max|x|))
    e = min(max(14 - E, -126), 126);
  }
  if (lane == 0) {
    float gw;
    if (grp_off) {  // grouped: the global of the group holding token row m
      int lo = 0, hi = n_groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_grp[mid] <= m) lo = mid; else hi = mid;
      }
      gw = (s_grp[lo] <= m && m < s_grp[lo + 1]) ? grp_global[lo] : 0.0f;
    } else {
      gw = *global;
    }
    tok_scale[m] = __fmul_rn(gw, __int_as_float((127 - e) << 23));
  }
  const float p2 = __int_as_float((127 + e) << 23);
  for (int64_t i = lane; i < nv; i += kT) {
    const uint4 v = src[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = __fmul_rn(__uint_as_float(w[j] << 16), p2);
      const float hi = __fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), p2);
      __half2 h = __floats2half2_rn(lo, hi);
      o[j] = *reinterpret_cast<uint32_t*>(&h);
    }
    d4[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------ weight rows
// Row copy into a TMA-readable stride (see WeightStage): one warp per row,
// in units of T (8 bytes for NVFP4 code rows, which K % 16 makes 8-byte
// multiples; 1 byte for block-scale rows).  Launched as a programmatic
// dependent: the weights may have been written by the kernel before it.
template <typename T>
__global__ void __launch_bounds__(256) stage_rows_kernel(const T* __restrict__ src, int64_t rows,
                                                         int64_t row_elems, T* __restrict__ dst,
                                                         int64_t dst_stride_elems) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows;
       r += warps) {
    const T* s = src + r * row_elems;
    T* d = dst + r * dst_stride_elems;
    for (int64_t j = lane; j < row_elems; j += 32) d[j] = s[j];
  }
}

cudaError_t stage_rows_launch(const uint8_t* src, int64_t rows, int64_t row_bytes, uint8_t* dst,
                              int64_t dst_stride, cudaStream_t stream) {
  const int sms = std::max(sm_count(), 1);
  const int64_t blocks = std::min<int64_t>((rows + 7) / 8, (int64_t)sms * 8);
  PdlLaunch l(dim3((unsigned)std::max<int64_t>(blocks, 1)), dim3(256), 0, stream);
  if (row_bytes % 8 == 0)
    return cudaLaunchKernelEx(&l.cfg, stage_rows_kernel<uint2>,
                              reinterpret_cast<const uint2*>(src), rows, row_bytes / 8,
                              reinterpret_cast<uint2*>(dst), dst_stride / 8);
  return cudaLaunchKernelEx(&l.cfg, stage_rows_kernel<uint8_t>, src, rows, row_bytes, dst,
                            dst_stride);
}

// Stage the weight rows that TMA cannot read in place (both copies are
// no-ops for K % 256 == 0, the usual lm_head width).
static cudaError_t stage_weights(const WeightStage& w, const uint8_t* packed,
                                 const uint8_t* scales, int64_t rows, int64_t K, uint8_t* ws,
                                 cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (w.packed)
    e = stage_rows_launch(packed, rows, K / 2, ws + w.packed_off, (int64_t)w.packed_stride, stream);
  if (e == cudaSuccess && w.scales)
    e = stage_rows_launch(scales, rows, K / 16, ws + w.scales_off, (int64_t)w.scales_stride,
                          stream);
  return e;
}

// Up to this many token rows the prep kernel gives each row a whole CTA.
constexpr int64_t kPrepWideRows = 256;

// ------------------------------------------------------------ host side
size_t lm_head_workspace_bytes(int64_t M, int64_t N, int64_t K, bool argmax) {
  const WsLayout L = ws_layout(M, N, K, std::max(sm_count(), 1), argmax, ActFormat::kF16);
  return weight_stage(N, K, L.total, true).total;
}

size_t lm_head_topk_workspace_bytes(int64_t M, int64_t N, int64_t K, int k) {
  const int sms = std::max(sm_count(), 1);
  if (M <= kTopkLogitsMaxM && topk_logits_fits(N)) {  // fp32 logits, then the selection
    const WsLayout L = ws_layout(M, N, K, sms, false, ActFormat::kF16);
    return weight_stage(N, K, topk_logits_layout(L.total, M, N).total, true).total;
  }
  const WsLayout L = ws_layout(M, N, K, sms, false, ActFormat::kF16, k);
  return weight_stage(N, K, L.total, true).total;
}

// out_mode: NVFP4_OUT_F32 / NVFP4_OUT_BF16 write logits[M, N] to `logits`;
// kOutArgmax writes token_ids[M] (and max_logits[M] unless null) instead;
// kOutTopk (topk_k > 0) writes token_ids[M, k] (and max_logits[M, k]).
static nvfp4_status lm_head_run(const void* x, int64_t M, int64_t K, const uint8_t* packed,
                                const uint8_t* scales, const float* global_scale, int64_t N,
                                void* logits, int out_mode, int64_t* token_ids,
                                float* max_logits, int topk_k, void* workspace,
                                cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const bool argmax = out_mode == kOutArgmax;
  // top-k of a few tokens: the fp32 logits are written and selected from;
  // of many tokens: thresholded candidates in the epilogue
  const bool topk_logits =
      out_mode == kOutTopk && M <= kTopkLogitsMaxM && topk_logits_fits(N);
  const bool topk = out_mode == kOutTopk && !topk_logits;
  const bool keys = argmax || topk;  // per-token lines the prep kernel clears
  const int BN = lm_head_token_tile(M);
  const int n_ttiles = (int)((M + BN - 1) / BN);
  const int64_t m_pad = (int64_t)n_ttiles * BN;
  const WsLayout L = ws_layout(M, N, K, sms, argmax, ActFormat::kF16, topk ? topk_k : 0);
  const TopkLogitsLayout TL = topk_logits_layout(L.total, M, N);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  __half* x16 = reinterpret_cast<__half*>(ws + L.x16);
  float* tok_scale = reinterpret_cast<float*>(ws + L.tok);
  uint32_t* split_cnt = reinterpret_cast<uint32_t*>(ws + L.cnt);
  uint32_t* split_ready = reinterpret_cast<uint32_t*>(ws + L.ready);
  float* split_part = reinterpret_cast<float*>(ws + L.part);
  const WeightStage wst = weight_stage(N, K, topk_logits ? TL.total : L.total, true);
  if (topk_logits) {
    out_mode = NVFP4_OUT_F32;
    logits = ws + TL.logits;
  }

  CUtensorMap tm_packed, tm_scales, tm_x;
  if (!encode_weight_maps(&tm_packed, &tm_scales, wst, packed, scales, N, K, ws) ||
      !encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x16, (uint64_t)K, (uint64_t)m_pad,
                 (uint64_t)K * 2, 64, (uint32_t)BN, CU_TENSOR_MAP_SWIZZLE_128B))
    return NVFP4_ERR_CUDA;
  if (stage_weights(wst, packed, scales, N, K, ws, stream) != cudaSuccess) return NVFP4_ERR_CUDA;

  // the counters, ready flags and the argmax counter are adjacent: the
  // prep kernel clears them all
  {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // few rows: a CTA per row (latency); many rows: a warp per row.  The
    // activation map covers whole token tiles and the prep kernel writes
    // the padding rows of the last one as zeros: a box mostly past the
    // map's last row (a single token in a 16-row tile) made every
    // activation load of the GEMM markedly slower than a box of rows
    // that exist (7 µs of a 59 µs call at M = 1)
    const bool wide = M <= kPrepWideRows;
    cfg.gridDim = dim3((unsigned)(wide ? m_pad : (m_pad + 7) / 8));
    cfg.blockDim = dim3(wide ? 128 : 256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, wide ? w4a16_prep_x_kernel<4> : w4a16_prep_x_kernel<1>,
                           static_cast<const uint16_t*>(x), M, K, m_pad,
                           global_scale, x16, tok_scale, status, split_cnt,
                           (int)((L.part - L.cnt) / 4),
                           keys ? reinterpret_cast<unsigned long long*>(ws + L.keys) : nullptr,
                           topk ? reinterpret_cast<uint32_t*>(ws + L.hist) : nullptr,
                           topk ? topk_hist_stride(N) : 0, nullptr, nullptr, 0) != cudaSuccess)
      return NVFP4_ERR_CUDA;
  }

  GemmArgs a = {};
  a.M = M;
  a.N = N;
  a.K = K;
  a.BN = BN;
  a.n_ttiles = n_ttiles;
  a.n_units = ((N + kRows - 1) / kRows) * n_ttiles;
  a.n_kb = (int)((K + kKB - 1) / kKB);  // the last stage's k past K reads zeros
  schedule_units(a, L.grid, kDecodeTailSkew);
  a.split_cnt = split_cnt;
  a.split_ready = split_ready;
  a.split_part = split_part;
  a.am_keys = keys ? reinterpret_cast<unsigned long long*>(ws + L.keys) : nullptr;
  a.am_done = argmax ? reinterpret_cast<uint32_t*>(ws + L.done) : nullptr;
  a.am_idx = token_ids;
  a.am_val = max_logits;
  if (topk) topk_args(a, ws, L, topk_k, N);
  a.row_scale = nullptr;
  a.grp_max = topk_logits ? reinterpret_cast<uint32_t*>(ws + TL.gmax) : nullptr;
  // decode-sized token tiles get a third A stage, six packed stages and a
  // third dequant warp per quadrant; 128-token tiles leave TMEM room for two
  // A stages only
  const bool deep = BN <= 64;
  const int stages = deep ? 3 : 2;

  // four accumulator buffers where TMEM has room for them (small token
  // tiles: short units then overlap their epilogues), else two
  a.dbuf_log2 = (4 * BN + stages * (kKB / 2) <= 512) ? 2u : 1u;
  a.tmem_cols = ((BN << a.dbuf_log2) + stages * (kKB / 2) <= 256) ? 256u : 512u;
  a.tok_scale = tok_scale;
  a.out = logits;
  a.status = status;
  const int grid = L.grid;  // min(SMs, units): every CTA's range spans >= one unit
  // programmatic dependent launch: the GEMM starts streaming weights while
  // the prep kernel is still running
  cudaError_t err;
  if (topk_logits)
    err = deep ? launch_gemm<kOutLogitsGroups, 3, 6, 3>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<kOutLogitsGroups, 2, 4, 2>(tm_packed, tm_scales, tm_x, a, grid, stream);
  else if (argmax)
    err = deep ? launch_gemm<kOutArgmax, 3, 6, 3>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<kOutArgmax, 2, 4, 2>(tm_packed, tm_scales, tm_x, a, grid, stream);
  else if (topk) {
    err = deep ? launch_gemm<kOutTopk, 3, 6, 3>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<kOutTopk, 2, 4, 2>(tm_packed, tm_scales, tm_x, a, grid, stream);
    if (err == cudaSuccess)
      err = topk_select_launch(a.am_keys, a.tk_grp, a.tk_cand, a.tk_hist, a.tk_hstride, M, N,
                               topk_k, token_ids, max_logits, stream);
  } else if (out_mode == NVFP4_OUT_BF16)
    err = deep ? launch_gemm<NVFP4_OUT_BF16, 3, 6, 3>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<NVFP4_OUT_BF16, 2, 4, 2>(tm_packed, tm_scales, tm_x, a, grid, stream);
  else
    err = deep ? launch_gemm<NVFP4_OUT_F32, 3, 6, 3>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<NVFP4_OUT_F32, 2, 4, 2>(tm_packed, tm_scales, tm_x, a, grid, stream);
  if (err == cudaSuccess && topk_logits)
    err = topk_logits_launch(reinterpret_cast<const float*>(ws + TL.logits), a.grp_max, M, N,
                             topk_k, token_ids, max_logits, stream);
  if (err != cudaSuccess || cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

nvfp4_status lm_head_launch(const void* x, int64_t M, int64_t K, const uint8_t* packed,
                            const uint8_t* scales, const float* global_scale, int64_t N,
                            void* logits, int out_mode, int64_t* token_ids, float* max_logits,
                            void* workspace, cudaStream_t stream) {
  return lm_head_run(x, M, K, packed, scales, global_scale, N, logits, out_mode, token_ids,
                     max_logits, 0, workspace, stream);
}

nvfp4_status lm_head_topk_launch(const void* x, int64_t M, int64_t K, const uint8_t* packed,
                                 const uint8_t* scales, const float* global_scale, int64_t N,
                                 int k, int64_t* token_ids, float* values, void* workspace,
                                 cudaStream_t stream) {
  return lm_head_run(x, M, K, packed, scales, global_scale, N, nullptr, kOutTopk, token_ids,
                     values, k, workspace, stream);
}

// ------------------------------------------------------------ grouped product
// Token tile of a grouped call: from the mean rows per group.
static int grouped_token_tile(int64_t M, int64_t n_groups) {
  const int64_t mean = std::max<int64_t>(1, (M + n_groups - 1) / n_groups);
  int bn = 16;  // a power of two (the device divides by shifting)
  while (bn < kMaxBN && bn < mean) bn *= 2;
  return bn;
}

// Units of a grouped call are at most weight tiles x (token tiles of M + one
// partial tile per group); the split-K arrays are sized for that grid.
static int64_t grouped_units_bound(int64_t M, int64_t N, int64_t n_groups, int BN) {
  return ((N + kRows - 1) / kRows) * ((M + BN - 1) / BN + n_groups);
}

size_t grouped_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
  const int BN = grouped_token_tile(M, n_groups);
  const int sms = std::max(sm_count(), 1);
  const int64_t units = grouped_units_bound(M, N, n_groups, BN);
  // the plain product's layout for M token rows and a grid of at most
  // min(SMs, unit bound); its token tile is never below the grouped one, so
  // the split-K partials fit
  const WsLayout L = ws_layout(M, units * kRows, K, sms, false, ActFormat::kF16);
  return weight_stage(n_groups * N, K, L.total, true).total;
}

nvfp4_status grouped_launch(const void* x, int64_t M, int64_t K, const int32_t* grp_off,
                            int64_t n_groups, const uint8_t* packed, const uint8_t* scales,
                            const float* grp_global, int64_t N, void* out, int out_dtype,
                            void* workspace, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const int BN = grouped_token_tile(M, n_groups);
  const int64_t units = grouped_units_bound(M, N, n_groups, BN);
  // same byte layout as grouped_workspace_bytes: token rows M (TMA zero-fills
  // past them), grid min(SMs, unit bound)
  const WsLayout L = ws_layout(M, units * kRows, K, sms, false, ActFormat::kF16);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  __half* x16 = reinterpret_cast<__half*>(ws + L.x16);
  float* tok_scale = reinterpret_cast<float*>(ws + L.tok);

  CUtensorMap tm_packed, tm_scales, tm_x;
  const int64_t rows = n_groups * N;
  const WeightStage wst = weight_stage(rows, K, L.total, true);
  if (!encode_weight_maps(&tm_packed, &tm_scales, wst, packed, scales, rows, K, ws) ||
      !encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x16, (uint64_t)K, (uint64_t)M,
                 (uint64_t)K * 2, 64, (uint32_t)BN, CU_TENSOR_MAP_SWIZZLE_128B))
    return NVFP4_ERR_CUDA;
  if (stage_weights(wst, packed, scales, rows, K, ws, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
  {
    const bool wide = M <= kPrepWideRows;
    PdlLaunch l(dim3((unsigned)(wide ? M : (M + 7) / 8)), dim3(wide ? 128 : 256), 0, stream);
    if (cudaLaunchKernelEx(&l.cfg, wide ? w4a16_prep_x_kernel<4> : w4a16_prep_x_kernel<1>,
                           static_cast<const uint16_t*>(x), M, K, M,
                           (const float*)nullptr, x16, tok_scale, status,
                           reinterpret_cast<uint32_t*>(ws + L.cnt), (int)((L.part - L.cnt) / 4),
                           (unsigned long long*)nullptr, (uint32_t*)nullptr, 0,
                           grp_off, grp_global,
                           (int)n_groups) != cudaSuccess)
      return NVFP4_ERR_CUDA;
  }
  GemmArgs a = {};
  a.M = M;
  a.N = N;
  a.K = K;
  a.BN = BN;
  a.n_ttiles = 1;
  a.n_kb = (int)((K + kKB - 1) / kKB);
  a.split_cnt = reinterpret_cast<uint32_t*>(ws + L.cnt);
  a.split_ready = reinterpret_cast<uint32_t*>(ws + L.ready);
  a.split_part = reinterpret_cast<float*>(ws + L.part);
  a.tok_scale = tok_scale;
  a.out = out;
  a.status = status;
  a.grp_off = grp_off;
  a.grp_global = grp_global;
  a.n_groups = (int)n_groups;
  const bool deep = BN <= 64;
  const int stages = deep ? 3 : 2;
  // four accumulator buffers where TMEM has room for them (small token
  // tiles: short units then overlap their epilogues), else two
  a.dbuf_log2 = (4 * BN + stages * (kKB / 2) <= 512) ? 2u : 1u;
  a.tmem_cols = ((BN << a.dbuf_log2) + stages * (kKB / 2) <= 256) ? 256u : 512u;
  const int grid = L.grid;
  cudaError_t err;
  if (out_dtype == NVFP4_OUT_BF16)
    err = deep ? launch_gemm<NVFP4_OUT_BF16, 3, 6, 3, true>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<NVFP4_OUT_BF16, 2, 4, 2, true>(tm_packed, tm_scales, tm_x, a, grid, stream);
  else
    err = deep ? launch_gemm<NVFP4_OUT_F32, 3, 6, 3, true>(tm_packed, tm_scales, tm_x, a, grid, stream)
               : launch_gemm<NVFP4_OUT_F32, 2, 4, 2, true>(tm_packed, tm_scales, tm_x, a, grid, stream);
  if (err != cudaSuccess || cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

}  // namespace nvfp4
