// w4a16_tc.cuh -- the persistent W4A16 product kernel and its launch, for the
// calls that end it differently: lm_head.cu stores the logits or keeps their
// argmax or top-k, cross_entropy.cu sums their exponentials, glu.cu joins the
// two halves of a gated block.
#pragma once

#include <cuda_fp16.h>

#include "gemm_common.cuh"

namespace nvfp4 {

// The epilogue of kOut (epilogue_role).
struct NoEpilogue {
  static constexpr bool kOwn = false, kPaired = false;
  static constexpr int kWideWarps = 4;
  static constexpr int kFirstPart = 0, kNextPart = 0;
};

constexpr int kKS = 256;            // k per packed/scale stage
constexpr int kFirstDqWarp = 3;

// Ring depths and the number of dequant warps per TMEM lane quadrant are
// template parameters of the GEMM:
//   token tiles of up to 64 (decode): 3 A/activation stages, 6 packed
//     stages, 3 warps per quadrant (TMEM: 2 x 64 accumulator columns +
//     3 x 128 A columns = 512);
//   token tiles of 128 (prefill): 2 A/activation stages, 4 packed stages,
//     2 warps per quadrant.
// A dequant warp takes every kDq-th stage.  An mbarrier parity wait for
// phase j is only sound once phase j-1 has completed; the warp itself has
// checked that for the slot's previous use only if that use was one of its
// own stages, i.e. if kDq divides the ring depth.
template <int kStages, int kPStages, int kDq>
struct GemmShape {
  static_assert(kStages % kDq == 0 && kPStages % kDq == 0,
                "dequant warps per quadrant must divide every ring depth they wait on");
  static constexpr int kDqWarps = 4 * kDq;
  static constexpr int kFirstEpiWarp = kFirstDqWarp + kDqWarps;
  static constexpr int kThreads = 32 * (kFirstEpiWarp + 4);
};
constexpr uint32_t kPackedStageBytes = kRows * (kKS / 2);   // 16384
constexpr uint32_t kScaleStageBytes = kRows * (kKS / 16);   // 2048


// ------------------------------------------------------------ the GEMM
// kOut: NVFP4_OUT_F32 / NVFP4_OUT_BF16 store the logits; kOutArgmax keeps
// only each token's largest logit and its vocabulary row; kOutTopk appends
// the candidates for each token's k largest (topk.cu selects them).
// kGrouped: the grouped (experts) product: weight rows e * N + n, token rows
// grouped by the offsets in p.grp_off, one global scale per group.
// Threads of one CTA: the shape's roles, plus the threshold warp in top-k mode.
template <int kOut, int kStages, int kPStages, int kDq>
constexpr int gemm_threads() {
  return GemmShape<kStages, kPStages, kDq>::kThreads + (kOut == kOutTopk ? 32 : 0);
}

// With an epilogue of a call's own the warps are whole warpgroups whose
// registers are split by what they do: for 128-token tiles, where that epilogue
// does more than store,
//   8 epilogue warps:  96 a thread at launch, then 40 for the warps that issue
//     copies and MMAs, 88 for dequant, 128 for the epilogue
//     (5 x 96 >= 40 + 2 x 88 + 2 x 128);
//   16 epilogue warps: 72 at launch, then 40, 72 and 80
//     (7 x 72 >= 40 + 2 x 72 + 4 x 80);
// and for small tiles, with three dequant warpgroups, 4 epilogue warps of 168
// (5 x 96 >= 40 + 3 x 88 + 168).  An epilogue instruction takes its warp 4 to 5
// cycles, so more warps are more of them, until they take the dequant warps'
// turns: see kManyWarpStages.
template <class E, int kStages>
constexpr int epi_warps() { return E::kOwn && kStages < 3 ? E::kWideWarps : 4; }

// Sums of up to so many stages end before an epilogue of 8 warps is done, and
// take 16.  1981 tokens of 66815 x 1040 (5 stages), logits' product of the
// cross entropy with P: 395 us with 8, 303 with 16; 2048 tokens of 43776 x 4096
// (16 stages) 465 and 470, the gated block of that size 283 and 290.
constexpr int kManyWarpStages = 12;

// Token tiles up to this take the deep rings and 4 epilogue warps.  One chunk of
// 16 tokens a unit needs no more; from two on more warps gain more than rings do:
// training calls of 37 tokens, 50257 x 1040 63 -> 52 us, 50257 x 4096 87 -> 80,
// the gated block's gradient of 64 tokens, 14336 x 4096 55 -> 50 (at most 0.5 us is
// lost, where a gated block of 2880 x 5120 takes 15).
constexpr int kDeepTokens = 16;

template <class E, int kOut, int kStages, int kPStages, int kDq>
constexpr int own_threads() {
  return E::kOwn ? 32 * (4 + 4 * kDq + epi_warps<E, kStages>())
                 : gemm_threads<kOut, kStages, kPStages, kDq>();
}

template <int kRegs>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// E: an epilogue of its own (see walk_epilogue) in place of the one of kOut.
// E::kPaired: the unit's 128 rows are 64 rows of the weight's first half and
// the 64 of the second half at the same place, 16 and 16 to a warp quadrant:
// lanes l and l + 16 of an epilogue warp hold such a pair.
template <int kOut, int kStages, int kPStages, int kDqPerQuad, bool kGrouped = false,
          class E = NoEpilogue>
__global__ void __launch_bounds__((own_threads<E, kOut, kStages, kPStages, kDqPerQuad>()), 1)
    w4a16_tc_kernel(const __grid_constant__ CUtensorMap tm_packed,
                    const __grid_constant__ CUtensorMap tm_scales,
                    const __grid_constant__ CUtensorMap tm_x, const GemmArgs p, const E own) {
  using Shape = GemmShape<kStages, kPStages, kDqPerQuad>;
  constexpr int kFirstDq = E::kOwn ? 4 : kFirstDqWarp;  // own: a whole warpgroup before
  constexpr int kFirstEpiWarp = kFirstDq + Shape::kDqWarps;
  constexpr int kEpiWarps = epi_warps<E, kStages>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int BN = p.BN;
  const uint32_t x_box_bytes = (uint32_t)BN * 128;  // one 64-k TMA box of the activations
  const uint32_t x_stage_bytes = (kKB / 64) * x_box_bytes;
  uint8_t* s_packed = smem;                                        // kPStages x 16 KB
  uint8_t* s_scales = s_packed + kPStages * kPackedStageBytes;     // kPStages x 2 KB
  uint8_t* s_x = s_scales + kPStages * kScaleStageBytes;           // kStages x BN*512
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_x + kStages * x_stage_bytes);
  uint64_t* p_full = bars;                 // packed/scale stage landed (TMA)
  uint64_t* p_empty = p_full + kPStages;   // packed/scale stage read by its 4 dequant warps
  uint64_t* s_full = p_empty + kPStages;   // A stage in TMEM (4 warps) + activation TMA landed
  uint64_t* s_empty = s_full + kStages;    // the MMAs reading stage s completed
  uint64_t* d_full = s_empty + kStages;   // accumulator buffer b holds a finished unit
  uint64_t* d_empty = d_full + 4;         // the epilogue has drained buffer b
  uint64_t* done_bar = d_empty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  uint64_t* i_full = done_bar + 2;  // own epilogue: token information of a unit
  uint64_t* i_empty = i_full + 2;
  static_assert(2 * (kStages + kPStages) + 8 + 2 + 4 <= 32);
  float* s_tok = reinterpret_cast<float*>(bars + 32);  // 4 epilogue warps x kMaxBN multipliers
  // argmax: the "last CTA" flag, then per epilogue warp the thresholds of
  // its current unit's tokens (lower bounds of each token's largest logit)
  int32_t* s_last = reinterpret_cast<int32_t*>(s_tok + 4 * kMaxBN);
  float* s_thr = reinterpret_cast<float*>(s_last + 4);
  // grouped: the schedule derived from the group offsets
  Sched* s_sched = reinterpret_cast<Sched*>(s_thr + 4 * kMaxBN);
  uint32_t* s_unit_pre = reinterpret_cast<uint32_t*>(s_sched + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(s_unit_pre + kMaxGroups + 1);
  uint2* s_grp_tab = reinterpret_cast<uint2*>(s_off + kMaxGroups + 1);  // 8-byte aligned

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if constexpr (kGrouped) {
    grouped_offsets_load(p, s_off);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(&p_full[i], 1);
      mbar_init(&p_empty[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_full[i], 4 + 1);
      mbar_init(&s_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], kEpiWarps);
    }
    mbar_init(done_bar, 1);
    if constexpr (E::kOwn) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&i_full[i], 1);
        mbar_init(&i_empty[i], kEpiWarps);
      }
    }
    *abort_flag = 0;
    if (kOut == kOutTopk) s_last[1] = 0;  // epilogue warps done (the region exists in this mode)
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if constexpr (kGrouped)
    if (warp == 0)
      grouped_sched_build(p, s_sched, s_unit_pre, s_off, s_grp_tab, (uint32_t)p.n_kb, lane);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_packed);
    tma_prefetch_desc(&tm_scales);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  // warp-uniform copy of the TMEM base (lets the compiler keep it uniform)
  const uint32_t tmem_base = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const uint32_t tmem_a = tmem_base + ((uint32_t)BN << p.dbuf_log2);  // A ring after the D buffers

  WaitCtl wc{p.status, abort_flag, kWaitLimitNs};
  Sched sc;
  if constexpr (kGrouped) sc = *s_sched; else sc = plain_sched(p);
  const uint32_t n_kb_u = (uint32_t)p.n_kb;
  // the producer and MMA loops below are warp-uniform; one elected lane
  // issues each TMA / tcgen05 instruction

  if (warp < kFirstDq) {
    if constexpr (E::kOwn) registers_down<40>();
  if (warp == 0) {
    // ---------------- packed codes + scales producer
    // a weight tile read once (one token tile) is not kept in L2; one read
    // by several token tiles in a row is
    const uint64_t pol_once = policy_evict_first(), pol_reused = policy_evict_last();
    if constexpr (E::kOwn)
      if (own.staged) grid_dependency_wait();  // the weight rows come from the kernel before
    uint32_t issued = 0, piece = 0;
    for_each_piece(sc, n_kb_u, [&](const Piece& pc) {
      const UnitGeom geo = unit_geom<kGrouped>(p, sc, pc.u, piece++);
      const int32_t n0 = (int32_t)geo.w_row;
      const uint64_t pol = geo.reused ? pol_reused : pol_once;  // packed codes
      for (uint32_t kb = pc.kb0; kb < pc.kb1; ++kb, ++issued) {
        const uint32_t st = issued % kPStages, ph = (issued / kPStages) & 1;
        if (!warp_wait(&p_empty[st], ph ^ 1, wc)) return false;
        if (elect_one()) {
          mbar_arrive_expect_tx(&p_full[st], kPackedStageBytes + kScaleStageBytes);
          if constexpr (E::kPaired) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int32_t y = n0 / 2 + half * (int32_t)own.half;
              tma_load_2d_hint(s_packed + st * kPackedStageBytes + half * (kPackedStageBytes / 2),
                               &tm_packed, kb * (kKS / 2), y, &p_full[st], pol);
              uint8_t* sd = s_scales + st * kScaleStageBytes + half * (kScaleStageBytes / 2);
              if (geo.reused)
                tma_load_2d_hint(sd, &tm_scales, kb * (kKS / 16), y, &p_full[st], pol_reused);
              else
                tma_load_2d(sd, &tm_scales, kb * (kKS / 16), y, &p_full[st]);
            }
          } else {
          tma_load_2d_hint(s_packed + st * kPackedStageBytes, &tm_packed, kb * (kKS / 2), n0,
                           &p_full[st], pol);
          // a stage takes 16 bytes of each 32-byte scale sector, the next
          // stage the other 16: scales read once keep the default policy
          // (evict-first would drop the sector before its second half is read)
          if (geo.reused)
            tma_load_2d_hint(s_scales + st * kScaleStageBytes, &tm_scales, kb * (kKS / 16), n0,
                             &p_full[st], pol_reused);
          else
            tma_load_2d(s_scales + st * kScaleStageBytes, &tm_scales, kb * (kKS / 16), n0,
                        &p_full[st]);
          }
        }
        __syncwarp();
      }
      return true;
    });
    drain_loads(p_full, kPStages, issued, 1, p.status);
  } else if (warp == 1) {
    // ---------------- activation producer (four 64-k boxes per stage)
    grid_dependency_wait();  // the rescaled activations come from the prep kernel
    const uint64_t pol = policy_evict_last();
    uint32_t issued = 0, piece = 0;
    for_each_piece(sc, n_kb_u, [&](const Piece& pc) {
      const int32_t t0 = (int32_t)unit_geom<kGrouped>(p, sc, pc.u, piece++).t0;
      for (uint32_t kb = pc.kb0; kb < pc.kb1; ++kb, ++issued) {
        const uint32_t st = issued % kStages, ph = (issued / kStages) & 1;
        if (!warp_wait(&s_empty[st], ph ^ 1, wc)) return false;
        if (elect_one()) {
          mbar_arrive_expect_tx(&s_full[st], x_stage_bytes);
          uint8_t* dst = s_x + st * x_stage_bytes;
#pragma unroll
          for (int b = 0; b < kKB / 64; ++b)
            tma_load_2d_hint(dst + b * x_box_bytes, &tm_x, kb * kKB + 64 * b, t0, &s_full[st],
                             pol);
        }
        __syncwarp();
      }
      return true;
    });
    drain_loads(s_full, kStages, issued, 5, p.status);
  } else if (warp == 2) {
    // ---------------- MMA issuer (whole warp; one elected lane issues).
    // One accumulator per piece, double buffered.
    const uint32_t idesc = idesc_f16_f32((uint32_t)BN);
    const uint64_t xdesc0 = smem_desc_sw128(smem_u32(s_x));
    const uint32_t box_desc = x_box_bytes >> 4;
    uint32_t g = 0;
    int64_t i = 0;
    for_each_piece(sc, n_kb_u, [&](const Piece& pc) {
      uint32_t buf = (uint32_t)(i & ((1 << p.dbuf_log2) - 1));
      uint32_t dph = (uint32_t)((i >> p.dbuf_log2) & 1);
      ++i;
      // grouped 128-token tiles: a group's last, partly filled tile takes MMAs
      // only as wide as its tokens, in 16-token steps (same box, 2048 tokens:
      // w13 134.9 -> 132.5 us, w2 89.2 -> 88.7 us; smaller tiles keep BN)
      uint32_t id = idesc;
      if constexpr (kGrouped) {
        if (BN == kMaxBN) {
          const UnitGeom geo = unit_geom<kGrouped>(p, sc, pc.u, (uint32_t)(i - 1));
          const int64_t live = geo.t_end - geo.t0;
          if (live < BN) id = idesc_f16_f32(live > 0 ? (uint32_t)((live + 15) / 16 * 16) : 16u);
        }
      }
      if (!warp_wait(&d_empty[buf], dph ^ 1, wc)) return false;
      tc_fence_after();
      uint32_t d_tmem = tmem_base + buf * BN;
      uint32_t part0 = pc.kb0, part1 = pc.kb0 + E::kFirstPart;  // this accumulator's stages
      for (uint32_t kb = pc.kb0; kb < pc.kb1; ++kb, ++g) {
        if constexpr (E::kFirstPart > 0) {
          if (kb == part1) {  // the next part, in the next accumulator
            if (elect_one()) tc_commit(&d_full[buf]);
            __syncwarp();
            part0 = kb;
            part1 = kb + E::kNextPart;
            buf = (uint32_t)(i & ((1 << p.dbuf_log2) - 1));
            dph = (uint32_t)((i >> p.dbuf_log2) & 1);
            ++i;
            if (!warp_wait(&d_empty[buf], dph ^ 1, wc)) return false;
            tc_fence_after();
            d_tmem = tmem_base + buf * BN;
          }
        }
        const uint32_t st = g % kStages, ph = (g / kStages) & 1;
        if (!warp_wait(&s_full[st], ph, wc)) return false;
        tc_fence_after();
        const uint64_t bdesc = xdesc0 + ((st * x_stage_bytes) >> 4);
        const uint32_t a_t = tmem_a + st * (kKB / 2);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk)
            tc_mma_ts(d_tmem, a_t + kk * 8, bdesc + (kk >> 2) * box_desc + 2 * (kk & 3), id,
                      (kb != part0) || (kk != 0));
          tc_commit(&s_empty[st]);
        }
        __syncwarp();
      }
      if (elect_one()) tc_commit(&d_full[buf]);
      __syncwarp();
      return true;
    });
    // this CTA has issued its last MMA: the next kernel in the stream may be
    // launched (it waits for this grid's completion before touching memory)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // every MMA issued above has completed once done_bar flips
    if (elect_one()) tc_commit(done_bar);
    __syncwarp();
    WaitCtl drain{p.status, abort_flag, 100000000ull};
    volatile int32_t zero = 0;
    drain.abort = &zero;
    mbar_wait(done_bar, 0, drain);
  } else if constexpr (E::kOwn) {  // warp 3
    token_info_role(p, sc, own, lane, i_full, i_empty, wc, reinterpret_cast<uint8_t*>(s_tok));
  }
  } else if (warp < kFirstEpiWarp) {
    if constexpr (E::kOwn && kEpiWarps != 16) registers_down<88>();
    // ---------------- dequant: one thread per vocabulary row.  The kDqPerQuad
    // warps of a TMEM lane quadrant take the 256-k stages in turn: wait for
    // the packed stage, convert 64 k at a time into 32 registers and store
    // them to the stage's TMEM columns, then signal the MMA warp.
    const int q = warp & 3;
    const int r = (warp - kFirstDq) >> 2;
    const int row = E::kPaired ? (lane & 16) * 4 + q * 16 + (lane & 15) : q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const int sw = row & 7;
    // this warp's stages are g = r, r + kDqPerQuad, ... of the CTA's sequence
    const uint32_t total = cta_stages(sc, n_kb_u);
    // NaN block scales (E4M3 S.1111.111: the "never loaded" sentinel of
    // `KNvfp4Static.process` on the page
    // "vllm/model_executor/layers/quantization/modelopt.py"): per byte,
    // (b & 0x7F) + 1 carries into bit 7 only for 0x7F / 0xFF, and never into
    // the next byte; the OR over the CTA's stages is tested once at the end
    uint32_t nan_seen = 0;
    bool ok = true;
    for (uint32_t g = (uint32_t)r; ok && g < total; g += kDqPerQuad) {
      const uint32_t ps = g % kPStages, pph = (g / kPStages) & 1;
      const uint32_t st = g % kStages, ph = (g / kStages) & 1;
      if (!warp_wait(&p_full[ps], pph, wc)) { ok = false; break; }
      const uint8_t* prow = s_packed + ps * kPackedStageBytes + row * (kKS / 2);
      const uint4 sc = *reinterpret_cast<const uint4*>(s_scales + ps * kScaleStageBytes +
                                                       row * (kKS / 16));
      const uint32_t scw[4] = {sc.x, sc.y, sc.z, sc.w};
      nan_seen |= ((sc.x & 0x7F7F7F7Fu) + 0x01010101u) | ((sc.y & 0x7F7F7F7Fu) + 0x01010101u) |
                  ((sc.z & 0x7F7F7F7Fu) + 0x01010101u) | ((sc.w & 0x7F7F7F7Fu) + 0x01010101u);
      const uint32_t ta = tmem_a + lane_off + st * (kKB / 2);
#pragma unroll
      for (int c4 = 0; c4 < kKB / 64; ++c4) {
        const uint4 c0 = *reinterpret_cast<const uint4*>(prow + (((2 * c4) ^ sw) << 4));
        const uint4 c1 = *reinterpret_cast<const uint4*>(prow + (((2 * c4 + 1) ^ sw) << 4));
        uint32_t s01, s23;
        scales4_to_f16(scw[c4], s01, s23);
        const uint32_t f0 = dup_lo(s01), f1 = dup_hi(s01), f2 = dup_lo(s23), f3 = dup_hi(s23);
        uint32_t v[32];
        dequant8(c0.x, f0, v + 0);
        dequant8(c0.y, f0, v + 4);
        dequant8(c0.z, f1, v + 8);
        dequant8(c0.w, f1, v + 12);
        dequant8(c1.x, f2, v + 16);
        dequant8(c1.y, f2, v + 20);
        dequant8(c1.z, f3, v + 24);
        dequant8(c1.w, f3, v + 28);
        if (c4 == 0 && !warp_wait(&s_empty[st], ph ^ 1, wc)) { ok = false; break; }
        tmem_st32(ta + c4 * 32, v);
      }
      if (!ok) break;
      // the packed stage has been read; the A stage is complete once the
      // TMEM stores land
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_empty[ps]);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_full[st]);
    }
    if (__any_sync(0xFFFFFFFFu, (nan_seen & 0x80808080u) != 0u) && lane == 0)
      raise_status(p.status, NVFP4_ERR_NONFINITE);
  } else if (warp < kFirstEpiWarp + kEpiWarps) {
    // ---------------- epilogue: one thread per vocabulary row, BN tokens
    if constexpr (E::kOwn) {
      registers_up<kEpiWarps == 16 ? 80 : kEpiWarps == 8 ? 128 : 168>();
      walk_epilogue<kEpiWarps>(p, sc, own, warp, warp - kFirstEpiWarp, lane, tmem_base, d_full,
                               d_empty, i_full, i_empty, wc, reinterpret_cast<uint8_t*>(s_tok));
    } else
      epilogue_role<kOut, false, kGrouped>(p, sc, warp, warp - kFirstEpiWarp, lane, tmem_base,
                                           d_full, d_empty, wc, s_tok, s_thr);
    if (kOut == kOutTopk && lane == 0) atomicAdd(s_last + 1, 1);  // this warp is done
  } else {
    // ---------------- top-k thresholds (only launched in top-k mode)
    topk_threshold_role(p, s_last + 1, lane);
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
  if constexpr (kOut == kOutArgmax) argmax_finish(p, 32 * kFirstEpiWarp, s_last);
}

// ------------------------------------------------------------ host side
static size_t gemm_smem_bytes(int BN, int stages, int pstages, bool argmax, bool grouped = false) {
  // ring buffers, then 256 B of barriers and flags, then the epilogue's
  // per-warp token multipliers (and, for argmax, a flag and per-warp
  // token thresholds; for the grouped product, after that region, its
  // schedule and the per-group unit prefix and token offsets)
  return 1024 + pstages * (size_t)(kPackedStageBytes + kScaleStageBytes) +
         stages * (size_t)BN * kKB * 2 + 256 + 4 * kMaxBN * sizeof(float) +
         (argmax || grouped ? 16 + 4 * kMaxBN * sizeof(float) : 0) +
         (grouped ? sizeof(Sched) + 2 * (kMaxGroups + 1) * sizeof(uint32_t) +
                        kGrpTab * sizeof(uint2) : 0);
}

// Launch one instantiation (programmatic dependent of the prep kernel).
template <int kOut, int kStages, int kPStages, int kDq, bool kGrouped = false>
static cudaError_t launch_gemm(const CUtensorMap& tm_packed, const CUtensorMap& tm_scales,
                               const CUtensorMap& tm_x, const GemmArgs& a, int grid,
                               cudaStream_t stream) {
  auto kern = w4a16_tc_kernel<kOut, kStages, kPStages, kDq, kGrouped>;
  constexpr bool kArgmax = kOut == kOutArgmax || kOut == kOutTopk;  // per-warp thresholds
  const size_t smem = gemm_smem_bytes(a.BN, kStages, kPStages, kArgmax, kGrouped);
  // the 3-stage shape only serves token tiles of up to 64
  constexpr int kMaxTileBN = kStages >= 3 ? 64 : kMaxBN;
  static std::atomic<uint64_t> limit_set{0};
  const cudaError_t attr_err =
      smem_limit_once(limit_set, reinterpret_cast<const void*>(kern),
                      gemm_smem_bytes(kMaxTileBN, kStages, kPStages, kArgmax, kGrouped));
  if (attr_err != cudaSuccess) return attr_err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(gemm_threads<kOut, kStages, kPStages, kDq>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_packed, tm_scales, tm_x, a, NoEpilogue{});
}

// The product with an epilogue of its own.
template <int kStages, int kPStages, int kDq, class E>
static cudaError_t launch_gemm_with(const E& own, const CUtensorMap& tm_packed,
                                    const CUtensorMap& tm_scales, const CUtensorMap& tm_x,
                                    const GemmArgs& a, int grid, cudaStream_t stream) {
  auto kern = w4a16_tc_kernel<NVFP4_OUT_F32, kStages, kPStages, kDq, false, E>;
  auto smem = [](int BN) {
    return 1024 + kPStages * (size_t)(kPackedStageBytes + kScaleStageBytes) +
           kStages * (size_t)BN * kKB * 2 + 256 + 2 * (size_t)E::kInfoBytes;
  };
  static_assert(E::kInfoBytes % 16 == 0);
  static std::atomic<uint64_t> limit_set{0};
  const cudaError_t err = smem_limit_once(limit_set, reinterpret_cast<const void*>(kern),
                                          smem(kStages >= 3 ? kDeepTokens : kMaxBN));
  if (err != cudaSuccess) return err;
  PdlLaunch l(dim3((unsigned)grid), dim3(own_threads<E, NVFP4_OUT_F32, kStages, kPStages, kDq>()),
              smem(a.BN), stream);
  return cudaLaunchKernelEx(&l.cfg, kern, tm_packed, tm_scales, tm_x, a, own);
}

// Tensor maps of the packed codes and block scales of `rows` weight rows:
// in place where the row length is a 16-byte multiple, else over the
// staged copy.  The map's extent is the real row length, so the TMA fills
// the k past K with zeros (code 0, scale 0: the weight is 0 there).
static inline bool encode_weight_maps(CUtensorMap* tm_packed, CUtensorMap* tm_scales,
                               const WeightStage& w, const uint8_t* packed, const uint8_t* scales,
                               int64_t rows, int64_t K, uint8_t* ws, uint32_t box_rows = kRows) {
  return encode_2d(tm_packed, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.packed ? ws + w.packed_off : packed,
                   (uint64_t)K / 2, (uint64_t)rows, w.packed ? w.packed_stride : (uint64_t)K / 2,
                   kKS / 2, box_rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_2d(tm_scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.scales ? ws + w.scales_off : scales,
                   (uint64_t)K / 16, (uint64_t)rows, w.scales ? w.scales_stride : (uint64_t)K / 16,
                   kKS / 16, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace nvfp4
