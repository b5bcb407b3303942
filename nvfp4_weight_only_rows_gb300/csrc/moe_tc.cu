// moe_tc.cu -- the expert layer of w4a16_moe on the FP4 tensor cores, with no
// dequantization: the block-scaled MMA (kind::mxf4nvf4) reads the NVFP4
// weights as they are stored, and the 16-bit activations are given to it as
// sums of NVFP4 values.
//
// A row v (a token's x, a pair's h) times a power of two that takes its
// largest magnitude to 2^10 .. 2^11 is split per 16 values into NVFP4 blocks,
// r_0 = v: s_i = e4m3(max|r_i| / 6), q_i = e2m1(r_i / s_i),
// r_{i+1} = 4 (r_i - s_i q_i).  The largest error of a code is its scale, so a
// piece leaves at most 0.177 of the block's maximum: six of them 3e-5 (for a
// bf16 result: 6e-7 rms, which moves it by 3e-5 of itself where fp32 sums in
// another order move it by 2e-5), eight 1e-6 (for an fp32 result).  The factor
// 4 keeps the residuals' scales off the E4M3 subnormals, and a block far below
// its row's maximum gets its first codes in a later piece: what is lost below
// the subnormals is 2e-8 of the row's maximum after six pieces, 1.3e-9 after
// eight (without it 6e-6, which one outlier channel of 3000 in a normal row
// turned into 3e-3 of the product).  The pieces of a pair are columns of the
// MMA's N side; their products, each exact, sum in fp32, and piece i's sum
// counts 4^-i.
//
// The layer is bound by HBM (9/16 byte a weight), and this way the SMs only
// move bytes: a 256-k stage of 128 weight rows is 18 KB, 800 cycles at the
// copy rate, and 4 MMAs of 16 to 64 cycles.
//
//   moe_prep_kernel     one CTA a token: pairs sorted by expert, tiles of up
//                       to `cap` pairs, pieces of x
//   moe_tc_kernel       gu = W13 x: persistent, the (tile, 128-row, stage)
//                       steps cut evenly over the SMs; a unit cut between
//                       CTAs leaves fp32 parts that its reader adds in order
//   moe_act_kernel      one CTA a pair: h and its pieces
//   moe_tc_kernel       y = W2 h
//   moe_tc_combine      out = sum over a token's slots, in slot order
// The products derive the tiles from the expert ids themselves, so that
// their weight loads start while the kernel before them still runs.
//
// Measured (bf16 result, H 2048, I 768, top 8 of 128): 64 tokens, 112 experts
// in use, 297 MB, 72.2 us (fp32 result 72.9), 6.9 and 6.0 TB/s between the products' first and last MMA,
// about 25 us of prep, h, combine, kernel boundaries and first loads around
// them.  5 tokens of H = I = 2880, top 4 of 32, 224 MB: 56.4 us.  193 tokens of
// 64 experts with I 720 and half the pairs elsewhere, 144 MB: 67.6 us (fp32
// result, tiles of 16 pairs, 71.5); the 14
// second tiles of experts with more than 20 pairs cost as much time as first
// ones, although they find their weights in L2.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gemm_common.cuh"

namespace nvfp4 {

constexpr int kPieces = 8;                  // columns of a pair for an fp32 result
constexpr int kPiecesBf16 = 6;              // ... for a bf16 one
constexpr int kTcMaxExperts = NVFP4_MOE_MAX_EXPERTS;
constexpr int kTcMaxK = 64;                 // slots of a token
constexpr uint32_t kTcAStage = 128 * 128;   // 128 rows x 256 codes
constexpr uint32_t kTcSfStage = 4 * 512;    // 4 atoms of 128 rows x 4 blocks
constexpr uint32_t kTcRow = 128;            // bytes of a piece in a stage
constexpr int kTcMaxRing = 8;
// Dynamic shared memory of a product's CTA: what lets a CTA of the prep kernel
// share its SM (64 of 152 CTAs began 5 us late without; 193 tokens: 67.7 us
// against 68.7 with 220 KB and one stage more).
constexpr size_t kTcSmem = 205 << 10;
constexpr int kTcMaxCap = 20;               // pairs of a tile
constexpr int64_t kTcMaxUnitK = 4096;       // largest K whose 128 rows of scales are loaded at once
constexpr int kTcSfCols = 32;               // TMEM columns of a stage's scales: A 16 + B 16

// What the kernels between the products know of a pair: where it lies.
struct __align__(16) TcPlace {
  int expert, tile, col, place;  // place in the order sorted by expert; -1: absent
};

// The routing as every CTA of a product derives it: pairs and tiles before
// each expert.
struct TcTables {
  int cnt[kTcMaxExperts];
  uint16_t off[kTcMaxExperts], tile[kTcMaxExperts + 1];  // at most 4096
};

struct TcTile {
  int expert, first, n;  // pairs first .. first + n - 1 in sorted order
};

// Named barrier `bar` of n threads.
__device__ __forceinline__ void tc_sync(int bar, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(n) : "memory");
}

// By the n threads tid = 0 .. n - 1 (whole warps) that meet at barrier `bar`.
// seen(i, e): pair i has expert e, or kTcNoExpert; meanwhile(): by the warps
// but the first, once every id was seen.
constexpr int kTcNoExpert = 0xFFFF;
template <typename Seen, typename Meanwhile>
__device__ __forceinline__ void tc_tables(const int32_t* ids, int P, int E, int cap, TcTables& s,
                                          int tid, int n, int bar, Seen seen, Meanwhile meanwhile) {
  const int lane = tid & 31;
  const int mine = tid < P ? __ldg(ids + tid) : -1;  // under way while the counts are cleared
  for (int e = tid; e < E; e += n) s.cnt[e] = 0;
  tc_sync(bar, n);
  auto count = [&](int i, int e) {
    const bool in = e >= 0 && e < E;
    if (in) atomicAdd(&s.cnt[e], 1);
    seen(i, in ? e : kTcNoExpert);
  };
  if (tid < P) count(tid, mine);
#pragma unroll 4
  for (int i = tid + n; i < P; i += n) count(i, __ldg(ids + i));
  tc_sync(bar, n);
  if (tid < 32) {
    // lane l takes `per` consecutive experts
    const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
    int both = 0;  // pairs | tiles << 16: at most 4096 of either
    for (int e = e0; e < e1; ++e) {
      const int c = s.cnt[e];
      both += c | ((c + cap - 1) / cap) << 16;
    }
    int incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    int off = (incl - both) & 0xFFFF, tiles = (incl - both) >> 16;
    for (int e = e0; e < e1; ++e) {
      const int c = s.cnt[e];
      s.off[e] = (uint16_t)off;
      s.tile[e] = (uint16_t)tiles;
      off += c;
      tiles += (c + cap - 1) / cap;
    }
    if (lane == 31) s.tile[E] = (uint16_t)tiles;
  } else {
    meanwhile();
  }
  tc_sync(bar, n);
}

__device__ __forceinline__ TcTile tc_tile(const TcTables& s, int E, int cap, int t) {
  int lo = 0, hi = E - 1;  // the last expert whose tiles begin at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tile[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int skip = (t - s.tile[lo]) * cap;
  return {lo, s.off[lo] + skip, min(cap, s.cnt[lo] - skip)};
}

struct TcArgs {
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  const float *g13, *g2;
  void* out;
  int M, k, H, I, E, P, cap, tiles_max, grid, pieces;
  int2* counts;                  // pairs, tiles
  TcPlace *by_pair, *by_place;
  uint8_t *act1, *sf1, *act2, *sf2;
  float *mul1, *mul2, *gu, *y, *part1, *part2;
  int32_t* status;
};

// ------------------------------------------------------------ the schedule
// S = units x stages steps over the first G = min(S, grid) CTAs (each has at
// least one), step x to the CTA b with S b / G <= x < S (b + 1) / G; unit u =
// tile x row tiles + row tile.
__host__ __device__ __forceinline__ int64_t tc_ctas(int64_t S, int64_t grid) {
  return S < grid ? S : grid;
}
__host__ __device__ __forceinline__ int64_t tc_bound(int64_t S, int64_t b, int64_t G) {
  return S * b / G;
}
__host__ __device__ __forceinline__ int tc_owner(int64_t S, int64_t x, int64_t G) {
  const int64_t a = (x + 1) * G - 1;  // at most S G
  if (S * G < (int64_t)1 << 32) return (int)((uint32_t)a / (uint32_t)S);
  return (int)(a / S);
}

// The part slot of CTA b for a unit it did not do alone: 1 if it began it.
__device__ __forceinline__ int tc_slot(int b, bool opened) { return 2 * b + (opened ? 1 : 0); }

// ------------------------------------------------------------ pieces
// A stage of a row, split: kSplitBytes of a warp's shared memory, [piece][128
// bytes of codes] and [piece][16 scales].  The loop is kept rolled, because
// this runs once and cold (unrolled, instruction fetch took longer than the
// work).  v: this lane's values 8 lane .. of the stage, already times the row's
// power of two.
constexpr float kResidualUp = 4.0f;  // a residual's factor before the next piece
constexpr int kSplitBytes = kPieces * (kTcRow + 16);

__device__ __forceinline__ void tc_split(float (&v)[8], int pieces, uint8_t* buf) {
  const int lane = threadIdx.x & 31;
  uint8_t* scales = buf + kPieces * kTcRow;
#pragma unroll 1
  for (int p = 0; p < pieces; ++p) {
    float a = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                    fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));  // the block's other half
    const uint32_t s8 = __nv_cvt_float_to_fp8(a * (1.0f / 6.0f), __NV_SATFINITE, __NV_E4M3);
    const float s =
        __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3)));
    // a quotient one ulp off may take the neighbouring code: its error is in
    // the residual like any other
    const float inv = s == 0.0f ? 0.0f : __fdividef(1.0f, s);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
    const uint32_t w = cvt_e2m1x8_signed(q);
    uint32_t h[4];
    e2m1x8_to_f16(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      v[2 * i] = kResidualUp * __fmaf_rn(-f.x, s, v[2 * i]);
      v[2 * i + 1] = kResidualUp * __fmaf_rn(-f.y, s, v[2 * i + 1]);
    }
    reinterpret_cast<uint32_t*>(buf + p * kTcRow)[lane] = w;
    if ((lane & 1) == 0) scales[p * 16 + (lane >> 1)] = (uint8_t)s8;
  }
  __syncwarp();
}

// One warp: a split stage to where the products read it, for the pair at d.
// Row n = pieces x d.col + p of the tile: 128 bytes in 16-byte pieces swizzled
// by the row (the MMA's 128-byte layout); its scales, row 32 a + b of atom j,
// at byte b 16 + a 4 of the atom.
__device__ __forceinline__ void tc_place(const uint8_t* buf, int pieces, int stage, const TcPlace& d,
                                         int P, int tiles_max, uint8_t* act, uint8_t* sf) {
  const int lane = threadIdx.x & 31;
  const int n0 = pieces * d.col;
  uint8_t* to = act + ((int64_t)stage * P + d.place) * pieces * kTcRow;
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // eight lanes a row, four rows at a time
    const int p = 4 * i + (lane >> 3), c = lane & 7;
    if (p < pieces)
      *reinterpret_cast<uint4*>(to + p * kTcRow + ((c ^ ((n0 + p) & 7)) << 4)) =
          *reinterpret_cast<const uint4*>(buf + p * kTcRow + c * 16);
  }
  const int p = lane & 7, n = n0 + p;
  if (p < pieces)
    *reinterpret_cast<uint32_t*>(sf + ((int64_t)stage * tiles_max + d.tile) * kTcSfStage +
                                 (lane >> 3) * 512 + (n & 31) * 16 + (n >> 5) * 4) =
        reinterpret_cast<const uint32_t*>(buf + kPieces * kTcRow)[p * 4 + (lane >> 3)];
}

// The power of two that takes a row's largest magnitude (bits mx) to 2^10 ..,
// and the multiplier that undoes it (NaN where the row is not finite).
__device__ __forceinline__ float tc_scale(uint32_t mx, float& undo) {
  const int e = max((int)(mx >> 23), 12);
  undo = e == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)(e - 10) << 23);
  return __uint_as_float((uint32_t)(264 - e) << 23);
}

// ------------------------------------------------------------ prep
// Half of the CTA splits the token's row while the other half finds where its
// pairs go.
constexpr int kPrepHalf = 256;

__global__ void __launch_bounds__(2 * kPrepHalf) moe_prep_kernel(const TcArgs p) {
  constexpr int kWarps = kPrepHalf / 32;
  __shared__ TcTables s_tab;
  __shared__ __align__(16) uint8_t s_buf[kWarps][kSplitBytes];
  __shared__ TcPlace s_dst[kTcMaxK];
  __shared__ int s_n;
  __shared__ uint32_t s_max;
  extern __shared__ __align__(16) uint8_t s_prep_mem[];
  uint16_t* s_ids = reinterpret_cast<uint16_t*>(s_prep_mem);  // of all pairs, whole 16 bytes
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, m = blockIdx.x;
  const bool splits = threadIdx.x < kPrepHalf;
  const int tid = splits ? threadIdx.x : threadIdx.x - kPrepHalf, warp = tid >> 5;
  const int n_stages = (p.H + 255) / 256;
  const uint4* row = reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.H);
  auto load = [&](int s) {
    const int i = 32 * s + lane;
    return i < p.H / 8 ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
  };
  float up = 0.0f, undo = 0.0f;
  int my_e = kTcNoExpert, my_rank = 0;
  auto split = [&](int s) {
    const uint4 r = load(s);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(u[q] << 16) * up;
      v[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u) * up;
    }
    tc_split(v, p.pieces, s_buf[warp]);
  };
  if (splits) {
    // stages warp, warp + 8, ..; the first of them is split ahead of the places
    uint32_t mx = 0;
    for (int s = warp; s < n_stages; s += kWarps) {
      const uint4 r = load(s);
      const uint32_t c = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu),
                                  __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
      mx = max(mx, max(c & 0xFFFFu, c >> 16));
    }
    mx = __reduce_max_sync(0xFFFFFFFFu, mx);
    if (tid == 0) s_max = 0u;
    tc_sync(1, kPrepHalf);
    if (lane == 0) atomicMax(&s_max, mx << 16);
    tc_sync(1, kPrepHalf);
    up = tc_scale(s_max, undo);
    if (warp < n_stages) split(warp);
  } else {
    // The place of pair i is its rank among its expert's pairs, counted from
    // the ids in shared memory (from global memory, one pair's after another:
    // 193 tokens of 8 2 us more).  Slot j is warp 1 + j % 7's, whose lane j / 7
    // keeps it.
    if (tid == 0) s_n = 0;
    tc_tables(p.ids, p.P, p.E, p.cap, s_tab, tid, kPrepHalf, 2,
              [&](int i, int e) { s_ids[i] = (uint16_t)e; },
              [&] {
                for (int j = warp - 1; j < p.k; j += kWarps - 1) {
                  const int i = m * p.k + j, e = s_ids[i];
                  const uint32_t ee = (uint32_t)e | (uint32_t)e << 16;
                  int bits = 0;
                  for (int b = 8 * lane; b < i; b += 256) {
                    const uint4 v = *reinterpret_cast<const uint4*>(s_ids + b);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                      const int left = i - (b + 2 * q);  // ids of this word before i
                      const uint32_t same = __vcmpeq2(w[q], ee);
                      bits += __popc(left >= 2 ? same : left == 1 ? same & 0xFFFFu : 0u);
                    }
                  }
                  const int rank = __reduce_add_sync(0xFFFFFFFFu, bits) >> 4;
                  if (lane == j / (kWarps - 1)) {
                    my_e = e;
                    my_rank = rank;
                  }
                }
              });
    if (m == 0 && tid == 0) {
      *p.status = NVFP4_OK;
      *p.counts = make_int2(s_tab.off[p.E - 1] + s_tab.cnt[p.E - 1], s_tab.tile[p.E]);
    }
    const int slot = warp - 1 + (kWarps - 1) * lane;
    if (warp > 0 && slot < p.k) {
      TcPlace d{0, 0, 0, -1};
      if (my_e != kTcNoExpert) {
        d = {my_e, s_tab.tile[my_e] + my_rank / p.cap, my_rank % p.cap, s_tab.off[my_e] + my_rank};
        p.by_place[d.place] = d;
        s_dst[atomicAdd(&s_n, 1)] = d;
      }
      p.by_pair[m * p.k + slot] = d;
    }
  }
  __syncthreads();
  // every warp places: the halves take alternate pairs of a split stage
  const int n_dst = s_n, first = splits ? 0 : 1;
  if (splits && tid < n_dst) p.mul1[s_dst[tid].place] = undo;
  for (int s = warp; s - warp < n_stages; s += kWarps) {
    if (s < n_stages)
      for (int j = first; j < n_dst; j += 2)
        tc_place(s_buf[warp], p.pieces, s, s_dst[j], p.P, p.tiles_max, p.act1, p.sf1);
    if (s - warp + kWarps < n_stages) {  // the next round (block-uniform)
      __syncthreads();
      if (splits && s + kWarps < n_stages) split(s + kWarps);
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------ the product
struct TcGemm {
  const int32_t* ids;
  const uint8_t *codes, *scales;
  int64_t rows;  // E N: rows of the whole tensor
  int N, K, E, cap, pieces, ring, P, tiles_max;
  int unit_scales;  // buffers for the scales of a unit's 128 rows; 0: a stage's at a time
  const uint8_t *act, *sf;
  const float* mul;
  float *dst, *part;
  int32_t* status;
};

// Where K / 2 bytes are no 16-byte multiple (K % 32 != 0), TMA cannot step
// from a row of codes to the next, but from one to the next but one: a stage's
// rows come as the even ones, which land where the MMA reads them (rows 0 to 63
// of the tile), and the odd ones, 8 bytes early, which four warps copy into
// place (rows 64 to 127).  193 tokens of 64 experts, I 720: 68.4 against 73.3
// us with 8-byte cp.async by those warps instead.
__device__ __forceinline__ int tc_row(bool tma, int r) {  // of tile row r, in memory
  return tma ? r : r < 64 ? 2 * r : 2 * r - 127;
}
constexpr uint32_t kTcOddRow = 128 + 16;              // bytes of an odd row, 8 before it among them
constexpr uint32_t kTcOddStage = 64 * kTcOddRow;

// Warps: 0 weight codes (and, per stage, scales), 1 MMA, 2 scales per unit,
// 3 activations, 4-7 epilogue, 8-11 scale layout, then the odd rows' copiers.
constexpr int kTcScaleWarps = 4;
constexpr int kTcThreads = 32 * (8 + kTcScaleWarps);
constexpr int kTcOddWarps = 4;
constexpr int kTcMaxUnits = 8;        // unit buffers of scales

struct TcPiece {
  int tile, rt, kb0, kb1;
};
// The CTA's steps [x0, x1) unit by unit.  One division at the start: three
// 64-bit ones a unit took a role longer than the three stages of a K of 768.
template <typename F>
__device__ __forceinline__ void tc_pieces(int x0, int x1, int n_st, int RT, F f) {
  const int u = x0 / n_st;
  TcPiece pc{u / RT, u % RT, x0 - u * n_st, 0};
  for (int left = x1 - x0; left > 0;) {
    pc.kb1 = min(n_st, pc.kb0 + left);
    if (!f(pc)) return;
    left -= pc.kb1 - pc.kb0;
    pc.kb0 = 0;
    if (++pc.rt == RT) {
      pc.rt = 0;
      ++pc.tile;
    }
  }
}

// 16 bytes of shared memory at any address, those past the first `valid` as
// zero (whole words around them are read).
__device__ __forceinline__ uint4 tc_lds16(uint32_t addr, int valid, bool aligned) {
  uint32_t w[5];
  if (aligned) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint32_t base = addr & ~3u, sh = (addr & 3u) * 8;
#pragma unroll
  for (int i = 0; i < 5; ++i)
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(base + 4 * i));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = __funnelshift_r(w[i], w[i + 1], sh);
    const int left = valid - 4 * i;
    if (left < 4) w[i] = left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The MMA's columns of a tile of n pairs (16 are its step), and the bytes of
// a full tile's stage (whole 8-row swizzle atoms).
__host__ __device__ __forceinline__ uint32_t tc_cols(int n, int pieces) {
  return (uint32_t)(n * pieces + 15) / 16 * 16;
}
__host__ __device__ __forceinline__ uint32_t tc_b_stage(int cap, int pieces) {
  return tc_cols(cap, pieces) * kTcRow;
}

__host__ __device__ __forceinline__ uint32_t tc_unit_bytes(int K) {
  return (uint32_t)align_up((size_t)128 * (K / 16) + 16, 128);
}

// An epilogue thread's row of a tile's n pairs, four at a time:
// out[c stride] = the sum of pair c's kNp columns, column q times 4^-q, from
// the smallest piece up, times its multiplier (lane c's mul).
template <int kNp>
__device__ __forceinline__ void tc_drain(uint32_t taddr, int n, float mul, bool store, float* out,
                                         int64_t stride) {
  constexpr int kAt = 4, kLoads = kAt * kNp / 8;
  static_assert(kAt * kNp % 8 == 0, "whole 8-column loads");
  for (int c = 0; c < n; c += kAt) {
    uint32_t v[kLoads][8];
    const int cols = min(kAt, n - c) * kNp;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (8 * i < cols) tmem_ld8(taddr + c * kNp + 8 * i, v[i]);
    tc_wait_ld();
#pragma unroll
    for (int h = 0; h < kAt; ++h) {
      const float m = __shfl_sync(0xFFFFFFFFu, mul, (c + h) & 31);
      if (c + h < n && store) {
        float sum = __uint_as_float(v[(h * kNp + kNp - 1) / 8][(h * kNp + kNp - 1) % 8]);
#pragma unroll
        for (int q = kNp - 2; q >= 0; --q)
          sum = __fmaf_rn(sum, 1.0f / kResidualUp,
                          __uint_as_float(v[(h * kNp + q) / 8][(h * kNp + q) % 8]));
        out[(c + h) * stride] = sum * m;
      }
    }
  }
}

// Registers: at most 112, so that a CTA of the prep kernel fits beside one of
// a product (the bound names more threads than there are).
template <bool kTma>
__global__ void __launch_bounds__(576, 1)
    moe_tc_kernel(const __grid_constant__ CUtensorMap tm_w,  // codes, or their even rows
                  const __grid_constant__ CUtensorMap tm_2,  // scales, or the odd rows
                  const TcGemm p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int ring = p.ring;
  const uint32_t b_stage = tc_b_stage(p.cap, p.pieces);
  uint8_t* s_a = smem;
  uint8_t* s_b = s_a + ring * kTcAStage;
  uint8_t* s_sfa = s_b + ring * b_stage;
  uint8_t* s_sfb = s_sfa + ring * kTcSfStage;
  uint8_t* s_odd = s_sfb + ring * kTcSfStage;
  // scales as stored: a slot a stage, or whole units
  uint8_t* s_raw = s_odd + (kTma ? 0 : ring * kTcOddStage);
  __shared__ TcTables s_tab;
  __shared__ uint64_t full[kTcMaxRing], empty[kTcMaxRing];
  __shared__ uint64_t raw_full[kTcMaxRing], raw_empty[kTcMaxUnits];
  __shared__ uint64_t odd_full[kTcMaxRing], d_full[2], d_empty[2], done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t s_abort;
  volatile int32_t* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ring; ++i) {
      mbar_init(&full[i], 2 + kTcScaleWarps + (kTma ? 0 : kTcOddWarps));
      mbar_init(&empty[i], 1);
      mbar_init(&odd_full[i], 1);
    }
    for (int i = 0; i < kTcMaxUnits; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kTcScaleWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);
    }
    mbar_init(&done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tma_prefetch_desc(&tm_w);
    if (!kTma || !p.unit_scales) tma_prefetch_desc(&tm_2);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tc_fence_before();
  }
  // The expert ids were complete before the kernel ahead of this one let it
  // start; its own results are waited for where they are read.
  tc_tables(p.ids, p.P, p.E, p.cap, s_tab, threadIdx.x, blockDim.x, 0, [](int, int) {}, [] {});
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);
  const WaitCtl wc{p.status, abort_flag, kWaitLimitNs};

  const int n_st = (p.K + 255) / 256, RT = (p.N + 127) / 128, nb = p.K / 16;
  const int64_t S = (int64_t)s_tab.tile[p.E] * RT * n_st;
  const int64_t G = tc_ctas(S, gridDim.x);
  const bool works = blockIdx.x < G;
  // at most 1024 tiles x 512 row tiles x 128 stages
  const int x0 = works ? (int)tc_bound(S, blockIdx.x, G) : 0;
  const int x1 = works ? (int)tc_bound(S, blockIdx.x + 1, G) : 0;
  // a tile is looked up once: its units follow one another
  int known = -1;
  TcTile tile{};
  auto tile_at = [&](int t) {
    if (t != known) {
      tile = tc_tile(s_tab, p.E, p.cap, t);
      known = t;
    }
    return tile;
  };

  if (warp == 0) {
    // ---------------- weight codes, and scales where they come per stage
    const uint64_t once = policy_evict_first();
    uint32_t issued = 0;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      const int r0 = tile_at(pc.tile).expert * p.N + pc.rt * 128;
      for (int kb = pc.kb0; kb < pc.kb1; ++kb, ++issued) {
        const uint32_t st = issued % ring, ph = (issued / ring) & 1;
        if (!warp_wait(&empty[st], ph ^ 1, wc)) return false;
        if (elect_one()) {
          if constexpr (kTma) {
            if (!p.unit_scales) {
              mbar_arrive_expect_tx(&raw_full[st], kTcSfStage);
              tma_load_2d_hint(s_raw + st * kTcSfStage, &tm_2, kb * 16, r0, &raw_full[st], once);
            }
            mbar_arrive_expect_tx(&full[st], kTcAStage);
            tma_load_2d_hint(s_a + st * kTcAStage, &tm_w, kb * 128, r0, &full[st], once);
          } else {
            mbar_arrive_expect_tx(&odd_full[st], kTcOddStage);
            tma_load_2d_hint(s_odd + st * kTcOddStage, &tm_2, kb * 128, r0 / 2, &odd_full[st],
                             once);
            mbar_arrive_expect_tx(&full[st], kTcAStage / 2);
            tma_load_2d_hint(s_a + st * kTcAStage, &tm_w, kb * 128, r0 / 2, &full[st], once);
          }
        }
        __syncwarp();
      }
      return true;
    });
    if (!kTma) drain_loads(odd_full, ring, issued, 0, p.status);
    else if (!p.unit_scales) drain_loads(raw_full, ring, issued, 0, p.status);
    // codes and activations of a stage land on one barrier, which the MMA
    // warp waits for; what an aborted call left in flight lands here
    if (*abort_flag) drain_loads(full, ring, issued, 0, p.status);
  } else if (warp == 3) {
    // ---------------- the pairs' pieces and their scales
    grid_dependency_wait();
    const uint64_t keep = policy_evict_last();
    uint32_t issued = 0;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      const TcTile t = tile_at(pc.tile);
      for (int kb = pc.kb0; kb < pc.kb1; ++kb, ++issued) {
        const uint32_t st = issued % ring, ph = (issued / ring) & 1;
        if (!warp_wait(&empty[st], ph ^ 1, wc)) return false;
        if (elect_one()) {
          const uint32_t bytes = (uint32_t)t.n * p.pieces * kTcRow;
          mbar_arrive_expect_tx(&full[st], bytes + kTcSfStage);
          bulk_load(s_b + st * b_stage, p.act + ((int64_t)kb * p.P + t.first) * p.pieces * kTcRow, bytes,
                    &full[st], keep);
          bulk_load(s_sfb + st * kTcSfStage, p.sf + ((int64_t)kb * p.tiles_max + pc.tile) * kTcSfStage,
                    kTcSfStage, &full[st], keep);
        }
        __syncwarp();
      }
      return true;
    });
    drain_loads(full, ring, issued, 0, p.status);
  } else if (warp == 2) {
    // ---------------- the scales of a unit's rows, one contiguous copy
    if (p.unit_scales) {
      const uint64_t once = policy_evict_first();
      uint32_t issued = 0;
      tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
        const uint32_t buf = issued % p.unit_scales, ph = (issued / p.unit_scales) & 1;
        if (!warp_wait(&raw_empty[buf], ph ^ 1, wc)) return false;
        const int64_t r0 = (int64_t)tile_at(pc.tile).expert * p.N + pc.rt * 128;
        if (elect_one()) {
          const uint32_t bytes = (uint32_t)min(128, p.N - pc.rt * 128) * nb;
          mbar_arrive_expect_tx(&raw_full[buf], bytes);
          bulk_load(s_raw + buf * tc_unit_bytes(p.K), p.scales + r0 * nb, bytes, &raw_full[buf], once);
        }
        __syncwarp();
        ++issued;
        return true;
      });
      drain_loads(raw_full, p.unit_scales, issued, 0, p.status);
    }
  } else if (warp == 1) {
    // ---------------- scales into TMEM, then one MMA per 64 k
    const uint64_t ad0 = smem_desc_sw128(smem_u32(s_a)), bd0 = smem_desc_sw128(smem_u32(s_b));
    const uint32_t n_cols = tc_cols(p.cap, p.pieces);
    const uint32_t sf_base = tmem + 2 * n_cols;
    uint32_t g = 0;
    int i = 0;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      const TcTile t = tile_at(pc.tile);
      // (columns past the tile's are computed from what the slot held before,
      // and read by nobody)
      const uint32_t idesc = idesc_e2m1_bs(tc_cols(t.n, p.pieces));
      const uint32_t buf = i & 1, dph = (i >> 1) & 1;
      ++i;
      if (!warp_wait(&d_empty[buf], dph ^ 1, wc)) return false;
      tc_fence_after();
      const uint32_t d = tmem + buf * n_cols;
      for (int kb = pc.kb0; kb < pc.kb1; ++kb, ++g) {
        const uint32_t st = g % ring, ph = (g / ring) & 1;
        if (!warp_wait(&full[st], ph, wc)) return false;
        tc_fence_after();
        const uint64_t ad = ad0 + ((st * kTcAStage) >> 4), bd = bd0 + ((st * b_stage) >> 4);
        const uint32_t sfa = sf_base + st * kTcSfCols, sfb = sfa + 16;
        const int n_at = min(4, (p.K - 256 * kb + 63) / 64);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j < n_at) {
              tc_cp_32x128b_x4(sfa + 4 * j, smem_u32(s_sfa + st * kTcSfStage + 512 * j));
              tc_cp_32x128b_x4(sfb + 4 * j, smem_u32(s_sfb + st * kTcSfStage + 512 * j));
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < n_at)
              tc_mma_fp4_bs(d, ad + 2 * j, bd + 2 * j, idesc, sfa + 4 * j, sfb + 4 * j,
                            (kb != pc.kb0) || (j != 0));
          tc_commit(&empty[st]);
        }
        __syncwarp();
      }
      if (elect_one()) tc_commit(&d_full[buf]);
      __syncwarp();
      return true;
    });
    // What comes next reads the prep kernel's places ahead of its own wait: a
    // CTA without work lets it start no sooner than that kernel is complete.
    grid_dependency_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (elect_one()) tc_commit(&done_bar);
    __syncwarp();
    volatile int32_t zero = 0;
    WaitCtl drain{p.status, &zero, 100000000ull};
    mbar_wait(&done_bar, 0, drain);
  } else if (warp < 8) {
    // ---------------- epilogue: a row a thread; a pair's pieces are summed
    grid_dependency_wait();  // the multipliers
    const int row = tc_row(kTma, (warp & 3) * 32 + lane);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    int i = 0, mul_of = -1;
    float mul = 0.0f;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      const TcTile t = tile_at(pc.tile);
      const uint32_t buf = i & 1, dph = (i >> 1) & 1;
      ++i;
      if (pc.tile != mul_of) {
        mul = lane < t.n ? __ldcg(p.mul + t.first + lane) : 0.0f;
        mul_of = pc.tile;
      }
      if (!warp_wait(&d_full[buf], dph, wc)) return false;
      tc_fence_after();
      const bool whole = pc.kb0 == 0 && pc.kb1 == n_st;
      const int n = pc.rt * 128 + row;
      float* out;
      int64_t stride;
      if (whole) {
        out = p.dst + (int64_t)t.first * p.N + n;
        stride = p.N;
      } else {
        out = p.part + (int64_t)tc_slot(blockIdx.x, pc.kb0 == 0) * p.cap * 128 + row;
        stride = 128;
      }
      const uint32_t d = tmem + buf * tc_cols(p.cap, p.pieces) + lane_off;
      if (p.pieces == kPiecesBf16)
        tc_drain<kPiecesBf16>(d, t.n, mul, n < p.N, out, stride);
      else
        tc_drain<kPieces>(d, t.n, mul, n < p.N, out, stride);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[buf]);
      return true;
    });
  } else if (warp < 8 + kTcScaleWarps) {
    // ---------------- weight scales from the order they are stored in to the
    // one tcgen05.cp reads (atom j, row 32 a + b: byte b 16 + a 4 of atom j);
    // warp a takes rows 32 a ..: one warp for all four took 1480 cycles a
    // stage where rows are not 16-byte multiples
    const int a = warp - 8, r = tc_row(kTma, 32 * a + lane);
    const bool aligned = !p.unit_scales || nb % 16 == 0;
    uint32_t bad = 0, it = 0, units = 0;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      const bool live = r < p.N - pc.rt * 128;  // a row of the unit
      const uint32_t buf = p.unit_scales ? units % p.unit_scales : 0;
      if (p.unit_scales && !warp_wait(&raw_full[buf], (units / p.unit_scales) & 1, wc)) return false;
      for (int kb = pc.kb0; kb < pc.kb1; ++kb, ++it) {
        const uint32_t st = it % ring, ph = (it / ring) & 1;
        if (!p.unit_scales && !warp_wait(&raw_full[st], ph, wc)) return false;
        const uint32_t from = p.unit_scales
                                  ? smem_u32(s_raw) + buf * tc_unit_bytes(p.K) + r * nb + 16 * kb
                                  : smem_u32(s_raw) + st * kTcSfStage + r * 16;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (live) v = tc_lds16(from, nb - 16 * kb, aligned);
        if (!warp_wait(&empty[st], ph ^ 1, wc)) return false;
        uint32_t* to = reinterpret_cast<uint32_t*>(s_sfa + st * kTcSfStage) + lane * 4 + a;
        to[0] = v.x;
        to[128] = v.y;
        to[256] = v.z;
        to[384] = v.w;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        bad |= bad_scales4(v.x) | bad_scales4(v.y) | bad_scales4(v.z) | bad_scales4(v.w);
      }
      ++units;
      __syncwarp();
      if (p.unit_scales && lane == 0) mbar_arrive(&raw_empty[buf]);
      return true;
    });
    if (__any_sync(0xFFFFFFFFu, bad != 0u)) {
      grid_dependency_wait();  // the prep kernel clears the status
      if (lane == 0) raise_status(p.status, NVFP4_ERR_NONFINITE);
    }
  } else if constexpr (!kTma) {
    // ---------------- the odd rows into place: eight lanes a row
    const int tid = threadIdx.x - kTcThreads, row = tid >> 3, c = tid & 7;
    uint32_t it = 0;
    tc_pieces(x0, x1, n_st, RT, [&](const TcPiece& pc) {
      for (int kb = pc.kb0; kb < pc.kb1; ++kb, ++it) {
        const uint32_t st = it % ring, ph = (it / ring) & 1;
        if (!warp_wait(&empty[st], ph ^ 1, wc) || !warp_wait(&odd_full[st], ph, wc)) return false;
        const uint32_t from = smem_u32(s_odd + st * kTcOddStage) + row * kTcOddRow + 8 + 16 * c;
        const uint32_t to = smem_u32(s_a + st * kTcAStage) + kTcAStage / 2 + row * 128 +
                            ((c ^ (row & 7)) << 4);
        uint32_t v[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 16 rows at a time
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                       : "=r"(v[q][0]), "=r"(v[q][1])
                       : "r"(from + q * 16 * kTcOddRow));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                       : "=r"(v[q][2]), "=r"(v[q][3])
                       : "r"(from + q * 16 * kTcOddRow + 8));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + q * 16 * 128),
                       "r"(v[q][0]), "r"(v[q][1]), "r"(v[q][2]), "r"(v[q][3])
                       : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
      return true;
    });
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ between the products
// The CTAs that share the unit of (tile, row tile), and where its sum lies.
struct TcSpan {
  int b0, b1;
};
__device__ __forceinline__ TcSpan tc_span(int64_t S, int grid, int n_st, int RT, int tile, int rt) {
  const int64_t x = ((int64_t)tile * RT + rt) * n_st;
  const int64_t G = tc_ctas(S, grid);
  return {tc_owner(S, x, G), tc_owner(S, x + n_st - 1, G)};
}

// Eight consecutive values of h a thread, so that a warp's are the stage it
// splits and stay in its registers (beyond 1024 threads they are computed
// again once the row's maximum is known).  CTAs this small (I of 768: 96
// threads) leave the next product's CTAs room beside them, whose weights are
// then under way while h is computed: 64 tokens 72.4 against 74.1 us with 256
// threads and h in shared memory.  Where there are more pairs than fit at once
// they start late (193 tokens of 8); a grid of what fits, looping, took 4% longer.
constexpr int kActMaxThreads = 1024;
static int act_threads(int64_t I) {
  return (int)std::min<int64_t>((I / 8 + 31) / 32 * 32, kActMaxThreads);
}

__global__ void __launch_bounds__(kActMaxThreads) moe_act_kernel(const TcArgs p) {
  // a split buffer a warp, the spans of the 2I / 128 row tiles
  extern __shared__ __align__(16) uint8_t s_act_mem[];
  __shared__ uint32_t s_max;
  const int n_threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = 2 * p.I, RT = (N + 127) / 128, n_st = (p.H + 255) / 256;
  uint8_t* buf = s_act_mem + warp * kSplitBytes;
  TcSpan* s_span = reinterpret_cast<TcSpan*>(s_act_mem + n_threads / 32 * kSplitBytes);
  // where a pair and its sums lie: written by the prep kernel, which was
  // complete before the product this kernel waits for began
  const int2 counts = __ldcg(p.counts);
  const int64_t S = (int64_t)counts.y * RT * n_st;
  const int64_t slot = (int64_t)p.cap * 128;
  const int q = blockIdx.x;
  const bool present = q < counts.x;
  TcPlace at{};
  if (present) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.by_place) + q);
    at = {v.x, v.y, v.z, q};
    for (int r = tid; r < RT; r += n_threads) s_span[r] = tc_span(S, p.grid, n_st, RT, at.tile, r);
  }
  if (tid == 0) s_max = 0u;
  __syncthreads();
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!present) return;
  const float g13 = __ldg(p.g13 + at.expert);
  // columns n .. n + 3 of gu: a unit that was cut has its parts added in order
  auto first = [&](int n, TcSpan sp) {
    return __ldcg(reinterpret_cast<const float4*>(
        sp.b0 == sp.b1 ? p.gu + (int64_t)q * N + n
                       : p.part1 + tc_slot(sp.b0, true) * slot + at.col * 128 + (n & 127)));
  };
  auto part = [&](int n, int b) {
    return __ldcg(reinterpret_cast<const float4*>(p.part1 + tc_slot(b, false) * slot +
                                                  at.col * 128 + (n & 127)));
  };
  auto values = [&](int i, float (&h)[8]) {
    float4 v[4];
    TcSpan sp[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {  // gate, up; i, i + 4
      const int n = (a & 1) * p.I + i + (a >> 1) * 4;
      sp[a] = s_span[n >> 7];
      v[a] = first(n, sp[a]);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int n = (a & 1) * p.I + i + (a >> 1) * 4;
      for (int b = sp[a].b0 + 1; b <= sp[a].b1; ++b) {
        const float4 o = part(n, b);
        v[a].x += o.x;
        v[a].y += o.y;
        v[a].z += o.z;
        v[a].w += o.w;
      }
    }
    auto act = [&](float g, float u) {
      g *= g13;
      return g / (1.0f + __expf(-g)) * (u * g13);
    };
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      h[4 * a] = act(v[2 * a].x, v[2 * a + 1].x);
      h[4 * a + 1] = act(v[2 * a].y, v[2 * a + 1].y);
      h[4 * a + 2] = act(v[2 * a].z, v[2 * a + 1].z);
      h[4 * a + 3] = act(v[2 * a].w, v[2 * a + 1].w);
    }
  };
  float h[8];
  uint32_t mx = 0;
  for (int i = 8 * tid; i < p.I; i += 8 * n_threads) {
    values(i, h);
#pragma unroll
    for (int a = 0; a < 8; ++a) mx = max(mx, __float_as_uint(h[a]) & 0x7FFFFFFFu);
  }
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  if (lane == 0) atomicMax(&s_max, mx);
  __syncthreads();
  float undo;
  const float up = tc_scale(s_max, undo);
  if (tid == 0) p.mul2[q] = undo;
  const int stages = (p.I + 255) / 256;
  for (int s = warp; s < stages; s += n_threads / 32) {
    const int i = 256 * s + 8 * lane;
    if (stages > n_threads / 32 && i < p.I) values(i, h);
#pragma unroll
    for (int a = 0; a < 8; ++a) h[a] = i < p.I ? h[a] * up : 0.0f;
    __syncwarp();
    tc_split(h, p.pieces, buf);
    tc_place(buf, p.pieces, s, at, p.P, p.tiles_max, p.act2, p.sf2);
  }
}

// out[m, :] = sum over the slots j of w[m, j] G2[e] y[pair], a 128-row tile of
// y a warp, four rows a lane.
template <bool kBf16>
__global__ void __launch_bounds__(256) moe_tc_combine_kernel(const TcArgs p) {
  const int lane = threadIdx.x & 31;
  const int RT = (p.H + 127) / 128, n_st = (p.I + 255) / 256;
  const int rt = blockIdx.x * 8 + (threadIdx.x >> 5), m = blockIdx.y;
  const int64_t S = (int64_t)__ldcg(p.counts).y * RT * n_st;
  const int n = rt * 128 + 4 * lane;
  const bool live = n < p.H;
  const int64_t slot = (int64_t)p.cap * 128;
  constexpr int kAt = 8;  // slots whose loads are in flight together
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = 0; j0 < p.k; j0 += kAt) {
    // lane j looks up slot j0 + j (what the prep kernel wrote: the first
    // round's ahead of the wait for the product)
    int4 at = make_int4(0, 0, 0, -1);
    TcSpan sp{0, 0};
    float w = 0.0f;
    if (lane < kAt && j0 + lane < p.k) {
      const int64_t i = (int64_t)m * p.k + j0 + lane;
      w = __ldg(p.weights + i);
      at = __ldcg(reinterpret_cast<const int4*>(p.by_pair) + i);
      if (at.w >= 0) {
        sp = tc_span(S, p.grid, n_st, RT, at.y, rt < RT ? rt : 0);
        w *= __ldg(p.g2 + at.x);
      }
    }
    if (j0 == 0) {
      grid_dependency_wait();
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    float4 v[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int place = __shfl_sync(0xFFFFFFFFu, at.w, j), col = __shfl_sync(0xFFFFFFFFu, at.z, j);
      const int b0 = __shfl_sync(0xFFFFFFFFu, sp.b0, j), b1 = __shfl_sync(0xFFFFFFFFu, sp.b1, j);
      v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (place >= 0 && live)
        v[j] = __ldcg(reinterpret_cast<const float4*>(
            b0 == b1 ? p.y + (int64_t)place * p.H + n
                     : p.part2 + tc_slot(b0, true) * slot + (int64_t)col * 128 + 4 * lane));
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int place = __shfl_sync(0xFFFFFFFFu, at.w, j), col = __shfl_sync(0xFFFFFFFFu, at.z, j);
      const int b0 = __shfl_sync(0xFFFFFFFFu, sp.b0, j), b1 = __shfl_sync(0xFFFFFFFFu, sp.b1, j);
      const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
      if (place < 0 || !live) continue;
      for (int b = b0 + 1; b <= b1; ++b) {
        const float4 o = __ldcg(reinterpret_cast<const float4*>(
            p.part2 + tc_slot(b, false) * slot + (int64_t)col * 128 + 4 * lane));
        v[j].x += o.x;
        v[j].y += o.y;
        v[j].z += o.z;
        v[j].w += o.w;
      }
      sum.x = __fmaf_rn(wj, v[j].x, sum.x);
      sum.y = __fmaf_rn(wj, v[j].y, sum.y);
      sum.z = __fmaf_rn(wj, v[j].z, sum.z);
      sum.w = __fmaf_rn(wj, v[j].w, sum.w);
    }
  }
  if (!live) return;
  const int64_t at = ((int64_t)m * p.H + n) >> 2;
  if constexpr (kBf16) {
    uint2 o;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(sum.y), "f"(sum.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(sum.w), "f"(sum.z));
    reinterpret_cast<uint2*>(p.out)[at] = o;
  } else {
    reinterpret_cast<float4*>(p.out)[at] = sum;
  }
}

// ------------------------------------------------------------ host side
struct TcLayout {
  size_t counts, by_pair, by_place, mul1, mul2, sf1, sf2, act1, act2, gu, y, part1, part2, total;
  int tiles_max;
};

// Pairs of a tile: 8 where no expert has more (unless a token names it
// twice), 16 where few do, else what 128 columns hold: a second tile of an
// expert reads its weights again, from L2, but in as many steps as the first.
static int tc_cap(int64_t P, int64_t M, int64_t E, int pieces) {
  return M <= 8 ? 8 : P <= 6 * E ? 16 : std::min(128 / pieces, kTcMaxCap);
}

static TcLayout tc_layout(int64_t M, int64_t k, int64_t H, int64_t I, int sms) {
  const int64_t P = M * k, cap = kTcMaxCap;  // either size of tile
  const int64_t st1 = (H + 255) / 256, st2 = (I + 255) / 256;
  TcLayout L;
  // every tile but one per expert is full
  L.tiles_max = (int)(std::min<int64_t>(P, kTcMaxExperts) + P / 8);
  size_t at = kWsHeader;
  auto put = [&](size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes, 256);
    return here;
  };
  L.counts = put(sizeof(int2));
  L.by_pair = put((size_t)P * sizeof(TcPlace));
  L.by_place = put((size_t)P * sizeof(TcPlace));
  L.mul1 = put((size_t)P * 4);
  L.mul2 = put((size_t)P * 4);
  L.sf1 = put((size_t)st1 * L.tiles_max * kTcSfStage);
  L.sf2 = put((size_t)st2 * L.tiles_max * kTcSfStage);
  L.act1 = put((size_t)st1 * P * kPieces * kTcRow);
  L.act2 = put((size_t)st2 * P * kPieces * kTcRow);
  L.gu = put((size_t)P * 2 * I * 4);
  L.y = put((size_t)P * H * 4);
  L.part1 = put((size_t)2 * sms * cap * 128 * 4);
  L.part2 = put((size_t)2 * sms * cap * 128 * 4);
  L.total = at;
  return L;
}

size_t moe_tc_workspace_bytes(int64_t M, int64_t k, int64_t H, int64_t I) {
  return tc_layout(M, k, H, I, std::max(sm_count(), 1)).total;
}

// Scales of a unit's rows are loaded at once, or per stage by TMA, whose row
// stride is a 16-byte multiple.
static bool tc_k_ok(int64_t K) { return K <= kTcMaxUnitK || K % 256 == 0; }
bool moe_tc_takes(int64_t k, int64_t H, int64_t I) {
  return k <= kTcMaxK && tc_k_ok(H) && tc_k_ok(I);
}

// The small kernels ask for the shared-memory split of the products: an SM
// changes its split only when it is idle, so a product's CTA could not start
// beside one of them, or had to wait for the change.
static cudaError_t tc_carveout_once(std::atomic<uint64_t>& done, const void* kern) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

static cudaError_t tc_gemm_launch(TcGemm g, int grid, cudaStream_t stream) {
  CUtensorMap tm = {}, tm_2 = {};
  const bool tma = g.K % 32 == 0;  // TMA steps from row to row
  // two units' scales, or as many as 20 KB hold: the next unit's are asked for
  // one buffer round ahead (K = 768, 64 tokens: 23 us with two)
  g.unit_scales = g.K > kTcMaxUnitK
                      ? 0
                      : std::max(2, std::min(kTcMaxUnits, (int)((20 << 10) / tc_unit_bytes(g.K))));
  const uint64_t row = (uint64_t)g.K / 2;
  if (tma ? !encode_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes, row, (uint64_t)g.rows, row, 128,
                       128, CU_TENSOR_MAP_SWIZZLE_128B)
          // (an even number of rows: N is a multiple of 16)
          : !encode_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes, row, (uint64_t)g.rows / 2,
                       2 * row, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
                !encode_2d(&tm_2, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes + row - 8, row + 8,
                           (uint64_t)g.rows / 2, 2 * row, kTcOddRow, 64,
                           CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorUnknown;
  if (!g.unit_scales &&  // (K % 256 == 0)
      !encode_2d(&tm_2, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.scales, (uint64_t)g.K / 16,
                 (uint64_t)g.rows, (uint64_t)g.K / 16, 16, 128, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorUnknown;
  // 24 to 47 KB a stage beside the units' scales: 3 to 7 stages
  const size_t stage =
      kTcAStage + tc_b_stage(g.cap, g.pieces) + (g.unit_scales ? 2 : 3) * (size_t)kTcSfStage +
      (tma ? 0 : kTcOddStage);
  const size_t units = g.unit_scales * (size_t)tc_unit_bytes(g.K);
  g.ring = (int)std::min<size_t>((kTcSmem - 1024 - units) / stage, kTcMaxRing);
  const size_t smem = 1024 + units + (size_t)g.ring * stage;
  static std::atomic<uint64_t> limit_set[2];
  auto kern = tma ? moe_tc_kernel<true> : moe_tc_kernel<false>;
  const cudaError_t err =
      smem_limit_once(limit_set[tma], reinterpret_cast<const void*>(kern), kTcSmem);
  if (err != cudaSuccess) return err;
  PdlLaunch l(dim3((unsigned)grid), dim3(kTcThreads + (tma ? 0 : 32 * kTcOddWarps)), smem, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, tm, tm_2, g);
}

nvfp4_status moe_tc_launch(const void* x, int64_t M, int64_t k, int64_t H, int64_t I, int64_t E,
                           const int32_t* ids, const float* weights, const uint8_t* p13,
                           const uint8_t* s13, const float* g13, const uint8_t* p2,
                           const uint8_t* s2, const float* g2, void* out, int out_dtype,
                           void* workspace, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return NVFP4_ERR_CUDA;
  const TcLayout L = tc_layout(M, k, H, I, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TcArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.ids = ids;
  a.weights = weights;
  a.g13 = g13;
  a.g2 = g2;
  a.out = out;
  a.M = (int)M;
  a.k = (int)k;
  a.H = (int)H;
  a.I = (int)I;
  a.E = (int)E;
  a.P = (int)(M * k);
  a.tiles_max = L.tiles_max;
  a.grid = sms;
  a.pieces = out_dtype == NVFP4_OUT_BF16 ? kPiecesBf16 : kPieces;
  a.cap = tc_cap(M * k, M, E, a.pieces);
  a.counts = reinterpret_cast<int2*>(ws + L.counts);
  a.by_pair = reinterpret_cast<TcPlace*>(ws + L.by_pair);
  a.by_place = reinterpret_cast<TcPlace*>(ws + L.by_place);
  a.act1 = ws + L.act1;
  a.sf1 = ws + L.sf1;
  a.act2 = ws + L.act2;
  a.sf2 = ws + L.sf2;
  a.mul1 = reinterpret_cast<float*>(ws + L.mul1);
  a.mul2 = reinterpret_cast<float*>(ws + L.mul2);
  a.gu = reinterpret_cast<float*>(ws + L.gu);
  a.y = reinterpret_cast<float*>(ws + L.y);
  a.part1 = reinterpret_cast<float*>(ws + L.part1);
  a.part2 = reinterpret_cast<float*>(ws + L.part2);
  a.status = reinterpret_cast<int32_t*>(ws);

  TcGemm g = {};
  g.cap = a.cap;
  g.pieces = a.pieces;
  g.ids = ids;
  g.E = a.E;
  g.P = a.P;
  g.tiles_max = a.tiles_max;
  g.status = a.status;
  TcGemm g1 = g, g2a = g;
  g1.codes = p13;
  g1.scales = s13;
  g1.rows = E * 2 * I;
  g1.N = (int)(2 * I);
  g1.K = (int)H;
  g1.act = a.act1;
  g1.sf = a.sf1;
  g1.mul = a.mul1;
  g1.dst = a.gu;
  g1.part = a.part1;
  g2a.codes = p2;
  g2a.scales = s2;
  g2a.rows = E * H;
  g2a.N = (int)H;
  g2a.K = (int)I;
  g2a.act = a.act2;
  g2a.sf = a.sf2;
  g2a.mul = a.mul2;
  g2a.dst = a.y;
  g2a.part = a.part2;

  cudaError_t err;
  {
    static std::atomic<uint64_t> split_set{0};
    err = tc_carveout_once(split_set, reinterpret_cast<const void*>(moe_prep_kernel));
    PdlLaunch l(dim3((unsigned)M), dim3(2 * kPrepHalf), align_up((size_t)a.P * 2, 16), stream);
    if (err == cudaSuccess) err = cudaLaunchKernelEx(&l.cfg, moe_prep_kernel, a);
  }
  if (err == cudaSuccess) err = tc_gemm_launch(g1, sms, stream);
  if (err == cudaSuccess) {
    const int threads = act_threads(I);
    const size_t smem =
        (size_t)threads / 32 * kSplitBytes + (size_t)((2 * I + 127) / 128) * sizeof(TcSpan);
    static std::atomic<uint64_t> split_set{0};
    err = tc_carveout_once(split_set, reinterpret_cast<const void*>(moe_act_kernel));
    if (err == cudaSuccess) {
      PdlLaunch l(dim3((unsigned)a.P), dim3(threads), smem, stream);
      err = cudaLaunchKernelEx(&l.cfg, moe_act_kernel, a);
    }
  }
  if (err == cudaSuccess) err = tc_gemm_launch(g2a, sms, stream);
  if (err == cudaSuccess) {
    const int RT = (int)((H + 127) / 128);
    const bool bf16 = out_dtype == NVFP4_OUT_BF16;
    auto kern = bf16 ? moe_tc_combine_kernel<true> : moe_tc_combine_kernel<false>;
    static std::atomic<uint64_t> split_set[2];
    err = tc_carveout_once(split_set[bf16], reinterpret_cast<const void*>(kern));
    PdlLaunch l(dim3((unsigned)((RT + 7) / 8), (unsigned)M), dim3(256), 0, stream);
    if (err == cudaSuccess) err = cudaLaunchKernelEx(&l.cfg, kern, a);
  }
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace nvfp4
