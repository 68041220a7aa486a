// few.cu -- the whole layer for a few tokens (T <= 16) in one cooperative kernel.
//
//   logits = x Wg^T (summed in fp64, rounded to fp32), the k experts of each
//   token and their weights as moe_router_topk;
//   y[t] = sum_j w[t,j] (silu(x W1e) * (x W3e)) W2e + shared(x[t]).
//
// With at most 16 tokens an expert sees one or two rows, so the layer is a
// stream of the chosen experts' weights through the SMs (bound by HBM: 3 d I
// weights an expert against 2 T operations a weight) and everything else is
// latency to be kept out of the stream's way.  One CTA per SM, four roles:
//   consumers (16 warps)  logits of a share of the experts, then the products
//                         and the two joins, with grid barriers between them;
//   producer (1 warp)     fills a ring of stages with weight tiles by TMA, ahead
//                         of the consumers and across the ends of pieces and
//                         phases: the shared expert's up projections need no
//                         routing and stream while it is found, and the first
//                         tiles of the down projections are in the ring before
//                         the barriers that the activations wait for;
//   columns (1 warp)      follows the tiles and brings the activations that go with
//                         them, several stages' at a time (bulk copies; copies of
//                         single stages, 128 bytes each, cost more than the
//                         weights: 710 instead of 455 us at T = 8 with 28 experts
//                         of 7168 x 2048 in bf16);
//   router (2 warps)      waits for all logits, finds the top-k (in every CTA)
//                         and the list of chosen experts and their rows; then
//                         brings the block scales of coded weights, and h's
//                         factors, beside the tiles (a consumer's own load one
//                         stage ahead comes too late: 0.6 us a stage of e4m3
//                         where HBM needs 0.37).
//
// Split of the work.  A segment is 128 output columns of one matrix of one
// expert, a unit the part of its contraction that one stage holds (16 KB of
// weights: 64 steps of bf16, 128 of e4m3, 256 of MXFP4), a chunk a run of at most
// 32 units of one segment.  CTAs claim chunks from a counter: SMs do not see the
// same bandwidth (with equal shares the slowest took 290 us for what others did
// in 230), and a claim is made a chunk ahead, so it costs nothing.  A chunk's
// sums go to a place of its own and who needs a segment adds its chunks in order:
// no floating-point atomics, and equal inputs give equal bits.
//
// Arithmetic: mma.sync m16n8k16 with the weights as the A operand (16 output
// columns by 16 steps, ldmatrix from the stage) and the activations as B's
// columns, 8 at a time.  (tcgen05 would pad the columns to 16 and could not take
// these codes unconverted; the tensor pipe is idle either way.)  Consumer warp w
// takes columns 16 (w % 8) of every second tile (w / 8): a tile's chain of waits,
// loads and MMAs is longer than the time HBM needs for one.
//   bf16 weights: x is bf16 as it comes; h is fp32 and goes in as three bf16
//   terms (8 bits each: 24 in all).
//   e4m3 and MXFP4 codes become fp16, which holds them exactly, by moving their
//   bits: exponent and mantissa read 2^-8 and 2^-14 times the code's value there,
//   made up in the sums' factors.  (The conversion instructions run at a sixteenth
//   of the rate; e4m3 MMAs are made of conversions and fp16 ones on this GPU, 2280
//   instructions a stage.)  x and h are fp16 too, times a power of two that puts
//   the largest of a token (of 128 values of h) between 2^14 and 2^15: a bf16 x
//   fits exactly down to 2^-28 of the largest and to 2^-39 of it below; h goes in
//   as two terms (22 bits).
// Block scales multiply fp32 sums.
#include <algorithm>
#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"
#include "few.h"

namespace moe {
namespace {

constexpr int kWarps = 16;  // consumers
constexpr int kThreads = 32 * kWarps;
constexpr int kRouterWarps = 2;  // 20 warps in all, which leaves a thread 96 registers
constexpr int kAllThreads = kThreads + 64 + 32 * kRouterWarps;
constexpr int kMaxNT = 3;       // 8-column B tiles of one pass
constexpr int kMaxCols = 8 * kMaxNT;
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = kFewMaxTokens * 32;  // T * k
constexpr uint32_t kTileBytes = 16384;

constexpr int kStages = 8;
constexpr uint32_t kColBytes = 16384;  // of a buffer of B columns; there are two

constexpr int kRedPitch = 17;  // floats of one B column of a warp pair's 16 output columns
constexpr int kRedFloats = 2 * kMaxCols * kRedPitch;  // of a pair of warps

struct Lists {  // what the routing leaves in shared memory
  int32_t idx[kMaxRows];      // [T][k]
  float w[kMaxRows];
  int16_t ent[kMaxRows];      // entries t * k + j ordered by expert, then token
  int16_t row_of[kMaxRows];   // the inverse
  int16_t expert[kMaxRows];   // distinct experts, ascending
  int16_t start[kMaxRows + 1];
  int16_t place[kMaxExperts];  // of an expert among the distinct ones
  int32_t counts[kMaxExperts];
  int n;                      // distinct experts
};

struct Control {
  uint64_t full[kStages], empty[kStages];
  uint64_t col_full[2], col_empty[2];
  // a stage's chunk is known, its tile on the way: two turns of the ring, since
  // who has no part in a stage may still be looking at it when the stage's place
  // is filled again, but not when the place after it is
  uint64_t issued[2 * kStages];
  uint64_t scaled[kStages];   // its scales are there
  uint64_t started;           // `first` is there
  int first;                  // first stage of the routed experts
  uint64_t ready;   // h is there, in all CTAs
  int chunk[2 * kStages];  // which chunk a stage belongs to; -1: the share is done
  uint64_t routed;  // the lists are there
  uint32_t abort, never;
};

__device__ __forceinline__ void consumer_sync() { ptx::named_barrier(9, kThreads); }
__device__ __forceinline__ void router_sync() { ptx::named_barrier(10, 32 * kRouterWarps); }

// ------------------------------------------------------------ grid barrier
// The consumers' writes so far are visible to who waits.
__device__ __forceinline__ void grid_arrive(uint32_t* bar) {
  consumer_sync();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(bar, 1u);
  }
}

// One thread's wait for all CTAs' arrivals.
__device__ __forceinline__ bool grid_poll(const uint32_t* bar, uint32_t* status, volatile uint32_t* abort) {
  const uint64_t t0 = ptx::globaltimer();
  uint32_t n = 0, seen;
  while (true) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(bar) : "memory");
    if (seen >= gridDim.x) break;
    if ((++n & 63u) == 0) {
      if (*abort) return false;
      if (ptx::globaltimer() - t0 > kWaitLimitNs) {
        raise_status(status, abort, kStatusTimeout);
        return false;
      }
    }
  }
  __threadfence();
  return true;
}

__device__ bool grid_wait(const uint32_t* bar, uint32_t* status, volatile uint32_t* abort) {
  if (threadIdx.x == 0) grid_poll(bar, status, abort);
  consumer_sync();
  return *abort == 0;
}

// Sum of a segment's chunks in order, four columns a lane, eight loads at a time.
__device__ __forceinline__ float4 sum_parts(const float* at, int parts) {
  const float4* v = reinterpret_cast<const float4*>(at) + (threadIdx.x & 31);
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = 0; i < parts; i += 8) {
    float4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < parts) b[j] = __ldcg(v + (i + j) * (kFewCols / 4));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j < parts) {
        a.x += b[j].x;
        a.y += b[j].y;
        a.z += b[j].z;
        a.w += b[j].w;
      }
    }
  }
  return a;
}

// ------------------------------------------------------------ tiles and columns
// The loads and MMAs of a stage are left to the compiler to arrange; these two keep
// them between the wait for the stage and its release.
__device__ __forceinline__ void after_wait(uint32_t& tile, uint32_t& cols) {
  asm volatile("" : "+r"(tile), "+r"(cols)::"memory");
}

template <int NT>
__device__ __forceinline__ void before_release(float (&acc)[NT][4]) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
    asm volatile("" : "+f"(acc[j][0]), "+f"(acc[j][1]), "+f"(acc[j][2]), "+f"(acc[j][3])::"memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Four e4m3 codes to two fp16 pairs, bytes (0, 2) and (1, 3), times 2^-8.  The
// code 0x7f, NaN, is not looked at (it reads 480).
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t& even, uint32_t& odd) {
  even = ((w << 8) & 0x80008000u) | ((w << 7) & 0x3f803f80u);
  odd = (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
}

// The same times 1 by the conversion instruction, NaN included.
__device__ __forceinline__ uint32_t e4m3_values(uint32_t two_codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two_codes));
  return r;
}

// Eight MXFP4 codes to four fp16 pairs, codes j and j + 4, times 2^-14.
__device__ __forceinline__ void mx_pairs(uint32_t w, uint32_t (&f)[4]) {
  f[0] = ((w << 12) & 0x80008000u) | ((w << 9) & 0x0e000e00u);
  f[1] = ((w << 8) & 0x80008000u) | ((w << 5) & 0x0e000e00u);
  f[2] = ((w << 4) & 0x80008000u) | ((w << 1) & 0x0e000e00u);
  f[3] = (w & 0x80008000u) | ((w >> 3) & 0x0e000e00u);
}

__device__ __forceinline__ void lds(uint32_t (&r)[4], uint32_t addr) {
  asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// Four scale bytes as 2^(byte - 127), 255 as NaN: through bf16, which holds them all.
__device__ __forceinline__ void scales_of(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  f[0] = ptx::bf16_lo(lo);
  f[1] = ptx::bf16_hi(lo);
  f[2] = ptx::bf16_lo(hi);
  f[3] = ptx::bf16_hi(hi);
}

// Values k and k + 1 (k even) of a column of fp16: in order, but for MXFP4 with
// steps 8c + j and 8c + j + 4 side by side, as the codes come apart.
template <int WT>
__device__ __forceinline__ void store_pair(uint16_t* column, int k, uint32_t v) {
  if (WT == kFewMxfp4) {
    uint16_t* to = column + (k & ~7) + 2 * (k & 3) + ((k >> 2) & 1);
    to[0] = (uint16_t)v;
    to[2] = (uint16_t)(v >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(column + k) = v;
  }
}

// One stage of a piece: a warp's sums for its 16 columns.  cols: the stage's part of
// the first B column, the others `pitch` bytes apart, up to column `last` (which
// stands in for those that do not exist: an MMA's columns do not mix).
// bf16: two boxes of 64 columns, [steps][64 columns].
template <int NT>
__device__ __forceinline__ void stage_bf16(uint32_t tile, uint32_t cols, int pitch, int last, float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t b[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) ldsm(b[j], cols + min(8 * j + r, last) * pitch + (32 * p + 8 * i) * 2);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 32 * p + 16 * q + (i >> 1) * 8 + r;
      const int chunk = (warp & 3) * 2 + (i & 1);
      uint32_t a[4];
      ldsm_t(a, tile + ((warp >> 2) & 1) * 8192 + k * 128 + ((chunk ^ (k & 7)) << 4));
#pragma unroll
      for (int j = 0; j < NT; ++j) mma_bf16(acc[j], a, b[j][2 * q], b[j][2 * q + 1]);
    }
  }
}

// e4m3: [steps][128 columns] codes; a 16-bit unit of ldmatrix is two columns of
// one step, so a register holds columns 2g and 2g + 1 of steps 2c and 2c + 1.
// True where the tile has a code 0x7f, whose sums are to be done again with NANS.
template <int NT, bool NANS>
__device__ __forceinline__ bool e4m3_sums(uint32_t tile, uint32_t cols, int pitch, int last, float (&part)[NT][4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7;
  uint32_t seen = 0;  // a byte's top bit, which adding 1 flips where the seven others are set
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[j][e] = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int k = 32 * q + 8 * i + r;
    uint32_t w[4], a[4][2];
    ldsm_t(w, tile + k * 128 + (((warp & 7) ^ (k & 7)) << 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (NANS) {
        a[e][0] = e4m3_values(__byte_perm(w[e], 0, 0x4420));
        a[e][1] = e4m3_values(__byte_perm(w[e], 0, 0x4431));
      } else {
        e4m3_pairs(w[e], a[e][0], a[e][1]);
        seen |= (w[e] + 0x01010101u) ^ w[e];
      }
    }
    const uint32_t a0[4] = {a[0][0], a[0][1], a[1][0], a[1][1]}, a1[4] = {a[2][0], a[2][1], a[3][0], a[3][1]};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t b[4];
      ldsm(b, cols + min(8 * j + r, last) * pitch + (32 * q + 8 * i) * 2);
      mma_f16(part[j], a0, b[0], b[1]);
      mma_f16(part[j], a1, b[2], b[3]);
    }
  }
  return (seen & 0x80808080u) != 0;
}

// f[j]: the block's scale times the columns' factor.
template <int NT>
__device__ __forceinline__ void stage_e4m3(uint32_t tile, uint32_t cols, int pitch, int last, const float (&f)[NT],
                                           float (&acc)[NT][4]) {
  float part[NT][4];
  float up = 256.0f;
  if (__any_sync(0xffffffffu, e4m3_sums<NT, false>(tile, cols, pitch, last, part))) {
    e4m3_sums<NT, true>(tile, cols, pitch, last, part);
    up = 1.0f;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(part[j][e], f[j] * up, acc[j][e]);
}

// MXFP4: [128 columns][steps / 2] codes, one half of the steps; lane (g, c) holds
// the eight codes 8c of a scale block for columns g and g + 8, whose scale bytes
// are in s[0], s[1].  f[j]: the columns' factor.
template <int NT>
__device__ __forceinline__ void stage_mxfp4(uint32_t tile, int half, uint32_t cols, int pitch, int last,
                                            const uint32_t (&s)[2], const float (&f)[NT], float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7, g = lane >> 2, c = lane & 3;
  const int n = (warp & 7) * 16 + (i & 1) * 8 + r;
  float sum[NT][4] = {};
  float s0[4], s1[4];
  scales_of(s[0], s0);
  scales_of(s[1], s1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {  // two scale blocks
    uint32_t w[4];
    const int chunk = half * 4 + 2 * p + (i >> 1);
    ldsm(w, tile + n * 128 + ((chunk ^ (n & 7)) << 4));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int blk = 2 * p + q;
      uint32_t x[4], y[4];
      mx_pairs(w[2 * q], x);
      mx_pairs(w[2 * q + 1], y);
      const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        lds(b, cols + min(8 * j + g, last) * pitch + (half * 128 + blk * 32 + 8 * c) * 2);
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_f16(part, a0, b[0], b[1]);
        mma_f16(part, a1, b[2], b[3]);
        sum[j][0] = fmaf(part[0], s0[blk], sum[j][0]);
        sum[j][1] = fmaf(part[1], s0[blk], sum[j][1]);
        sum[j][2] = fmaf(part[2], s1[blk], sum[j][2]);
        sum[j][3] = fmaf(part[3], s1[blk], sum[j][3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(sum[j][e], f[j] * 16384.0f, acc[j][e]);
}

// ------------------------------------------------------------ shares and pieces
// B columns that a row of h takes.
__host__ __device__ constexpr int terms(int weights) { return weights == kFewBf16 ? 3 : 2; }

// A chunk, or one pass over it: units [step0, step1) of 128 output columns of
// one matrix, for `rows` rows of `group` B columns each.
struct Piece {
  int mat;     // 0: W1, 1: W3, 2: W2
  int expert;  // slice of the routed weights
  int col0, step0, step1;
  int first;   // place of the first row in the list (shared expert: token)
  int rows, group;
  bool again;  // the weights are read by another pass too
  float* out;  // sums of the first row, [128]
  int64_t ld;  // to the next row's
};

// Up projections: segments are (expert, W1 or W3, column block), the shared
// expert sees every token in order.  Down projections: segments are (expert,
// column block) and B holds the terms of each row's h.  Sums lie as [row][matrix]
// [column block][chunk of the segment][128].
template <int WT, bool SHARED, bool DOWN>
struct Share {
  int K, N, blocks, steps, per_expert, total;
  FewSplit split;
  float* buf;
  __device__ __forceinline__ Share(const FewParams& p, const Lists& ls) {
    const int inner = SHARED ? p.S : p.I;
    K = DOWN ? inner : p.d;
    N = DOWN ? p.d : inner;
    blocks = N / kFewCols;
    steps = (K + few_unit_steps(WT) - 1) / few_unit_steps(WT);
    per_expert = DOWN ? blocks : 2 * blocks;
    split = SHARED ? (DOWN ? p.split_dn_s : p.split_up_s) : (DOWN ? p.split_dn_r : p.split_up_r);
    buf = SHARED ? (DOWN ? p.dn_s : p.up_s) : (DOWN ? p.dn_r : p.up_r);
    total = (SHARED ? 1 : ls.n) * per_expert * split.parts;
  }
  __device__ __forceinline__ Piece chunk(const FewParams& p, const Lists& ls, int id) const {
    Piece q;
    const int seg = id / split.parts, part = id - seg * split.parts;
    const int ei = seg / per_expert, in = seg - ei * per_expert;
    q.mat = DOWN ? 2 : in >= blocks ? 1 : 0;
    q.col0 = (in - (q.mat == 1 ? blocks : 0)) * kFewCols;
    q.step0 = part * split.units;
    q.step1 = min(steps, q.step0 + split.units);
    q.expert = SHARED ? 0 : ls.expert[ei];
    q.first = SHARED ? 0 : ls.start[ei];
    q.rows = SHARED ? p.T : ls.start[ei + 1] - q.first;
    q.group = DOWN ? terms(WT) : 1;
    q.again = q.rows > kPass;
    q.ld = (int64_t)per_expert * split.parts * kFewCols;
    q.out = buf + q.first * q.ld + ((int64_t)in * split.parts + part) * kFewCols;
    return q;
  }
  // Rows of a pass: at most 8 in the down projections (more read the weights
  // again, from L2 mostly: only the shared expert and crowded small layers have
  // them).
  static constexpr int kPass = DOWN ? 8 : kFewMaxTokens;
  template <typename F>
  __device__ __forceinline__ bool passes(Piece q, F f) const {
    const int all = q.rows;
    for (int r0 = 0; r0 < all; r0 += kPass) {
      q.rows = min(kPass, all - r0);
      if (!f(q)) return false;
      q.first += kPass;
      q.out += kPass * q.ld;
    }
    return true;
  }
};

// How many units' columns a buffer takes for a piece, and the columns' distance
// in bytes: a pad keeps the reads of 8 columns off each other's banks.
template <int WT>
struct ColumnPlan {
  static constexpr int kUnitBytes = 2 * few_unit_steps(WT);
  static constexpr int kPad = WT == kFewMxfp4 ? 64 : 16;
  int units, pitch;
  __device__ __forceinline__ explicit ColumnPlan(const Piece& q) {
    const int cols = q.rows * q.group;
    units = min(q.step1 - q.step0, ((int)kColBytes / cols - kPad) / kUnitBytes);
    pitch = units * kUnitBytes + kPad;
  }
};
// every piece has room for one unit's columns
static_assert((int)kColBytes / kMaxCols >= 2 * 64 + 16 && (int)kColBytes / 16 >= 2 * 256 + 64, "B columns");

// The rings' positions: stages and column buffers handed over so far, and which
// phase of its `scaled` barrier each stage is in (only routed stages have one).
struct Ring {
  int n = 0, cols = 0;
  uint32_t scaled = 0;
};

// What goes with a stage's tile of codes: MXFP4's scale bytes of both halves of
// the steps for each of the 128 columns, and a factor for each row of h (e4m3: for
// each row, the block's scale times it) and half.
struct StageScales {
  uint32_t words[kFewCols][2];
  float factor[8][2];
};

struct Smem {
  StageScales* scales;
  uint8_t* stages;
  uint8_t* cols;
  float* red;
  Control* c;
};

// ------------------------------------------------------------ producer
// The weight tile of unit `step` of a piece.
template <int WT, bool SHARED>
__device__ __forceinline__ void load_tile(const FewMaps& m, const FewParams& p, const Piece& q, int step, uint8_t* to,
                                          uint64_t* bar, uint64_t policy) {
  const CUtensorMap* map = SHARED ? &m.shared[q.mat] : &m.routed[q.mat];
  if (WT == kFewBf16) {
    ptx::tma_load_3d(to, map, bar, q.col0, step * 64, q.expert, policy);
    ptx::tma_load_3d(to + 8192, map, bar, q.col0 + 64, step * 64, q.expert, policy);
  } else if (WT == kFewE4m3) {
    ptx::tma_load_3d(to, map, bar, q.col0, step * 128, q.expert, policy);
  } else {
    const int N = q.mat == 2 ? p.d : p.I;
    ptx::tma_load_2d(to, map, bar, step * 128, q.expert * N + q.col0, policy);
  }
}

template <int WT, bool SHARED, bool DOWN>
__device__ bool produce(const FewMaps& m, const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring,
                        uint32_t* counter) {
  const int lane = threadIdx.x & 31;
  const uint64_t once = ptx::policy_evict_first(), more = ptx::policy_evict_normal();
  Control& c = *sm.c;
  const Share<WT, SHARED, DOWN> share(p, ls);
  auto slot_free = [&] {
    if (warp_wait(&c.empty[ring.n % kStages], ((ring.n / kStages) & 1) ^ 1, &c.abort)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  int id = blockIdx.x;
  while (id < share.total) {
    int claimed = 0;
    if (lane == 0) claimed = (int)atomicAdd(counter, 1u) + gridDim.x;  // used after this chunk
    const bool ok = share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      for (int step = q.step0; step < q.step1; ++step, ++ring.n) {
        const int s = ring.n % kStages;
        if (!slot_free()) return false;
        if (lane == 0) {
          c.chunk[ring.n % (2 * kStages)] = id;
          ptx::mbar_arrive(&c.issued[ring.n % (2 * kStages)]);
          ptx::mbar_arrive_expect_tx(&c.full[s], kTileBytes);
          load_tile<WT, SHARED>(m, p, q, step, sm.stages + s * kTileBytes, &c.full[s], q.again ? more : once);
        }
        __syncwarp();
      }
      return true;
    });
    if (!ok) return false;
    id = __shfl_sync(0xffffffffu, claimed, 0);
  }
  if (!slot_free()) return false;
  if (lane == 0) {
    c.chunk[ring.n % (2 * kStages)] = -1;
    ptx::mbar_arrive(&c.issued[ring.n % (2 * kStages)]);
    ptx::mbar_arrive(&c.full[ring.n % kStages]);
  }
  ++ring.n;
  return true;
}

// ------------------------------------------------------------ columns
template <int WT, bool SHARED, bool DOWN>
__device__ bool bring_columns(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int kSteps = few_unit_steps(WT);
  const int lane = threadIdx.x & 31;
  const Share<WT, SHARED, DOWN> share(p, ls);
  Control& c = *sm.c;
  auto wait = [&](uint64_t* bar, int n) {
    if (warp_wait(bar, n & 1, &c.abort)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  // a stage is also released by this warp, so that its chunk is still to be read
  auto next_stage = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.empty[ring.n % kStages]);
    ++ring.n;
  };
  int id = blockIdx.x < share.total ? (int)blockIdx.x : -1;  // the first chunk needs no tile to be known by
  while (true) {
    if (id < 0) {
      if (!wait(&c.issued[ring.n % (2 * kStages)], ring.n / (2 * kStages))) return false;
      next_stage();
      return true;
    }
    const bool ok = share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      const ColumnPlan<WT> plan(q);
      const int cols = q.rows * q.group;
      const uint8_t* src = nullptr;
      if (lane < cols) {
        if (DOWN)
          src = (SHARED ? p.h_s : p.h_r) + ((int64_t)q.first * terms(WT) + lane) * share.K * 2;
        else
          src = (WT == kFewBf16 ? p.x : p.x16) + (SHARED ? q.first + lane : ls.ent[q.first + lane] / p.k) * (int64_t)p.d * 2;
      }
      for (int step = q.step0; step < q.step1; ++step) {
        if ((step - q.step0) % plan.units == 0) {
          const int buf = ring.cols & 1;
          if (!wait(&c.col_empty[buf], (ring.cols >> 1) + 1)) return false;
          const int last = min(q.step1, step + plan.units);
          const uint32_t bytes = 2 * (min(share.K, last * kSteps) - step * kSteps);
          if (lane == 0) ptx::mbar_arrive_expect_tx(&c.col_full[buf], bytes * cols);
          __syncwarp();
          if (lane < cols)
            bulk_load(ptx::smem_u32(sm.cols) + buf * kColBytes + lane * plan.pitch, src + step * kSteps * 2, bytes,
                      &c.col_full[buf]);
          ++ring.cols;
        }
        if (!wait(&c.issued[ring.n % (2 * kStages)], ring.n / (2 * kStages))) return false;
        next_stage();
      }
      return true;
    });
    if (!ok || !wait(&c.issued[ring.n % (2 * kStages)], ring.n / (2 * kStages))) return false;
    id = c.chunk[ring.n % (2 * kStages)];
  }
}

// ------------------------------------------------------------ scales
// The scales of a routed share, by the router's warps: MXFP4's by all 64 threads,
// two columns each, e4m3's by the first warp.
template <int WT, bool DOWN>
__device__ bool bring_scales(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int kGroup = 4;  // units whose loads go together
  const int lane = threadIdx.x & 31;
  const int tid = threadIdx.x - kAllThreads + 32 * kRouterWarps;
  const Share<WT, false, DOWN> share(p, ls);
  Control& c = *sm.c;
  auto wait = [&](int n) {
    if (warp_wait(&c.issued[n % (2 * kStages)], (n / (2 * kStages)) & 1, &c.abort)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  auto hand_over = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.scaled[ring.n % kStages]);
    ++ring.n;
  };
  const int words = share.K / 128;
  int id = blockIdx.x < share.total ? (int)blockIdx.x : -1;
  while (true) {
    if (id < 0) {
      if (!wait(ring.n)) return false;
      hand_over();
      return true;
    }
    const bool ok = share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      const uint8_t* scales = q.mat == 0 ? p.s1 : q.mat == 1 ? p.s3 : p.s2;
      for (int step0 = q.step0; step0 < q.step1; step0 += kGroup) {
        if constexpr (WT == kFewE4m3) {
          // lane 8 u + r: unit u of the group, row r of the piece
          const int step = step0 + (lane >> 3), row = lane & 7;
          float f = 0.0f;
          if (step < q.step1) {
            f = __ldg(reinterpret_cast<const float*>(scales) +
                      ((int64_t)q.expert * (share.K / 128) + step) * (share.N / 128) + q.col0 / 128);
            if (DOWN && row < q.rows) f *= __ldcg(p.h_scale + (int64_t)(q.first + row) * (share.K / 128) + step);
          }
          for (int u = 0; u < kGroup && step0 + u < q.step1; ++u) {
            if (!wait(ring.n)) return false;
            if ((lane >> 3) == u && tid < 32) {
              float* to = sm.scales[ring.n % kStages].factor[row];
              to[0] = f;
              to[1] = f;
            }
            hand_over();
          }
        } else {
          uint32_t w[kGroup][2][2];
          float f[kGroup];
          const int row = (tid >> 1) & 7, half = tid & 1;
#pragma unroll
          for (int u = 0; u < kGroup; ++u) {
            const int step = step0 + u;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t* at = reinterpret_cast<const uint32_t*>(scales) +
                                   ((int64_t)q.expert * share.N + q.col0 + tid + 64 * i) * words + 2 * step;
              if (step >= q.step1) {
                w[u][i][0] = w[u][i][1] = 0u;
              } else if ((words & 1) == 0) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
                w[u][i][0] = v.x;
                w[u][i][1] = v.y;
              } else {
                w[u][i][0] = __ldg(at);
                w[u][i][1] = 2 * step + 1 < words ? __ldg(at + 1) : 0u;
              }
            }
            f[u] = 1.0f;
            if (DOWN && tid < 16 && row < q.rows && step < q.step1 && 2 * step + half < words)
              f[u] = __ldcg(p.h_scale + (int64_t)(q.first + row) * words + 2 * step + half);
          }
#pragma unroll
          for (int u = 0; u < kGroup; ++u) {
            if (step0 + u < q.step1) {
              if (!wait(ring.n)) return false;
              StageScales& to = sm.scales[ring.n % kStages];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint2*>(to.words[tid + 64 * i]) = make_uint2(w[u][i][0], w[u][i][1]);
              if (tid < 16) to.factor[row][half] = f[u];
              hand_over();
            }
          }
        }
      }
      return true;
    });
    if (!ok || !wait(ring.n)) return false;
    id = c.chunk[ring.n % (2 * kStages)];
  }
}

// ------------------------------------------------------------ consumers
template <int WT, int NT, bool DOWN>
__device__ __forceinline__ void consume_piece(const FewParams& p, const Piece& q, int K, const Smem& sm, Ring& ring) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3, team = warp >> 3;
  Control& ct = *sm.c;
  float acc[NT][4] = {};
  const ColumnPlan<WT> plan(q);
  const int last = q.rows * q.group - 1;
  int left = 0;  // units whose columns are in the buffer
  uint32_t cols = 0;
  // A wait that fails raises the abort flag, which ends all later ones at once, and
  // the piece goes on with whatever the buffers hold: its barriers need every
  // warp, and the share ends at the next chunk.
  auto arrived = [&](uint64_t* bar, uint32_t parity) {
    if (!ptx::wait_bounded(bar, parity, &ct.abort)) raise_status(p.status, &ct.abort, kStatusTimeout);
  };
  for (int step = q.step0; step < q.step1; ++step) {
    if (left == 0) {
      const int buf = ring.cols & 1;
      arrived(&ct.col_full[buf], (ring.cols >> 1) & 1);
      cols = ptx::smem_u32(sm.cols) + buf * kColBytes;
      left = min(plan.units, q.step1 - step);
    }
    const int slot = ring.n % kStages;
    if ((ring.n & 1) == team) {
      arrived(&ct.full[slot], (ring.n / kStages) & 1);
      uint32_t tile = ptx::smem_u32(sm.stages) + slot * kTileBytes;
      if constexpr (WT == kFewBf16) {
        after_wait(tile, cols);
        stage_bf16<NT>(tile, cols, plan.pitch, last, acc);
      } else {
        arrived(&ct.scaled[slot], (ring.scaled >> slot) & 1);
        after_wait(tile, cols);
        const StageScales& sc = sm.scales[slot];
        const int halves = WT == kFewMxfp4 && 2 * step + 1 < K / 128 ? 2 : 1;  // MXFP4's last unit may be half of one
        for (int h = 0; h < halves; ++h) {
          float f[NT];  // of the row that columns 2c and 2c + 1 belong to
#pragma unroll
          for (int j = 0; j < NT; ++j)
            f[j] = sc.factor[DOWN && NT <= 2 ? 4 * j + c : 0][h];
          if constexpr (WT == kFewE4m3) {
            stage_e4m3<NT>(tile, cols, plan.pitch, last, f, acc);
          } else {
            const uint32_t s[2] = {sc.words[(warp & 7) * 16 + g][h], sc.words[(warp & 7) * 16 + g + 8][h]};
            stage_mxfp4<NT>(tile, h, cols, plan.pitch, last, s, f, acc);
          }
        }
      }
      before_release<NT>(acc);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ct.empty[slot]);
    }
    if (WT != kFewBf16) ring.scaled ^= 1u << slot;
    cols += ColumnPlan<WT>::kUnitBytes;
    ++ring.n;
    if (--left == 0) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ct.col_empty[ring.cols & 1]);
      ++ring.cols;
    }
  }
  // the two teams' sums, and the terms of each row, are joined by the
  // pair of warps that has these 16 columns
  const int pair = warp & 7;
  float* red = sm.red + pair * kRedFloats;
  const int lo = WT == kFewE4m3 ? 2 * g : g, hi = WT == kFewE4m3 ? 2 * g + 1 : g + 8;
  float* to = red + team * kMaxCols * kRedPitch;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    to[(8 * j + 2 * c) * kRedPitch + lo] = acc[j][0];
    to[(8 * j + 2 * c + 1) * kRedPitch + lo] = acc[j][1];
    to[(8 * j + 2 * c) * kRedPitch + hi] = acc[j][2];
    to[(8 * j + 2 * c + 1) * kRedPitch + hi] = acc[j][3];
  }
  ptx::named_barrier(1 + pair, 64);
  for (int i = team * 32 + lane; i < q.rows * 16; i += 64) {
    const int r = i >> 4, col = i & 15;
    float a = 0.0f;
    for (int t = 0; t < q.group; ++t) {
      const float* x = red + (r * q.group + t) * kRedPitch + col;
      a += x[0] + x[kMaxCols * kRedPitch];
    }
    q.out[r * q.ld + pair * 16 + col] = a;
  }
  ptx::named_barrier(1 + pair, 64);
}

template <int WT, bool SHARED, bool DOWN>
__device__ bool consume(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  const Share<WT, SHARED, DOWN> share(p, ls);
  Control& ct = *sm.c;
  volatile uint32_t* abort = &ct.abort;
  while (true) {
    const int at = ring.n % (2 * kStages);
    const bool there = warp_wait(&ct.issued[at], (ring.n / (2 * kStages)) & 1, &ct.abort);
    if (!there) raise_status(p.status, &ct.abort, kStatusTimeout);
    // both warps of a pair take the chunk or neither
    if (!ptx::named_barrier_and(1 + ((threadIdx.x >> 5) & 7), 64, there && *abort == 0)) return false;
    const int id = ct.chunk[at];
    if (id < 0) {
      const int slot = ring.n % kStages;
      if (WT != kFewBf16) {  // the scales' warps still read the mark
        if (!ptx::wait_bounded(&ct.scaled[slot], (ring.scaled >> slot) & 1, &ct.abort))
          raise_status(p.status, &ct.abort, kStatusTimeout);
        ring.scaled ^= 1u << slot;
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0 && (ring.n & 1) == (threadIdx.x >> 8)) ptx::mbar_arrive(&ct.empty[slot]);
      ++ring.n;
      return true;
    }
    share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      const int cols = q.rows * q.group;
      if (cols <= 8)
        consume_piece<WT, 1, DOWN>(p, q, share.K, sm, ring);
      else if (cols <= 16 || terms(WT) == 2)
        consume_piece<WT, 2, DOWN>(p, q, share.K, sm, ring);
      else
        consume_piece<WT, terms(WT) == 2 ? 2 : 3, DOWN>(p, q, share.K, sm, ring);
      return true;
    });
  }
}

// ------------------------------------------------------------ router
// Logits of this CTA's experts: 8 warps for an expert and a few tokens, sums in fp64 (the products
// of two bf16 values are exact there and the sum is good to 2^-53 of its
// terms), rounded once.
__device__ void logits_share(const FewParams& p, double* red) {
  constexpr int kG = 4;  // tokens of a job at most; fewer where there are CTAs for it
  const int group = min(kG, (p.E * p.T + 2 * (int)gridDim.x - 1) / (2 * (int)gridDim.x));
  const int groups = (p.T + group - 1) / group;
  const int half = threadIdx.x >> 8, tid = threadIdx.x & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = p.d / 8;
  for (int job0 = blockIdx.x * 2; job0 < p.E * groups; job0 += gridDim.x * 2) {
    const int job = job0 + half;  // E is even, and so is their number
    const int e = job % p.E, t0 = job / p.E * group, n = min(group, p.T - t0);
    double acc[kG] = {};
    for (int v = tid; v < nv; v += 256) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.Wg + (int64_t)e * p.d * 2) + v);
      uint4 xv[kG];
#pragma unroll
      for (int t = 0; t < kG; ++t)
        if (t < n) xv[t] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + t) * p.d * 2) + v);
      const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
      double w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = (double)ptx::bf16_lo(ww[i]);
        w[2 * i + 1] = (double)ptx::bf16_hi(ww[i]);
      }
#pragma unroll
      for (int t = 0; t < kG; ++t) {
        if (t < n) {
          const uint32_t xx[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t] = fma(w[2 * i], (double)ptx::bf16_lo(xx[i]), acc[t]);
            acc[t] = fma(w[2 * i + 1], (double)ptx::bf16_hi(xx[i]), acc[t]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kG; ++t) {
      if (t < n) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        if (lane == 0) red[warp * kG + t] = acc[t];
      }
    }
    consumer_sync();
    if (tid < n) {
      double a = 0.0;
#pragma unroll
      for (int w = 0; w < 8; ++w) a += red[(half * 8 + w) * kG + tid];
      p.logits[(int64_t)(t0 + tid) * p.E + e] = (float)a;
    }
    consumer_sync();
  }
}

// Doubles in the order of unsigned numbers, -0 as 0 and NaN as the lowest.
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ double of_ordered(uint64_t b) {
  return __longlong_as_double((long long)((b >> 63) ? b & 0x7fffffffffffffffull : ~b));
}

// Lowest index among the lanes' largest keys (index 0x7fffffff: no candidate).
__device__ __forceinline__ int warp_best(uint64_t key, int idx) {
  const bool in = idx != 0x7fffffff;
  const uint32_t hi = in ? (uint32_t)(key >> 32) : 0u, top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = in && hi == top ? (uint32_t)key : 0u, low = __reduce_max_sync(0xffffffffu, lo);
  return (int)__reduce_min_sync(0xffffffffu, in && hi == top && (uint32_t)key == low ? (uint32_t)idx : 0x7fffffffu);
}

// The k experts of token t and their weights, by one warp.  Scores that decide
// the selection are fp64 (of the fp32 logits); a NaN score ranks last.
__device__ void choose(const FewParams& p, Lists& ls, int t, uint64_t* key, float* logit) {
  const int lane = threadIdx.x & 31;
  const float* l = p.logits + (int64_t)t * p.E;
#pragma unroll 8
  for (int e = lane; e < p.E; e += 32) logit[e] = __ldcg(l + e);
  for (int e = lane; e < p.E; e += 32) {
    const double v = (double)logit[e];
    key[e] = ordered(p.route == 0 ? v : 1.0 / (1.0 + exp(-v)) + (p.bias ? (double)__ldg(p.bias + e) : 0.0));
  }
  __syncwarp();
  uint32_t taken = 0;  // bit v: expert 32 v + lane is out
  if (p.route == 1) {
    const int size = p.E / p.n_group;
    uint64_t mine = 0;
    int group = 0x7fffffff;
    if (lane < p.n_group) {
      uint64_t used = 0;
      double sum = 0.0;
      for (int r = 0; r < p.group_topn; ++r) {
        int bi = -1;
        uint64_t bv = 0;
        for (int i = 0; i < size; ++i)
          if (!((used >> i) & 1) && (bi < 0 || key[lane * size + i] > bv)) {
            bi = i;
            bv = key[lane * size + i];
          }
        used |= 1ull << bi;
        sum += bv == 0 ? -__longlong_as_double(0x7ff0000000000000ll) : of_ordered(bv);
      }
      mine = ordered(sum);
      group = lane;
    }
    uint32_t kept = 0;
    for (int r = 0; r < p.topk_group; ++r) {
      const int b = warp_best(mine, group);
      kept |= 1u << b;
      if (lane == b) group = 0x7fffffff;
    }
    for (int e = lane, v = 0; e < p.E; e += 32, ++v)
      if (!((kept >> (e / size)) & 1)) taken |= 1u << v;
  }
  // each lane holds its best; only the lane that gave one away looks again
  uint64_t best = 0;
  int at = 0x7fffffff;
  auto look = [&] {
    at = 0x7fffffff;
    for (int e = lane, v = 0; e < p.E; e += 32, ++v)
      if (!((taken >> v) & 1) && (at == 0x7fffffff || key[e] > best)) {
        best = key[e];
        at = e;
      }
  };
  look();
  int my_idx = 0;
  for (int j = 0; j < p.k; ++j) {
    const int b = warp_best(best, at);
    if (at == b) {
      taken |= 1u << (b >> 5);
      look();
    }
    if (lane == j) my_idx = b;
  }
  const int top = __shfl_sync(0xffffffffu, my_idx, 0);
  float w;
  if (p.route == 0) {
    const float e = lane < p.k ? expf(logit[my_idx] - logit[top]) : 0.0f;
    float den = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    w = e / den;
  } else {
    const double s = lane < p.k ? 1.0 / (1.0 + exp(-(double)logit[my_idx])) : 0.0;
    double den = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    w = (float)((double)p.route_scale * s / den);
  }
  if (lane < p.k) {
    ls.idx[t * p.k + lane] = my_idx;
    ls.w[t * p.k + lane] = w;
  }
  __syncwarp();
}

// Routing of all tokens and the lists of chosen experts and their rows, by the
// router's warps.
__device__ void route(const FewParams& p, Lists& ls, uint64_t* keys) {
  constexpr int kThreads = 32 * kRouterWarps;
  const int tid = threadIdx.x - kAllThreads + kThreads;
  const int warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < p.E; e += kThreads) ls.counts[e] = 0;
  for (int t = warp; t < p.T; t += kRouterWarps)
    choose(p, ls, t, keys + warp * p.E, reinterpret_cast<float*>(keys + kRouterWarps * p.E) + warp * p.E);
  router_sync();
  const int n = p.T * p.k;
  for (int i = tid; i < n; i += kThreads) atomicAdd(&ls.counts[ls.idx[i]], 1);
  router_sync();
  if (warp == 0) {
    int chosen = 0, rows = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int cnt = ls.counts[e0 + lane];
      const uint32_t any = __ballot_sync(0xffffffffu, cnt > 0);
      int before = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const int total = __shfl_sync(0xffffffffu, before, 31);
      if (cnt > 0) {
        const int at = chosen + __popc(any & ((1u << lane) - 1u));
        ls.expert[at] = (int16_t)(e0 + lane);
        ls.start[at] = (int16_t)(rows + before - cnt);
        ls.place[e0 + lane] = (int16_t)at;
      }
      chosen += __popc(any);
      rows += total;
    }
    if (lane == 0) {
      ls.start[chosen] = (int16_t)rows;
      ls.n = chosen;
    }
  }
  router_sync();
  for (int i = tid; i < n; i += kThreads) {
    const int e = ls.idx[i];
    int at = ls.start[ls.place[e]];
    for (int q = 0; q < i; ++q) at += ls.idx[q] == e ? 1 : 0;
    ls.ent[at] = (int16_t)i;
    ls.row_of[i] = (int16_t)at;
  }
  if (blockIdx.x == 0) {
    for (int i = tid; i < n; i += kThreads) {
      if (p.idx_out) p.idx_out[i] = ls.idx[i];
      if (p.w_out) p.w_out[i] = ls.w[i];
    }
    if (p.counts_out)
      for (int e = tid; e < p.E; e += kThreads) p.counts_out[e] = ls.counts[e];
  }
  router_sync();
}

// ------------------------------------------------------------ between the products
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// The three bf16 terms of v: its upper 8 bits, the next 8, and the rest.
__device__ __forceinline__ void terms_of(float v, uint32_t (&t)[3]) {
  const uint32_t b = __float_as_uint(v);
  t[0] = b >> 16;
  if ((b & 0x7f800000u) == 0x7f800000u) {  // infinities and NaN stand alone
    if ((b & 0x007fffffu) != 0) t[0] |= 0x40u;
    t[1] = t[2] = 0;
    return;
  }
  const float r = v - __uint_as_float(b & 0xffff0000u);
  t[1] = __float_as_uint(r) >> 16;
  const float q = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  t[2] = __float_as_uint(q) >> 16;
}

// The power of two 2^(14 - e) for a largest magnitude of exponent e, as the factor
// and its inverse; both normal numbers.
__device__ __forceinline__ void fp16_factor(uint32_t top, float& factor, float& inverse) {
  const uint32_t field = max(top >> 23, 15u);
  factor = __uint_as_float((268u - field) << 23);
  inverse = __uint_as_float((field - 14u) << 23);
}

// Bits of |v| where v is finite, 0 otherwise.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

__device__ __forceinline__ uint32_t fp16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float fp16_lo(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)v)); }
__device__ __forceinline__ float fp16_hi(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)(v >> 16))); }

// x of this CTA's tokens in fp16, for the routed experts' codes.
template <int WT>
__device__ void fp16_tokens(const FewParams& p, uint32_t* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = gridDim.x - 1 - blockIdx.x; t < p.T; t += gridDim.x) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(p.x + (int64_t)t * p.d * 2);
    uint32_t top = 0;
    for (int i = threadIdx.x; i < p.d / 2; i += kThreads) {
      const uint32_t v = __ldg(x + i);
      top = max(top, max(finite_bits(ptx::bf16_lo(v)), finite_bits(ptx::bf16_hi(v))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[warp] = top;
    consumer_sync();
    top = red[lane & (kWarps - 1)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float factor, inverse;
    fp16_factor(top, factor, inverse);
    if (threadIdx.x == 0) p.x_scale[t] = inverse;
    uint16_t* to = reinterpret_cast<uint16_t*>(p.x16 + (int64_t)t * p.d * 2);
    for (int i = threadIdx.x; i < p.d / 2; i += kThreads) {
      const uint32_t v = __ldg(x + i);
      store_pair<WT>(to, 2 * i, fp16_pair(ptx::bf16_lo(v) * factor, ptx::bf16_hi(v) * factor));
    }
    consumer_sync();
  }
}

// Four values of h, columns k to k + 3, to a row's three bf16 terms [3][K].
__device__ __forceinline__ void store_terms(uint8_t* to, int K, int k, const float (&h)[4]) {
  uint32_t t[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) terms_of(h[i], t[i]);
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *reinterpret_cast<uint2*>(to + ((int64_t)q * K + k) * 2) =
        make_uint2(t[0][q] | (t[1][q] << 16), t[2][q] | (t[3][q] << 16));
}

// The same as two fp16 terms [2][K]; the second of an infinity or NaN is none.
template <int WT>
__device__ __forceinline__ void store_terms16(uint8_t* to, int K, int k, const float (&h)[4], float factor) {
  uint16_t* column = reinterpret_cast<uint16_t*>(to);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = h[2 * i] * factor, b = h[2 * i + 1] * factor;
    const uint32_t first = fp16_pair(a, b);
    const float ra = finite_bits(a) == (__float_as_uint(a) & 0x7fffffffu) ? a - fp16_lo(first) : 0.0f;
    const float rb = finite_bits(b) == (__float_as_uint(b) & 0x7fffffffu) ? b - fp16_hi(first) : 0.0f;
    store_pair<WT>(column, k + 2 * i, first);
    store_pair<WT>(column + K, k + 2 * i, fp16_pair(ra, rb));
  }
}

// h of every row, four columns a lane and 128 a warp.
template <int WT>
__device__ void activations(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kWarps;
  const int rows = p.T * p.k;
  const int rb = p.I / kFewCols, sb = p.S / kFewCols;
  const int jobs = rows * rb + p.T * sb;
  for (int job = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; job < jobs; job += warps) {
    const bool shared = job >= rows * rb;
    const int j = shared ? job - rows * rb : job;
    const int blocks = shared ? sb : rb;
    const int row = j / blocks, block = j % blocks;
    float f = 1.0f;
    if (!shared && WT != kFewBf16) f = __ldcg(p.x_scale + ls.ent[row] / p.k);
    const float* buf = shared ? p.up_s : p.up_r;
    const int parts = shared ? p.split_up_s.parts : p.split_up_r.parts;
    const float4 g = sum_parts(buf + ((int64_t)(row * 2) * blocks + block) * parts * kFewCols, parts);
    const float4 u = sum_parts(buf + ((int64_t)(row * 2 + 1) * blocks + block) * parts * kFewCols, parts);
    const float h[4] = {gated(g.x * f, u.x * f), gated(g.y * f, u.y * f), gated(g.z * f, u.z * f), gated(g.w * f, u.w * f)};
    const int k = block * kFewCols + 4 * lane;
    if (shared) {
      store_terms(p.h_s + (int64_t)row * 3 * p.S * 2, p.S, k, h);
    } else if constexpr (WT == kFewBf16) {
      store_terms(p.h_r + (int64_t)row * 3 * p.I * 2, p.I, k, h);
    } else {
      uint32_t top = max(max(finite_bits(h[0]), finite_bits(h[1])), max(finite_bits(h[2]), finite_bits(h[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      float factor, inverse;
      fp16_factor(top, factor, inverse);
      if (lane == 0) p.h_scale[(int64_t)row * rb + block] = inverse;
      store_terms16<WT>(p.h_r + (int64_t)row * 2 * p.I * 2, p.I, k, h, factor);
    }
  }
}

// y: routed rows in slot order, then the shared expert's.
__device__ void combine(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kWarps;
  const int blocks = p.d / kFewCols;
  const int jobs = p.T * blocks;
  for (int job = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; job < jobs; job += warps) {
    const int t = job / blocks, block = job % blocks;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
      const int i = t * p.k + j;
      const float w = ls.w[i];
      const int parts = p.split_dn_r.parts;
      const float4 o = sum_parts(p.dn_r + ((int64_t)ls.row_of[i] * blocks + block) * parts * kFewCols, parts);
      y.x = fmaf(w, o.x, y.x);
      y.y = fmaf(w, o.y, y.y);
      y.z = fmaf(w, o.z, y.z);
      y.w = fmaf(w, o.w, y.w);
    }
    if (p.S > 0) {
      const int parts = p.split_dn_s.parts;
      const float4 o = sum_parts(p.dn_s + ((int64_t)t * blocks + block) * parts * kFewCols, parts);
      y.x += o.x;
      y.y += o.y;
      y.z += o.z;
      y.w += o.w;
    }
    const int64_t at = (int64_t)t * p.d + block * kFewCols + 4 * lane;
    if (p.y_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
          make_uint2(ptx::pack_bf16x2(y.x, y.y), ptx::pack_bf16x2(y.z, y.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = y;
  }
}

// ------------------------------------------------------------ the kernel
template <int RT>
__global__ void __launch_bounds__(kAllThreads, 1)
    few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ FewMaps maps) {
  extern __shared__ uint8_t dyn[];
  __shared__ Lists ls;
  __shared__ Control ct;
  Smem sm;
  sm.stages = align_1024(dyn);
  sm.cols = sm.stages + kStages * kTileBytes;
  sm.red = reinterpret_cast<float*>(sm.cols + 2 * kColBytes);
  sm.c = &ct;
  // the router's keys, and where it is done, the scales
  uint64_t* keys = reinterpret_cast<uint64_t*>(sm.red + 8 * kRedFloats);
  sm.scales = reinterpret_cast<StageScales*>(keys);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&ct.full[s], 1);
      ptx::mbar_init(&ct.empty[s], kWarps / 2 + 1);
      ptx::mbar_init(&ct.issued[s], 1);
      ptx::mbar_init(&ct.issued[s + kStages], 1);
      ptx::mbar_init(&ct.scaled[s], kRouterWarps);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ct.col_full[b], 1);
      ptx::mbar_init(&ct.col_empty[b], kWarps);
    }
    ptx::mbar_init(&ct.ready, 1);
    ptx::mbar_init(&ct.started, 1);
    ptx::mbar_init(&ct.routed, 32 * kRouterWarps);
    ct.abort = 0u;
    ct.never = 0u;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
  }
  __syncthreads();
  volatile uint32_t* abort = &ct.abort;

  if (warp == kWarps) {
    // ---------------------------------------------- producer
    Ring ring;
    if ((threadIdx.x & 31) < 3) {
      ptx::prefetch_tmap(&maps.routed[threadIdx.x & 31]);
      if (p.S > 0) ptx::prefetch_tmap(&maps.shared[threadIdx.x & 31]);
    }
    bool ok = true;
    if (p.S > 0) ok = produce<kFewBf16, true, false>(maps, p, ls, sm, ring, p.bar + 4);
    if (ok && !warp_wait(&ct.routed, 0, abort)) {
      raise_status(p.status, abort, kStatusTimeout);
      ok = false;
    }
    ok = ok && __all_sync(0xffffffffu, *abort == 0);  // the router gave up: there are no lists
    if ((threadIdx.x & 31) == 0) {
      ct.first = ring.n;
      ptx::mbar_arrive(&ct.started);
    }
    if (ok) ok = produce<RT, false, false>(maps, p, ls, sm, ring, p.bar + 5);
    if (ok) ok = produce<RT, false, true>(maps, p, ls, sm, ring, p.bar + 6);
    if (ok && p.S > 0) produce<kFewBf16, true, true>(maps, p, ls, sm, ring, p.bar + 7);
    // every issued copy must land before the CTA may exit
    if ((threadIdx.x & 31) == 0)
      for (int j = ring.n > kStages ? ring.n - kStages : 0; j < ring.n; ++j)
        if (!ptx::wait_bounded(&ct.full[j % kStages], (j / kStages) & 1, &ct.never))
          raise_status(p.status, abort, kStatusTimeout);
  } else if (warp == kWarps + 1) {
    // ---------------------------------------------- columns
    Ring ring;
    bool ok = true;
    auto wait = [&](uint64_t* bar) {
      if (warp_wait(bar, 0, abort) && __all_sync(0xffffffffu, *abort == 0)) {
        ptx::fence_proxy_async_all();  // x in fp16 and h were written by ordinary stores
        return true;
      }
      raise_status(p.status, abort, kStatusTimeout);
      return false;
    };
    if (p.S > 0) ok = bring_columns<kFewBf16, true, false>(p, ls, sm, ring);
    ok = ok && wait(&ct.routed) && bring_columns<RT, false, false>(p, ls, sm, ring);
    ok = ok && wait(&ct.ready) && bring_columns<RT, false, true>(p, ls, sm, ring);
    if (ok && p.S > 0) bring_columns<kFewBf16, true, true>(p, ls, sm, ring);
    // every issued copy must land before the CTA may exit
    for (int j = ring.cols > 2 ? ring.cols - 2 : 0; j < ring.cols; ++j)
      if (!ptx::wait_bounded(&ct.col_full[j & 1], (j >> 1) & 1, &ct.never))
        raise_status(p.status, abort, kStatusTimeout);
  } else if (warp > kWarps) {
    // ---------------------------------------------- router
    if (threadIdx.x == kThreads + 64) grid_poll(p.bar + 0, p.status, abort);
    router_sync();
    if (*abort == 0) route(p, ls, keys);
    ptx::mbar_arrive(&ct.routed);
    if constexpr (RT != kFewBf16) {
      auto wait = [&](uint64_t* bar) {
        return warp_wait(bar, 0, abort) && __all_sync(0xffffffffu, *abort == 0);
      };
      // both warps are done with the keys, and the share has begun
      Ring ring;
      if (wait(&ct.routed) && wait(&ct.started)) {
        ring.n = ct.first;
        if (bring_scales<RT, false>(p, ls, sm, ring) && wait(&ct.ready)) bring_scales<RT, true>(p, ls, sm, ring);
      }
    }
  } else {
    // ---------------------------------------------- consumers
    Ring ring;
    logits_share(p, reinterpret_cast<double*>(sm.red));
    if (RT != kFewBf16) {
      fp16_tokens<RT>(p, reinterpret_cast<uint32_t*>(sm.red));
      ptx::fence_proxy_async_all();  // bulk copies will read them
    }
    grid_arrive(p.bar + 0);
    bool ok = true;
    if (p.S > 0) ok = consume<kFewBf16, true, false>(p, ls, sm, ring);
    // all consumers agree on whether there are lists
    ok = ptx::named_barrier_and(9, kThreads, ok && ptx::wait_bounded(&ct.routed, 0, abort) && *abort == 0);
    if (ok) ok = consume<RT, false, false>(p, ls, sm, ring);
    grid_arrive(p.bar + 1);
    if (grid_wait(p.bar + 1, p.status, abort)) {
      activations<RT>(p, ls);
      ptx::fence_proxy_async_all();  // bulk copies will read h
      grid_arrive(p.bar + 2);
      if (grid_wait(p.bar + 2, p.status, abort)) {
        if (threadIdx.x == 0) ptx::mbar_arrive(&ct.ready);
        if (consume<RT, false, true>(p, ls, sm, ring) && p.S > 0) consume<kFewBf16, true, true>(p, ls, sm, ring);
        grid_arrive(p.bar + 3);
        if (grid_wait(p.bar + 3, p.status, abort)) combine(p, ls);
      }
    }
  }
}

template <int RT>
cudaError_t launch(const FewParams& p, const FewMaps& maps, int sms, cudaStream_t stream) {
  // stages, the pairs' joins, the columns, a routing key and a logit per expert and router warp
  const size_t smem = 1024 + kStages * kTileBytes + 2 * kColBytes + 8 * kRedFloats * 4 + 
                      std::max((size_t)kRouterWarps * p.E * 12, kStages * sizeof(StageScales));
  auto kernel = few_kernel<RT>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  void* args[] = {const_cast<FewParams*>(&p), const_cast<FewMaps*>(&maps)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(sms),
                                     dim3(kAllThreads), args, smem, stream);
}

}  // namespace

cudaError_t launch_few(const FewParams& p, const FewMaps& maps, int weights, int sms, cudaStream_t stream) {
  switch (weights) {
    case kFewBf16: return launch<kFewBf16>(p, maps, sms, stream);
    case kFewE4m3: return launch<kFewE4m3>(p, maps, sms, stream);
    default: return launch<kFewMxfp4>(p, maps, sms, stream);
  }
}

}  // namespace moe
