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
//                         of the consumers and across the ends of chunks and
//                         phases: the shared expert's up projections need no
//                         routing and stream while it is found, and the first
//                         tiles of the down projections are in the ring before
//                         the barriers that the activations wait for;
//   columns (1 warp)      follows the tiles and brings the activations that go with
//                         them (for bf16 weights several stages' at a time, by bulk
//                         copies: single stages' copies of 128 bytes cost more than
//                         the weights, 710 instead of 455 us at T = 8 with 28
//                         experts of 7168 x 2048);
//   router (2 warps)      makes x's terms for coded weights, waits for all logits,
//                         finds the top-k (of more than two tokens some CTAs do, and
//                         tell the others) and the list of chosen experts and their
//                         rows.
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
// Arithmetic.
//   bf16 weights: mma.sync m16n8k16 with the weights as the A operand (16 output
//   columns by 16 steps, ldmatrix from the stage) and the activations as B's
//   columns, 8 at a time.  Consumer warp w takes columns 16 (w % 8) of every second
//   tile (w / 8): a tile's chain of waits, loads and MMAs is longer than the time
//   HBM needs for one.  x is bf16 as it comes; h is fp32 and goes in as three bf16
//   terms (8 bits each: 24 in all).
//   e4m3 and MXFP4 weights: tcgen05.mma takes the codes as they are, M = 128
//   output columns, kind::f8f6f4 and kind::mxf4 (with its block scales).  It wants
//   activations of the same kind, so these go in as sums of rounded terms, each
//   term one more B column that rounds what the ones before left: x in three e4m3
//   terms and h in six (4 bits each, after a power of two has put the largest of
//   128 values between 2^7 and 2^8), or both in twelve MXFP4 terms (2 bits each,
//   every block of 32 with a scale of its own): 24 bits of a block's largest value
//   in h, and for e4m3 2^-25 of it in x.  The columns cost nothing beside the
//   weights, and no code is converted: mma.sync needs fp16 operands made of the
//   codes, which bound the kernel at 2.6 (MXFP4) and 3.9 TB/s (e4m3).  An infinity
//   has no code and goes in as NaN.
//   The consumers share the work on codes out: four warps drain the accumulators,
//   two threads issue MMAs, and eight warps (MXFP4) bring the scales to TMEM, or one
//   (e4m3) the factors of the sums.
//
// Measured in runs of calls, d = 7168, inner 2048, top-8 of 32 with a shared expert,
// T = 8 (28 experts): bf16 382 us, 6.7 TB/s and the measured copy rate of HBM; e4m3
// 248 us, 5.3 TB/s (230 us with the MMAs and terms left out: its tiles' rows of 128
// bytes); MXFP4 176 us, 4.2 TB/s (159 us without them and the scales).  T = 1: 136, 101
// and 75 us, of which the phases outside the streams (router, four barriers of 2 us,
// activations, combine) take some 25.
//
// Waits.  Every wait ends after a limit.  Who gives up raises the CTA's abort flag, which
// ends the CTA's other waits, and releases nothing more; the CTA then misses the grid's
// next barrier, so that the others give up too and y is not written.  Before the CTA
// goes, its copies and MMAs under way have landed.
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
constexpr int kMaxStages = 8;

// The ring of a call with these routed weights: beside a tile of codes a stage
// holds up to 64 rows of 128 bytes of the activations' terms.
template <int RT>
struct Cfg {
  static constexpr bool kCoded = RT != kFewBf16;
  static constexpr int kStages = kCoded ? 6 : kMaxStages;
  static constexpr uint32_t kStageBytes = kTileBytes + (kCoded ? 8192 : 0);
  static constexpr uint32_t kColBytes = kCoded ? 8192 : 16384;  // of a buffer of B columns; there are two
};

// Terms of the activations for coded weights: rows that x and h take in the arrays
// (whole swizzle atoms), and terms that are in use.
constexpr int kTermRows8 = few_term_rows(kFewE4m3), kTermRows4 = few_term_rows(kFewMxfp4);
constexpr int kXTerms8 = 3, kHTerms8 = 6, kTerms4 = 12;

constexpr int kRedPitch = 17;  // floats of one B column of a warp pair's 16 output columns
constexpr int kRedFloats = 2 * kMaxCols * kRedPitch;  // of a pair of warps

// TMEM of coded calls: four accumulators (e4m3: each of a unit, whose sums get their
// scales in registers; MXFP4: in pairs, each of a pass's every second unit), then
// MXFP4's scales, 8 columns of the weights' and 8 of the terms' for each stage.
constexpr int kAccCols = 64, kAccs = 4;
constexpr int kIssuers = 2;  // threads that issue MMAs
constexpr int kSfCols = 16;
// e4m3: factors of a pass, [8 rows][32 units], for this many passes in turn.  When a
// stage is filled the one before it in its place has been multiplied, so that the
// accumulators up to kAccs stages before that are drained: the passes 11 before are
// done with.
constexpr int kFactors = 12;
constexpr size_t kExchangeBytes = 4 * 8 * (128 + 64) * 4;  // two groups of 4 units' scales for each team, or factors
static_assert(kExchangeBytes >= kFactors * 256 * 4, "room for the factors");
template <int RT>
constexpr int kTmemCols = RT == kFewE4m3 ? 256 : 512;

struct Lists {  // what the routing leaves in shared memory
  int32_t idx[kMaxRows];      // [T][k]
  float w[kMaxRows];
  int16_t ent[kMaxRows];      // entries t * k + j ordered by expert, then token
  int16_t row_of[kMaxRows];   // the inverse
  int16_t expert[kMaxRows];   // distinct experts, ascending
  int16_t start[kMaxRows + 1];
  int32_t counts[kMaxExperts];
  int n;                      // distinct experts
};

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t col_full[2], col_empty[2];
  // a stage's chunk is known, its tile on the way: two turns of the ring, since
  // who has no part in a stage may still be looking at it when the stage's place
  // is filled again, but not when the place after it is
  uint64_t issued[2 * kMaxStages];
  uint64_t scaled[kFactors];    // MXFP4: a stage's scales are in TMEM; e4m3: a pass's factors are there
  uint64_t acc_full[kAccs], acc_empty[kAccs];
  uint64_t landed[kIssuers];  // a call that gave up: the MMAs issued so far are done
  uint64_t ready;   // h is there, in all CTAs
  uint64_t routed;  // the lists are there
  int chunk[2 * kMaxStages];  // which chunk a stage belongs to; -1: the share is done
  // what an accumulator holds: of e4m3 a pass's first unit (-1) or the one of this
  // number, of MXFP4 nothing (0) or sums
  int acc_chunk[kAccs], acc_pass[kAccs], acc_what[kAccs];
  int position;  // stages handed over when a coded share ended
  uint32_t tmem, abort, never;
};

__device__ __forceinline__ void consumer_sync() { ptx::named_barrier(9, kThreads); }
__device__ __forceinline__ void router_sync() { ptx::named_barrier(10, 32 * kRouterWarps); }

// ------------------------------------------------------------ grid barrier
// The consumers' writes so far are visible to who waits.  A CTA one of whose consumers
// gave up (and raised the flag before it came here) is missed: the others must not read
// what it has not written.  (A call: inlined it took the coded layers 1% longer, at T = 8
// e4m3 252.7 instead of 248.3 us and MXFP4 178.0 instead of 175.6.)
__device__ __noinline__ void grid_arrive(uint32_t* bar, const volatile uint32_t* abort) {
  consumer_sync();
  if (threadIdx.x == 0 && *abort == 0) {
    __threadfence();
    atomicAdd(bar, 1u);
  }
}

// One thread's wait for `count` CTAs' arrivals.
__device__ __forceinline__ bool grid_poll(const uint32_t* bar, uint32_t count, uint32_t* status,
                                          volatile uint32_t* abort) {
  const uint64_t t0 = ptx::globaltimer();
  uint32_t n = 0, seen;
  while (true) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(bar) : "memory");
    if (seen >= count) break;
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

// All consumers' wait: they go on, or none of them.
__device__ bool grid_wait(const uint32_t* bar, uint32_t* status, volatile uint32_t* abort) {
  if (threadIdx.x == 0) grid_poll(bar, gridDim.x, status, abort);
  return ptx::named_barrier_and(9, kThreads, *abort == 0);
}

// The code between the products runs once or twice a call and is not in any cache
// then: it is kept short, and its loads in batches.
__device__ __forceinline__ void add(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// `count` arrivals at once.
__device__ __forceinline__ void mbar_arrive_many(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(ptx::smem_u32(bar)), "r"(count) : "memory");
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

// ------------------------------------------------------------ shares and pieces
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
    q.group = DOWN ? 3 : 1;
    q.again = q.rows > kPass;
    q.ld = (int64_t)per_expert * split.parts * kFewCols;
    q.out = buf + q.first * q.ld + ((int64_t)in * split.parts + part) * kFewCols;
    return q;
  }
  // Rows of a pass: 24 bf16 columns or 64 rows of terms (more rows read the weights
  // again, from L2 mostly: only the shared expert and crowded small layers have
  // them).
  static constexpr int kPass = WT == kFewBf16 ? (DOWN ? kMaxCols / 3 : kFewMaxTokens) : 64 / few_term_rows(WT);
  static __device__ __forceinline__ void cut(Piece& q, int all, int r0) {
    q.rows = min(kPass, all - r0);
    q.first += r0;
    q.out += r0 * q.ld;
  }
  template <typename F>
  __device__ __forceinline__ bool passes(const Piece& whole, F f) const {
    for (int r0 = 0; r0 < whole.rows; r0 += kPass) {
      Piece q = whole;
      cut(q, whole.rows, r0);
      if (!f(q)) return false;
    }
    return true;
  }
};

// bf16 columns: how many units' a buffer takes for a piece, and their distance in
// bytes: a pad keeps the reads of 8 columns off each other's banks.
template <int RT>
struct ColumnPlan {
  static constexpr int kUnitBytes = 2 * few_unit_steps(kFewBf16);
  static constexpr int kPad = 16;
  int units, pitch;
  __device__ __forceinline__ explicit ColumnPlan(const Piece& q) {
    const int cols = q.rows * q.group;
    units = min(q.step1 - q.step0, ((int)Cfg<RT>::kColBytes / cols - kPad) / kUnitBytes);
    pitch = units * kUnitBytes + kPad;
  }
  static_assert((int)Cfg<RT>::kColBytes / kMaxCols >= kUnitBytes + kPad, "room for one unit's columns");
};

// The rings' positions: stages and column buffers handed over so far, and
// accumulators.
struct Ring {
  int n = 0, cols = 0, accs = 0;
};

struct Smem {
  uint8_t* stages;
  uint8_t* cols;
  float* red;
  uint32_t* exchange;  // MXFP4: groups of scales on their way from rows to lanes; e4m3: factors
  Control* c;
};

template <int RT>
__device__ __forceinline__ bool wait_issued(Control& c, int n) {
  constexpr int kTurns = 2 * Cfg<RT>::kStages;
  return warp_wait(&c.issued[n % kTurns], (n / kTurns) & 1, &c.abort);
}

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

template <int WT, int RT, bool SHARED, bool DOWN>
__device__ bool produce(const FewMaps& m, const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring,
                        uint32_t* counter) {
  constexpr int S = Cfg<RT>::kStages;
  const int lane = threadIdx.x & 31;
  const uint64_t once = ptx::policy_evict_first(), more = ptx::policy_evict_normal();
  Control& c = *sm.c;
  const Share<WT, SHARED, DOWN> share(p, ls);
  auto slot_free = [&] {
    if (warp_wait(&c.empty[ring.n % S], ((ring.n / S) & 1) ^ 1, &c.abort)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  // MXFP4: the next chunk's scale bytes to L2, a line or two of each of its 128 rows.
  // Read when they are needed, in pieces of 32 bytes, they held the stages up: 54
  // experts at T = 16 took 311 instead of 293 us.  (Bulk prefetches of whole rows
  // went through the unit that has the tiles to load: 397 us.)
  auto fetch_scales = [&](int id) {
    if (WT != kFewMxfp4 || id >= share.total) return;
    const Piece q = share.chunk(p, ls, id);
    const int pitch = share.K / 32, from = q.step0 * 8, end = min(q.step1 * 8, pitch);
    const uint8_t* scales = (q.mat == 0 ? p.s1 : q.mat == 1 ? p.s3 : p.s2) +
                            ((int64_t)q.expert * share.N + q.col0 + lane) * pitch;
    for (int i = 0; i < 4; ++i)  // rows lane + 32 i
      for (int o = from; o < end; o += 64)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(scales + (int64_t)(32 * i) * pitch + o) : "memory");
  };
  int id = blockIdx.x;
  while (id < share.total) {
    int claimed = 0;
    if (lane == 0) claimed = (int)atomicAdd(counter, 1u) + gridDim.x;  // used after this chunk
    bool fetched = WT != kFewMxfp4;
    const bool ok = share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      // the columns' warp adds the terms to a stage of codes; tests have stages wait for
      // more than comes
      uint32_t bytes = kTileBytes + (WT == kFewBf16 ? 0 : q.rows * few_term_rows(WT) * 128) + p.missing;
      if (DOWN && !SHARED && blockIdx.x == 0) bytes += p.missing_down;
      for (int step = q.step0; step < q.step1; ++step, ++ring.n) {
        const int s = ring.n % S;
        if (!slot_free()) return false;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&c.full[s], bytes);
          c.chunk[ring.n % (2 * S)] = id;
          ptx::mbar_arrive(&c.issued[ring.n % (2 * S)]);
          load_tile<WT, SHARED>(m, p, q, step, sm.stages + s * Cfg<RT>::kStageBytes, &c.full[s], q.again ? more : once);
        }
        __syncwarp();
        if (!fetched && (step == q.step0 + 1 || step == q.step1 - 1)) {
          fetch_scales(__shfl_sync(0xffffffffu, claimed, 0));
          fetched = true;
        }
      }
      return true;
    });
    if (!ok) return false;
    id = __shfl_sync(0xffffffffu, claimed, 0);
  }
  if (!slot_free()) return false;
  if (lane == 0) {
    c.chunk[ring.n % (2 * S)] = -1;
    ptx::mbar_arrive(&c.issued[ring.n % (2 * S)]);
    ptx::mbar_arrive(&c.full[ring.n % S]);
  }
  ++ring.n;
  return true;
}

// ------------------------------------------------------------ columns
// Walks a share's chunks: f for every pass, ring.n being its first stage.
template <int WT, int RT, bool SHARED, bool DOWN, typename F>
__device__ __forceinline__ bool follow_chunks(const FewParams& p, const Lists& ls, const Smem& sm, const Ring& ring,
                                              F f) {
  const Share<WT, SHARED, DOWN> share(p, ls);
  Control& c = *sm.c;
  int id = blockIdx.x < share.total ? (int)blockIdx.x : -1;  // the first chunk needs no tile to be known by
  while (id >= 0) {
    if (!share.passes(share.chunk(p, ls, id), f)) return false;
    if (!wait_issued<RT>(c, ring.n)) {
      if ((threadIdx.x & 31) == 0) raise_status(p.status, &c.abort, kStatusTimeout);
      return false;
    }
    id = c.chunk[ring.n % (2 * Cfg<RT>::kStages)];
  }
  return true;
}

// The columns of bf16 shares.  A stage is also released by this warp, so that its
// chunk is still to be read when it gets there.
template <int RT, bool SHARED, bool DOWN>
__device__ bool bring_columns(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int kSteps = few_unit_steps(kFewBf16);
  const int lane = threadIdx.x & 31;
  const int K = DOWN ? (SHARED ? p.S : p.I) : p.d;
  Control& c = *sm.c;
  auto give_up = [&] {
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  auto next_stage = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.empty[ring.n % Cfg<RT>::kStages]);
    ++ring.n;
  };
  const bool ok = follow_chunks<kFewBf16, RT, SHARED, DOWN>(p, ls, sm, ring, [&](const Piece& q) {
    const ColumnPlan<RT> plan(q);
    const int cols = q.rows * q.group;
    const uint8_t* src = nullptr;
    if (lane < cols) {
      if (DOWN)
        src = (SHARED ? p.h_s : p.h_r) + ((int64_t)q.first * 3 + lane) * K * 2;
      else
        src = p.x + (SHARED ? q.first + lane : ls.ent[q.first + lane] / p.k) * (int64_t)p.d * 2;
    }
    for (int step = q.step0; step < q.step1; ++step) {
      if ((step - q.step0) % plan.units == 0) {
        const int buf = ring.cols & 1;
        if (!warp_wait(&c.col_empty[buf], ((ring.cols >> 1) & 1) ^ 1, &c.abort)) return give_up();
        const uint32_t bytes = 2 * kSteps * (min(q.step1, step + plan.units) - step);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&c.col_full[buf], bytes * cols);
        __syncwarp();
        if (lane < cols)
          bulk_load(ptx::smem_u32(sm.cols) + buf * Cfg<RT>::kColBytes + lane * plan.pitch, src + step * kSteps * 2,
                    bytes, &c.col_full[buf]);
        ++ring.cols;
      }
      if (!wait_issued<RT>(c, ring.n)) return give_up();
      next_stage();
    }
    return true;
  });
  if (!ok || !wait_issued<RT>(c, ring.n)) return give_up();
  next_stage();  // the mark of the end
  return true;
}

// The terms of coded shares, into the stages themselves: a row's are one or two
// swizzle atoms of 8 rows.
template <int RT, bool DOWN>
__device__ bool bring_terms(const FewMaps& m, const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int S = Cfg<RT>::kStages, kRows = few_term_rows(RT);
  const int lane = threadIdx.x & 31;
  const uint64_t policy = ptx::policy_evict_normal();
  Control& c = *sm.c;
  auto give_up = [&] {
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  // this warp's release of a stage, and those of the consumer warps that have no part
  // in coded shares (the MMAs' completion is the last, and e4m3's factors have one of
  // their own)
  auto next_stage = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive_many(&c.empty[ring.n % S], RT == kFewE4m3 ? 7 : 8);
    ++ring.n;
  };
  const bool ok = follow_chunks<RT, RT, false, DOWN>(p, ls, sm, ring, [&](const Piece& q) {
    int row = 0;
    if (lane < q.rows) row = (DOWN ? q.first + lane : ls.ent[q.first + lane] / p.k) * kRows;
    for (int step = q.step0; step < q.step1; ++step) {
      if (!wait_issued<RT>(c, ring.n)) return give_up();
      const int s = ring.n % S;
      if (lane < q.rows)
        ptx::tma_load_2d(sm.stages + s * Cfg<RT>::kStageBytes + kTileBytes + lane * kRows * 128,
                         DOWN ? &m.h_terms : &m.x_terms, &c.full[s], step * 128, row, policy);
      next_stage();
    }
    return true;
  });
  if (!ok || !wait_issued<RT>(c, ring.n)) return give_up();
  next_stage();
  return true;
}

// ------------------------------------------------------------ consumers: bf16
template <int RT, int NT>
__device__ __forceinline__ void consume_piece(const FewParams& p, const Piece& q, const Smem& sm, Ring& ring) {
  constexpr int S = Cfg<RT>::kStages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3, team = warp >> 3;
  Control& ct = *sm.c;
  float acc[NT][4] = {};
  const ColumnPlan<RT> plan(q);
  const int last = q.rows * q.group - 1;
  int left = 0;  // units whose columns are in the buffer
  uint32_t cols = 0;
  // A wait that fails raises the abort flag, which ends all later ones at once, and
  // the piece goes on with whatever the buffers hold: its barriers need every
  // warp, and the share ends at the next chunk.  But the warp releases nothing more:
  // a stage or buffer whose copies have not landed must not be armed again, which
  // counts its barrier below zero.
  bool releases = lane == 0;
  auto arrived = [&](uint64_t* bar, uint32_t parity) {
    if (!ptx::wait_bounded(bar, parity, &ct.abort)) {
      raise_status(p.status, &ct.abort, kStatusTimeout);
      releases = false;
    }
  };
  auto release = [&](uint64_t* bar) {
    __syncwarp();
    if (releases) ptx::mbar_arrive(bar);
  };
  for (int step = q.step0; step < q.step1; ++step) {
    if (left == 0) {
      const int buf = ring.cols & 1;
      arrived(&ct.col_full[buf], (ring.cols >> 1) & 1);
      cols = ptx::smem_u32(sm.cols) + buf * Cfg<RT>::kColBytes;
      left = min(plan.units, q.step1 - step);
    }
    const int slot = ring.n % S;
    if ((ring.n & 1) == team) {
      arrived(&ct.full[slot], (ring.n / S) & 1);
      uint32_t tile = ptx::smem_u32(sm.stages) + slot * Cfg<RT>::kStageBytes;
      after_wait(tile, cols);
      // Sums of a tile alone (four MMAs), which are then added up rounding to nearest:
      // the tensor core cuts off what its accumulator does not hold, and over all of
      // a chunk that put y 1.2e-6 off.
      float sums[NT][4] = {};
      stage_bf16<NT>(tile, cols, plan.pitch, last, sums);
      before_release<NT>(sums);
      release(&ct.empty[slot]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += sums[j][i];
    }
    cols += ColumnPlan<RT>::kUnitBytes;
    ++ring.n;
    if (--left == 0) {
      release(&ct.col_empty[ring.cols & 1]);
      ++ring.cols;
    }
  }
  // the two teams' sums, and the terms of each row, are joined by the pair of warps
  // that has these 16 columns
  const int pair = warp & 7;
  float* red = sm.red + pair * kRedFloats;
  float* to = red + team * kMaxCols * kRedPitch;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    to[(8 * j + 2 * c) * kRedPitch + g] = acc[j][0];
    to[(8 * j + 2 * c + 1) * kRedPitch + g] = acc[j][1];
    to[(8 * j + 2 * c) * kRedPitch + g + 8] = acc[j][2];
    to[(8 * j + 2 * c + 1) * kRedPitch + g + 8] = acc[j][3];
  }
  ptx::named_barrier(1 + pair, 64);
  for (int i = team * 32 + lane; i < q.rows * 16; i += 64) {
    const int r = i >> 4, col = i & 15;
    // An infinite weight makes the leading term's sum infinite, and NaN of the sums of the
    // lower terms where those are zero: the leading one is the sum then.
    float a = 0.0f;
    for (int t = 0; t < q.group && fabsf(a) < __uint_as_float(0x7f800000u); ++t) {
      const float* x = red + (r * q.group + t) * kRedPitch + col;
      a += x[0] + x[kMaxCols * kRedPitch];
    }
    q.out[r * q.ld + pair * 16 + col] = a;
  }
  ptx::named_barrier(1 + pair, 64);
}

template <int RT, bool SHARED, bool DOWN>
__device__ bool consume(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int S = Cfg<RT>::kStages;
  const Share<kFewBf16, SHARED, DOWN> share(p, ls);
  Control& ct = *sm.c;
  volatile uint32_t* abort = &ct.abort;
  while (true) {
    const bool there = wait_issued<RT>(ct, ring.n);
    if (!there) raise_status(p.status, &ct.abort, kStatusTimeout);
    // both warps of a pair take the chunk or neither
    if (!ptx::named_barrier_and(1 + ((threadIdx.x >> 5) & 7), 64, there && *abort == 0)) return false;
    const int id = ct.chunk[ring.n % (2 * S)];
    if (id < 0) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0 && (ring.n & 1) == (threadIdx.x >> 8)) ptx::mbar_arrive(&ct.empty[ring.n % S]);
      ++ring.n;
      return true;
    }
    share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      const int cols = q.rows * q.group;
      if (cols <= 8)
        consume_piece<RT, 1>(p, q, sm, ring);
      else if (cols <= 16)
        consume_piece<RT, 2>(p, q, sm, ring);
      else
        consume_piece<RT, 3>(p, q, sm, ring);
      return true;
    });
  }
}

// ------------------------------------------------------------ consumers: codes
// kind::f8f6f4 instruction descriptor: fp32 accumulator (bits 4-5 = 1), A and B
// e4m3 (0), A MN-major (bit 15: weights lie [steps][columns]), B K-major, N >> 3 at
// bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_e4m3(int N) {
  return (1u << 4) | (1u << 15) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// kind::mxf4: A and B e2m1 (bits 7-9 and 10-11 = 1), both K-major, ue8m0 scales (bit
// 23), M >> 7 at bits 27-28, and which pair of a TMEM word's four scale bytes to
// use, bits 29-30 (A) and 4-5 (B).
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t pair) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | ((pair * 2) << 29) |
         ((pair * 2) << 4);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Issues a share's MMAs.  A thread does all of it, since with a warp's other lanes
// waiting beside each issue a stage took half as long again; and an MMA takes its
// thread some 70 cycles, so two threads have every second stage each, with
// accumulators of their own.
template <int RT, bool DOWN>
__device__ bool issue_mmas(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring, int who) {
  constexpr int S = Cfg<RT>::kStages;
  // the stage that was in a stage's place was this thread's too, so its barrier is
  // never waited for a turn early
  static_assert(S % kIssuers == 0 && kAccs % kIssuers == 0, "stages and accumulators of its own");
  Control& c = *sm.c;
  const uint32_t base = ptx::smem_u32(sm.stages);
  const uint64_t a_desc = ptx::sdesc_sw128(base, 16, 1024), b_desc = ptx::sdesc_sw128(base + kTileBytes, 16, 1024);
  const int K = DOWN ? p.I : p.d;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ptx::wait_bounded(bar, parity, &c.abort)) return true;
    raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  // an accumulator is handed over when its MMAs are done and its labels are there
  auto take = [&](int acc) { return wait(&c.acc_empty[acc % kAccs], ((acc / kAccs) & 1) ^ 1); };
  auto hand_over = [&](int acc, int id, int pass, int what) {
    const int b = acc % kAccs;
    ptx::mma_commit(&c.acc_full[b]);
    c.acc_chunk[b] = id;
    c.acc_pass[b] = pass;
    c.acc_what[b] = what;
    ptx::mbar_arrive(&c.acc_full[b]);
  };
  const Share<RT, false, DOWN> share(p, ls);
  while (true) {
    if (!wait(&c.issued[ring.n % (2 * S)], (ring.n / (2 * S)) & 1)) return false;
    const int id = c.chunk[ring.n % (2 * S)];
    if (id < 0) break;
    int pass = 0;
    const bool ok = share.passes(share.chunk(p, ls, id), [&](const Piece& q) {
      const int N = (q.rows * few_term_rows(RT) + 15) & ~15;
      if constexpr (RT == kFewE4m3) {
        const uint32_t idesc = idesc_e4m3(N);
        for (int step = q.step0; step < q.step1; ++step, ++ring.n, ++ring.accs) {
          if (ring.accs % kIssuers != who) continue;
          const int s = ring.n % S;
          if (!take(ring.accs) || !wait(&c.full[s], (ring.n / S) & 1)) return false;
          ptx::tc_fence_after();
          const uint32_t off = s * (Cfg<RT>::kStageBytes >> 4);
          const uint64_t a = a_desc + off, b = b_desc + off;
          const uint32_t d = c.tmem + (ring.accs % kAccs) * kAccCols;
          // 32 steps: 32 rows of the tile, 32 bytes of a term's row
          mma_e4m3(d, a, b, idesc, 0u);
          mma_e4m3(d, a + (4096 >> 4), b + 2, idesc, 1u);
          mma_e4m3(d, a + (8192 >> 4), b + 4, idesc, 1u);
          mma_e4m3(d, a + (12288 >> 4), b + 6, idesc, 1u);
          ptx::mma_commit(&c.empty[s]);
          hand_over(ring.accs, id, pass, step == q.step0 ? -1 : step - q.step0);
        }
      } else {
        const uint32_t id0 = idesc_mxf4(N, 0), id1 = idesc_mxf4(N, 1);
        const int acc = ring.accs + who;
        const uint32_t d = c.tmem + (acc % kAccs) * kAccCols;
        if (!take(acc)) return false;
        uint32_t more = 0;
        for (int step = q.step0; step < q.step1; ++step, ++ring.n) {
          if (ring.n % kIssuers != who) continue;
          const int s = ring.n % S;
          // every stage of a coded share has scales: its own count of them
          if (!wait(&c.full[s], (ring.n / S) & 1) || !wait(&c.scaled[s], (ring.cols >> s) & 1)) return false;
          ring.cols ^= 1 << s;
          ptx::tc_fence_after();
          const uint32_t off = s * (Cfg<RT>::kStageBytes >> 4);
          const uint64_t a = a_desc + off, b = b_desc + off;
          const uint32_t sf = c.tmem + kAccs * kAccCols + s * kSfCols;
          mma_mxf4(d, a, b, id0, sf, sf + 8, more);
          mma_mxf4(d, a + 2, b + 2, id1, sf, sf + 8, 1u);
          if (K - step * 256 > 128) {  // else the last unit is half of one
            mma_mxf4(d, a + 4, b + 4, id0, sf + 4, sf + 12, 1u);
            mma_mxf4(d, a + 6, b + 6, id1, sf + 4, sf + 12, 1u);
          }
          ptx::mma_commit(&c.empty[s]);
          more = 1;
        }
        hand_over(acc, id, pass, more);
        ring.accs += kIssuers;
      }
      ++pass;
      return true;
    });
    if (!ok) return false;
  }
  // the end is told once, or by MXFP4's accumulators, which go in pairs, both
  const bool mine = ring.accs % kIssuers == who;
  const int acc = RT == kFewE4m3 ? ring.accs : ring.accs + who;
  if (RT == kFewMxfp4 || mine) {
    if (!take(acc)) return false;
    hand_over(acc, -1, 0, 0);
  }
  if (mine) {
    ptx::mbar_arrive(&c.empty[ring.n % S]);
    c.position = ring.n + 1;
  }
  ring.accs += RT == kFewE4m3 ? 1 : kIssuers;
  return true;
}

// 16 consecutive TMEM columns of this thread's lane as fp32.
__device__ __forceinline__ void load_sums(uint32_t tmem, float (&v)[16]) {
  uint32_t r[16];
  ptx::tmem_ld16(tmem, r);
  ptx::tmem_ld_wait(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Drains a share's accumulators (four warps; a thread has one output column).
template <int RT, bool DOWN>
__device__ bool drain(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = threadIdx.x & 127;
  Control& c = *sm.c;
  const Share<RT, false, DOWN> share(p, ls);
  float sums[RT == kFewE4m3 ? 8 : 4];  // of each row
  Piece q = {};
  while (true) {
    const int b = ring.accs % kAccs;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (warp_wait(bar, parity, &c.abort)) return true;
      if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
      return false;
    };
    if (!wait(&c.acc_full[b], (ring.accs / kAccs) & 1)) return false;
    ptx::tc_fence_after();
    const int id = c.acc_chunk[b], what = c.acc_what[b];
    const bool second = RT == kFewMxfp4 && (ring.accs & 1) != 0;  // of a pair
    const uint32_t acc = c.tmem + ((uint32_t)((warp & 3) * 32) << 16) + b * kAccCols;
    auto release = [&] {
      ptx::tc_fence_before();
      ptx::mbar_arrive(&c.acc_empty[b]);
      ++ring.accs;
    };
    if (id < 0) {
      release();
      if (RT == kFewMxfp4 && !second) continue;
      return true;
    }
    if (RT == kFewMxfp4 ? !second : what < 0) {  // the pass's first
      q = share.chunk(p, ls, id);
      share.cut(q, q.rows, c.acc_pass[b] * share.kPass);
#pragma unroll
      for (int r = 0; r < share.kPass; ++r) sums[r] = 0.0f;
    }
    if constexpr (RT == kFewMxfp4) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r < q.rows && what) {
          float v[16];
          load_sums(acc + r * 16, v);
          // the last terms, the smallest, first
          float a = 0.0f;
#pragma unroll
          for (int t = kTerms4 - 1; t >= 0; --t) a += v[t];
          sums[r] += a;
        }
      }
      release();
      if (second) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < q.rows) q.out[r * q.ld + col] = sums[r];
      }
    } else {
      const int slot = ring.cols % kFactors;
      const float* factors = reinterpret_cast<const float*>(sm.exchange) + slot * 256;
      if (what < 0 && !wait(&c.scaled[slot], (ring.cols / kFactors) & 1)) return false;
      const int unit = max(what, 0);
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        if (r < q.rows) {
          float v[16];
          load_sums(acc + r * 8, v);
          constexpr int kT = DOWN ? kHTerms8 : kXTerms8;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float a = 0.0f;
#pragma unroll
            for (int t = kT - 1; t >= 0; --t) a = fmaf(a, 0.0625f, v[8 * i + t]);
            sums[r + i] = fmaf(a, factors[(r + i) * 32 + unit], sums[r + i]);
          }
        }
      }
      release();
      if (unit == q.step1 - q.step0 - 1) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < q.rows) q.out[r * q.ld + col] = sums[r];
        ++ring.cols;
      }
    }
  }
}

// e4m3: the factors of a share's passes (one warp, a lane per unit): the scale of a
// block of weights times the power of two that undoes the scaling of a row's terms.
// It reads no stage, but releases each: who waits for `issued` and holds no stage back
// can fall two turns of the ring behind and wait for a phase that is gone.
template <bool DOWN>
__device__ bool bring_factors(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  constexpr int RT = kFewE4m3;
  const int lane = threadIdx.x & 31;
  Control& c = *sm.c;
  const Share<RT, false, DOWN> share(p, ls);
  auto issued = [&] {
    if (p.late_factors) __nanosleep(20000);  // a test's: more than a pass takes
    if (wait_issued<RT>(c, ring.n)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  auto next_stage = [&] {
    if (!issued()) return false;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.empty[ring.n % Cfg<RT>::kStages]);
    ++ring.n;
    return true;
  };
  const bool ok = follow_chunks<RT, RT, false, DOWN>(p, ls, sm, ring, [&](const Piece& q) {
    const int unit = min(q.step0 + lane, share.steps - 1);
    const uint8_t* scales = q.mat == 0 ? p.s1 : q.mat == 1 ? p.s3 : p.s2;
    const float f = __ldg(reinterpret_cast<const float*>(scales) +
                          ((int64_t)q.expert * share.steps + unit) * share.blocks + q.col0 / 128);
    float v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      v[r] = 0.0f;
      if (r < q.rows) {
        const int row = DOWN ? q.first + r : ls.ent[q.first + r] / p.k;
        v[r] = __ldcg((DOWN ? p.h_scale : p.x_scale) + (int64_t)row * share.steps + unit);
      }
    }
    if (!issued()) return false;  // the place is free once the pass's first stage is on its way
    const int slot = ring.cols % kFactors;
    float* to = reinterpret_cast<float*>(sm.exchange) + slot * 256 + lane;
#pragma unroll
    for (int r = 0; r < 8; ++r) to[r * 32] = f * v[r];
    ptx::mbar_arrive(&c.scaled[slot]);
    ++ring.cols;
    for (int step = q.step0; step < q.step1; ++step)
      if (!next_stage()) return false;
    return true;
  });
  return ok && next_stage();  // the mark of the end
}

// MXFP4: a share's scales to TMEM (two teams of four warps, which take groups of
// units in turn), row r of 128 in lane r % 32 of
// column r / 32 in all lane quarters, four blocks of 32 steps to a word.  Thread r
// reads row r of the weights and of the terms, and the rows go through shared memory to the lanes that store them.
template <bool DOWN>
__device__ bool bring_scales(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring, int team) {
  constexpr int RT = kFewMxfp4, S = Cfg<RT>::kStages, kGroup = 4, kRows = 128 + 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = threadIdx.x & 127;
  Control& c = *sm.c;
  const Share<RT, false, DOWN> share(p, ls);
  const int words = share.K / 128;  // of a row, four scales each
  const uint8_t* terms = DOWN ? p.h_term_scales : p.x_term_scales;
  int buf = 2 * team, group = 0;
  bool ok = true;
  // A warp whose wait failed goes on without: the others need it at the barriers.
  // They leave together at the end of a chunk.
  auto issued = [&] {
    if (ok && !wait_issued<RT>(c, ring.n)) {
      if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
      ok = false;
    }
    return ok;
  };
  auto pass = [&](const Piece& q) {
    const uint8_t* scales = q.mat == 0 ? p.s1 : q.mat == 1 ? p.s3 : p.s2;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(scales) + ((int64_t)q.expert * share.N + q.col0 + r) * words;
    const uint32_t* x = nullptr;
    if (r < q.rows * kTermRows4) {
      const int row = DOWN ? q.first + r / kTermRows4 : ls.ent[q.first + r / kTermRows4] / p.k;
      x = reinterpret_cast<const uint32_t*>(terms) + ((int64_t)row * kTermRows4 + r % kTermRows4) * words;
    }
    uint32_t a[2 * kGroup], t[2 * kGroup];
    const bool wide = words % 4 == 0 && q.step0 % 2 == 0;
    auto load = [&](int step0) {
      if (wide) {
#pragma unroll
        for (int i = 0; i < 2 * kGroup; i += 4) {
          const bool have = 2 * step0 + i < words && step0 < q.step1;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          const uint4 y = have ? __ldg(reinterpret_cast<const uint4*>(w + 2 * step0 + i)) : zero;
          const uint4 z = have && x ? __ldcg(reinterpret_cast<const uint4*>(x + 2 * step0 + i)) : zero;
          a[i] = y.x, a[i + 1] = y.y, a[i + 2] = y.z, a[i + 3] = y.w;
          t[i] = z.x, t[i + 1] = z.y, t[i + 2] = z.z, t[i + 3] = z.w;
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < 2 * kGroup; ++i) {
        const int at = 2 * step0 + i;
        const bool have = at < words && step0 < q.step1;
        a[i] = have ? __ldg(w + at) : 0u;
        t[i] = have && x ? __ldcg(x + at) : 0u;
      }
    };
    load((group & 1) == team ? q.step0 : q.step0 + kGroup);
    for (int step0 = q.step0; step0 < q.step1; step0 += kGroup) {
      if ((group++ & 1) != team) {
        ring.n += min(kGroup, q.step1 - step0);
        continue;
      }
      uint32_t* ex = sm.exchange + buf * (2 * kGroup * kRows);
#pragma unroll
      for (int i = 0; i < 2 * kGroup; ++i) {
        ex[i * kRows + r] = a[i];
        if (r < 64) ex[i * kRows + 128 + r] = t[i];
      }
      load(step0 + 2 * kGroup);  // the next ones are on their way meanwhile
      ptx::named_barrier(11 + team, 128);
      for (int u = 0; u < kGroup && step0 + u < q.step1; ++u, ++ring.n) {
        uint32_t v[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t* line = ex + (2 * u + h) * kRows + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * h + j] = line[32 * j];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[8 + 4 * h + j] = j < 2 ? line[128 + 32 * j] : 0u;
        }
        if (!issued()) continue;
        ptx::tc_fence_after();
        const uint32_t to = c.tmem + ((uint32_t)((warp & 3) * 32) << 16) + kAccs * kAccCols + (ring.n % S) * kSfCols;
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
            "%14, %15, %16};" ::"r"(to),
            "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
            "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
            : "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.scaled[ring.n % S]);
      }
      buf ^= 1;
    }
    return true;
  };
  int id = blockIdx.x < share.total ? (int)blockIdx.x : -1;
  while (id >= 0) {
    share.passes(share.chunk(p, ls, id), pass);
    if (!ptx::named_barrier_and(11 + team, 128, issued())) return false;
    id = c.chunk[ring.n % (2 * S)];
  }
  ++ring.n;  // the mark of the end
  return true;
}

// The consumers' part in a routed share, whose warps take different roles for
// coded weights.
template <int RT, bool DOWN>
__device__ bool consume_routed(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring, Ring& coded) {
  if constexpr (RT == kFewBf16) {
    return consume<RT, false, DOWN>(p, ls, sm, ring);
  } else {
    const int warp = threadIdx.x >> 5;
    bool ok = true;
    if (warp < 4) {
      ok = drain<RT, DOWN>(p, ls, sm, coded);
    } else if (RT == kFewMxfp4 && (warp < 8 || warp >= 12)) {
      coded.n = ring.n;
      ok = bring_scales<DOWN>(p, ls, sm, coded, warp >= 12);
    } else if (warp < 8) {
      if (RT == kFewE4m3 && warp == 4) {
        coded.n = ring.n;
        ok = bring_factors<DOWN>(p, ls, sm, coded);
      }
    } else if (warp < 8 + kIssuers) {
      coded.n = ring.n;
      if ((threadIdx.x & 31) == 0) ok = issue_mmas<RT, DOWN>(p, ls, sm, coded, warp - 8);
      __syncwarp();
    }
    return ok;
  }
}

// ------------------------------------------------------------ router
// Logits of this CTA's experts: 8 warps for an expert and a few tokens, sums in fp64
// (the products of two bf16 values are exact there and the sum is good to 2^-53 of
// its terms), rounded once.
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
// router's warps.  With more tokens than these the first CTAs choose, two tokens
// each, and tell the others: a token takes a warp some 2.5 us, a barrier 2.
__device__ void route(const FewParams& p, Lists& ls, uint64_t* keys, volatile uint32_t* abort) {
  constexpr int kThreads = 32 * kRouterWarps;
  const int tid = threadIdx.x - kAllThreads + kThreads;
  const int warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < p.E; e += kThreads) ls.counts[e] = 0;
  const int n = p.T * p.k;
  const bool apart = p.T > kRouterWarps;
  const int choosers = min((int)gridDim.x, (p.T + kRouterWarps - 1) / kRouterWarps);
  const int end = apart && blockIdx.x >= choosers ? 0 : p.T;
  for (int t = (apart ? blockIdx.x * kRouterWarps : 0) + warp; t < end; t += (apart ? choosers : 1) * kRouterWarps) {
    choose(p, ls, t, keys + warp * p.E, reinterpret_cast<float*>(keys + kRouterWarps * p.E) + warp * p.E);
    if (apart && lane < p.k) {
      p.chosen[t * p.k + lane] = ls.idx[t * p.k + lane];
      p.chosen_w[t * p.k + lane] = ls.w[t * p.k + lane];
    }
  }
  router_sync();
  if (apart) {
    if (tid == 0) {
      if (blockIdx.x < choosers) {
        __threadfence();
        atomicAdd(p.bar + 9, 1u);
      }
      grid_poll(p.bar + 9, choosers, p.status, abort);
    }
    if (!ptx::named_barrier_and(10, kThreads, *abort == 0)) return;
    for (int i = tid; i < n; i += kThreads) {
      ls.idx[i] = __ldcg(p.chosen + i);
      ls.w[i] = __ldcg(p.chosen_w + i);
    }
    router_sync();
  }
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
      uint32_t* filled = reinterpret_cast<uint32_t*>(keys);  // the keys are done with
      if (cnt > 0) {
        filled[e0 + lane] = rows + before - cnt;
        const int at = chosen + __popc(any & ((1u << lane) - 1u));
        ls.expert[at] = (int16_t)(e0 + lane);
        ls.start[at] = (int16_t)(rows + before - cnt);
      }
      chosen += __popc(any);
      rows += total;
    }
    if (lane == 0) {
      ls.start[chosen] = (int16_t)rows;
      ls.n = chosen;
    }
  }
  if (warp == 0) {
    // rows of an expert in the entries' order
    volatile uint32_t* filled = reinterpret_cast<uint32_t*>(keys);
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane, e = i < n ? ls.idx[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      if (e >= 0) {
        const int at = filled[e] + __popc(same & ((1u << lane) - 1u));
        ls.ent[at] = (int16_t)i;
        ls.row_of[i] = (int16_t)at;
      }
      __syncwarp();
      if (e >= 0 && (same >> lane) == 1u) filled[e] += __popc(same);
      __syncwarp();
    }
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

// Bits of |v| where v is finite, 0 otherwise.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
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

// Two values as e4m3, the first in the low byte, and back as fp16.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_values(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
  return r;
}

__device__ __forceinline__ float fp16_lo(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)v)); }
__device__ __forceinline__ float fp16_hi(uint32_t v) { return __half2float(__ushort_as_half((uint16_t)(v >> 16))); }

// A warp's 128 values, four a lane from step k on, of row `row` with K steps, as
// e4m3 terms [row][kTermRows8][K] and the power of two that undoes their scaling.
template <int N>
__device__ __forceinline__ void store_e4m3_terms(uint8_t* terms, float* scale, int64_t row, int K, int k,
                                                 const float (&value)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, finite_bits(value[i]));
  top = __reduce_max_sync(0xffffffffu, top);
  // 2^(7 - e) for a largest magnitude of exponent e, and its inverse: normal numbers
  const uint32_t field = max(top >> 23, 8u);
  const float factor = __uint_as_float((261u - field) << 23);
  if ((threadIdx.x & 31) == 0) scale[row * (K / 128) + k / 128] = __uint_as_float((field - 7u) << 23);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool finite = (__float_as_uint(value[i]) & 0x7f800000u) != 0x7f800000u;
    v[i] = finite ? value[i] * factor : __uint_as_float(0x7fffffffu);
  }
  uint8_t* to = terms + row * kTermRows8 * K + k;
#pragma unroll 1  // code that runs once a call costs its fetch: unrolled, h took twice as long
  for (int t = 0; t < N; ++t) {
    const uint32_t q0 = e4m3_pair(v[0], v[1]), q1 = e4m3_pair(v[2], v[3]);
    *reinterpret_cast<uint32_t*>(to + (int64_t)t * K) = q0 | (q1 << 16);
    const uint32_t b0 = e4m3_values(q0), b1 = e4m3_values(q1);
    v[0] = (v[0] - fp16_lo(b0)) * 16.0f;
    v[1] = (v[1] - fp16_hi(b0)) * 16.0f;
    v[2] = (v[2] - fp16_lo(b1)) * 16.0f;
    v[3] = (v[3] - fp16_hi(b1)) * 16.0f;
  }
}

// The same as MXFP4 terms, codes [row][kTermRows4][K / 2] and scale bytes
// [row][kTermRows4][K / 32]: each term takes the scale of what is left of its block
// (as moe_mx_quantise chooses one) and rounds that.
__device__ __forceinline__ void store_mxfp4_terms(uint8_t* terms, uint8_t* scales, int64_t row, int K, int k,
                                                  const float (&value)[4]) {
  float v[4] = {value[0], value[1], value[2], value[3]};
  uint8_t* codes = terms + row * kTermRows4 * (K / 2) + k / 2;
  uint8_t* bytes = scales + row * kTermRows4 * (K / 32) + k / 32;
#pragma unroll 1
  for (int t = 0; t < kTerms4; ++t) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t field = top >> 23;
    const uint32_t s = top >= 0x7f800000u ? 255u : top == 0 ? 127u : field > 2 ? field - 2 : 0u;
    const float inverse = s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
    const float unit = s == 0 ? __uint_as_float(1u << 22) : __uint_as_float(s << 23);
    uint32_t q = 0;
    float back[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c, f;
      asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
          : "=r"(c)
          : "f"(v[2 * i + 1] * inverse), "f"(v[2 * i] * inverse));
      asm("{\n\t.reg .b8 q;\n\tcvt.u8.u32 q, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;\n\t}" : "=r"(f) : "r"(c));
      q |= c << (8 * i);
      back[2 * i] = fp16_lo(f);
      back[2 * i + 1] = fp16_hi(f);
    }
    if (s == 255u) q = 0;  // the scale is NaN: all of the block is, here and in all later terms
    *reinterpret_cast<uint16_t*>(codes + (int64_t)t * (K / 2)) = (uint16_t)q;
    if ((threadIdx.x & 7) == 0) bytes[(int64_t)t * (K / 32)] = (uint8_t)s;
    if (s != 255u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(-back[i], unit, v[i]);
    }
  }
}

// The terms of x, 128 values a warp, by the routers' warps of all CTAs.
template <int RT>
__device__ void token_terms(const FewParams& p) {
  const int lane = threadIdx.x & 31;
  const int blocks = p.d / 128, jobs = p.T * blocks;
  const int warp = (threadIdx.x >> 5) - (kAllThreads / 32 - kRouterWarps);
  for (int job = warp * gridDim.x + blockIdx.x; job < jobs; job += gridDim.x * kRouterWarps) {
    const int t = job / blocks, k = (job - t * blocks) * 128 + 4 * lane;
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p.x + ((int64_t)t * p.d + k) * 2));
    const float x[4] = {ptx::bf16_lo(v.x), ptx::bf16_hi(v.x), ptx::bf16_lo(v.y), ptx::bf16_hi(v.y)};
    if (RT == kFewE4m3)
      store_e4m3_terms<kXTerms8>(p.x_terms, p.x_scale, t, p.d, k, x);
    else
      store_mxfp4_terms(p.x_terms, p.x_term_scales, t, p.d, k, x);
  }
}

// h of every row, four columns a lane and 128 a warp.
template <int RT>
__device__ void activations(const FewParams& p) {
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
    const float* buf = shared ? p.up_s : p.up_r;
    const int parts = shared ? p.split_up_s.parts : p.split_up_r.parts;
    // sums of the segments' chunks in order, four columns a lane
    float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
    const float* from = buf + ((int64_t)(row * 2) * blocks + block) * parts * kFewCols + 4 * lane;
    const int64_t second = (int64_t)blocks * parts * kFewCols;
#pragma unroll 4
    for (int i = 0; i < parts; ++i, from += kFewCols) {
      add(g, __ldcg(reinterpret_cast<const float4*>(from)));
      add(u, __ldcg(reinterpret_cast<const float4*>(from + second)));
    }
    const float h[4] = {gated(g.x, u.x), gated(g.y, u.y), gated(g.z, u.z), gated(g.w, u.w)};
    const int k = block * kFewCols + 4 * lane;
    if (shared)
      store_terms(p.h_s + (int64_t)row * 3 * p.S * 2, p.S, k, h);
    else if (RT == kFewBf16)
      store_terms(p.h_r + (int64_t)row * 3 * p.I * 2, p.I, k, h);
    else if (RT == kFewE4m3)
      store_e4m3_terms<kHTerms8>(p.h_r, p.h_scale, row, p.I, k, h);
    else
      store_mxfp4_terms(p.h_r, p.h_term_scales, row, p.I, k, h);
  }
}

// y: routed rows' chunks in order, slots inside, then the shared expert's.
__device__ void combine(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kWarps;
  const int blocks = p.d / kFewCols;
  const int jobs = p.T * blocks;
  for (int job = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; job < jobs; job += warps) {
    const int t = job / blocks, block = job % blocks;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int parts = p.split_dn_r.parts;
#pragma unroll 1
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      const float* from[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = t * p.k + min(j0 + j, p.k - 1);
        from[j] = p.dn_r + ((int64_t)ls.row_of[i] * blocks + block) * parts * kFewCols + 4 * lane;
        w[j] = ls.w[i];
      }
      const int n = p.k - j0;
#pragma unroll 1
      for (int i = 0; i < parts; ++i) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) v[j] = __ldcg(reinterpret_cast<const float4*>(from[j] + i * kFewCols));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < n) {
            y.x = fmaf(w[j], v[j].x, y.x);
            y.y = fmaf(w[j], v[j].y, y.y);
            y.z = fmaf(w[j], v[j].z, y.z);
            y.w = fmaf(w[j], v[j].w, y.w);
          }
        }
      }
    }
    if (p.S > 0) {
      const int own = p.split_dn_s.parts;
      const float* from = p.dn_s + ((int64_t)t * blocks + block) * own * kFewCols + 4 * lane;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int i = 0; i < own; ++i) add(o, __ldcg(reinterpret_cast<const float4*>(from + i * kFewCols)));
      add(y, o);
    }
    const int64_t at = (int64_t)t * p.d + block * kFewCols + 4 * lane;
    if (p.y_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
          make_uint2(ptx::pack_bf16x2(y.x, y.y), ptx::pack_bf16x2(y.z, y.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = y;
  }
}

// Waits for the last copies of a ring of `size` barriers that was armed `n` times.  All
// were issued before the first wait, so that its limit is the limit of all of them.
__device__ __noinline__ void land_copies(uint64_t* bars, int size, int n, Control& c, uint32_t* status) {
  for (int j = max(0, n - size); j < n; ++j) {
    if (!ptx::wait_bounded(&bars[j % size], (j / size) & 1, &c.never)) {
      raise_status(status, &c.abort, kStatusTimeout);
      return;
    }
  }
}

// Of a whole call the accumulators' drain has seen every MMA done.  Of one that gave up
// they must land before TMEM and the CTA go: each issuer waits for its own.  (A call:
// inlined, it moved the code of the e4m3 layer so that T = 8 took 254 instead of 249 us.)
__device__ __noinline__ void land_mmas(Control& c, uint32_t* status) {
  const int who = (int)(threadIdx.x >> 5) - 8;
  if (who < 0 || who >= kIssuers || (threadIdx.x & 31) != 0) return;
  ptx::mma_commit(&c.landed[who]);
  if (!ptx::wait_bounded(&c.landed[who], 0, &c.never)) raise_status(status, &c.abort, kStatusTimeout);
}

// ------------------------------------------------------------ the kernel
template <int RT>
__global__ void __launch_bounds__(kAllThreads, 1)
    few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ FewMaps maps) {
  extern __shared__ uint8_t dyn[];
  __shared__ Lists ls;
  __shared__ Control ct;
  constexpr int S = Cfg<RT>::kStages;
  constexpr bool kCoded = Cfg<RT>::kCoded;
  Smem sm;
  sm.stages = align_1024(dyn);
  sm.cols = sm.stages + S * Cfg<RT>::kStageBytes;
  sm.red = reinterpret_cast<float*>(sm.cols + 2 * Cfg<RT>::kColBytes);
  // the router's keys, and where it is done, scales on their way
  uint64_t* keys = reinterpret_cast<uint64_t*>(sm.red + 8 * kRedFloats);
  sm.exchange = reinterpret_cast<uint32_t*>(keys);
  sm.c = &ct;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFactors; ++s) ptx::mbar_init(&ct.scaled[s], RT == kFewE4m3 ? 32 : 128);
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(&ct.full[s], 1);
      // 8 consumer warps and the columns' warp, or, of a coded share's stage, that
      // one for 7 or 8 (with e4m3 the factors' warp has its own) and the MMAs
      ptx::mbar_init(&ct.empty[s], kWarps / 2 + 1);
      ptx::mbar_init(&ct.issued[s], 1);
      ptx::mbar_init(&ct.issued[s + S], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ct.col_full[b], 1);
      ptx::mbar_init(&ct.col_empty[b], kWarps);
    }
    for (int b = 0; b < kAccs; ++b) {
      ptx::mbar_init(&ct.acc_full[b], 2);
      ptx::mbar_init(&ct.acc_empty[b], 128);
    }
    for (int i = 0; i < kIssuers; ++i) ptx::mbar_init(&ct.landed[i], 1);
    ptx::mbar_init(&ct.ready, 1);
    ptx::mbar_init(&ct.routed, 32 * kRouterWarps);
    ct.abort = 0u;
    ct.position = 0;  // in range where a share ends early
    ct.never = 0u;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
  }
  if (kCoded && warp == 8) {
    ptx::tmem_alloc(&ct.tmem, kTmemCols<RT>);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  volatile uint32_t* abort = &ct.abort;

  if (warp == kWarps) {
    // ---------------------------------------------- producer
    Ring ring;
    if ((threadIdx.x & 31) < 3) {
      ptx::prefetch_tmap(&maps.routed[threadIdx.x & 31]);
      if (p.S > 0) ptx::prefetch_tmap(&maps.shared[threadIdx.x & 31]);
    }
    bool ok = true;
    if (p.S > 0) ok = produce<kFewBf16, RT, true, false>(maps, p, ls, sm, ring, p.bar + 4);
    if (ok && !warp_wait(&ct.routed, 0, abort)) {
      raise_status(p.status, abort, kStatusTimeout);
      ok = false;
    }
    ok = ok && __all_sync(0xffffffffu, *abort == 0);  // the router gave up: there are no lists
    if (ok) ok = produce<RT, RT, false, false>(maps, p, ls, sm, ring, p.bar + 5);
    if (ok) ok = produce<RT, RT, false, true>(maps, p, ls, sm, ring, p.bar + 6);
    if (ok && p.S > 0) produce<kFewBf16, RT, true, true>(maps, p, ls, sm, ring, p.bar + 7);
    // every issued copy must land before the CTA may exit
    if ((threadIdx.x & 31) == 0) land_copies(ct.full, S, ring.n, ct, p.status);
  } else if (warp == kWarps + 1) {
    // ---------------------------------------------- columns
    Ring ring;
    bool ok = true;
    auto wait = [&](uint64_t* bar) {
      if (warp_wait(bar, 0, abort) && __all_sync(0xffffffffu, *abort == 0)) {
        ptx::fence_proxy_async_all();  // x's and h's terms were written by ordinary stores
        return true;
      }
      raise_status(p.status, abort, kStatusTimeout);
      return false;
    };
    if (p.S > 0) ok = bring_columns<RT, true, false>(p, ls, sm, ring);
    if constexpr (kCoded) {
      ok = ok && wait(&ct.routed) && bring_terms<RT, false>(maps, p, ls, sm, ring);
      ok = ok && wait(&ct.ready) && bring_terms<RT, true>(maps, p, ls, sm, ring);
    } else {
      ok = ok && wait(&ct.routed) && bring_columns<RT, false, false>(p, ls, sm, ring);
      ok = ok && wait(&ct.ready) && bring_columns<RT, false, true>(p, ls, sm, ring);
    }
    if (ok && p.S > 0) bring_columns<RT, true, true>(p, ls, sm, ring);
    // every issued copy must land before the CTA may exit
    land_copies(ct.col_full, 2, ring.cols, ct, p.status);
  } else if (warp > kWarps) {
    // ---------------------------------------------- router
    if constexpr (kCoded) {
      token_terms<RT>(p);
      ptx::fence_proxy_async_all();  // TMA will read them
      router_sync();
    }
    if (threadIdx.x == kThreads + 64) {
      if (kCoded) {
        __threadfence();
        atomicAdd(p.bar + 8, 1u);
      }
      grid_poll(p.bar + 0, gridDim.x, p.status, abort);
      if (kCoded) grid_poll(p.bar + 8, gridDim.x, p.status, abort);
    }
    if (ptx::named_barrier_and(10, 32 * kRouterWarps, *abort == 0)) route(p, ls, keys, abort);
    ptx::mbar_arrive(&ct.routed);
  } else {
    // ---------------------------------------------- consumers
    Ring ring, coded;
    logits_share(p, reinterpret_cast<double*>(sm.red));
    grid_arrive(p.bar + 0, abort);
    bool ok = true, whole = false;
    if (p.S > 0) ok = consume<RT, true, false>(p, ls, sm, ring);
    // all consumers agree on whether there are lists
    ok = ptx::named_barrier_and(9, kThreads, ok && ptx::wait_bounded(&ct.routed, 0, abort) && *abort == 0);
    if (ok) consume_routed<RT, false>(p, ls, sm, ring, coded);
    grid_arrive(p.bar + 1, abort);
    if (grid_wait(p.bar + 1, p.status, abort)) {
      if (kCoded) ring.n = ct.position;
      activations<RT>(p);
      ptx::fence_proxy_async_all();  // bulk copies will read h
      grid_arrive(p.bar + 2, abort);
      if (grid_wait(p.bar + 2, p.status, abort)) {
        if (threadIdx.x == 0) ptx::mbar_arrive(&ct.ready);
        consume_routed<RT, true>(p, ls, sm, ring, coded);
        if (p.S > 0) {
          if (kCoded) {
            // the ring's position is known to the warp that issued the MMAs
            consumer_sync();
            ring.n = ct.position;
          }
          consume<RT, true, true>(p, ls, sm, ring);
        }
        grid_arrive(p.bar + 3, abort);
        whole = grid_wait(p.bar + 3, p.status, abort);
        if (whole) combine(p, ls);
      }
    }
    if (kCoded && !whole) land_mmas(ct, p.status);
  }
  if constexpr (kCoded) {
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
      ptx::tc_fence_after();
      ptx::tmem_dealloc(ct.tmem, kTmemCols<RT>);
    }
  }
}

template <int RT>
cudaError_t launch(const FewParams& p, const FewMaps& maps, int sms, cudaStream_t stream) {
  // stages, the columns, the pairs' joins; a routing key and a logit per expert and
  // router warp, or the scales' exchange
  auto bytes = [](size_t experts) {
    return 1024 + Cfg<RT>::kStages * Cfg<RT>::kStageBytes + 2 * Cfg<RT>::kColBytes + 8 * kRedFloats * 4 +
           std::max<size_t>(kRouterWarps * experts * 12, Cfg<RT>::kCoded ? kExchangeBytes : 0);
  };
  const size_t smem = bytes(p.E);
  auto kernel = few_kernel<RT>;
  // the most that any call takes: a limit of its own could be lowered by another
  // thread's call before this one's launch
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(kMaxExperts));
  if (err != cudaSuccess) return err;
  void* args[] = {const_cast<FewParams*>(&p), const_cast<FewMaps*>(&maps)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(sms), dim3(kAllThreads), args, smem,
                                     stream);
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
