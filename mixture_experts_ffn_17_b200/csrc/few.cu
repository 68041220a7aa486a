// few.cu -- the whole layer for a few tokens (T <= 16) in one cooperative kernel.
//
//   logits = x Wg^T (summed in fp64, rounded to fp32), the k experts of each
//   token and their weights as moe_router_topk;
//   y[t] = sum_j w[t,j] (silu(x W1e) * (x W3e)) W2e + shared(x[t]).
//
// With at most 16 tokens an expert sees one or two rows, so the layer is a
// stream of the chosen experts' weights through the SMs (bound by HBM: 3 d I
// weights an expert against 2 T operations a weight) and everything else is
// latency to be kept out of the stream's way.  One CTA per SM, three roles:
//   consumers (16 warps)  logits of a share of the experts, then the products
//                         and the two joins, with grid barriers between them;
//   producer (1 warp)     fills a ring of stages with weight tiles (TMA) and the
//                         matching columns of activations (bulk copies), ahead
//                         of the consumers and across the ends of pieces and
//                         phases: the shared expert's up projections need no
//                         routing and stream while it is found, and the first
//                         tiles of the down projections are in the ring before
//                         the barriers that the activations wait for;
//   router (4 warps)      waits for all logits, finds the top-k (in every CTA)
//                         and the list of chosen experts and their rows.
//
// Split of the work.  A segment is 128 output columns of one matrix of one
// expert, a unit the part of its contraction that one stage holds (16 KB of
// weights: 64 steps of bf16, 128 of e4m3, 256 of MXFP4).  The units of all
// segments lie on one line that is cut into equal shares, one a CTA, so every
// SM streams the same number of bytes whatever the number of experts; a share's
// part of one segment is a piece, and its sums go to slot (segment + CTA) of a
// buffer (unique: along the line each piece raises one of the two by one).  Who
// consumes a segment adds its pieces in CTA order: no atomics, and equal inputs
// give equal bits.
//
// Arithmetic: mma.sync m16n8k16 with the weights as the A operand (16 output
// columns by 16 steps, ldmatrix from the stage) and the activations as B's
// columns, 8 at a time.  (tcgen05 would pad the columns to 16 and could not take
// these codes unconverted; the tensor pipe is idle either way.)  Consumer warp w
// takes columns 16 (w % 8) of a tile and one half of its steps (w / 8).  e4m3
// and MXFP4 codes become bf16 exactly: their exponent and mantissa bits are
// moved to bf16's and the exponent's offset is made up by an exact
// multiplication with a power of two.  x is bf16; h is fp32 and goes in as three
// bf16 terms (8 bits each: 24 in all), so its rounding costs nothing against
// fp32.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "few.h"

namespace moe {
namespace {

constexpr int kWarps = 16;  // consumers
constexpr int kThreads = 32 * kWarps;
constexpr int kRouterWarps = 4;
constexpr int kAllThreads = kThreads + 32 + 32 * kRouterWarps;
constexpr int kMaxNT = 3;       // 8-column B tiles of one pass
constexpr int kMaxCols = 8 * kMaxNT;
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = kFewMaxTokens * 32;  // T * k
constexpr uint32_t kTileBytes = 16384;

// Steps of the contraction that a stage holds, the distance of its B columns in
// bytes (2 steps + a pad that keeps their reads off each other's banks), and the
// stages that fit beside the rest.
template <int WT>
struct Unit {
  static constexpr int kSteps = few_unit_steps(WT);
  static constexpr int kPitch = WT == kFewMxfp4 ? 2 * kSteps + 64 : 2 * kSteps + 16;
  static constexpr uint32_t kBytes = (kTileBytes + kMaxCols * kPitch + 1023) / 1024 * 1024;
  static constexpr int kStages = WT == kFewBf16 ? 8 : WT == kFewE4m3 ? 7 : 5;
};

// Router warps that choose experts at the same time (a key per expert each).
__host__ __device__ constexpr int choosers(int E) { return E <= 512 ? kRouterWarps : kRouterWarps / 2; }

constexpr int kRedPitch = 17;  // floats of one B column of a warp pair's 16 output columns
constexpr int kRedFloats = 2 * kMaxCols * kRedPitch;  // of a pair of warps

struct Lists {  // what the routing leaves in shared memory
  int32_t idx[kMaxRows];      // [T][k]
  float w[kMaxRows];
  int16_t ent[kMaxRows];      // entries t * k + j ordered by expert, then token
  int16_t row_of[kMaxRows];   // the inverse
  int16_t expert[kMaxRows];   // distinct experts, ascending
  int16_t start[kMaxRows + 1];
  int16_t seg_of[kMaxExperts];  // place of an expert among the distinct ones
  int32_t counts[kMaxExperts];
  int n;                      // distinct experts
};

struct Control {
  uint64_t full[9], empty[9];
  uint64_t routed;  // the lists are there
  uint64_t ready;   // h is there, in all CTAs
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

// ------------------------------------------------------------ the line of units
// The host admits only calls whose units * CTAs fit 32 bits.
struct Line {
  uint32_t units;
  uint32_t steps;  // units of a segment
  __device__ Line(int segs, int s) : units((uint32_t)segs * (uint32_t)s), steps((uint32_t)s) {}
  __device__ uint32_t begin(uint32_t cta) const { return units * cta / gridDim.x; }
  // the CTA whose share holds unit u
  __device__ uint32_t owner(uint32_t u) const { return ((u + 1) * gridDim.x - 1) / units; }
};

// Sum of a segment's pieces, four columns at `col` of row `row` of `rows`.
__device__ __forceinline__ float4 sum_pieces(const float* buf, const Line& L, uint32_t seg, int rows, int row, int col) {
  const uint32_t u0 = seg * L.steps, u1 = u0 + L.steps;
  const uint32_t c1 = L.owner(u1 - 1);
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (uint32_t c = L.owner(u0); c <= c1; ++c) {
    if (max(L.begin(c), u0) >= min(L.begin(c + 1), u1)) continue;  // an empty share
    const float4 v = __ldcg(reinterpret_cast<const float4*>(buf + ((int64_t)(seg + c) * rows + row) * kFewCols + col));
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  return a;
}

// ------------------------------------------------------------ tiles and columns
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void lds(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// Two e4m3 codes in bytes 1 and 3 to bf16x2: sign to bit 15, the seven other
// bits to exponent and mantissa; 2^120 makes up the exponents' offsets (127 -
// 7), exactly and for subnormal codes too.  The code 0x7f is NaN.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t v) {
  const uint32_t m = (v >> 4) & 0x07f007f0u;
  uint32_t r = mul_bf16x2((v & 0x80008000u) | m, 0x7b807b80u);
  if (((m + 0x00100010u) & 0x08000800u) != 0) {  // a magnitude of 0x7f in either half
    if ((m & 0xffffu) == 0x07f0u) r |= 0x00007fffu;
    if ((m >> 16) == 0x07f0u) r |= 0x7fff0000u;
  }
  return r;
}

// Codes j and j + 4 of eight MXFP4 codes to bf16x2, times `scale` (2^126 and
// the block's scale in each half): the three low bits go to the ends of
// exponent and mantissa, which reads 2^-126 times the code's value.
template <int J>
__device__ __forceinline__ uint32_t mx_pair(uint32_t w, uint32_t scale) {
  const uint32_t s = J == 3 ? w : w << (12 - 4 * J);
  const uint32_t m = J <= 1 ? w << (6 - 4 * J) : w >> (4 * J - 6);
  return mul_bf16x2((s & 0x80008000u) | (m & 0x01c001c0u), scale);
}

// One stage of a piece: this warp's sums over its half of the steps.
// bf16: two boxes of 64 columns, [steps][64 columns].
template <int NT>
__device__ __forceinline__ void stage_bf16(uint32_t tile, uint32_t cols, float (&acc)[NT][4]) {
  constexpr int P = Unit<kFewBf16>::kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7;
  const int k0 = (warp >> 3) * 32;
  uint32_t b[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) ldsm(b[j], cols + (8 * j + r) * P + (k0 + 8 * i) * 2);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int k = k0 + 16 * q + (i >> 1) * 8 + r;
    const int chunk = (warp & 3) * 2 + (i & 1);
    uint32_t a[4];
    ldsm_t(a, tile + ((warp >> 2) & 1) * 8192 + k * 128 + ((chunk ^ (k & 7)) << 4));
#pragma unroll
    for (int j = 0; j < NT; ++j) mma(acc[j], a, b[j][2 * q], b[j][2 * q + 1]);
  }
}

// e4m3: [steps][128 columns] codes; a 16-bit unit of ldmatrix is two columns of
// one step, so a register holds columns 2g and 2g + 1 of steps 2c and 2c + 1.
template <int NT>
__device__ __forceinline__ void stage_e4m3(uint32_t tile, uint32_t cols, float scale, float (&acc)[NT][4]) {
  constexpr int P = Unit<kFewE4m3>::kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7;
  float part[NT][4] = {};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int k0 = (warp >> 3) * 64 + 32 * q;
    const int k = k0 + 8 * i + r;
    uint32_t w[4];
    ldsm_t(w, tile + k * 128 + (((warp & 7) ^ (k & 7)) << 4));
    uint32_t a0[4] = {e4m3_pair(w[0] << 8), e4m3_pair(w[0]), e4m3_pair(w[1] << 8), e4m3_pair(w[1])};
    uint32_t a1[4] = {e4m3_pair(w[2] << 8), e4m3_pair(w[2]), e4m3_pair(w[3] << 8), e4m3_pair(w[3])};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t b[4];
      ldsm(b, cols + (8 * j + r) * P + (k0 + 8 * i) * 2);
      mma(part[j], a0, b[0], b[1]);
      mma(part[j], a1, b[2], b[3]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(part[j][e], scale, acc[j][e]);
}

// MXFP4: [128 columns][steps / 2] codes; lane (g, c) holds the eight codes 8c of
// a scale block for columns g and g + 8, whose scale bytes are in s[0], s[1].
template <int NT>
__device__ __forceinline__ void stage_mxfp4(uint32_t tile, uint32_t cols, const uint32_t (&s)[2], float (&acc)[NT][4]) {
  constexpr int P = Unit<kFewMxfp4>::kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 3, r = lane & 7, g = lane >> 2, c = lane & 3;
  const int half = warp >> 3;
  const int n = (warp & 7) * 16 + (i & 1) * 8 + r;
#pragma unroll
  for (int p = 0; p < 2; ++p) {  // two scale blocks
    uint32_t w[4];
    const int chunk = half * 4 + 2 * p + (i >> 1);
    ldsm(w, tile + n * 128 + ((chunk ^ (n & 7)) << 4));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int blk = 2 * p + q;
      // 2^(byte - 127 + 126) as bf16x2; a scale of 4 or more would leave
      // bf16's range there and takes a second multiplication by 2^(byte - 128)
      const uint32_t v0 = (s[0] >> (8 * blk)) & 255u, v1 = (s[1] >> (8 * blk)) & 255u;
      const uint32_t m0 = (min(v0, 128u) + 126u) * 0x00800080u, m1 = (min(v1, 128u) + 126u) * 0x00800080u;
      const uint32_t x = w[2 * q], y = w[2 * q + 1];
      uint32_t a0[4] = {mx_pair<0>(x, m0), mx_pair<0>(y, m1), mx_pair<1>(x, m0), mx_pair<1>(y, m1)};
      uint32_t a1[4] = {mx_pair<2>(x, m0), mx_pair<2>(y, m1), mx_pair<3>(x, m0), mx_pair<3>(y, m1)};
      if (__any_sync(0xffffffffu, max(v0, v1) > 128u)) {
        const uint32_t n0 = v0 == 255u ? 0x7fff7fffu : ((v0 > 128u ? v0 - 128u : 0u) + 127u) * 0x00800080u;
        const uint32_t n1 = v1 == 255u ? 0x7fff7fffu : ((v1 > 128u ? v1 - 128u : 0u) + 127u) * 0x00800080u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a0[e] = mul_bf16x2(a0[e], (e & 1) ? n1 : n0);
          a1[e] = mul_bf16x2(a1[e], (e & 1) ? n1 : n0);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        lds(b, cols + (8 * j + g) * P + (half * 128 + blk * 32 + 8 * c) * 2);
        mma(acc[j], a0, __byte_perm(b[0], b[2], 0x5410), __byte_perm(b[0], b[2], 0x7632));
        mma(acc[j], a1, __byte_perm(b[1], b[3], 0x5410), __byte_perm(b[1], b[3], 0x7632));
      }
    }
  }
}

// ------------------------------------------------------------ shares and pieces
// One pass over a piece: units [step0, step1) of 128 output columns of one
// matrix, for `rows` rows of `group` B columns each.
struct Piece {
  int mat;     // 0: W1, 1: W3, 2: W2
  int expert;  // slice of the routed weights
  int col0, step0, step1;
  int first;   // up: place of the first row in the list; down: row of h
  int rows, group;
  bool again;  // the weights are read by another pass too
  float* out;  // [rows][128]
};

// Calls f for every pass of this CTA's share, in order, until it returns false.
// Up projections: segments are (expert, W1 or W3, column block), the shared
// expert sees every token in order.  Down projections: segments are (expert,
// column block) and B holds the three terms of each row's h, at most 8 rows a
// pass (more read the weights again, from L2 mostly: only the shared expert and
// crowded small layers have them).
template <int WT, bool SHARED, bool DOWN, typename F>
__device__ __forceinline__ bool for_pieces(const FewParams& p, const Lists& ls, F f) {
  const int inner = SHARED ? p.S : p.I;
  const int K = DOWN ? inner : p.d;
  const int blocks = (DOWN ? p.d : inner) / kFewCols;
  const int per_expert = DOWN ? blocks : 2 * blocks;
  float* buf = SHARED ? (DOWN ? p.dn_s : p.up_s) : (DOWN ? p.dn_r : p.up_r);
  const Line L((SHARED ? 1 : ls.n) * per_expert, (K + Unit<WT>::kSteps - 1) / Unit<WT>::kSteps);
  const uint32_t end = L.begin(blockIdx.x + 1);
  for (uint32_t u = L.begin(blockIdx.x); u < end;) {
    const uint32_t seg = u / L.steps;
    Piece q;
    q.step0 = (int)(u - seg * L.steps);
    q.step1 = (int)min(L.steps, q.step0 + (end - u));
    u += q.step1 - q.step0;
    const int ei = (int)(seg / per_expert), in = (int)seg - ei * per_expert;
    q.mat = DOWN ? 2 : in >= blocks ? 1 : 0;
    q.col0 = (in - (q.mat == 1 ? blocks : 0)) * kFewCols;
    q.expert = SHARED ? 0 : ls.expert[ei];
    const int first = SHARED ? (DOWN ? p.T * p.k : 0) : ls.start[ei];
    const int all = SHARED ? p.T : ls.start[ei + 1] - ls.start[ei];
    float* out = buf + (int64_t)(seg + blockIdx.x) * p.T * kFewCols;
    constexpr int kPass = DOWN ? kMaxCols / 3 : kFewMaxTokens;
    q.group = DOWN ? 3 : 1;
    q.again = all > kPass;
    for (int r0 = 0; r0 < all; r0 += kPass) {
      q.first = first + r0;
      q.rows = min(kPass, all - r0);
      q.out = out + r0 * kFewCols;
      if (!f(q)) return false;
    }
  }
  return true;
}

// The ring's position: stages handed over so far.
struct Ring {
  int n = 0;
};

struct Smem {
  uint8_t* stages;
  float* red;
  Control* c;
};

// ------------------------------------------------------------ producer
template <int WT, int RT>
__device__ __forceinline__ uint8_t* stage_at(const Smem& sm, int s) {
  return sm.stages + s * Unit<RT>::kBytes;
}

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

// Streams a share.  early: as many tiles as the ring holds go ahead of the
// activations' columns, which follow when `ready` completes.
template <int WT, int RT, bool SHARED, bool DOWN>
__device__ bool produce(const FewMaps& m, const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring, bool early) {
  constexpr int S = Unit<RT>::kStages;
  constexpr int kSteps = Unit<WT>::kSteps;
  constexpr int kPitch = Unit<WT>::kPitch;
  const int lane = threadIdx.x & 31;
  const uint64_t once = ptx::policy_evict_first(), more = ptx::policy_evict_normal();
  const int K = DOWN ? (SHARED ? p.S : p.I) : p.d;
  Control& c = *sm.c;
  auto columns = [&](const Piece& q, int step, int slot) {
    const int n = lane;
    if (n >= q.rows * q.group) return;
    const uint16_t* src = DOWN ? p.h + ((int64_t)q.first * 3 + n) * p.ld_h
                               : p.x + (int64_t)(SHARED ? n : ls.ent[q.first + n] / p.k) * p.d;
    bulk_load(ptx::smem_u32(stage_at<WT, RT>(sm, slot)) + kTileBytes + n * kPitch, src + step * kSteps,
              2 * min(kSteps, K - step * kSteps), &c.full[slot]);
  };
  auto tile = [&](const Piece& q, int step, int slot) {
    if (lane == 0) {
      const uint32_t cols = q.rows * q.group * 2 * min(kSteps, K - step * kSteps);
      ptx::mbar_arrive_expect_tx(&c.full[slot], kTileBytes + cols);
      load_tile<WT, SHARED>(m, p, q, step, stage_at<WT, RT>(sm, slot), &c.full[slot], q.again ? more : once);
    }
    __syncwarp();
  };
  auto slot_free = [&](int n) {
    if (ptx::wait_bounded(&c.empty[n % S], ((n / S) & 1) ^ 1, &c.abort)) return true;
    if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
    return false;
  };
  int ahead = 0;
  if (early) {
    int n = ring.n;
    if (!for_pieces<WT, SHARED, DOWN>(p, ls, [&](const Piece& q) {
          for (int step = q.step0; step < q.step1 && ahead < S; ++step, ++ahead, ++n) {
            if (!slot_free(n)) return false;
            tile(q, step, n % S);
          }
          return ahead < S;
        }) &&
        c.abort)
      return false;
    if (!ptx::wait_bounded(&c.ready, 0, &c.abort)) {
      if (lane == 0) raise_status(p.status, &c.abort, kStatusTimeout);
      return false;
    }
    ptx::fence_proxy_async_all();  // h was written by ordinary stores
  }
  return for_pieces<WT, SHARED, DOWN>(p, ls, [&](const Piece& q) {
    for (int step = q.step0; step < q.step1; ++step, ++ring.n) {
      if (ahead > 0) {
        --ahead;
      } else {
        if (!slot_free(ring.n)) return false;
        tile(q, step, ring.n % S);
      }
      columns(q, step, ring.n % S);
    }
    return true;
  });
}

// ------------------------------------------------------------ consumers
template <int WT, int RT, int NT>
__device__ __forceinline__ bool consume_piece(const FewParams& p, const Piece& q, const uint8_t* scales, int K, int N,
                                              const Smem& sm, Ring& ring) {
  constexpr int S = Unit<RT>::kStages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  Control& ct = *sm.c;
  float acc[NT][4] = {};
  // scales of the next unit are fetched while this one is multiplied
  const float* sf = nullptr;
  const uint32_t* sw = nullptr;
  float f = 0.0f;
  uint32_t s[2] = {0u, 0u};
  int64_t sld = 0;
  const int half = warp >> 3;
  if constexpr (WT == kFewE4m3) {
    sld = N / 128;
    sf = reinterpret_cast<const float*>(scales) + (int64_t)q.expert * (K / 128) * sld + q.col0 / 128;
    f = __ldg(sf + q.step0 * sld);
  } else if constexpr (WT == kFewMxfp4) {
    sld = K / 128;  // words of four scales in a row
    sw = reinterpret_cast<const uint32_t*>(scales) +
         ((int64_t)q.expert * N + q.col0 + (warp & 7) * 16 + g) * sld + half;
    if (2 * q.step0 + half < sld) {
      s[0] = __ldg(sw + 2 * q.step0);
      s[1] = __ldg(sw + 8 * sld + 2 * q.step0);
    }
  }
  for (int step = q.step0; step < q.step1; ++step, ++ring.n) {
    float f1 = 0.0f;
    uint32_t s1[2] = {0u, 0u};
    if (step + 1 < q.step1) {
      if constexpr (WT == kFewE4m3) f1 = __ldg(sf + (step + 1) * sld);
      if constexpr (WT == kFewMxfp4) {
        if (2 * (step + 1) + half < sld) {
          s1[0] = __ldg(sw + 2 * (step + 1));
          s1[1] = __ldg(sw + 8 * sld + 2 * (step + 1));
        }
      }
    }
    const int slot = ring.n % S;
    if (!ptx::wait_bounded(&ct.full[slot], (ring.n / S) & 1, &ct.abort)) {
      raise_status(p.status, &ct.abort, kStatusTimeout);
      return false;
    }
    const uint32_t tile = ptx::smem_u32(stage_at<WT, RT>(sm, slot)), cols = tile + kTileBytes;
    if constexpr (WT == kFewBf16) stage_bf16<NT>(tile, cols, acc);
    if constexpr (WT == kFewE4m3) stage_e4m3<NT>(tile, cols, f, acc);
    if constexpr (WT == kFewMxfp4) {
      if (2 * step + half < sld) stage_mxfp4<NT>(tile, cols, s, acc);  // the last unit may be half of one
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&ct.empty[slot]);
    f = f1;
    s[0] = s1[0];
    s[1] = s1[1];
  }
  // the two halves of the steps, and the terms of each row, are joined by the
  // pair of warps that has these 16 columns
  const int pair = warp & 7;
  float* red = sm.red + pair * kRedFloats;
  const int lo = WT == kFewE4m3 ? 2 * g : g, hi = WT == kFewE4m3 ? 2 * g + 1 : g + 8;
  float* to = red + half * kMaxCols * kRedPitch;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    to[(8 * j + 2 * c) * kRedPitch + lo] = acc[j][0];
    to[(8 * j + 2 * c + 1) * kRedPitch + lo] = acc[j][1];
    to[(8 * j + 2 * c) * kRedPitch + hi] = acc[j][2];
    to[(8 * j + 2 * c + 1) * kRedPitch + hi] = acc[j][3];
  }
  ptx::named_barrier(1 + pair, 64);
  for (int i = half * 32 + lane; i < q.rows * 16; i += 64) {
    const int r = i >> 4, col = i & 15;
    float a = 0.0f;
    for (int t = 0; t < q.group; ++t) {
      const float* x = red + (r * q.group + t) * kRedPitch + col;
      a += x[0] + x[kMaxCols * kRedPitch];
    }
    q.out[r * kFewCols + pair * 16 + col] = a;
  }
  ptx::named_barrier(1 + pair, 64);
  return true;
}

template <int WT, int RT, bool SHARED, bool DOWN>
__device__ bool consume(const FewParams& p, const Lists& ls, const Smem& sm, Ring& ring) {
  const int inner = SHARED ? p.S : p.I;
  const int K = DOWN ? inner : p.d, N = DOWN ? p.d : inner;
  return for_pieces<WT, SHARED, DOWN>(p, ls, [&](const Piece& q) {
    const uint8_t* scales = q.mat == 0 ? p.s1 : q.mat == 1 ? p.s3 : p.s2;
    const int cols = q.rows * q.group;
    if (cols <= 8) return consume_piece<WT, RT, 1>(p, q, scales, K, N, sm, ring);
    if (cols <= 16) return consume_piece<WT, RT, 2>(p, q, scales, K, N, sm, ring);
    return consume_piece<WT, RT, 3>(p, q, scales, K, N, sm, ring);
  });
}

// ------------------------------------------------------------ router
// Logits of this CTA's experts: 8 warps an expert, sums in fp64 (the products
// of two bf16 values are exact there and the sum is good to 2^-53 of its
// terms), rounded once.
__device__ void logits_share(const FewParams& p, double* red) {
  const int half = threadIdx.x >> 8, tid = threadIdx.x & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = p.d / 8;
  for (int e0 = blockIdx.x * 2; e0 < p.E; e0 += gridDim.x * 2) {
    const int e = e0 + half;  // E is even
    double acc[kFewMaxTokens];
#pragma unroll
    for (int t = 0; t < kFewMaxTokens; ++t) acc[t] = 0.0;
    for (int v = tid; v < nv; v += 256) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.Wg + (int64_t)e * p.d) + v);
      const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
      double w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = (double)ptx::bf16_lo(ww[i]);
        w[2 * i + 1] = (double)ptx::bf16_hi(ww[i]);
      }
#pragma unroll
      for (int t = 0; t < kFewMaxTokens; ++t) {
        if (t < p.T) {
          const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.d) + v);
          const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t] = fma(w[2 * i], (double)ptx::bf16_lo(xx[i]), acc[t]);
            acc[t] = fma(w[2 * i + 1], (double)ptx::bf16_hi(xx[i]), acc[t]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kFewMaxTokens; ++t) {
      if (t < p.T) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        if (lane == 0) red[warp * kFewMaxTokens + t] = acc[t];
      }
    }
    consumer_sync();
    if (tid < p.T) {
      double a = 0.0;
#pragma unroll
      for (int w = 0; w < 8; ++w) a += red[(half * 8 + w) * kFewMaxTokens + tid];
      p.logits[(int64_t)tid * p.E + e] = (float)a;
    }
    consumer_sync();
  }
}

struct Best {
  double key;
  int idx;
};

__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double k = __shfl_xor_sync(0xffffffffu, b.key, o);
    const int i = __shfl_xor_sync(0xffffffffu, b.idx, o);
    if (k > b.key || (k == b.key && i < b.idx)) b = Best{k, i};
  }
  return b;
}

// The k experts of token t and their weights, by one warp.  Scores that decide
// the selection are fp64 (of the fp32 logits); a NaN score ranks last.
__device__ void choose(const FewParams& p, Lists& ls, int t, double* key) {
  const int lane = threadIdx.x & 31;
  const double kLow = -__longlong_as_double(0x7ff0000000000000ll);
  const float* l = p.logits + (int64_t)t * p.E;
  for (int e = lane; e < p.E; e += 32) {
    const double v = (double)__ldcg(l + e);
    double s = p.route == 0 ? v : 1.0 / (1.0 + exp(-v)) + (p.bias ? (double)__ldg(p.bias + e) : 0.0);
    key[e] = s != s ? kLow : s;
  }
  __syncwarp();
  uint32_t taken = 0;  // bit v: expert 32 v + lane is out
  if (p.route == 1) {
    const int size = p.E / p.n_group;
    Best mine{kLow, 0x7fffffff};
    if (lane < p.n_group) {
      uint64_t used = 0;
      double sum = 0.0;
      for (int r = 0; r < p.group_topn; ++r) {
        int bi = -1;
        double bv = kLow;
        for (int i = 0; i < size; ++i)
          if (!((used >> i) & 1) && (bi < 0 || key[lane * size + i] > bv)) {
            bi = i;
            bv = key[lane * size + i];
          }
        used |= 1ull << bi;
        sum += bv;
      }
      mine = Best{sum, lane};
    }
    uint32_t kept = 0;
    for (int r = 0; r < p.topk_group; ++r) {
      const Best b = warp_best(mine);
      kept |= 1u << b.idx;
      if (lane == b.idx) mine = Best{kLow, 0x7fffffff};
    }
    for (int e = lane, v = 0; e < p.E; e += 32, ++v)
      if (!((kept >> (e / size)) & 1)) taken |= 1u << v;
  }
  int my_idx = 0;
  for (int j = 0; j < p.k; ++j) {
    Best b{kLow, 0x7fffffff};
    for (int e = lane, v = 0; e < p.E; e += 32, ++v)
      if (!((taken >> v) & 1) && (key[e] > b.key || (key[e] == b.key && e < b.idx))) b = Best{key[e], e};
    b = warp_best(b);
    if ((b.idx & 31) == lane) taken |= 1u << (b.idx >> 5);
    if (lane == j) my_idx = b.idx;
  }
  const int top = __shfl_sync(0xffffffffu, my_idx, 0);
  float w;
  if (p.route == 0) {
    const float e = lane < p.k ? expf(__ldcg(l + my_idx) - __ldcg(l + top)) : 0.0f;
    float den = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    w = e / den;
  } else {
    const double s = lane < p.k ? 1.0 / (1.0 + exp(-(double)__ldcg(l + my_idx))) : 0.0;
    double den = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    w = (float)((double)p.route_scale * s / den);
  }
  if (lane < p.k) {
    ls.idx[t * p.k + lane] = my_idx;
    ls.w[t * p.k + lane] = w;
  }
}

// Routing of all tokens and the lists of chosen experts and their rows, by the
// router's warps.
__device__ void route(const FewParams& p, Lists& ls, double* keys) {
  constexpr int kThreads = 32 * kRouterWarps;
  const int tid = threadIdx.x - kAllThreads + kThreads;
  const int warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < p.E; e += kThreads) ls.counts[e] = 0;
  const int n_choose = choosers(p.E);
  for (int t = warp; warp < n_choose && t < p.T; t += n_choose) choose(p, ls, t, keys + (int64_t)warp * p.E);
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
        ls.seg_of[e0 + lane] = (int16_t)at;
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
    int at = ls.start[ls.seg_of[e]];
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

// h of every row, four columns a lane.
template <int WT>
__device__ void activations(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int rows = p.T * p.k;
  const int rb = p.I / kFewCols, sb = p.S / kFewCols;
  const int64_t jobs = (int64_t)rows * rb + (int64_t)p.T * sb;
  const Line Lr(ls.n * 2 * rb, (p.d + Unit<WT>::kSteps - 1) / Unit<WT>::kSteps);
  const Line Ls(2 * sb, p.d / Unit<kFewBf16>::kSteps);
  for (int64_t job = (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x; job < jobs; job += warps) {
    const bool shared = job >= (int64_t)rows * rb;
    const int64_t j = shared ? job - (int64_t)rows * rb : job;
    const int blocks = shared ? sb : rb;
    const int row = (int)(j / blocks), block = (int)(j % blocks);
    uint32_t seg = block;
    int at = row;
    if (!shared) {
      const int ei = ls.seg_of[ls.idx[ls.ent[row]]];
      seg += (uint32_t)(ei * 2 * blocks);
      at = row - ls.start[ei];
    }
    const float* buf = shared ? p.up_s : p.up_r;
    const Line& L = shared ? Ls : Lr;
    const float4 g = sum_pieces(buf, L, seg, p.T, at, 4 * lane);
    const float4 u = sum_pieces(buf, L, seg + blocks, p.T, at, 4 * lane);
    const float h[4] = {gated(g.x, u.x), gated(g.y, u.y), gated(g.z, u.z), gated(g.w, u.w)};
    uint32_t t[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) terms_of(h[i], t[i]);
    uint16_t* to = p.h + (int64_t)(shared ? rows + row : row) * 3 * p.ld_h + block * kFewCols + 4 * lane;
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint2*>(to + (int64_t)q * p.ld_h) = make_uint2(t[0][q] | (t[1][q] << 16), t[2][q] | (t[3][q] << 16));
  }
}

// y: routed rows in slot order, then the shared expert's.
template <int WT>
__device__ void combine(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int blocks = p.d / kFewCols;
  const Line Lr(ls.n * blocks, (p.I + Unit<WT>::kSteps - 1) / Unit<WT>::kSteps);
  const Line Ls(blocks, p.S > 0 ? p.S / Unit<kFewBf16>::kSteps : 1);
  const int64_t jobs = (int64_t)p.T * blocks;
  for (int64_t job = (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x; job < jobs; job += warps) {
    const int t = (int)(job / blocks), block = (int)(job % blocks);
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < p.k; ++j) {
      const int i = t * p.k + j;
      const int ei = ls.seg_of[ls.idx[i]];
      const float w = ls.w[i];
      const float4 o = sum_pieces(p.dn_r, Lr, (uint32_t)(ei * blocks + block), p.T, ls.row_of[i] - ls.start[ei], 4 * lane);
      y.x = fmaf(w, o.x, y.x);
      y.y = fmaf(w, o.y, y.y);
      y.z = fmaf(w, o.z, y.z);
      y.w = fmaf(w, o.w, y.w);
    }
    if (p.S > 0) {
      const float4 o = sum_pieces(p.dn_s, Ls, block, p.T, t, 4 * lane);
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
  constexpr int S = Unit<RT>::kStages;
  Smem sm;
  sm.stages = align_1024(dyn);
  sm.red = reinterpret_cast<float*>(sm.stages + S * Unit<RT>::kBytes);
  sm.c = &ct;
  double* keys = reinterpret_cast<double*>(sm.red + 8 * kRedFloats);  // the router's, or partial logits
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(&ct.full[s], 1);
      ptx::mbar_init(&ct.empty[s], kWarps);
    }
    ptx::mbar_init(&ct.routed, 32 * kRouterWarps);
    ptx::mbar_init(&ct.ready, 1);
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
    bool ok = true;
    if (p.S > 0) ok = produce<kFewBf16, RT, true, false>(maps, p, ls, sm, ring, false);
    if (ok && !ptx::wait_bounded(&ct.routed, 0, abort)) {
      raise_status(p.status, abort, kStatusTimeout);
      ok = false;
    }
    ok = ok && *abort == 0;  // the router gave up: there are no lists
    if (ok) ok = produce<RT, RT, false, false>(maps, p, ls, sm, ring, false);
    // the routed share first: it is there in every call
    if (ok) ok = produce<RT, RT, false, true>(maps, p, ls, sm, ring, true);
    if (ok && p.S > 0) produce<kFewBf16, RT, true, true>(maps, p, ls, sm, ring, false);
    // every issued copy must land before the CTA may exit (tiles that went
    // ahead of a wait that failed have landed long before its limit)
    if ((threadIdx.x & 31) == 0)
      for (int j = ring.n > S ? ring.n - S : 0; j < ring.n; ++j)
        if (!ptx::wait_bounded(&ct.full[j % S], (j / S) & 1, &ct.never)) raise_status(p.status, abort, kStatusTimeout);
  } else if (warp > kWarps) {
    // ---------------------------------------------- router
    if (threadIdx.x == kThreads + 32) grid_poll(p.bar + 0, p.status, abort);
    router_sync();
    if (*abort == 0) route(p, ls, keys);
    ptx::mbar_arrive(&ct.routed);
  } else {
    // ---------------------------------------------- consumers
    Ring ring;
    logits_share(p, reinterpret_cast<double*>(sm.red));
    grid_arrive(p.bar + 0);
    bool ok = true;
    if (p.S > 0) ok = consume<kFewBf16, RT, true, false>(p, ls, sm, ring);
    ok = ok && ptx::wait_bounded(&ct.routed, 0, abort) && *abort == 0;
    if (ok) ok = consume<RT, RT, false, false>(p, ls, sm, ring);
    grid_arrive(p.bar + 1);
    if (grid_wait(p.bar + 1, p.status, abort)) {
      activations<RT>(p, ls);
      ptx::fence_proxy_async_all();  // h is read by bulk copies
      grid_arrive(p.bar + 2);
      if (grid_wait(p.bar + 2, p.status, abort)) {
        if (threadIdx.x == 0) ptx::mbar_arrive(&ct.ready);
        if (consume<RT, RT, false, true>(p, ls, sm, ring) && p.S > 0)
          consume<kFewBf16, RT, true, true>(p, ls, sm, ring);
        grid_arrive(p.bar + 3);
        if (grid_wait(p.bar + 3, p.status, abort)) combine<RT>(p, ls);
      }
    }
  }
}

template <int RT>
cudaError_t launch(const FewParams& p, const FewMaps& maps, int sms, cudaStream_t stream) {
  // stages, the pairs' joins, one routing key per expert and choosing warp
  const size_t smem = 1024 + Unit<RT>::kStages * Unit<RT>::kBytes + 8 * kRedFloats * 4 + (size_t)choosers(p.E) * p.E * 8;
  auto kernel = few_kernel<RT>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  void* args[] = {const_cast<FewParams*>(&p), const_cast<FewMaps*>(&maps)};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(std::min(sms, kFewMaxSms)),
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
