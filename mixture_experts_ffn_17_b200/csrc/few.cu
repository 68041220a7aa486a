// few.cu -- the whole layer for a few tokens (T <= 16) in one cooperative kernel.
//
//   logits = x Wg^T (summed in fp64, rounded to fp32), the k experts of each
//   token and their weights as moe_router_topk;
//   y[t] = sum_j w[t,j] (silu(x W1e) * (x W3e)) W2e + shared(x[t]).
//
// With at most 16 tokens an expert sees one or two rows, so the layer is a
// stream of the chosen experts' weights through the SMs (bound by HBM: 3 d I
// weights an expert against 2 T operations a weight) and everything else is
// latency.  One CTA per SM walks all steps, with grid barriers between them:
//   0  logits of a share of the experts; then, before waiting, this CTA's
//      share of the shared expert's up projections, which need no routing
//   1  top-k in every CTA (redundantly), the list of chosen experts and their
//      rows; this CTA's share of the routed up projections
//   2  h = silu(g) * u from the partial sums, as three bf16 terms
//   3  this CTA's share of the down projections
//   4  y from the partial sums
//
// Split of the work.  A segment is 128 output columns of one matrix of one
// expert, a unit 128 steps of its contraction.  The units of all segments lie
// on one line that is cut into equal shares, one a CTA, so every SM streams the
// same number of bytes whatever the number of experts; a share's part of one
// segment is a piece, and its sums go to slot (segment + CTA) of a buffer
// (unique: along the line each piece raises one of the two by one).  Who
// consumes a segment adds its pieces in CTA order: no atomics, and equal inputs
// give equal bits.
//
// Arithmetic: mma.sync m16n8k16 with the weights as the A operand (16 output
// columns by 16 steps) taken from global memory straight into registers, and
// the tokens as the 8 columns of B.  The order of the 16 steps inside an MMA is
// free as long as A and B agree, so lane (g, c) takes steps 4c..4c+3 of columns
// 8g..8g+7: one wide load a step, and pairs of steps are joined by byte
// permutes.  (tcgen05 would need the weights in shared memory and at least 8
// more columns; the tensor work here is a few percent either way.)  e4m3 and
// MXFP4 codes become bf16 exactly: their exponent and mantissa bits are moved
// to bf16's and the exponent's offset is made up by an exact multiplication
// with a power of two.  x is bf16; h is fp32 and goes in as three bf16 terms
// (8 bits each: 24 in all), so its rounding costs nothing against fp32.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "few.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNT = 3;       // 8-column B tiles of one pass
constexpr int kRedPitch = 129;  // floats of one B column in the CTA's reduction buffer
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = kFewMaxTokens * 32;  // T * k

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
  uint32_t abort;
};

// ------------------------------------------------------------ grid barrier
__device__ __forceinline__ void grid_arrive(uint32_t* bar) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(bar, 1u);
  }
}

__device__ bool grid_wait(uint32_t* bar, uint32_t* status, uint32_t* abort) {
  if (threadIdx.x == 0) {
    const uint64_t t0 = ptx::globaltimer();
    uint32_t n = 0;
    uint32_t seen;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(bar) : "memory");
      if (seen >= gridDim.x) break;
      if ((++n & 63u) == 0 && ptx::globaltimer() - t0 > kWaitLimitNs) {
        atomicOr(status, kStatusTimeout);
        *abort = 1u;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
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

// ------------------------------------------------------------ matrix pieces
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ uint2 load_stream8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
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

// The B operand's columns of this lane: for column tile j, lane (g, c) reads
// column 8 j + g; null where there is none.
struct Columns {
  const uint16_t* p[kMaxNT];
};

// This warp's part of a piece for weights [K, N] (bf16 or e4m3): units of 128
// rows by 128 columns; the warp takes 64 of the columns and 16 of the rows.
template <int WT, int NT>
__device__ __forceinline__ void rows_piece(const uint8_t* W, int64_t N, int col0, int step0, int step1,
                                           const float* scale, int64_t scale_ld, const Columns& B,
                                           float (&acc)[4][NT][4]) {
  constexpr int U = NT == 1 ? 4 : 2;  // units in flight, as registers allow
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int k_in = (warp >> 1) * 16 + 4 * c;
  const int64_t size = WT == kFewBf16 ? 2 : 1;
  const uint8_t* base = W + ((int64_t)k_in * N + col0 + (warp & 1) * 64 + 8 * g) * size;
  for (int s0 = step0; s0 < step1; s0 += U) {
    uint4 a4[WT == kFewBf16 ? U : 1][4];
    uint2 a2[WT == kFewBf16 ? 1 : U][4];
    uint2 b[U][NT];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u < step1) {
        const uint8_t* p = base + (int64_t)(s0 + u) * kFewStep * N * size;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (WT == kFewBf16)
            a4[u][r] = load_stream(p + r * N * size);
          else
            a2[u][r] = load_stream8(p + r * N * size);
        }
        if (WT == kFewE4m3) sc[u] = __ldg(scale + (s0 + u) * scale_ld);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[u][j] = B.p[j] ? *reinterpret_cast<const uint2*>(B.p[j] + (s0 + u) * kFewStep + k_in) : make_uint2(0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u < step1) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t f[4];
          if (WT == kFewBf16) {
            const uint32_t w0 = (&a4[u][0].x)[t], w1 = (&a4[u][1].x)[t], w2 = (&a4[u][2].x)[t], w3 = (&a4[u][3].x)[t];
            f[0] = __byte_perm(w0, w1, 0x5410);
            f[1] = __byte_perm(w0, w1, 0x7632);
            f[2] = __byte_perm(w2, w3, 0x5410);
            f[3] = __byte_perm(w2, w3, 0x7632);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma(acc[t][j], f, b[u][j].x, b[u][j].y);
          } else {
            const uint32_t w0 = t < 2 ? a2[u][0].x : a2[u][0].y, w1 = t < 2 ? a2[u][1].x : a2[u][1].y;
            const uint32_t w2 = t < 2 ? a2[u][2].x : a2[u][2].y, w3 = t < 2 ? a2[u][3].x : a2[u][3].y;
            const uint32_t lo = (t & 1) ? 0x6020u : 0x4000u, hi = (t & 1) ? 0x7030u : 0x5010u;
            f[0] = e4m3_pair(__byte_perm(w0, w1, lo));
            f[1] = e4m3_pair(__byte_perm(w0, w1, hi));
            f[2] = e4m3_pair(__byte_perm(w2, w3, lo));
            f[3] = e4m3_pair(__byte_perm(w2, w3, hi));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma(part, f, b[u][j].x, b[u][j].y);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(part[i], sc[u], acc[t][j][i]);
            }
          }
        }
      }
    }
  }
}

// The same for MXFP4 weights [N, K / 2]: the warp takes 16 of the 128 output
// columns (rows of W) and every second unit; lane (g, c) reads scale block c
// of the unit for columns g and g + 8.
template <int NT>
__device__ __forceinline__ void codes_piece(const uint8_t* W, const uint8_t* scales, int64_t K, int col0, int step0,
                                            int step1, const Columns& B, float (&acc)[NT][4]) {
  constexpr int U = NT == 1 ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int64_t n = col0 + (warp & 7) * 16 + g;
  const uint8_t* base = W + n * (K / 2) + c * 16;
  const uint8_t* sbase = scales + n * (K / 32) + c;
  for (int s0 = step0 + (warp >> 3); s0 < step1; s0 += 2 * U) {
    uint4 a[U][2];
    uint32_t sc[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + 2 * u;
      if (s < step1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          a[u][r] = load_stream(base + (int64_t)r * 8 * (K / 2) + (int64_t)s * (kFewStep / 2));
          sc[u][r] = __ldg(sbase + (int64_t)r * 8 * (K / 32) + (int64_t)s * (kFewStep / 32));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + 2 * u;
      if (s < step1) {
        // 2^(byte - 127 + 126) as bf16x2; a scale of 4 or more would leave
        // bf16's range there and takes a second multiplication by 2^(byte - 128)
        uint32_t m[2], over = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t first = min(sc[u][r], 128u);
          const uint32_t e = first + 126u;  // exponent field of 2^(first - 127 + 126)
          m[r] = (e << 7) | (e << 23);
          over |= sc[u][r] > 128u ? 1u : 0u;
        }
        const bool big = __any_sync(0xffffffffu, over != 0);
        uint32_t m2[2] = {0x3f803f80u, 0x3f803f80u};
        if (big) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t v = sc[u][r];
            const uint32_t e = v == 255u ? 0xffu : (v > 128u ? v - 128u : 0u) + 127u;
            m2[r] = v == 255u ? 0x7fff7fffu : (e << 7) | (e << 23);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t w0 = (&a[u][0].x)[q], w1 = (&a[u][1].x)[q];
          uint32_t f0[4] = {mx_pair<0>(w0, m[0]), mx_pair<0>(w1, m[1]), mx_pair<1>(w0, m[0]), mx_pair<1>(w1, m[1])};
          uint32_t f1[4] = {mx_pair<2>(w0, m[0]), mx_pair<2>(w1, m[1]), mx_pair<3>(w0, m[0]), mx_pair<3>(w1, m[1])};
          if (big) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f0[i] = mul_bf16x2(f0[i], m2[i & 1]);
              f1[i] = mul_bf16x2(f1[i], m2[i & 1]);
            }
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 b = B.p[j] ? *reinterpret_cast<const uint4*>(B.p[j] + (int64_t)s * kFewStep + c * 32 + q * 8)
                                   : make_uint4(0u, 0u, 0u, 0u);
            mma(acc[j], f0, __byte_perm(b.x, b.z, 0x5410), __byte_perm(b.x, b.z, 0x7632));
            mma(acc[j], f1, __byte_perm(b.y, b.w, 0x5410), __byte_perm(b.y, b.w, 0x7632));
          }
        }
      }
    }
  }
}

// One matrix as a piece sees it.
struct Matrix {
  const uint8_t* W;  // bf16 / e4m3 [K, N], MXFP4 [N, K / 2]
  const uint8_t* s;
  int64_t K, N;
};

// A piece for `cols` columns of B, its sums to out [cols / group][128]: every
// `group` columns (the terms of one row) are added.
template <int WT, int NT>
__device__ __noinline__ void piece(const Matrix& M, int col0, int step0, int step1, const Columns& B, int rows,
                                   int group, float* out, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  constexpr int kParts = WT == kFewMxfp4 ? 2 : kWarps / 2;  // warps that share a column
  if (WT == kFewMxfp4) {
    float acc[NT][4] = {};
    codes_piece<NT>(M.W, M.s, M.K, col0, step0, step1, B, acc);
    float* to = red + (warp >> 3) * (8 * NT * kRedPitch) + (warp & 7) * 16 + g;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) to[(8 * j + 2 * c + (i & 1)) * kRedPitch + (i >> 1) * 8] = acc[j][i];
  } else {
    float acc[4][NT][4] = {};
    const float* s = WT == kFewE4m3 ? reinterpret_cast<const float*>(M.s) + col0 / 128 : nullptr;
    rows_piece<WT, NT>(M.W, M.N, col0, step0, step1, s, M.N / 128, B, acc);
    float* to = red + (warp >> 1) * (8 * NT * kRedPitch) + (warp & 1) * 64 + 8 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(8 * j + 2 * c + (i & 1)) * kRedPitch + 2 * t + (i >> 1)] = acc[t][j][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kFewCols; i += kThreads) {
    const int r = i / kFewCols, col = i % kFewCols;
    float a = 0.0f;
    for (int q = 0; q < group; ++q)
#pragma unroll
      for (int p = 0; p < kParts; ++p) a += red[(p * 8 * NT + r * group + q) * kRedPitch + col];
    out[(int64_t)r * kFewCols + col] = a;
  }
  __syncthreads();
}

template <int WT>
__device__ __forceinline__ void piece_any(const Matrix& M, int col0, int step0, int step1, const Columns& B, int rows,
                                          int group, float* out, float* red) {
  const int nt = (rows * group + 7) / 8;
  if (nt <= 1)
    piece<WT, 1>(M, col0, step0, step1, B, rows, group, out, red);
  else if (nt == 2)
    piece<WT, 2>(M, col0, step0, step1, B, rows, group, out, red);
  else
    piece<WT, 3>(M, col0, step0, step1, B, rows, group, out, red);
}

// This CTA's share of the up projections: segments are (expert, W1 or W3,
// column block).  Shared expert: every token, in order.
template <int WT, bool SHARED>
__device__ void up_share(const FewParams& p, const Lists& ls, float* buf, float* red) {
  const int N = SHARED ? p.S : p.I;
  const int blocks = N / kFewCols;
  const Line L((SHARED ? 1 : ls.n) * 2 * blocks, p.d / kFewStep);
  const int g = (threadIdx.x & 31) >> 2;
  const uint32_t end = L.begin(blockIdx.x + 1);
  for (uint32_t u = L.begin(blockIdx.x); u < end;) {
    const uint32_t seg = u / L.steps;
    const int step0 = (int)(u - seg * L.steps);
    const int step1 = (int)min(L.steps, step0 + (end - u));
    u += step1 - step0;
    const int block = (int)(seg % blocks);
    const int mat = (int)(seg / blocks) & 1;
    const int ei = (int)(seg / (2 * blocks));
    const int first = SHARED ? 0 : ls.start[ei];
    const int rows = SHARED ? p.T : ls.start[ei + 1] - first;
    Columns B;
#pragma unroll
    for (int j = 0; j < kMaxNT; ++j) {
      const int n = 8 * j + g;
      const int t = SHARED ? n : n < rows ? ls.ent[first + n] / p.k : 0;
      B.p[j] = n < rows ? p.x + (int64_t)t * p.d : nullptr;
    }
    Matrix M{SHARED ? (mat ? p.W3s : p.W1s) : (mat ? p.W3 : p.W1), mat ? p.s3 : p.s1, p.d, N};
    if (!SHARED) {
      const int64_t e = ls.expert[ei], n = (int64_t)p.d * p.I;
      M.W += WT == kFewBf16 ? 2 * e * n : WT == kFewE4m3 ? e * n : e * n / 2;
      M.s += WT == kFewE4m3 ? e * (n / 16384) * 4 : WT == kFewMxfp4 ? e * n / 32 : 0;
    }
    piece_any<WT>(M, block * kFewCols, step0, step1, B, rows, 1, buf + (int64_t)(seg + blockIdx.x) * p.T * kFewCols, red);
  }
}

// This CTA's share of the down projections: segments are (expert, column
// block); the B columns are the three terms of each row's h, at most 8 rows a
// pass (more read the weights again, from L2 mostly: only the shared expert
// and crowded small layers have them).
template <int WT, bool SHARED>
__device__ void down_share(const FewParams& p, const Lists& ls, float* buf, float* red) {
  const int K = SHARED ? p.S : p.I;
  const int blocks = p.d / kFewCols;
  const Line L((SHARED ? 1 : ls.n) * blocks, K / kFewStep);
  const int g = (threadIdx.x & 31) >> 2;
  const uint32_t end = L.begin(blockIdx.x + 1);
  for (uint32_t u = L.begin(blockIdx.x); u < end;) {
    const uint32_t seg = u / L.steps;
    const int step0 = (int)(u - seg * L.steps);
    const int step1 = (int)min(L.steps, step0 + (end - u));
    u += step1 - step0;
    const int block = (int)(seg % blocks);
    const int ei = (int)(seg / blocks);
    const int first = SHARED ? p.T * p.k : ls.start[ei];
    const int all = SHARED ? p.T : ls.start[ei + 1] - first;
    Matrix M{SHARED ? p.W2s : p.W2, p.s2, K, p.d};
    if (!SHARED) {
      const int64_t e = ls.expert[ei], n = (int64_t)p.d * p.I;
      M.W += WT == kFewBf16 ? 2 * e * n : WT == kFewE4m3 ? e * n : e * n / 2;
      M.s += WT == kFewE4m3 ? e * (n / 16384) * 4 : WT == kFewMxfp4 ? e * n / 32 : 0;
    }
    for (int r0 = 0; r0 < all; r0 += 8) {
      const int rows = min(8, all - r0);
      Columns B;
#pragma unroll
      for (int j = 0; j < kMaxNT; ++j) {
        const int n = 8 * j + g;
        B.p[j] = n < 3 * rows ? p.h + ((int64_t)(first + r0) * 3 + n) * p.ld_h : nullptr;
      }
      piece_any<WT>(M, block * kFewCols, step0, step1, B, rows, 3,
                    buf + ((int64_t)(seg + blockIdx.x) * p.T + r0) * kFewCols, red);
    }
  }
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
    __syncthreads();
    if (tid < p.T) {
      double a = 0.0;
#pragma unroll
      for (int w = 0; w < 8; ++w) a += red[(half * 8 + w) * kFewMaxTokens + tid];
      p.logits[(int64_t)tid * p.E + e] = (float)a;
    }
    __syncthreads();
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

// Routing of all tokens and the lists of chosen experts and their rows.
__device__ void route(const FewParams& p, Lists& ls, double* keys) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kThreads) ls.counts[e] = 0;
  if (warp < p.T) choose(p, ls, warp, keys + (int64_t)warp * p.E);
  __syncthreads();
  const int n = p.T * p.k;
  for (int i = threadIdx.x; i < n; i += kThreads) atomicAdd(&ls.counts[ls.idx[i]], 1);
  __syncthreads();
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
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int e = ls.idx[i];
    int at = ls.start[ls.seg_of[e]];
    for (int q = 0; q < i; ++q) at += ls.idx[q] == e ? 1 : 0;
    ls.ent[at] = (int16_t)i;
    ls.row_of[i] = (int16_t)at;
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      if (p.idx_out) p.idx_out[i] = ls.idx[i];
      if (p.w_out) p.w_out[i] = ls.w[i];
    }
    if (p.counts_out)
      for (int e = threadIdx.x; e < p.E; e += kThreads) p.counts_out[e] = ls.counts[e];
  }
  __syncthreads();
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
__device__ void activations(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int rows = p.T * p.k;
  const int rb = p.I / kFewCols, sb = p.S / kFewCols;
  const int64_t jobs = (int64_t)rows * rb + (int64_t)p.T * sb;
  const Line Lr(ls.n * 2 * rb, p.d / kFewStep);
  const Line Ls(2 * sb, p.d / kFewStep);
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
__device__ void combine(const FewParams& p, const Lists& ls) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int blocks = p.d / kFewCols;
  const Line Lr(ls.n * blocks, p.I / kFewStep);
  const Line Ls(blocks, p.S > 0 ? p.S / kFewStep : 1);
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

template <int WT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Lists ls;
  float* red = reinterpret_cast<float*>(dyn);
  double* keys = reinterpret_cast<double*>(dyn);
  if (threadIdx.x == 0) ls.abort = 0;

  logits_share(p, keys);
  grid_arrive(p.bar + 0);
  if (p.S > 0) up_share<kFewBf16, true>(p, ls, p.up_s, red);
  if (!grid_wait(p.bar + 0, p.status, &ls.abort)) return;

  route(p, ls, keys);
  up_share<WT, false>(p, ls, p.up_r, red);
  grid_arrive(p.bar + 1);
  if (!grid_wait(p.bar + 1, p.status, &ls.abort)) return;

  activations(p, ls);
  grid_arrive(p.bar + 2);
  if (!grid_wait(p.bar + 2, p.status, &ls.abort)) return;

  if (p.S > 0) down_share<kFewBf16, true>(p, ls, p.dn_s, red);
  down_share<WT, false>(p, ls, p.dn_r, red);
  grid_arrive(p.bar + 3);
  if (!grid_wait(p.bar + 3, p.status, &ls.abort)) return;

  combine(p, ls);
}

}  // namespace

size_t few_smem_bytes(const FewParams& p, int weights) {
  // the CTA's reduction buffer for the widest pass (the shared expert's is
  // bf16 whatever the routed weights), or the tokens' routing keys
  const size_t red = (size_t)(kWarps / 2) * 8 * kMaxNT * kRedPitch * 4;
  (void)weights;
  return std::max(red, (size_t)p.T * p.E * 8);
}

cudaError_t launch_few(const FewParams& p, int weights, int sms, cudaStream_t stream) {
  const size_t smem = few_smem_bytes(p, weights);
  auto kernel = weights == kFewBf16   ? few_kernel<kFewBf16>
                : weights == kFewE4m3 ? few_kernel<kFewE4m3>
                                      : few_kernel<kFewMxfp4>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  FewParams q = p;
  void* args[] = {&q};
  return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(std::min(sms, kFewMaxSms)),
                                     dim3(kThreads), args, smem, stream);
}

}  // namespace moe
