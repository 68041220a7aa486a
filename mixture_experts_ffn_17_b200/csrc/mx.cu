// mx.cu -- MXFP4 quantisation of rows and of weight matrices, and reading back.
//
// MXFP4 (OCP MX specification): 32 consecutive values along the contraction
// share a scale 2^(s - 127), one byte s, and each value is a 4-bit e2m1 code
// of magnitude 0, 0.5, 1, 1.5, 2, 3, 4 or 6.  With m the largest magnitude of
// a block,
//   s = max(0, floor(log2 m) - 2 + 127)   (127 where m = 0, 255 where the
//                                          block holds a NaN or an infinity),
//   code = the value of the grid nearest v / 2^(s - 127), ties to the even
//          code, magnitudes above 6 taken as 6.
// floor(log2 m) + 127 is the exponent field of m in fp32, so s = field - 2,
// and the inverse scale 2^(127 - s) is a normal fp32 number for every s that
// can arise (its field is 254 - s, 2 to 254): the product v 2^(127 - s) is
// exact where it is not far below the smallest code, and the only rounding is
// the conversion's.
//
// All three kernels move bytes and are bound by HBM (per value 2 or 4 bytes on
// the wide side, 17/32 on the narrow one), but for silu(g) * u of bf16 values, whose
// exponential and reciprocal keep the SMs busy (70% of the issue slots, DRAM 43%):
// 32768 x 7168 take 269 us in bf16, 4.0 TB/s, and 315 us in fp32, 6.4 TB/s.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "mx.h"

namespace moe {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte of a block whose largest magnitude has these fp32 bits (NaN and
// infinities have the largest bits of all, so the maximum over the bits finds
// them too).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= kInfBits) return 255u;
  if (top == 0) return 127u;
  const uint32_t field = top >> 23;
  return field > 2 ? field - 2 : 0u;
}

// 2^(127 - s); 0 for s = 255, whose codes are all zero.
__device__ __forceinline__ float inverse_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// Codes of eight values, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float inv, bool bad) {
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b;
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
        : "=r"(b)
        : "f"(v[2 * i + 1] * inv), "f"(v[2 * i] * inv));
    c |= b << (8 * i);
  }
  return bad ? 0u : c;
}

__device__ __forceinline__ uint32_t top_bits(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}

// Eight consecutive values at element `at`.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (VEC) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(q));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = ptx::bf16_lo(w[i]);
        v[2 * i + 1] = ptx::bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)__ldg(q + i) << 16);
    }
  } else {
    const float* q = static_cast<const float*>(p) + at;
    if (VEC) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(q)), b = __ldg(reinterpret_cast<const float4*>(q) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldg(q + i);
    }
  }
}

// silu(g) * u, silu(g) = g / (1 + e^-g) = g e^g / (1 + e^g), of which the form whose
// exponential is at most 1 is taken: the denominator stays between 1 and 2, where the fast
// reciprocal is good, and silu(g) small instead of 0 down to the smallest fp32 numbers.
// The exponential is good to one step of fp32 (2^-149 at least), the sum, the reciprocal
// and the products add some five halves.  silu(g) first: g * u may overflow where it does
// not.
__device__ __forceinline__ float gated(float g, float u) {
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? g * e : g) * __fdividef(1.0f, 1.0f + e) * u;
}

// Groups of 8 values in flight per thread: 2048 threads of an SM with 16 bytes each
// do not cover HBM's latency (58% of its rate, with 64 bytes 84%).
template <bool BF16, bool GATED>
constexpr int kGroups = (BF16 ? 4 : 2) / (GATED ? 2 : 1);

// One thread quantises 8 values of a group, four neighbouring threads a block: their
// largest magnitude is joined by two shuffles.  Loads are 16 bytes wide (VEC: base
// and row stride allow it) and a warp's codes one 128-byte line.  DENSE: rows follow
// one another, so that a group's place needs no division.
template <bool BF16, bool VEC, bool GATED, bool DENSE>
__global__ void __launch_bounds__(256)
    mx_quantise_kernel(const void* __restrict__ src, const void* __restrict__ up, int64_t groups, int per_row,
                       int64_t ld, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int U = kGroups<BF16, GATED>;
  grid_dependency_wait();
  // groups is a multiple of 4, so the four threads of a block leave together
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * U;
  for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x * U; g0 < groups; g0 += stride) {
    float v[U][8], w[GATED ? U : 1][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * 256 + threadIdx.x;
      if (g < groups) {
        int64_t at = g * 8;
        if (!DENSE) {
          const int64_t row = groups <= 0xffffffffll ? (int64_t)((uint32_t)g / (uint32_t)per_row) : g / per_row;
          at = row * ld + (g - row * per_row) * 8;
        }
        load8<BF16, VEC>(src, at, v[u]);
        if (GATED) load8<BF16, VEC>(up, at, w[u % (GATED ? U : 1)]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = w[u % (GATED ? U : 1)][i] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * 256 + threadIdx.x;
      if (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = gated(v[u][i], w[u % (GATED ? U : 1)][i]);
      }
      uint32_t top = top_bits(v[u]);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t s = scale_byte(top);
      if (g < groups) {
        codes[g] = codes_of(v[u], inverse_scale(s), s == 255u);
        if ((threadIdx.x & 3) == 0) scales[g >> 2] = (uint8_t)s;
      }
    }
  }
}

// W [K, N] of one expert to codes along K: a CTA takes 256 rows by 64 columns,
// warp w the 32 rows of one scale block and lane l columns 2l and 2l + 1, so
// loads are whole rows (a 128-byte line a warp in bf16) and the maximum of a
// block stays in a thread.  The codes go through shared memory, so that each
// column leaves as 128 consecutive bytes.
constexpr int kWRows = 256, kWCols = 64;
constexpr int kWPitch = kWRows / 2 + 16;  // bytes of a column's codes in shared memory

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256)
    mx_quantise_weights_kernel(const void* __restrict__ W, int K, int N, uint8_t* __restrict__ codes,
                               uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t sh_codes[kWCols * kWPitch];
  __shared__ uint8_t sh_scales[kWCols][kWRows / kMxBlock];
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t e = blockIdx.z;
  const int k_base = blockIdx.y * kWRows;
  const int n_base = blockIdx.x * kWCols;
  const int k0 = k_base + warp * kMxBlock;
  const int n0 = n_base + 2 * lane;
  if (k0 < K) {
    // bf16 values stay packed, two columns to a register: half the registers, so
    // twice the threads, whose loads are in flight
    uint32_t raw[BF16 ? kMxBlock : 1];
    float fa[BF16 ? 1 : kMxBlock], fb[BF16 ? 1 : kMxBlock];
    const int64_t at = (e * K + k0) * (int64_t)N + n0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      const int64_t p = at + (int64_t)i * N;
      if (BF16) {
        const uint16_t* q = static_cast<const uint16_t*>(W) + p;
        uint32_t r = 0;
        if (VEC) {  // N even and the base aligned: n0 < N implies n0 + 1 < N
          if (n0 < N) r = __ldg(reinterpret_cast<const uint32_t*>(q));
        } else {
          if (n0 < N) r = __ldg(q);
          if (n0 + 1 < N) r |= (uint32_t)__ldg(q + 1) << 16;
        }
        raw[i % (BF16 ? kMxBlock : 1)] = r;
      } else {
        const float* q = static_cast<const float*>(W) + p;
        float2 r = make_float2(0.0f, 0.0f);
        if (VEC) {
          if (n0 < N) r = __ldg(reinterpret_cast<const float2*>(q));
        } else {
          if (n0 < N) r.x = __ldg(q);
          if (n0 + 1 < N) r.y = __ldg(q + 1);
        }
        fa[i % (BF16 ? 1 : kMxBlock)] = r.x;
        fb[i % (BF16 ? 1 : kMxBlock)] = r.y;
      }
    }
    auto left = [&](int i) { return BF16 ? ptx::bf16_lo(raw[i % (BF16 ? kMxBlock : 1)]) : fa[i % (BF16 ? 1 : kMxBlock)]; };
    auto right = [&](int i) { return BF16 ? ptx::bf16_hi(raw[i % (BF16 ? kMxBlock : 1)]) : fb[i % (BF16 ? 1 : kMxBlock)]; };
    uint32_t ta = 0, tb = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      ta = max(ta, __float_as_uint(left(i)) & 0x7fffffffu);
      tb = max(tb, __float_as_uint(right(i)) & 0x7fffffffu);
    }
    const uint32_t sa = scale_byte(ta), sb = scale_byte(tb);
    const float ia = inverse_scale(sa), ib = inverse_scale(sb);
    uint32_t ca[4], cb[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8], w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = left(8 * q + i);
        w[i] = right(8 * q + i);
      }
      ca[q] = codes_of(v, ia, sa == 255u);
      cb[q] = codes_of(w, ib, sb == 255u);
    }
    uint8_t* to = sh_codes + 2 * lane * kWPitch + warp * 16;
    *reinterpret_cast<uint4*>(to) = make_uint4(ca[0], ca[1], ca[2], ca[3]);
    *reinterpret_cast<uint4*>(to + kWPitch) = make_uint4(cb[0], cb[1], cb[2], cb[3]);
    sh_scales[2 * lane][warp] = (uint8_t)sa;
    sh_scales[2 * lane + 1][warp] = (uint8_t)sb;
  }
  __syncthreads();
  const int blocks = min(kWRows, K - k_base) / kMxBlock;  // scale blocks of this tile
  for (int i = threadIdx.x; i < kWCols * 8; i += 256) {
    const int col = i >> 3, kb = i & 7;
    if (n_base + col < N && kb < blocks) {
      const int64_t row = e * N + n_base + col;
      *reinterpret_cast<uint4*>(codes + row * (K / 2) + (k_base / 2 + kb * 16)) =
          *reinterpret_cast<const uint4*>(sh_codes + col * kWPitch + kb * 16);
      scales[row * (K / kMxBlock) + k_base / kMxBlock + kb] = sh_scales[col][kb];
    }
  }
}

// One thread reads 8 codes, 16 or 32 consecutive bytes of output, of each of
// kReads groups.  The codes come apart in pairs j and j + 4 whose exponent and
// mantissa bits, moved to bf16's, read 2^-126 times their value; two exact
// multiplications make up for that and apply the scale (bf16 holds every value
// and every scale), and byte permutes put neighbours together.
constexpr int kReads = 8;

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(256)
    mx_dequantise_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t groups,
                         void* __restrict__ dst) {
  grid_dependency_wait();
  const int64_t stride = (int64_t)gridDim.x * blockDim.x * kReads;
  for (int64_t b0 = (int64_t)blockIdx.x * blockDim.x * kReads; b0 < groups; b0 += stride) {
    const int64_t g0 = b0 + threadIdx.x;
    uint32_t c[kReads], s[kReads];
#pragma unroll
    for (int u = 0; u < kReads; ++u) {
      const int64_t g = g0 + u * 256;
      if (g < groups) {
        c[u] = __ldg(codes + g);
        s[u] = __ldg(scales + (g >> 2));
      }
    }
#pragma unroll
    for (int u = 0; u < kReads; ++u) {
      const int64_t g = g0 + u * 256;
      const uint32_t lanes = __ballot_sync(0xffffffffu, g < groups);
      if (g >= groups) continue;
      const uint32_t w = c[u];
      uint32_t p[4] = {((w << 12) & 0x80008000u) | ((w << 6) & 0x01c001c0u),
                       ((w << 8) & 0x80008000u) | ((w << 2) & 0x01c001c0u),
                       ((w << 4) & 0x80008000u) | ((w >> 2) & 0x01c001c0u), (w & 0x80008000u) | ((w >> 6) & 0x01c001c0u)};
      // 2^(s - 127) as bf16, 2^-127 as its subnormal; 255 is NaN
      const uint32_t f = s[u] == 255u ? 0x7fffu : s[u] == 0 ? 0x0040u : s[u] << 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = mul_bf16x2(mul_bf16x2(p[i], 0x7e807e80u), f * 0x00010001u);
      const uint32_t o[4] = {__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                             __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)};
      if (BF16) {
        static_cast<uint4*>(dst)[g] = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        // two neighbouring threads write one's 32 bytes and then the other's, so
        // that each store fills whole sectors
        const bool odd = threadIdx.x & 1;
        const uint32_t give0 = odd ? o[0] : o[2], give1 = odd ? o[1] : o[3];
        const uint32_t got0 = __shfl_xor_sync(lanes, give0, 1), got1 = __shfl_xor_sync(lanes, give1, 1);
        float4* to = static_cast<float4*>(dst) + 2 * (g & ~(int64_t)1) + (odd ? 1 : 0);
        const uint32_t a0 = odd ? got0 : o[0], a1 = odd ? got1 : o[1], b0 = odd ? o[2] : got0, b1 = odd ? o[3] : got1;
        to[0] = make_float4(ptx::bf16_lo(a0), ptx::bf16_hi(a0), ptx::bf16_lo(a1), ptx::bf16_hi(a1));
        to[2] = make_float4(ptx::bf16_lo(b0), ptx::bf16_hi(b0), ptx::bf16_lo(b1), ptx::bf16_hi(b1));
      }
    }
  }
}

// CTAs for `items` threads' work.
int grid_for(int64_t items, int sms) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((items + 255) / 256, (int64_t)sms * 16));
}

template <bool BF16, bool VEC, bool GATED>
cudaError_t launch_quantise(const void* src, const void* up, int64_t groups, int per_row, int64_t ld, uint8_t* codes,
                            uint8_t* scales, int sms, cudaStream_t stream) {
  constexpr int U = kGroups<BF16, GATED>;
  const dim3 grid(grid_for((groups + U - 1) / U, sms));
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  auto kernel = ld == (int64_t)per_row * 8 ? mx_quantise_kernel<BF16, VEC, GATED, true>
                                           : mx_quantise_kernel<BF16, VEC, GATED, false>;
  return launch_chained(kernel, grid, dim3(256), 0, stream, src, up, groups, per_row, ld, c, scales);
}

template <bool BF16, bool VEC>
cudaError_t launch_quantise(const void* src, const void* up, int64_t groups, int per_row, int64_t ld, uint8_t* codes,
                            uint8_t* scales, int sms, cudaStream_t stream) {
  return up ? launch_quantise<BF16, VEC, true>(src, up, groups, per_row, ld, codes, scales, sms, stream)
            : launch_quantise<BF16, VEC, false>(src, up, groups, per_row, ld, codes, scales, sms, stream);
}

}  // namespace

cudaError_t launch_mx_quantise(const void* src, const void* up, bool bf16, int64_t rows, int cols, int64_t ld,
                               uint8_t* codes, uint8_t* scales, int sms, cudaStream_t stream) {
  const int64_t groups = rows * (cols / 8);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(up) |
                         (uintptr_t)(ld * (bf16 ? 2 : 4));
  const bool vec = (bits & 15u) == 0;
  if (bf16)
    return vec ? launch_quantise<true, true>(src, up, groups, cols / 8, ld, codes, scales, sms, stream)
               : launch_quantise<true, false>(src, up, groups, cols / 8, ld, codes, scales, sms, stream);
  return vec ? launch_quantise<false, true>(src, up, groups, cols / 8, ld, codes, scales, sms, stream)
             : launch_quantise<false, false>(src, up, groups, cols / 8, ld, codes, scales, sms, stream);
}

cudaError_t launch_mx_quantise_weights(const void* W, bool bf16, int E, int K, int N, uint8_t* codes, uint8_t* scales,
                                       cudaStream_t stream) {
  const dim3 grid((N + kWCols - 1) / kWCols, (K + kWRows - 1) / kWRows, E);
  const bool vec = N % 2 == 0 && (reinterpret_cast<uintptr_t>(W) & (bf16 ? 3u : 7u)) == 0;
  auto kernel = bf16 ? (vec ? mx_quantise_weights_kernel<true, true> : mx_quantise_weights_kernel<true, false>)
                     : (vec ? mx_quantise_weights_kernel<false, true> : mx_quantise_weights_kernel<false, false>);
  return launch_chained(kernel, grid, dim3(256), 0, stream, W, K, N, codes, scales);
}

cudaError_t launch_mx_dequantise(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, void* dst,
                                 bool bf16, int sms, cudaStream_t stream) {
  const int64_t groups = rows * (cols / 8);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  return launch_chained(bf16 ? mx_dequantise_kernel<true> : mx_dequantise_kernel<false>,
                        dim3(grid_for((groups + kReads - 1) / kReads, sms)), dim3(256), 0, stream, c, scales, groups,
                        dst);
}

}  // namespace moe
