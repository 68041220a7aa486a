// grad.cu -- global norm of a set of gradient tensors, and clipping by it.
//
//   norm   = sqrt(sum over all tensors and elements of g^2)
//   factor = min(1, max_norm / (norm + 1e-6)),   out = factor * g
//
// Two passes over memory: grad_square_kernel reads every tensor once and
// leaves one fp64 partial sum per CTA; the next launch (one per 120 tensors)
// has every CTA add the partials in the same fixed order, so that all of them
// hold the same norm without a further launch, an atomic or a counter, and
// scales.  Clipping in place with factor 1 returns without touching the
// tensors.  Both passes are bound by HBM: the floor is one read for the norm
// and one read and one write for the scaling.  The scaling walks the chunks
// in the opposite order, so that what the norm read last is still in L2.
//
// Sums: the 4 or 8 squares of one 16-byte vector are added in fp32 and the
// result goes to an fp64 accumulator: at most 4 (fp32) or 7 roundings of 2^-24
// in a sum of squares, half as much in the norm.  With every square in fp64
// norm and clipping of 750M bf16 values took 899 us instead of 736 (conversions;
// with the fp64 numbers made from the bits 758, with the fp32 sums' errors
// carried along 760).  A vector whose sum
// leaves [1e-30, 1e30] is done again in fp64 element by element, so neither
// tiny gradients vanish nor large ones overflow; all-zero vectors (experts no
// token chose) are skipped.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "grad.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;  // 16-byte vectors in flight per thread

template <bool BF16>
struct Elem {
  static constexpr int kVec = BF16 ? 8 : 4;                       // elements per 16 bytes
  static constexpr int64_t kChunk = (int64_t)kThreads * kUnroll * kVec;  // elements per CTA step
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Which tensor chunk c of this launch belongs to.
__device__ __forceinline__ int tensor_of(const GradBatch& b, uint32_t c) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <bool BF16>
__device__ __forceinline__ double square_of(const uint4& v) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  float f[Elem<BF16>::kVec];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      f[2 * i] = ptx::bf16_lo(r[i]);
      f[2 * i + 1] = ptx::bf16_hi(r[i]);
    } else {
      f[i] = __uint_as_float(r[i]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < Elem<BF16>::kVec; ++i) s = fmaf(f[i], f[i], s);
  if (s >= 1e-30f && s <= 1e30f) return (double)s;
  const uint32_t mag = BF16 ? 0x7fff7fffu : 0x7fffffffu;
  if ((((r[0] | r[1]) | (r[2] | r[3])) & mag) == 0) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < Elem<BF16>::kVec; ++i) d = fma((double)f[i], (double)f[i], d);
  return d;
}

template <bool BF16>
__device__ __forceinline__ double square_one(const void* p, int64_t i) {
  const float f = BF16 ? bf16_value(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  return (double)f * (double)f;
}

// Elements before the first 16-byte boundary of a tensor.
template <bool BF16>
__device__ __forceinline__ int64_t head_of(const void* p, int64_t count) {
  const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (BF16 ? 2 : 4);
  return h < count ? h : count;
}

// Sum of squares of chunk c of one tensor, this thread's part.  Chunk c holds
// the kChunk elements from head + c * kChunk on; chunk 0 also the head.
template <bool BF16>
__device__ double chunk_squares(const void* p, int64_t count, uint32_t c) {
  constexpr int kVec = Elem<BF16>::kVec;
  const int64_t head = head_of<BF16>(p, count);
  double acc = 0.0;
  if (c == 0 && threadIdx.x < head) acc += square_one<BF16>(p, threadIdx.x);
  const int64_t lo = head + (int64_t)c * Elem<BF16>::kChunk;
  const int64_t left = count - lo;
  if (left <= 0) return acc;
  const int64_t n = left < Elem<BF16>::kChunk ? left : Elem<BF16>::kChunk;
  const int nv = (int)(n / kVec);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + lo * (BF16 ? 2 : 4));
  if (nv == kThreads * kUnroll) {
    uint4 r[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) r[i] = __ldg(v + i * kThreads + threadIdx.x);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) acc += square_of<BF16>(r[i]);
  } else {
    for (int i = threadIdx.x; i < nv; i += kThreads) acc += square_of<BF16>(__ldg(v + i));
    const int tail = (int)(n - (int64_t)nv * kVec);
    if (threadIdx.x < tail) acc += square_one<BF16>(p, lo + (int64_t)nv * kVec + threadIdx.x);
  }
  return acc;
}

// Sum over the CTA, the same in every thread; fixed order.
__device__ double block_sum(double a, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
  return s;
}

__global__ void __launch_bounds__(kThreads)
    grad_square_kernel(const __grid_constant__ GradBatch b, double* __restrict__ part) {
  __shared__ double sh[kThreads / 32];
  grid_dependency_wait();
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < b.first[b.n]; c += gridDim.x) {
    const int t = tensor_of(b, c);
    acc += b.bf16[t] ? chunk_squares<true>(b.src[t], b.count[t], c - b.first[t])
                     : chunk_squares<false>(b.src[t], b.count[t], c - b.first[t]);
  }
  const double s = block_sum(acc, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm from all partials: every thread of every CTA gets the same value.
__device__ double norm_of(const double* __restrict__ part, int nparts, double* sh) {
  double a = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) a += part[i];
  return sqrt(block_sum(a, sh));
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const double* __restrict__ part, int nparts, float* __restrict__ norm_out) {
  __shared__ double sh[kThreads / 32];
  grid_dependency_wait();
  const double norm = norm_of(part, nparts, sh);
  if (threadIdx.x == 0) *norm_out = (float)norm;
}

// fp32 product rounded once to the tensor's type.
template <bool BF16>
__device__ __forceinline__ uint4 scaled(const uint4& v, float f) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = BF16 ? ptx::pack_bf16x2(ptx::bf16_lo(r[i]) * f, ptx::bf16_hi(r[i]) * f)
                : __float_as_uint(__uint_as_float(r[i]) * f);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool BF16>
__device__ __forceinline__ void scale_one(const void* s, void* d, int64_t i, float f) {
  if (BF16)
    static_cast<uint16_t*>(d)[i] =
        (uint16_t)ptx::pack_bf16x2(bf16_value(static_cast<const uint16_t*>(s)[i]) * f, 0.0f);
  else
    static_cast<float*>(d)[i] = static_cast<const float*>(s)[i] * f;
}

template <bool BF16>
__device__ void chunk_scale(const void* s, void* d, int64_t count, uint32_t c, float f) {
  constexpr int kVec = Elem<BF16>::kVec;
  const int64_t head = head_of<BF16>(s, count);
  if (c == 0 && threadIdx.x < head) scale_one<BF16>(s, d, threadIdx.x, f);
  const int64_t lo = head + (int64_t)c * Elem<BF16>::kChunk;
  const int64_t left = count - lo;
  if (left <= 0) return;
  const int64_t n = left < Elem<BF16>::kChunk ? left : Elem<BF16>::kChunk;
  if (((reinterpret_cast<uintptr_t>(s) ^ reinterpret_cast<uintptr_t>(d)) & 15u) != 0) {
    // source and destination sit differently within 16 bytes: element by element
    for (int64_t i = threadIdx.x; i < n; i += kThreads) scale_one<BF16>(s, d, lo + i, f);
    return;
  }
  const int nv = (int)(n / kVec);
  const int64_t at = lo * (BF16 ? 2 : 4);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(s) + at);
  uint4* w = reinterpret_cast<uint4*>(static_cast<uint8_t*>(d) + at);
  if (nv == kThreads * kUnroll) {
    uint4 r[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) r[i] = v[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) w[i * kThreads + threadIdx.x] = scaled<BF16>(r[i], f);
  } else {
    for (int i = threadIdx.x; i < nv; i += kThreads) w[i] = scaled<BF16>(v[i], f);
    const int tail = (int)(n - (int64_t)nv * kVec);
    if (threadIdx.x < tail) scale_one<BF16>(s, d, lo + (int64_t)nv * kVec + threadIdx.x, f);
  }
}

__global__ void __launch_bounds__(kThreads)
    grad_scale_kernel(const __grid_constant__ GradBatch b, const double* __restrict__ part, int nparts, float max_norm,
                      float* __restrict__ norm_out) {
  __shared__ double sh[kThreads / 32];
  grid_dependency_wait();
  const double norm = norm_of(part, nparts, sh);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double ratio = (double)max_norm / (norm + 1e-6);
  const float f = ratio >= 1.0 ? 1.0f : (float)ratio;  // a NaN norm gives a NaN factor
  if (f == 1.0f && b.in_place) return;
  const uint32_t total = b.first[b.n];
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const uint32_t c = total - 1 - i;
    const int t = tensor_of(b, c);
    if (f == 1.0f && b.src[t] == b.dst[t]) continue;
    if (b.bf16[t])
      chunk_scale<true>(b.src[t], b.dst[t], b.count[t], c - b.first[t], f);
    else
      chunk_scale<false>(b.src[t], b.dst[t], b.count[t], c - b.first[t], f);
  }
}

}  // namespace

int64_t grad_chunks(int64_t count, bool bf16) {
  const int64_t ch = bf16 ? Elem<true>::kChunk : Elem<false>::kChunk;
  return count > 0 ? (count + ch - 1) / ch : 0;
}

int grad_grid(uint32_t chunks, int ctas) { return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, ctas)); }

cudaError_t launch_grad_squares(const GradBatch& b, double* part, int grid, cudaStream_t stream) {
  return launch_chained(grad_square_kernel, dim3(grid), dim3(kThreads), 0, stream, b, part);
}

cudaError_t launch_grad_norm(const double* part, int nparts, float* norm_out, cudaStream_t stream) {
  return launch_chained(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, part, nparts, norm_out);
}

cudaError_t launch_grad_scale(const GradBatch& b, const double* part, int nparts, float max_norm, float* norm_out,
                              int grid, cudaStream_t stream) {
  return launch_chained(grad_scale_kernel, dim3(grid), dim3(kThreads), 0, stream, b, part, nparts, max_norm, norm_out);
}

}  // namespace moe
