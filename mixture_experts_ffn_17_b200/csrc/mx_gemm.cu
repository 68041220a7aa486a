// mx_gemm.cu -- grouped product of MXFP4 rows with MXFP4 expert weights.
//
//   Y[r, n] = sum_k A[r, k] W[e, n, k]   for offsets[e] <= r < offsets[e + 1],
//
// both operands as 4-bit codes with a scale byte per 32 values of k, on
// tcgen05.mma kind::mxf4 (64 steps of k an instruction, scales applied by the
// tensor core, fp32 accumulation in TMEM).
//
// The operands change sides: 128 rows of W (output columns) are the M = 128
// side and up to 192 token rows the N side, in multiples of 16.  A decode batch
// has one or two rows an expert, and a tile then costs its weights' bytes and
// 16 columns of tensor work instead of a 128-row tile of padding; and lane i of
// the accumulator holds output column i, so a warp's store of one token's
// values is one contiguous run.
//
// Persistent CTAs, one per SM, over tiles (token tile of an expert, 128 output
// columns), the column blocks of one token tile next to each other: the tokens
// stay in L2 and the weights stream.  Roles: a producer thread (TMA, 256 steps
// of k = 128 bytes a row and stage, 128-byte swizzle), four warps that bring the
// scale bytes, an MMA thread, and four warps that drain the accumulators (two, so
// that draining overlaps the next tile).
//
// Scales.  The tensor core takes them from TMEM: row r of 128 in lane r % 32 (the
// same in all four lane quarters) of column r / 32, the four bytes of a word being
// four blocks of 32 steps.  The scale warps read their row-major arrays, four
// stages' worth of a row (32 bytes) at a time and a group ahead, exchange rows
// through shared memory and store each quarter with tcgen05.st.  (tcgen05.cp from
// shared memory spreads them too, but runs in the MMAs' own queue: 404 instead of
// 295 us for a decode batch of 512 rows, 226 experts of 7168 x 2048.)
// TMEM: 2 x 192 accumulator columns and 24 columns of scales a stage.
//
// Bound: HBM by the weights (17/32 byte a value) up to several hundred rows an
// expert.  Measured: 512 rows, 226 experts of 7168 x 2048: 297 us, 0.92 of the copy
// rate; 32768 rows, 256 experts of 2048 x 7168, loads as e^(z/2): 491 us in a run of ten
// calls at 1965 MHz (0.78), 564 us in a run of 4000 at 1477 MHz, under the power cap;
// 32768 rows, 8 experts of 7168 x 2048: 252 to 265 us, 3.6 to 3.8 PFLOP/s.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "mx.h"

namespace moe {
namespace {

constexpr int kStages = 5;
constexpr int kTok = kMxTileTokens;  // token rows of a tile
constexpr int kM = 128;              // output columns of a tile
constexpr int kK = 256;              // steps of k of a stage
constexpr uint32_t kWBytes = kM * kK / 2;
constexpr uint32_t kTBytes = kTok * kK / 2;
constexpr uint32_t kStageBytes = kWBytes + kTBytes;
static_assert(kStageBytes % 1024 == 0, "stages stay aligned for the 128-byte swizzle");
constexpr int kSfCols = 8 + 16;  // TMEM columns of a stage's scales: 2 x 4 of the weights, 2 x 8 of the tokens
constexpr int kGroup = 4;        // stages whose scales are read together
constexpr int kSfRows = kM + kTok;
constexpr int kTmemCols = 512;
static_assert(2 * kTok + kStages * kSfCols <= kTmemCols, "TMEM columns");
constexpr size_t kSmem = kStages * kStageBytes + 1024 + 2 * 2 * kGroup * kSfRows * 4;
static_assert(kSmem + sizeof(int) * (kMxMaxExperts + 40) <= 232448, "shared memory");
constexpr int kThreads = 320;  // 4 epilogue warps, 4 scale warps, producer, MMA
constexpr uint32_t kOne4 = 0x7f7f7f7fu;  // four scales of 1

struct Tile {
  int64_t row0;
  int e, nb, rows;
};

// kind::mxf4 instruction descriptor: A and B e2m1 (bits 7-9 and 10-11 = 1),
// N >> 3 at bits 17-22, ue8m0 scales (bit 23), M >> 7 at bits 27-28, and which
// pair of a TMEM word's four scale bytes to use, bits 29-30 (A) and 4-5 (B).
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t pair) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | ((pair * 2) << 29) |
         ((pair * 2) << 4);
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

// Eight columns of this warp's lane quarter.
__device__ __forceinline__ void store_scales(uint32_t tmem, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(tmem), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

struct Shared {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
  uint32_t tmem, abort, never;
  int tiles;                          // token tiles
  int first[kMxMaxExperts + 1];       // first token tile of each expert
};

// Rows of expert e, with offsets outside [0, R] or descending read as none.
__device__ __forceinline__ int64_t segment(const MxProduct& p, int e, int64_t* start) {
  const int64_t a = __ldg(p.offsets + e), b = __ldg(p.offsets + e + 1);
  *start = a;
  return a < 0 || b > p.rows || b < a ? 0 : b - a;
}

// The CTA's tiles: every gridDim.x-th, by steps instead of divisions and searches
// (each role walks them in its own single thread or warps).
struct Walk {
  int t, tt, nb, e;  // tile, token tile, column block, expert
  __device__ __forceinline__ Walk(const MxProduct& p) : t(blockIdx.x), e(0) {
    tt = t / (p.N / kM);
    nb = t - tt * (p.N / kM);
  }
  __device__ __forceinline__ void next(int dt, int dn, int blocks) {
    t += gridDim.x;
    tt += dt;
    nb += dn;
    if (nb >= blocks) {
      nb -= blocks;
      ++tt;
    }
  }
  // the expert whose token tiles hold tt (t < total: there is one)
  __device__ __forceinline__ Tile tile(const MxProduct& p, const Shared& sh) {
    while (sh.first[e + 1] <= tt) ++e;
    int64_t start;
    const int64_t rows = segment(p, e, &start);
    const int64_t skip = (int64_t)(tt - sh.first[e]) * kTok;
    return Tile{start + skip, e, nb, (int)min((int64_t)kTok, rows - skip)};
  }
};

__device__ __forceinline__ int padded(int rows) { return (rows + 15) & ~15; }

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA16,
                      const __grid_constant__ CUtensorMap tmA64, const __grid_constant__ MxProduct p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* stage0 = align_1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sh.full[s], 1 + 128);
      ptx::mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&sh.tfull[b], 1);
      ptx::mbar_init(&sh.tempty[b], 128);
    }
    ptx::mbar_init(&sh.done, 1);
    sh.abort = 0u;
    sh.never = 0u;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
  }
  if (warp == 9) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  grid_dependency_wait();  // offsets and codes come from earlier kernels
  // token tiles of each expert, then their running sum
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    int64_t start;
    sh.first[e] = (int)((segment(p, e, &start) + kTok - 1) / kTok);
    if (blockIdx.x == 0) {
      const int64_t b = __ldg(p.offsets + e + 1);
      if (start < 0 || b > p.rows || b < start) atomicOr(p.status, kStatusBounds);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int n = e0 + lane < p.E ? sh.first[e0 + lane] : 0;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (e0 + lane < p.E) sh.first[e0 + lane] = base + sum - n;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      sh.tiles = base;
      sh.first[p.E] = base;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile uint32_t* abort = &sh.abort;
  const int total = sh.tiles * (p.N / kM);
  const int nk = (p.K + kK - 1) / kK;
  const int blocks = p.N / kM, dt = (int)gridDim.x / blocks, dn = (int)gridDim.x - dt * blocks;
  Walk walk(p);

  if (warp == 8) {
    // ------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol_w = ptx::policy_evict_first(), pol_t = ptx::policy_evict_normal();
      int kg = 0;
      bool ok = true;
      for (; ok && walk.t < total; walk.next(dt, dn, blocks)) {
        const Tile ti = walk.tile(p, sh);
        const int wrow = ti.e * p.N + ti.nb * kM;
        const bool small = ti.rows <= 48;  // boxes of 16 rows, else of 64
        const int boxes = small ? (ti.rows + 15) / 16 : (ti.rows + 63) / 64;
        const uint32_t box_bytes = (small ? 16 : 64) * kK / 2;
        for (int kb = 0; kb < nk; ++kb, ++kg) {
          const int s = kg % kStages;
          if (!ptx::wait_bounded(&sh.empty[s], ((kg / kStages) & 1) ^ 1, abort)) {
            raise_status(p.status, abort, kStatusTimeout);
            ok = false;
            break;
          }
          uint8_t* st = stage0 + s * kStageBytes;
          ptx::mbar_arrive_expect_tx(&sh.full[s], kWBytes + boxes * box_bytes);
          if (p.withhold) continue;
          ptx::tma_load_2d(st, &tmW, &sh.full[s], kb * (kK / 2), wrow, pol_w);
          for (int b = 0; b < boxes; ++b)
            ptx::tma_load_2d(st + kWBytes + b * box_bytes, small ? &tmA16 : &tmA64, &sh.full[s], kb * (kK / 2),
                             (int)ti.row0 + b * (small ? 16 : 64), pol_t);
        }
      }
      // every issued copy must land before the CTA may exit; all were issued before the
      // first wait, so that its limit is the limit of all of them
      for (int j = (kg > kStages ? kg - kStages : 0); j < kg; ++j) {
        if (!ptx::wait_bounded(&sh.full[j % kStages], (j / kStages) & 1, &sh.never)) {
          raise_status(p.status, abort, kStatusTimeout);
          break;
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------ MMA
    if (lane == 0) {
      int kg = 0, use = 0;
      bool ok = true;
      const uint32_t base = ptx::smem_u32(stage0);
      const uint64_t w_desc = ptx::sdesc_sw128(base, 16, 1024), x_desc = ptx::sdesc_sw128(base + kWBytes, 16, 1024);
      for (; ok && walk.t < total; walk.next(dt, dn, blocks)) {
        const Tile ti = walk.tile(p, sh);
        const int b = use & 1;
        if (!ptx::wait_bounded(&sh.tempty[b], ((use >> 1) & 1) ^ 1, abort)) {
          raise_status(p.status, abort, kStatusTimeout);
          break;
        }
        ptx::tc_fence_after();
        const int N = padded(ti.rows);
        const uint32_t d = tmem + b * kTok;
        const uint32_t id0 = idesc_mxf4(N, 0), id1 = idesc_mxf4(N, 1);
        for (int kb = 0; kb < nk; ++kb, ++kg) {
          const int s = kg % kStages;
          if (!ptx::wait_bounded(&sh.full[s], (kg / kStages) & 1, abort)) {
            raise_status(p.status, abort, kStatusTimeout);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          // descriptors differ from the first stage's in their address field alone
          const uint32_t off = s * (kStageBytes >> 4);
          const uint64_t w = w_desc + off, x = x_desc + off;
          const uint32_t sf = tmem + 2 * kTok + s * kSfCols;
          const bool whole = p.K - kb * kK > kK / 2;  // else one 128-step half holds data
          mma_mxf4(d, w, x, id0, sf, sf + 8, kb != 0 ? 1u : 0u);
          mma_mxf4(d, w + 2, x + 2, id1, sf, sf + 8, 1u);
          if (whole) {
            mma_mxf4(d, w + 4, x + 4, id0, sf + 4, sf + 16, 1u);
            mma_mxf4(d, w + 6, x + 6, id1, sf + 4, sf + 16, 1u);
          }
          ptx::mma_commit(&sh.empty[s]);
        }
        if (!ok) break;
        ptx::mma_commit(&sh.tfull[b]);
        ++use;
      }
      ptx::mma_commit(&sh.done);
      if (!ptx::wait_bounded(&sh.done, 0, &sh.never)) raise_status(p.status, abort, kStatusTimeout);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ scales
    // Thread r reads row r of the weights and rows r and r + 128 of the tokens.
    const int r = threadIdx.x - 128;
    const int words = p.K / 128;  // of four scales in a row
    const bool wide = words % 4 == 0;
    uint32_t* exchange = reinterpret_cast<uint32_t*>(stage0 + kStages * kStageBytes);  // [2][8 words][rows]
    uint32_t q[3][2 * kGroup];
    auto row_words = [&](uint32_t (&v)[2 * kGroup], const uint8_t* base, int64_t row, int k0, bool have) {
      const uint32_t* a = reinterpret_cast<const uint32_t*>(base) + row * words + k0;
#pragma unroll
      for (int i = 0; i < 2 * kGroup; i += 4) {
        if (wide) {
          const uint4 x = have && k0 + i < words ? __ldg(reinterpret_cast<const uint4*>(a + i))
                                                 : make_uint4(kOne4, kOne4, kOne4, kOne4);
          v[i] = x.x;
          v[i + 1] = x.y;
          v[i + 2] = x.z;
          v[i + 3] = x.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i + j] = have && k0 + i + j < words ? __ldg(a + i + j) : kOne4;
        }
      }
    };
    auto fetch = [&](const Tile& ti, int kb0) {
      row_words(q[0], p.w_scales, (int64_t)ti.e * p.N + ti.nb * kM + r, 2 * kb0, true);
      row_words(q[1], p.a_scales, ti.row0 + r, 2 * kb0, r < ti.rows);
      row_words(q[2], p.a_scales, ti.row0 + r + 128, 2 * kb0, r + 128 < ti.rows);
    };
    int kg = 0, buf = 0;
    bool ok = true;
    Tile ti{}, next{};
    if (walk.t < total) {
      next = walk.tile(p, sh);
      fetch(next, 0);
    }
    // a warp whose wait failed goes on without waiting: the others need it at the
    // barrier
    while (walk.t < total) {
      ti = next;
      for (int kb0 = 0; kb0 < nk; kb0 += kGroup) {
        uint32_t* ex = exchange + buf * (2 * kGroup * kSfRows);
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) {
          ex[i * kSfRows + r] = q[0][i];
          ex[i * kSfRows + kM + r] = q[1][i];
          if (r + 128 < kTok) ex[i * kSfRows + kM + 128 + r] = q[2][i];
        }
        // the next group, of this tile or the next one
        if (kb0 + kGroup < nk) {
          fetch(ti, kb0 + kGroup);
        } else {
          walk.next(dt, dn, blocks);
          if (walk.t < total) {
            next = walk.tile(p, sh);
            fetch(next, 0);
          }
        }
        ptx::named_barrier(1, 128);
        for (int i = 0; i < kGroup && kb0 + i < nk; ++i, ++kg) {
          const int s = kg % kStages;
          uint32_t w[8], a[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t* line = ex + (2 * i + h) * kSfRows + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * h + j] = line[32 * j];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[h][j] = 32 * j < kTok ? line[kM + 32 * j] : kOne4;
          }
          if (ok && !warp_wait(&sh.empty[s], ((kg / kStages) & 1) ^ 1, abort)) {
            raise_status(p.status, abort, kStatusTimeout);
            ok = false;
          }
          if (!ok) continue;
          ptx::tc_fence_after();
          const uint32_t sf = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 2 * kTok + s * kSfCols;
          store_scales(sf, w);
          store_scales(sf + 8, a[0]);
          store_scales(sf + 16, a[1]);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          ptx::tc_fence_before();
          ptx::mbar_arrive(&sh.full[s]);
        }
        buf ^= 1;
      }
    }
  } else {
    // ------------------------------------------------ epilogue
    int use = 0;
    for (; walk.t < total; walk.next(dt, dn, blocks)) {
      const Tile ti = walk.tile(p, sh);
      const int b = use & 1;
      if (!warp_wait(&sh.tfull[b], (use >> 1) & 1, abort)) {
        raise_status(p.status, abort, kStatusTimeout);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(warp * 32) << 16) + b * kTok;
      const int64_t col = ti.nb * kM + warp * 32 + lane;
      for (int c0 = 0; c0 < ti.rows; c0 += 32) {
        uint32_t v[32];
        ptx::tmem_ld32(acc + c0, v);
        ptx::tmem_ld_wait(v);
        if (c0 + 32 >= ti.rows) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&sh.tempty[b]);
        }
        const int n = ti.rows - c0;
        const int64_t to = (ti.row0 + c0) * (int64_t)p.N + col;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j < n) {
            if (BF16)
              static_cast<uint16_t*>(p.Y)[to + j * (int64_t)p.N] =
                  (uint16_t)ptx::pack_bf16x2(__uint_as_float(v[j]), 0.0f);
            else
              static_cast<float*>(p.Y)[to + j * (int64_t)p.N] = __uint_as_float(v[j]);
          }
        }
      }
      ++use;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_mx_product(const CUtensorMap& tmW, const CUtensorMap& tmA16, const CUtensorMap& tmA64,
                              const MxProduct& p, bool y_bf16, int sms, cudaStream_t stream) {
  auto kernel = y_bf16 ? mx_product_kernel<true> : mx_product_kernel<false>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (err != cudaSuccess) return err;
  return launch_chained(kernel, dim3(sms), dim3(kThreads), kSmem, stream, tmW, tmA16, tmA64, p);
}

}  // namespace moe
