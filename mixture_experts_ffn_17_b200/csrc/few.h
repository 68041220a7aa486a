// few.h -- host-side declarations of the few-token layer kernel.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

// Two tiles of eight B columns.  Up to here the layer is ahead of moe_forward, 8 of 256
// experts of 7168 x 2048 at T = 1, 4 and 16: bf16 144, 419 and 1238 us against 368, 482
// and 1310, e4m3 108, 270 and 796 us against 321, 553 and 1509.
constexpr int kFewMaxTokens = 16;
constexpr int kFewCols = 128;    // output columns of a segment

// How a call's routed expert weights are held.
enum FewWeights : int { kFewBf16 = 0, kFewE4m3 = 1, kFewMxfp4 = 2 };

// Steps of the contraction in a work unit: 16 KB of 128 columns' weights.
constexpr int few_unit_steps(int weights) { return weights == kFewBf16 ? 64 : weights == kFewE4m3 ? 128 : 256; }

// Rows that a row of x or h takes as terms: whole swizzle atoms of 8 rows.
constexpr int few_term_rows(int weights) { return weights == kFewMxfp4 ? 16 : 8; }

// How a segment's units are cut into chunks.
struct FewSplit {
  int parts, units;  // chunks of a segment, units of a chunk (the last may have fewer)
};

// The cut for `segs` segments of `steps` units at most: about 16 chunks a CTA,
// so that CTAs that are ahead take more of them, of 8 to 32 units (a chunk's end
// costs about one unit's time), and a chunk a CTA where there is less work.
// Made for 148 CTAs whatever the device, so that results do not depend on it.
// Chunks start at multiples of `whole` units.
inline FewSplit few_split(int64_t segs, int steps, int whole) {
  constexpr int64_t kCtas = 148;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (segs < 1 || steps < 1) return FewSplit{1, 1};  // nothing to cut
  const int64_t total = segs * steps, least = up(total, kCtas);
  int64_t units = up(total, 16 * kCtas);
  if (units < 8) units = least < 8 ? least : 8;
  if (units > 32) units = 32;
  if (units > steps) units = steps;
  units = up(up(steps, up(steps, units)), whole) * whole;
  return FewSplit{(int)up(steps, units), (int)units};
}

struct FewParams {
  int T, d, E, k, I, S;  // S = 0: no shared expert
  int route, n_group, topk_group, group_topn;
  float route_scale;
  int y_bf16;
  const uint8_t* x;  // bf16 [T, d]
  const uint8_t* Wg;
  const float* bias;  // may be null
  const uint8_t *s1, *s3, *s2;  // fp32 block scales or scale bytes
  void* y;
  int32_t* idx_out;    // may be null
  float* w_out;        // may be null
  int32_t* counts_out; // may be null
  uint32_t* status;
  // arrivals at the grid's barriers, claimed chunks (4 each), x's terms, choosers; zero before the launch
  uint32_t* bar;
  int32_t* chosen;     // [T, k] experts and weights, on their way between CTAs
  float* chosen_w;
  FewSplit split_up_r, split_up_s, split_dn_r, split_dn_s;
  float* logits;       // [T, E]
  float *up_r, *up_s, *dn_r, *dn_s;  // the chunks' sums, [row][segment][part][kFewCols]
  uint8_t* h_r;        // the routed rows' activations: [T * k][3][I] bf16 terms, or terms as x_terms
  uint8_t* h_s;        // [T][3][S] bf16 terms
  // coded weights: terms of x, [T][few_term_rows][d] e4m3 or [..][d / 2] MXFP4 codes
  uint8_t* x_terms;
  float *x_scale, *h_scale;                // e4m3: the power of two that undoes the scaling of 128 values
  uint8_t *x_term_scales, *h_term_scales;  // MXFP4: [row][few_term_rows][K / 32]
  // for tests: e4m3's factors' warp is held up before every stage; bytes that never come
  // of every tile, and of the first CTA's tiles of the routed down products
  bool late_factors;
  uint32_t missing, missing_down;
};

// Tensor maps of W1, W3 and W2, all with the 128-byte swizzle.  bf16: [E, K, N]
// in boxes of 64 steps by 64 columns; e4m3: [E, K, N] bytes in boxes of 128 by
// 128; MXFP4: [E * N, K / 2] bytes in boxes of 128 columns by 256 steps.  Terms:
// [rows, bytes of K] in boxes of few_term_rows by 128.
struct FewMaps {
  CUtensorMap routed[3], shared[3], x_terms, h_terms;
};

cudaError_t launch_few(const FewParams& p, const FewMaps& maps, int weights, int sms, cudaStream_t stream);

}  // namespace moe
