// ops_api.cu -- host side of the few-token layer, the MXFP4 operators and the
// gradient norm: argument checks, workspace layouts and launch sequences.
#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "api_internal.h"
#include "few.h"
#include "grad.h"
#include "moe.h"
#include "moe_internal.h"
#include "mx.h"

namespace moe {
namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool ws_ok(const void* ws, size_t bytes, size_t need) { return ws && bytes >= need && aligned(ws, kAlign); }

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<uint8_t*>(ws) + off);
}

#define MOE_CUDA(call)                              \
  do {                                              \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

// ------------------------------------------------------------ few tokens
int few_weights(const moe_shape& s) {
  return s.w_dtype == MOE_BF16 ? kFewBf16 : s.w_dtype == MOE_E4M3 ? kFewE4m3 : kFewMxfp4;
}

struct FewLayout {
  FewSplit split_up_r, split_up_s, split_dn_r, split_dn_s;
  size_t logits, up_r, up_s, dn_r, dn_s, h_r, h_s, x_terms, x_scale, h_scale, x_term_scales, h_term_scales;
  size_t chosen, chosen_w, total;
};

FewLayout few_layout(const moe_shape& s) {
  FewLayout L{};
  const int64_t T = s.T, rows = T * s.k, experts = std::min<int64_t>(s.E, rows);
  const int unit = few_unit_steps(few_weights(s)), unit_s = few_unit_steps(kFewBf16);
  const int64_t bi = s.inter / kFewCols, bs = s.shared_inter / kFewCols, bd = s.d / kFewCols;
  const int whole = few_weights(s) == kFewMxfp4 ? 2 : 1;  // chunks' scales on 16-byte boundaries
  L.split_up_r = few_split(experts * 2 * bi, (s.d + unit - 1) / unit, whole);
  L.split_up_s = few_split(2 * bs, s.d / unit_s, 1);
  L.split_dn_r = few_split(experts * bd, (s.inter + unit - 1) / unit, whole);
  L.split_dn_s = few_split(bd, s.shared_inter / unit_s, 1);
  size_t off = kAlign;  // the status word and the counters
  auto take = [&](size_t bytes) {
    const size_t here = off;
    off += (bytes + kAlign - 1) / kAlign * kAlign;
    return here;
  };
  auto sums = [&](int64_t segs, const FewSplit& sp) { return (size_t)(segs * sp.parts) * kFewCols * 4; };
  L.logits = take((size_t)T * s.E * 4);
  L.up_r = take(sums(rows * 2 * bi, L.split_up_r));
  L.up_s = take(sums(T * 2 * bs, L.split_up_s));
  L.dn_r = take(sums(rows * bd, L.split_dn_r));
  L.dn_s = take(s.shared_inter > 0 ? sums(T * bd, L.split_dn_s) : 0);
  // bytes of a step in all of a row's terms
  const int kind = few_weights(s);
  const int64_t twice = kind == kFewBf16 ? 12 : few_term_rows(kind) * (kind == kFewE4m3 ? 2 : 1);
  const bool coded = kind != kFewBf16;
  L.h_r = take((size_t)(rows * s.inter * twice / 2));
  L.h_s = take((size_t)T * 3 * s.shared_inter * 2);
  L.x_terms = take(coded ? (size_t)(T * s.d * twice / 2) : 0);
  L.x_scale = take(kind == kFewE4m3 ? (size_t)T * bd * 4 : 0);
  L.h_scale = take(kind == kFewE4m3 ? (size_t)rows * bi * 4 : 0);
  L.x_term_scales = take(kind == kFewMxfp4 ? (size_t)T * few_term_rows(kind) * (s.d / kMxBlock) : 0);
  L.h_term_scales = take(kind == kFewMxfp4 ? (size_t)rows * few_term_rows(kind) * (s.inter / kMxBlock) : 0);
  L.chosen = take((size_t)rows * 4);
  L.chosen_w = take((size_t)rows * 4);
  L.total = off;
  return L;
}

// MOE_DEBUG_LATE_FACTORS=1 in the environment holds up the warp that brings the
// e4m3 factors (tests of the ring: the others must wait for it).
bool debug_late_factors() {
  const char* v = std::getenv("MOE_DEBUG_LATE_FACTORS");
  return v && v[0] == '1';
}

// MOE_DEBUG_WITHHOLD_LOADS=1 withholds the product's loads and a part of every tile of
// the few-token layer, 2 of one CTA's tiles in its routed down products (tests: the
// waits run out and the call reports MOE_ERR_DEVICE_TIMEOUT).
int debug_withhold() {
  const char* v = std::getenv("MOE_DEBUG_WITHHOLD_LOADS");
  return v && (v[0] == '1' || v[0] == '2') ? v[0] - '0' : 0;
}

moe_status check_few(const moe_shape* shape) {
  if (!shape) return MOE_ERR_INVALID_ARG;
  moe_shape s = *shape;
  if (s.w_dtype == MOE_MXFP4) s.w_dtype = MOE_BF16;  // the other limits are the same
  const moe_status v = check_shape(&s);
  if (v != MOE_OK) return v;
  if (s.T > kFewMaxTokens) return MOE_ERR_UNSUPPORTED;
  // chunk numbers are 32 bits, with room for one claim more from every CTA
  const FewLayout L = few_layout(*shape);
  const int64_t experts = std::min<int64_t>(s.E, s.T * s.k), limit = (int64_t)1 << 30;
  if (experts * 2 * (s.inter / kFewCols) * L.split_up_r.parts >= limit ||
      experts * (s.d / kFewCols) * L.split_dn_r.parts >= limit)
    return MOE_ERR_UNSUPPORTED;
  // and so are the rows of the tensor maps
  if ((int64_t)s.E * std::max(s.d, s.inter) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ------------------------------------------------------------ gradients
// Ranges that a clipping call writes, the norm's among them, must be disjoint from all
// others.
bool ranges_overlap(const moe_tensor* t, int n, const float* norm_out) {
  struct Range {
    uintptr_t begin, end;
    bool write;
  };
  Range r[2 * kGradMaxTensors + 1];
  int m = 0;
  const uintptr_t norm = reinterpret_cast<uintptr_t>(norm_out);
  if (norm_out) r[m++] = Range{norm, norm + sizeof(float), true};
  for (int i = 0; i < n; ++i) {
    if (t[i].count == 0) continue;
    const uintptr_t bytes = (uintptr_t)t[i].count * (t[i].dtype == MOE_BF16 ? 2 : 4);
    const uintptr_t src = reinterpret_cast<uintptr_t>(t[i].data);
    const uintptr_t dst = t[i].out ? reinterpret_cast<uintptr_t>(t[i].out) : src;
    r[m++] = Range{dst, dst + bytes, true};
    if (dst != src) r[m++] = Range{src, src + bytes, false};
  }
  std::sort(r, r + m, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t written = 0, used = 0;  // furthest ends so far
  for (int i = 0; i < m; ++i) {
    if (r[i].begin < (r[i].write ? used : written)) return true;
    used = std::max(used, r[i].end);
    if (r[i].write) written = std::max(written, r[i].end);
  }
  return false;
}

moe_status check_tensors(const moe_tensor* t, int n, bool clip, const float* norm_out) {
  if (n < 0 || (n > 0 && !t)) return MOE_ERR_INVALID_ARG;
  if (n > kGradMaxTensors) return MOE_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    if (t[i].count < 0 || (t[i].dtype != MOE_F32 && t[i].dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    if (t[i].count > (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    if (t[i].count == 0) continue;
    const uintptr_t size = t[i].dtype == MOE_BF16 ? 2 : 4;
    if (!t[i].data || !aligned(t[i].data, size)) return MOE_ERR_INVALID_ARG;
    if (clip && t[i].out && !aligned(t[i].out, size)) return MOE_ERR_INVALID_ARG;
  }
  return clip && ranges_overlap(t, n, norm_out) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int grad_batches(int n) { return std::max(1, (n + kGradBatch - 1) / kGradBatch); }

size_t grad_ws_bytes(int n) { return (size_t)grad_batches(n) * kGradMaxSms * kGradNormCtas * sizeof(double); }

bool fill_batch(GradBatch& b, const moe_tensor* t, int n, int first) {
  b.n = std::min(kGradBatch, n - first);
  b.in_place = true;
  int64_t chunks = 0;
  for (int i = 0; i < b.n; ++i) {
    const moe_tensor& x = t[first + i];
    b.src[i] = x.data;
    b.dst[i] = x.out ? x.out : x.data;
    b.in_place = b.in_place && b.dst[i] == x.data;
    b.count[i] = x.count;
    b.bf16[i] = x.dtype == MOE_BF16;
    b.first[i] = (uint32_t)chunks;
    chunks += grad_chunks(x.count, x.dtype == MOE_BF16);
    if (chunks >= (int64_t)1 << 31) return false;
  }
  b.first[b.n] = (uint32_t)chunks;
  return true;
}

// The norm's partial sums of every batch; *parts receives their number.
moe_status grad_squares(const moe_tensor* t, int n, double* part, int sms, int* parts, cudaStream_t st) {
  *parts = 0;
  for (int b = 0; b < grad_batches(n); ++b) {
    GradBatch batch;
    if (!fill_batch(batch, t, n, b * kGradBatch)) return MOE_ERR_UNSUPPORTED;
    const int grid = grad_grid(batch.first[batch.n], sms * kGradNormCtas);
    MOE_CUDA(launch_grad_squares(batch, part + *parts, grid, st));
    *parts += grid;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_size(const moe_shape* shape) {
  if (check_few(shape) != MOE_OK) return 0;
  return few_layout(*shape).total;
}

moe_status moe_forward_few(const moe_shape* shape, const void* x, const void* Wg, const float* bias, const void* W1,
                           const void* W3, const void* W2, const void* s1, const void* s3, const void* s2,
                           const void* W1s, const void* W3s, const void* W2s, void* y, int32_t* topk_idx_out,
                           float* topk_w_out, int32_t* counts_out, void* ws, size_t ws_bytes, void* stream) {
  const moe_status v = check_few(shape);
  if (v != MOE_OK) return v;
  const moe_shape& s = *shape;
  if (!x || !Wg || !W1 || !W3 || !W2 || !y) return MOE_ERR_INVALID_ARG;
  if (s.shared_inter > 0 && (!W1s || !W3s || !W2s)) return MOE_ERR_INVALID_ARG;
  if (s.w_dtype != MOE_BF16 && (!s1 || !s3 || !s2)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, Wg, bias, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, y, topk_idx_out, topk_w_out, counts_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  const FewLayout L = few_layout(s);
  if (!ws_ok(ws, ws_bytes, L.total)) return MOE_ERR_WORKSPACE;
  if (s.T == 0) return MOE_OK;
  FewParams p{};
  p.T = (int)s.T;
  p.d = s.d;
  p.E = s.E;
  p.k = s.k;
  p.I = s.inter;
  p.S = s.shared_inter;
  p.route = s.route;
  p.n_group = s.n_group;
  p.topk_group = s.topk_group;
  p.group_topn = s.group_topn;
  p.route_scale = s.route_scale;
  p.y_bf16 = s.y_dtype == MOE_BF16;
  auto bytes = [](const void* q) { return static_cast<const uint8_t*>(q); };
  p.x = bytes(x);
  p.Wg = bytes(Wg);
  p.bias = s.route == MOE_ROUTE_SIGMOID_GROUP ? bias : nullptr;
  p.s1 = bytes(s1);
  p.s3 = bytes(s3);
  p.s2 = bytes(s2);
  p.y = y;
  p.idx_out = topk_idx_out;
  p.w_out = topk_w_out;
  p.counts_out = counts_out;
  p.status = at<uint32_t>(ws, 0);
  p.bar = at<uint32_t>(ws, 64);
  p.split_up_r = L.split_up_r;
  p.split_up_s = L.split_up_s;
  p.split_dn_r = L.split_dn_r;
  p.split_dn_s = L.split_dn_s;
  p.logits = at<float>(ws, L.logits);
  p.up_r = at<float>(ws, L.up_r);
  p.up_s = at<float>(ws, L.up_s);
  p.dn_r = at<float>(ws, L.dn_r);
  p.dn_s = at<float>(ws, L.dn_s);
  p.h_r = at<uint8_t>(ws, L.h_r);
  p.h_s = at<uint8_t>(ws, L.h_s);
  p.chosen = at<int32_t>(ws, L.chosen);
  p.chosen_w = at<float>(ws, L.chosen_w);
  p.x_terms = at<uint8_t>(ws, L.x_terms);
  p.x_scale = at<float>(ws, L.x_scale);
  p.h_scale = at<float>(ws, L.h_scale);
  p.x_term_scales = at<uint8_t>(ws, L.x_term_scales);
  p.h_term_scales = at<uint8_t>(ws, L.h_term_scales);
  p.late_factors = debug_late_factors();
  p.missing = debug_withhold() == 1 ? 16 : 0;
  p.missing_down = debug_withhold() == 2 ? 16 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // before the maps: the driver makes none in a thread that has no context yet, and
  // this call gives it one
  MOE_CUDA(cudaMemsetAsync(ws, 0, kAlign, st));
  const int weights = few_weights(s);
  FewMaps maps{};
  const void* routed[] = {W1, W3, W2};
  const void* shared[] = {W1s, W3s, W2s};
  for (int i = 0; i < 3; ++i) {
    const uint64_t K = i == 2 ? s.inter : s.d, N = i == 2 ? s.d : s.inter;
    const bool made = weights == kFewBf16   ? map_bf16_tiles(&maps.routed[i], routed[i], N, K, s.E)
                      : weights == kFewE4m3 ? map_byte_tiles(&maps.routed[i], routed[i], N, K, s.E)
                                            : map_bytes(&maps.routed[i], routed[i], K / 2, N * s.E, 128);
    if (!made) return MOE_ERR_CUDA;
    if (s.shared_inter > 0 && !map_bf16_tiles(&maps.shared[i], shared[i], i == 2 ? s.d : s.shared_inter,
                                              i == 2 ? s.shared_inter : s.d, 1))
      return MOE_ERR_CUDA;
  }
  if (weights != kFewBf16) {
    const int rows = few_term_rows(weights), per_byte = weights == kFewMxfp4 ? 2 : 1;
    if (!map_bytes(&maps.x_terms, p.x_terms, s.d / per_byte, (uint64_t)s.T * rows, rows) ||
        !map_bytes(&maps.h_terms, p.h_r, s.inter / per_byte, (uint64_t)s.T * s.k * rows, rows))
      return MOE_ERR_CUDA;
  }
  MOE_CUDA(launch_few(p, maps, weights, device_sms(), st));
  return MOE_OK;
}

moe_status moe_mx_quantise(const void* src, const void* up, int src_dtype, int64_t rows, int cols, int64_t ld,
                           void* codes, void* scales, void* stream) {
  if (rows < 0 || cols <= 0 || ld < cols || (src_dtype != MOE_F32 && src_dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (cols % kMxBlock != 0) return MOE_ERR_UNSUPPORTED;
  if (rows > ((int64_t)1 << 56) / ld) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const uintptr_t size = src_dtype == MOE_BF16 ? 2 : 4;
  if (!src || !codes || !scales || !aligned(src, size) || !aligned(up, size) || !aligned(codes, 16) ||
      !aligned(scales, 16))
    return MOE_ERR_INVALID_ARG;
  MOE_CUDA(launch_mx_quantise(src, up, src_dtype == MOE_BF16, rows, cols, ld, static_cast<uint8_t*>(codes),
                              static_cast<uint8_t*>(scales), device_sms(), static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_mx_quantise_weights(const void* W, int src_dtype, int E, int K, int N, void* codes, void* scales,
                                   void* stream) {
  if (E < 0 || K <= 0 || N <= 0 || (src_dtype != MOE_F32 && src_dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (K % kMxBlock != 0 || E > 65535 || K > (1 << 23)) return MOE_ERR_UNSUPPORTED;
  if (E == 0) return MOE_OK;
  if (!W || !codes || !scales || !aligned(W, src_dtype == MOE_BF16 ? 2 : 4) || !aligned(codes, 16) ||
      !aligned(scales, 16))
    return MOE_ERR_INVALID_ARG;
  MOE_CUDA(launch_mx_quantise_weights(W, src_dtype == MOE_BF16, E, K, N, static_cast<uint8_t*>(codes),
                                      static_cast<uint8_t*>(scales), static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_mx_dequantise(const void* codes, const void* scales, int64_t rows, int cols, void* dst, int dst_dtype,
                             void* stream) {
  if (rows < 0 || cols <= 0 || (dst_dtype != MOE_F32 && dst_dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (cols % kMxBlock != 0 || rows > ((int64_t)1 << 56) / cols) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !dst || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(dst, 16))
    return MOE_ERR_INVALID_ARG;
  MOE_CUDA(launch_mx_dequantise(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, cols,
                                dst, dst_dtype == MOE_BF16, device_sms(), static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

size_t moe_mx_product_workspace_size(int64_t rows, int E) {
  if (rows < 0 || rows >= (int64_t)1 << 31 || E <= 0 || E > kMxMaxExperts) return 0;
  return kAlign;
}

moe_status moe_mx_grouped_product(int64_t rows, int E, int K, int N, const void* A, const void* A_scales,
                                  const int32_t* offsets, const void* W, const void* W_scales, void* Y, int y_dtype,
                                  void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || E <= 0 || K <= 0 || N <= 0 || (y_dtype != MOE_F32 && y_dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0 || N % 128 != 0 || E > kMxMaxExperts || rows >= (int64_t)1 << 31 ||
      (int64_t)E * N >= (int64_t)1 << 31 ||
      (rows / kMxTileTokens + E) * (N / 128) >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  const void* ptrs[] = {A, A_scales, offsets, W, W_scales, Y};
  for (const void* p : ptrs)
    if (!aligned(p, 16) || (rows > 0 && !p)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, moe_mx_product_workspace_size(rows, E))) return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOE_CUDA(cudaMemsetAsync(ws, 0, 4, st));
  if (rows == 0) return MOE_OK;
  CUtensorMap w, a16, a64;
  if (!map_bytes(&w, W, K / 2, (uint64_t)E * N, 128) || !map_bytes(&a16, A, K / 2, rows, 16) ||
      !map_bytes(&a64, A, K / 2, rows, 64))
    return MOE_ERR_CUDA;
  MxProduct p{};
  p.rows = rows;
  p.E = E;
  p.K = K;
  p.N = N;
  p.a_scales = static_cast<const uint8_t*>(A_scales);
  p.w_scales = static_cast<const uint8_t*>(W_scales);
  p.offsets = offsets;
  p.Y = Y;
  p.status = at<uint32_t>(ws, 0);
  p.withhold = debug_withhold() == 1;
  MOE_CUDA(launch_mx_product(w, a16, a64, p, y_dtype == MOE_BF16, device_sms(), st));
  return MOE_OK;
}

size_t moe_grad_workspace_size(int n) {
  if (n < 0 || n > kGradMaxTensors) return 0;
  return grad_ws_bytes(n);
}

moe_status moe_grad_norm(const moe_tensor* tensors, int n, float* norm_out, void* ws, size_t ws_bytes, void* stream) {
  const moe_status v = check_tensors(tensors, n, false, norm_out);
  if (v != MOE_OK) return v;
  if (!norm_out || !aligned(norm_out, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, grad_ws_bytes(n))) return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int parts = 0;
  double* part = at<double>(ws, 0);
  const moe_status r = grad_squares(tensors, n, part, std::min(device_sms(), kGradMaxSms), &parts, st);
  if (r != MOE_OK) return r;
  MOE_CUDA(launch_grad_norm(part, parts, norm_out, st));
  return MOE_OK;
}

moe_status moe_grad_clip(const moe_tensor* tensors, int n, float max_norm, float* norm_out, void* ws, size_t ws_bytes,
                         void* stream) {
  const moe_status v = check_tensors(tensors, n, true, norm_out);
  if (v != MOE_OK) return v;
  if (!(max_norm >= 0.0f) || !aligned(norm_out, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, grad_ws_bytes(n))) return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int parts = 0;
  double* part = at<double>(ws, 0);
  const int sms = std::min(device_sms(), kGradMaxSms);
  const moe_status r = grad_squares(tensors, n, part, sms, &parts, st);
  if (r != MOE_OK) return r;
  // the last batch first: the norm read it last
  for (int b = grad_batches(n) - 1; b >= 0; --b) {
    GradBatch batch;
    fill_batch(batch, tensors, n, b * kGradBatch);
    MOE_CUDA(launch_grad_scale(batch, part, parts, max_norm, b == 0 ? norm_out : nullptr,
                               grad_grid(batch.first[batch.n], sms * kGradScaleCtas), st));
  }
  return MOE_OK;
}

}  // extern "C"
