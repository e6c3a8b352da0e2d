// sq_api_w4.cu -- the C ABI of the 4-bit weight and expert-routing entry
// points: host-side argument checks and dispatch, as in sq_api.cu.
#include <math.h>

#include "../../include/sq.h"
#include "sq_w4.h"

using namespace sq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }  // NULL is aligned

sq_status launched(cudaError_t e) {
  if (e == cudaSuccess) return SQ_OK;
  cudaGetLastError();
  // more blocks than a grid holds
  return e == cudaErrorInvalidConfiguration ? SQ_ERR_UNSUPPORTED_SHAPE : SQ_ERR_CUDA;
}

sq_status context(sq_stream_t stream, Ctx* c) { return static_cast<sq_status>(call_context(stream, c)); }

sq_status check_weight(const void* w4, int64_t N, int64_t K, int group, int has_zero, W4Weight* w) {
  if (!w4 || N <= 0 || K <= 0) return SQ_ERR_INVALID_ARG;
  if (K > SQ_MAX_K) return SQ_ERR_K_OVERFLOW;
  if (K % 16 != 0 || N > SQ_W4_MAX_N) return SQ_ERR_UNSUPPORTED_SHAPE;
  if (group != 32 && group != 64 && group != 128) return SQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(w4)) return SQ_ERR_MISALIGNED;
  w->data = static_cast<uint8_t*>(const_cast<void*>(w4));
  w->N = N;
  w->K = K;
  w->group = group;
  w->zero = has_zero != 0;
  return SQ_OK;
}

sq_status check_experts(int64_t E) {
  if (E <= 0) return SQ_ERR_INVALID_ARG;
  return E > SQ_MOE_MAX_EXPERTS ? SQ_ERR_UNSUPPORTED_SHAPE : SQ_OK;
}

}  // namespace

extern "C" {

size_t sq_w4_packed_bytes(int64_t N, int64_t K, int group, int has_zero) {
  W4Weight w;
  static const uint64_t any[2] __attribute__((aligned(16))) = {0, 0};
  if (check_weight(any, N, K, group, has_zero, &w) != SQ_OK) return 0;
  return static_cast<size_t>(w.bytes());
}

sq_status sq_quantize_weight_w4(const void* w_f16, int64_t N, int64_t K, const float* s, int group, int has_zero,
                                void* w4, sq_stream_t stream) {
  W4Weight w;
  if (!w_f16) return SQ_ERR_INVALID_ARG;
  sq_status st = check_weight(w4, N, K, group, has_zero, &w);
  if (st != SQ_OK) return st;
  if (!aligned16(w_f16) || !aligned16(s)) return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  return launched(launch_w4_quantize(static_cast<const __half*>(w_f16), s, w, c));
}

sq_status sq_w4_pack(const uint8_t* codes, const void* scales_f16, const uint8_t* zeros, int64_t N, int64_t K,
                     int group, void* w4, sq_stream_t stream) {
  W4Weight w;
  if (!codes || !scales_f16) return SQ_ERR_INVALID_ARG;
  sq_status st = check_weight(w4, N, K, group, zeros != nullptr, &w);
  if (st != SQ_OK) return st;
  if (!aligned16(codes) || !aligned16(scales_f16) || !aligned16(zeros)) return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  return launched(launch_w4_pack(codes, static_cast<const __half*>(scales_f16), zeros, w, c));
}

sq_status sq_w4_dequantize(const void* w4, int64_t N, int64_t K, int group, int has_zero, void* w_out_f16,
                           sq_stream_t stream) {
  W4Weight w;
  if (!w_out_f16) return SQ_ERR_INVALID_ARG;
  sq_status st = check_weight(w4, N, K, group, has_zero, &w);
  if (st != SQ_OK) return st;
  if (!aligned16(w_out_f16)) return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  return launched(launch_w4_dequantize(w, static_cast<__half*>(w_out_f16), c));
}

sq_status sq_w4a16_linear(const void* x_f16, int64_t M, int64_t ldx, const void* w4, int64_t N, int64_t K, int group,
                          int has_zero, const void* bias_f16, int relu, void* y_f16, sq_stream_t stream) {
  W4Product p{};
  if (!x_f16 || !y_f16 || M <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_weight(w4, N, K, group, has_zero, &p.w);
  if (st != SQ_OK) return st;
  if (ldx < K) return SQ_ERR_INVALID_ARG;
  if (ldx % 8 != 0 || !aligned16(x_f16) || !aligned16(bias_f16) || !aligned16(y_f16)) return SQ_ERR_MISALIGNED;
  if (M > 0x7fffffffLL) return SQ_ERR_UNSUPPORTED_SHAPE;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  p.x = static_cast<const __half*>(x_f16);
  p.ldx = ldx;
  p.M = M;
  p.bias = static_cast<const __half*>(bias_f16);
  p.relu = relu != 0;
  p.y = static_cast<__half*>(y_f16);
  p.E = 1;
  p.div = 1;
  return launched(launch_w4_product(p, c));
}

sq_status sq_w4a16_experts(const void* x_f16, int64_t rows, int64_t ldx, const void* w4, int64_t E, int64_t N,
                           int64_t K, int group, int has_zero, const void* bias_f16, int relu,
                           const int32_t* offsets, const int32_t* order, int64_t pairs, int64_t pairs_per_row,
                           void* y, int y_f32, sq_stream_t stream) {
  W4Product p{};
  if (!x_f16 || !y || !offsets || !order || rows <= 0 || pairs <= 0 || pairs_per_row <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_experts(E);
  if (st != SQ_OK) return st;
  if ((st = check_weight(w4, N, K, group, has_zero, &p.w)) != SQ_OK) return st;
  if (ldx < K) return SQ_ERR_INVALID_ARG;
  if (rows > 0x7fffffffLL || pairs > 0x7fffffffLL || pairs_per_row > 0x7fffffffLL) return SQ_ERR_UNSUPPORTED_SHAPE;
  if ((pairs - 1) / pairs_per_row >= rows) return SQ_ERR_INVALID_ARG;  // the last pair's row does not exist
  if (ldx % 8 != 0 || !aligned16(x_f16) || !aligned16(bias_f16) || !aligned16(y) || !aligned16(offsets) ||
      !aligned16(order))
    return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  p.x = static_cast<const __half*>(x_f16);
  p.ldx = ldx;
  p.M = pairs;
  p.bias = static_cast<const __half*>(bias_f16);
  p.relu = relu != 0;
  if (y_f32)
    p.y32 = static_cast<float*>(y);
  else
    p.y = static_cast<__half*>(y);
  p.offsets = offsets;
  p.order = order;
  p.E = static_cast<int>(E);
  p.div = static_cast<int>(pairs_per_row);
  return launched(launch_w4_product(p, c));
}

sq_status sq_moe_route(const void* logits, int logits_f16, int64_t T, int64_t E, int64_t ld, const float* bias,
                       int sigmoid, int n_group, int topk_group, int group_top, int topk, int renormalize, float scale,
                       int32_t* ids, float* weights, sq_stream_t stream) {
  if (!logits || !ids || !weights || T <= 0 || topk <= 0 || n_group <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_experts(E);
  if (st != SQ_OK) return st;
  if (ld < E || E % n_group != 0 || topk_group <= 0 || topk_group > n_group || group_top < 1 || group_top > 2)
    return SQ_ERR_INVALID_ARG;
  if (topk > topk_group * (E / n_group) || group_top > E / n_group || !isfinite(scale)) return SQ_ERR_INVALID_ARG;
  if (topk > SQ_MOE_MAX_TOPK || n_group > 32 || T > 0x7fffffffLL / topk) return SQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights)) return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  RouteArgs a{};
  a.logits = logits;
  a.half = logits_f16 != 0;
  a.T = T;
  a.ld = ld;
  a.E = static_cast<int>(E);
  a.topk = topk;
  a.sigmoid = sigmoid != 0;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.group_top = group_top;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  return launched(launch_moe_route(a, c));
}

size_t sq_moe_plan_workspace_bytes(int64_t pairs, int64_t E) {
  if (pairs <= 0 || pairs > 0x7fffffffLL || check_experts(E) != SQ_OK) return 0;
  return moe_plan_workspace_bytes(pairs, static_cast<int>(E));
}

sq_status sq_moe_plan(const int32_t* ids, int64_t pairs, int64_t E, int32_t* offsets, int32_t* order, void* workspace,
                      size_t ws_bytes, sq_stream_t stream) {
  if (!ids || !offsets || !order || pairs <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_experts(E);
  if (st != SQ_OK) return st;
  if (pairs > 0x7fffffffLL) return SQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(ids) || !aligned16(offsets) || !aligned16(order)) return SQ_ERR_MISALIGNED;
  const size_t need = moe_plan_workspace_bytes(pairs, static_cast<int>(E));
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace))) return SQ_ERR_WORKSPACE;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  return launched(launch_moe_plan(ids, pairs, static_cast<int>(E), offsets, order, static_cast<int32_t*>(workspace), c));
}

sq_status sq_moe_combine(const void* y_pairs, int pairs_f32, const int32_t* ids, const float* weights, int64_t T,
                         int64_t topk, int64_t N, int64_t E, void* y_f16, sq_stream_t stream) {
  if (!y_pairs || !ids || !weights || !y_f16 || T <= 0 || topk <= 0 || N <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_experts(E);
  if (st != SQ_OK) return st;
  if (topk > SQ_MOE_MAX_TOPK || N > 0x7fffffffLL || T > 0x7fffffffLL / topk || T > (0x7fffffffLL * 128) / N)
    return SQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(y_pairs) || !aligned16(ids) || !aligned16(weights) || !aligned16(y_f16)) return SQ_ERR_MISALIGNED;
  Ctx c;
  if ((st = context(stream, &c)) != SQ_OK) return st;
  return launched(launch_moe_combine(pairs_f32 ? nullptr : static_cast<const __half*>(y_pairs),
                                     pairs_f32 ? static_cast<const float*>(y_pairs) : nullptr, ids, weights, T,
                                     static_cast<int>(topk), N, static_cast<int>(E), static_cast<__half*>(y_f16), c));
}

}  // extern "C"
