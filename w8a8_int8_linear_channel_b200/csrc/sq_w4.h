// sq_w4.h -- the 4-bit weight format and the launchers of its kernels and of
// the expert-routing kernels, shared between the C-ABI layer (sq_api_w4.cu)
// and the kernel files.  Not part of the public ABI.
#pragma once

#include <atomic>

#include "sq_internal.h"

namespace sq {

// A packed weight is a row-major grid of tiles of 128 output channels x 128
// k, each one contiguous record:
//   codes   8192 bytes: channel r's 64 bytes at 64 r.  Its 16-byte chunk c
//           (0..3) lies at position c ^ ((r >> 1) & 3) and holds four 32-bit
//           words; word w holds k = 32 w + 8 c + (0..7), element 2 i in bits
//           4 i .. 4 i + 3 and element 2 i + 1 sixteen bits higher.
//   scales  fp16 [128][128 / group]
//   zeros   uint8 [128][128 / group]   (only with zero points)
// Why this layout: one contiguous record is one bulk copy; a masked word is a
// pair of neighbouring k (the two halves of an fp16 pair); the four lanes of
// a quarter of an mma fragment read the four chunks of a row, and every
// group of 32 or more k is made of whole words of all four lanes; the XOR
// keeps both a warp's rows-by-chunks read and a thread-per-row read free of
// shared-memory bank conflicts.
// Channels past N and k past K hold the value zero (scale 0).
constexpr int kW4Rows = 128;
constexpr int kW4K = 128;
constexpr int kW4CodeBytes = kW4Rows * kW4K / 2;

__host__ __device__ constexpr int w4_record_bytes(int group, bool zero) {
  return kW4CodeBytes + kW4Rows * (kW4K / group) * (zero ? 3 : 2);
}

struct W4Weight {
  uint8_t* data;
  int64_t N, K;
  int group;      // 32, 64 or 128
  bool zero;      // zero points present (else 8)
  __host__ __device__ int64_t nt() const { return (N + kW4Rows - 1) / kW4Rows; }
  __host__ __device__ int64_t kt() const { return (K + kW4K - 1) / kW4K; }
  int64_t bytes() const { return nt() * kt() * w4_record_bytes(group, zero); }
};

// Per kernel and device, once: allows `smem` bytes of dynamic shared memory.  A
// launch of a few microseconds should not ask the runtime for it every time.
struct KernelSetup {
  std::atomic<bool> done[64];
};
inline cudaError_t kernel_setup(KernelSetup& k, const void* kernel, size_t smem, int device) {
  if (k.done[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) k.done[device].store(true, std::memory_order_release);
  return e;
}

cudaError_t launch_w4_pack(const uint8_t* codes, const __half* scales, const uint8_t* zeros, const W4Weight& w,
                           const Ctx& c);
cudaError_t launch_w4_quantize(const __half* src, const float* s, const W4Weight& w, const Ctx& c);
cudaError_t launch_w4_dequantize(const W4Weight& w, __half* out, const Ctx& c);

// y = x W^T with a packed W.  Dense: M tokens.  Experts (offsets != NULL): the
// pairs order[offsets[e] .. offsets[e + 1]) use weight e, pair p reads x row
// p / div and writes y row p; M is the number of pairs.
struct W4Product {
  const __half* x;
  int64_t ldx, M;
  W4Weight w;
  const __half* bias;  // [N] or [E, N] or NULL
  int relu;
  __half* y;    // fp16 [M, N] or NULL
  float* y32;   // fp32 [M, N] or NULL
  const int32_t* offsets;
  const int32_t* order;
  int E;
  int div;
};
cudaError_t launch_w4_product(const W4Product& p, const Ctx& c);
cudaError_t launch_w4_stream(const W4Product& p, const Ctx& c);                // few tokens per weight tile
cudaError_t launch_w4_gemm(const W4Product& p, const Ctx& c, int64_t tokens);  // more; tokens per tile on average
// Blocks of bt tokens: exactly, or for experts the most that any routing of
// the pairs can need (CTAs of blocks that do not exist leave at once).
int64_t w4_blocks(const W4Product& p, int bt);

// Expert routing (k_moe.cu).
struct RouteArgs {
  const void* logits;
  int half;
  int64_t T, ld;
  int E, topk, sigmoid, n_group, topk_group, group_top, renormalize;
  double scale;
  const float* bias;
  int32_t* ids;
  float* weights;
};
cudaError_t launch_moe_route(const RouteArgs& a, const Ctx& c);
size_t moe_plan_workspace_bytes(int64_t P, int E);
cudaError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* order, int32_t* ws,
                            const Ctx& c);
cudaError_t launch_moe_combine(const __half* y16, const float* y32, const int32_t* ids, const float* weights,
                               int64_t T, int topk, int64_t N, int E, __half* y, const Ctx& c);

}  // namespace sq
