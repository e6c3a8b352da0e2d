// sq_w4.cuh -- device code shared by the 4-bit weight kernels.
#pragma once

#include "sq_ptx.cuh"
#include "sq_w4.h"

namespace sq {

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16
// bytes), completion counted on `bar` in bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// mbar_wait whose tries suspend the warp (up to 2 us each) instead of polling:
// with up to seven warps on a scheduler (two CTAs of fourteen on an SM) the
// waiting ones must not take issue slots.
__device__ __forceinline__ bool w4_wait(uint32_t bar, uint32_t parity, uint64_t budget_ns, uint32_t* status,
                                        volatile uint32_t* abort) {
  if (mbar_try_wait_hint(bar, parity, 2000)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_hint(bar, parity, 2000)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > budget_ns) {
      atomicCAS(status, DEV_OK, DEV_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// The same by a whole warp, which is converged on return with one answer: the
// .sync.aligned instructions (tcgen05, mma, barrier.cluster) that follow a wait
// must not meet a warp whose lanes left the wait at different times.
__device__ __forceinline__ bool w4_wait_warp(uint32_t bar, uint32_t parity, uint64_t budget_ns, uint32_t* status,
                                             volatile uint32_t* abort) {
  return __all_sync(0xffffffffu, w4_wait(bar, parity, budget_ns, status, abort));
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t mask_or(uint32_t v, uint32_t mask) {
  uint32_t r;  // (v & mask) | 0x64006400
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(r) : "r"(v), "r"(mask));
  return r;
}

// The eight codes of a word minus their zero point as four fp16 pairs.  The
// bits 0x6400 | q are the number 1024 + q, 0x6400 | 16 q is 1024 + 16 q: one
// subtraction (bias_lo = 1024 + z) or one fused multiply-add by 1/16
// (bias_hi = -(64 + z)) gives q - z, both exact.
__device__ __forceinline__ void dequant(uint32_t word, uint32_t bias_lo, uint32_t bias_hi, uint32_t (&h)[4]) {
  const uint32_t up = word >> 8;
  constexpr uint32_t kSixteenth = 0x2C002C00u;  // 1/16, twice
  h[0] = hsub2(mask_or(word, 0x000F000Fu), bias_lo);
  h[1] = hfma2(mask_or(word, 0x00F000F0u), kSixteenth, bias_hi);
  h[2] = hsub2(mask_or(up, 0x000F000Fu), bias_lo);
  h[3] = hfma2(mask_or(up, 0x00F000F0u), kSixteenth, bias_hi);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t cluster_id_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Block number `block` of the token blocks of all experts in order (ceil(n_e /
// bt) blocks of expert e): its expert (-1: there is no such block), first plan
// entry and token count.  Warp-collective; every lane gets the answer.
__device__ __forceinline__ int w4_find_block(const W4Product& p, int block, int bt, int lane, int* start, int* count) {
  constexpr int kAhead = 4;  // loads in flight (256 experts, one token, a layer: 21.5 us, one at a time 24.0)
  int before = 0;
  int lows[kAhead], highs[kAhead];
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int q = e0 / 32 % kAhead;
    if (q == 0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + 32 * i + lane;
        lows[i] = e < p.E ? p.offsets[e] : 0;
        highs[i] = e < p.E ? p.offsets[e + 1] : 0;
      }
    }
    int lo = lows[0], hi = highs[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) lows[i] = lows[i + 1], highs[i] = highs[i + 1];
    // offsets that no plan wrote must not lead out of the order array
    lo = max(lo, 0);
    hi = static_cast<int>(min(static_cast<int64_t>(hi), p.M));
    const int mine = hi > lo ? (hi - lo - 1) / bt + 1 : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const int rel = block - before;
    const unsigned hit = __ballot_sync(0xffffffffu, rel >= inc - mine && rel < inc);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int first = __shfl_sync(0xffffffffu, lo, src) + (rel - __shfl_sync(0xffffffffu, inc - mine, src)) * bt;
      const int left = __shfl_sync(0xffffffffu, hi, src) - first;
      *start = first;
      *count = left < bt ? left : bt;
      return e0 + src;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return -1;
}

}  // namespace sq
