// k_w4_weight.cu -- making and reading packed 4-bit weights: quantization of
// an fp16 weight in groups, packing of codes a caller already has, and the
// fp16 values of a packed weight.  A warp handles one channel's 128 k of one
// tile; lane l owns k = 4 l .. 4 l + 3.
#include "sq_ptx.cuh"
#include "sq_w4.h"

namespace sq {
namespace {

constexpr int kWarps = 8;

// Two neighbouring lanes hold the eight codes of one packed word (4 each, in
// the low nibbles c[0..3]); the even lane returns the word.
__device__ __forceinline__ uint32_t pack_word(const uint32_t (&c)[4], int lane) {
  // element 2 i -> bits 4 i, element 2 i + 1 -> bits 16 + 4 i; lane parity = upper four elements
  const int i = (lane & 1) * 2;
  uint32_t v = (c[0] << (4 * i)) | (c[1] << (16 + 4 * i)) | (c[2] << (4 * i + 4)) | (c[3] << (20 + 4 * i));
  return v | __shfl_xor_sync(0xffffffffu, v, 1);
}

// Byte offset in a record of the word that lane l's k (4 l ..) fall into.
__device__ __forceinline__ int word_offset(int r, int lane) {
  const int k = 4 * lane;
  const int w = k >> 5, c = (k >> 3) & 3;
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + 4 * w;
}

// v rounded to n significant bits, ties to even (v >= 0).  Adding and
// subtracting 2^(24 - n) * ulp-scaled magnitudes is done on the bits: the
// rounding increment carries into the exponent as it should.
__device__ __forceinline__ float round_bits(float v, int n) {
  uint32_t b = __float_as_uint(v);
  if (b >= 0x7f800000u || v == 0.0f) return v;
  const int drop = 24 - n;
  const uint32_t half = (1u << (drop - 1)) - 1u + ((b >> drop) & 1u);
  return __uint_as_float((b + half) & ~((1u << drop) - 1u));
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Code of v at scale s and zero point z (an integer value), clamped to
// [lo, hi]; IEEE division, ties to even.  A NaN and every value of a group
// whose scale is 0 or Inf get the zero point.
__device__ __forceinline__ uint32_t code_of(float v, float s, float z, float lo, float hi) {
  if (!(s > 0.0f) || isinf(s) || isnan(v)) return static_cast<uint32_t>(z);
  const float q = __fadd_rn(rintf(__fdiv_rn(v, s)), z);
  return static_cast<uint32_t>(fminf(fmaxf(q, lo), hi));
}

// HBM-bound: reads 2 bytes and writes half a byte per weight.
template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_quantize(const __half* __restrict__ src, const float* __restrict__ fold, uint8_t* __restrict__ out,
                  int64_t N, int64_t K, int64_t KT, int64_t tasks) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); task < tasks;
       task += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t n = task / KT, kt = task - n * KT;
    const int r = static_cast<int>(n & (kW4Rows - 1));
    uint8_t* rec = out + ((n >> 7) * KT + kt) * REC;
    const int64_t k = kt * kW4K + 4 * lane;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n < N && k < K) {
      const uint2 raw = *reinterpret_cast<const uint2*>(src + n * K + k);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
      if (fold) {
        const float4 f = *reinterpret_cast<const float4*>(fold + k);
        // the folded weight is an fp16 tensor, as in the INT8 quantizer
        v[0] = __half2float(__float2half_rn(__fmul_rn(v[0], f.x)));
        v[1] = __half2float(__float2half_rn(__fmul_rn(v[1], f.y)));
        v[2] = __half2float(__float2half_rn(__fmul_rn(v[2], f.z)));
        v[3] = __half2float(__float2half_rn(__fmul_rn(v[3], f.w)));
      }
    }
    float s, z;
    uint32_t c[4];
    if (ZERO) {
      // fmaxf drops a NaN, so it never sets a range
      float hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), 0.0f);
      float lo = fmaxf(fmaxf(fmaxf(-v[0], -v[1]), fmaxf(-v[2], -v[3])), 0.0f);
      hi = group_max<G / 4>(hi);
      lo = group_max<G / 4>(lo);
      // 7 significant bits: |q - z| <= 15 takes 4, so (q - z) * s fits fp16's 11
      s = __half2float(__float2half_rn(round_bits(__fdiv_rn(__fadd_rn(hi, lo), 15.0f), 7)));
      z = (s > 0.0f && !isinf(s)) ? fminf(rintf(__fdiv_rn(lo, s)), 15.0f) : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = code_of(v[i], s, z, 0.0f, 15.0f);
    } else {
      float m = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), 0.0f);
      m = group_max<G / 4>(m);
      // 8 significant bits: |q| <= 7 takes 3, so q * s fits fp16's 11
      s = __half2float(__float2half_rn(round_bits(__fdiv_rn(m, 7.0f), 8)));
      z = 8.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = code_of(v[i], s, z, 1.0f, 15.0f);
    }
    const uint32_t word = pack_word(c, lane);
    if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(rec + word_offset(r, lane)) = word;
    if ((lane & (G / 4 - 1)) == 0) {
      const int g = lane / (G / 4);
      *reinterpret_cast<__half*>(rec + kW4CodeBytes + (r * NG + g) * 2) = __float2half_rn(s);
      if (ZERO) rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + g] = static_cast<uint8_t>(z);
    }
  }
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_pack(const uint8_t* __restrict__ codes, const __half* __restrict__ scales,
              const uint8_t* __restrict__ zeros, uint8_t* __restrict__ out, int64_t N, int64_t K, int64_t KT,
              int64_t tasks) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int lane = threadIdx.x & 31;
  const int64_t groups = (K + G - 1) / G;
  griddep_wait();
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); task < tasks;
       task += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t n = task / KT, kt = task - n * KT;
    const int r = static_cast<int>(n & (kW4Rows - 1));
    uint8_t* rec = out + ((n >> 7) * KT + kt) * REC;
    const int64_t k = kt * kW4K + 4 * lane;
    const int64_t g = k / G;
    uint32_t z = ZERO ? 0u : 8u;
    __half s = __float2half_rn(0.0f);
    if (n < N && g < groups) {
      s = scales[n * groups + g];
      if (ZERO) z = zeros[n * groups + g] & 15u;
    }
    uint32_t c[4] = {z, z, z, z};
    if (n < N && k < K) {
      const uint32_t raw = *reinterpret_cast<const uint32_t*>(codes + n * K + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = (raw >> (8 * i)) & 15u;
    }
    const uint32_t word = pack_word(c, lane);
    if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(rec + word_offset(r, lane)) = word;
    if ((lane & (G / 4 - 1)) == 0) {
      const int gi = lane / (G / 4);
      *reinterpret_cast<__half*>(rec + kW4CodeBytes + (r * NG + gi) * 2) = s;
      if (ZERO) rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + gi] = static_cast<uint8_t>(z);
    }
  }
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_dequantize(const uint8_t* __restrict__ in, __half* __restrict__ out, int64_t N, int64_t K, int64_t KT,
                    int64_t tasks) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); task < tasks;
       task += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t n = task / KT, kt = task - n * KT;
    const int r = static_cast<int>(n & (kW4Rows - 1));
    const uint8_t* rec = in + ((n >> 7) * KT + kt) * REC;
    const int64_t k = kt * kW4K + 4 * lane;
    if (k >= K) continue;
    const int g = lane / (G / 4);
    const float s = __half2float(*reinterpret_cast<const __half*>(rec + kW4CodeBytes + (r * NG + g) * 2));
    const float z = ZERO ? static_cast<float>(rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + g]) : 8.0f;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(rec + word_offset(r, lane)) >> ((lane & 1) * 8);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t q = (word >> ((i >> 1) * 4 + (i & 1) * 16)) & 15u;
      v[i] = __fmul_rn(__fsub_rn(static_cast<float>(q), z), s);
    }
    __half2 h[2] = {__floats2half2_rn(v[0], v[1]), __floats2half2_rn(v[2], v[3])};
    *reinterpret_cast<uint2*>(out + n * K + k) = *reinterpret_cast<uint2*>(h);
  }
}

// One warp per (channel, tile) task, up to 8 resident blocks per SM; longer
// task lists loop.
unsigned grid_for(int64_t tasks, const Ctx& c) {
  const int64_t blocks = (tasks + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(c.num_sms) * 64;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

}  // namespace

#define SQ_W4_DISPATCH(w, CALL)                        \
  do {                                                 \
    if ((w).zero) {                                    \
      if ((w).group == 32) return CALL(32, true);      \
      if ((w).group == 64) return CALL(64, true);      \
      return CALL(128, true);                          \
    }                                                  \
    if ((w).group == 32) return CALL(32, false);       \
    if ((w).group == 64) return CALL(64, false);       \
    return CALL(128, false);                           \
  } while (0)

cudaError_t launch_w4_pack(const uint8_t* codes, const __half* scales, const uint8_t* zeros, const W4Weight& w,
                           const Ctx& c) {
  const int64_t tasks = w.nt() * kW4Rows * w.kt();
#define SQ_CALL(G, Z)                                                                                        \
  launch_pdl(k_w4_pack<G, Z>, dim3(grid_for(tasks, c)), dim3(kWarps * 32), 0, c.stream, codes, scales, zeros, \
             w.data, w.N, w.K, w.kt(), tasks)
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_quantize(const __half* src, const float* s, const W4Weight& w, const Ctx& c) {
  const int64_t tasks = w.nt() * kW4Rows * w.kt();
#define SQ_CALL(G, Z)                                                                                           \
  launch_pdl(k_w4_quantize<G, Z>, dim3(grid_for(tasks, c)), dim3(kWarps * 32), 0, c.stream, src, s, w.data, w.N, \
             w.K, w.kt(), tasks)
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_dequantize(const W4Weight& w, __half* out, const Ctx& c) {
  const int64_t tasks = w.N * w.kt();
#define SQ_CALL(G, Z)                                                                                             \
  launch_pdl(k_w4_dequantize<G, Z>, dim3(grid_for(tasks, c)), dim3(kWarps * 32), 0, c.stream,                     \
             static_cast<const uint8_t*>(w.data), out, w.N, w.K, w.kt(), tasks)
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

}  // namespace sq
