// k_w4_weight.cu -- making and reading packed 4-bit weights: quantization of
// an fp16 weight in groups, packing of codes a caller already has, and the
// fp16 values of a packed weight.  All three are bound by HBM when they are
// written so that nothing but the eight values of a packed word is computed
// per thread: a warp takes two channels, 16 lanes each, lane l the k = 8 l ..
// 8 l + 7 of a tile (one 16-byte load or store, one packed word), and walks
// along K with the next tile's load in flight.
#include "sq_w4.cuh"

namespace sq {
namespace {

constexpr int kWarps = 8;

constexpr int kRowsPerBlock = 2 * kWarps;

// Byte offset in a record of the word with k = 8 l .. 8 l + 7 of channel r.
__device__ __forceinline__ int word_offset(int r, int l) { return r * 64 + (((l & 3) ^ ((r >> 1) & 3)) << 4) + 4 * (l >> 2); }

// Element 2 i in bits 4 i .., element 2 i + 1 sixteen bits higher; c[] < 16.
__device__ __forceinline__ uint32_t pack_word(const uint32_t (&c)[8]) {
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= c[2 * i] << (4 * i) | c[2 * i + 1] << (16 + 4 * i);
  return v;
}

// The tiles [t0, t1) of K that this block's row of the grid takes.
struct Span {
  int t0, t1;
};
__device__ __forceinline__ Span k_span(int KT) {
  const int64_t y = blockIdx.y, n = gridDim.y;
  return {static_cast<int>(KT * y / n), static_cast<int>(KT * (y + 1) / n)};
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

// Codes clamp(rint(v / s) + z, lo, hi) (lo, hi and z are integers, so clamping
// first is the same), division exact as IEEE's, ties to
// even; a NaN and every value of a group whose scale is 0 or Inf get z.
// v * (1 / s) is off by at most 2^-22 |v / s| < 2^-17, so it rounds like the
// quotient unless it lies that close to a half; only then is the division done
// (about one weight in ten thousand).
__device__ __forceinline__ void codes_of(const float (&v)[8], float s, float z, float lo, float hi, uint32_t (&c)[8]) {
  if (!(s > 0.0f) || isinf(s)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = static_cast<uint32_t>(z);
    return;
  }
  const float inv = __frcp_rn(s);
  // Adding 1.5 * 2^23 rounds to an integer (ties to even) and leaves its low
  // bits in the mantissa; rintf would go through the slow conversion pipe.
  constexpr float kMagic = 12582912.0f;
  const float top = __fadd_rn(hi, -z), bottom = __fadd_rn(lo, -z);
  float d[8], far = 1.0f;  // the smallest distance of a quotient's fraction from a half
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fminf(fmaxf(__fmul_rn(v[i], inv), bottom), top);
    d[i] = __fadd_rn(t, kMagic);
    far = fminf(far, fabsf(__fadd_rn(fabsf(__fadd_rn(t, -__fadd_rn(d[i], -kMagic))), -0.5f)));
  }
  // (a NaN lost its sign to the clamp; an inv of Inf, from a subnormal scale, makes NaN and clamped values)
  bool unsure = !(far > 0x1p-12f) || isinf(inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) unsure |= isnan(v[i]);
  if (unsure) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      d[i] = __fadd_rn(isnan(v[i]) ? 0.0f : fminf(fmaxf(__fdiv_rn(v[i], s), bottom), top), kMagic);
  }
  const uint32_t zi = static_cast<uint32_t>(z);
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = (__float_as_uint(d[i]) + zi) & 15u;
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_quantize(const __half* __restrict__ src, const float* __restrict__ fold, uint8_t* __restrict__ out,
                  int64_t N, int64_t K, int KT) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int l = threadIdx.x & 15;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 4);
  const int r = static_cast<int>(n & (kW4Rows - 1));
  const Span sp = k_span(KT);
  griddep_wait();
  uint8_t* rec = out + ((n >> 7) * KT + sp.t0) * REC;
  const __half* row = src + n * K + 8 * l;
  auto load = [&](int kt) {
    const int64_t k = static_cast<int64_t>(kt) * kW4K;
    return kt < sp.t1 && n < N && k + 8 * l < K ? ld_stream(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
  };
  uint4 next = load(sp.t0);
  for (int kt = sp.t0; kt < sp.t1; ++kt, rec += REC) {
    const uint4 raw = next;
    next = load(kt + 1);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(reinterpret_cast<const __half2*>(&raw)[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
    if (fold) {
      const int64_t k = static_cast<int64_t>(kt) * kW4K + 8 * l;
      if (k < K) {
        // the folded weight is an fp16 tensor, as in the INT8 quantizer
        const float4 f0 = *reinterpret_cast<const float4*>(fold + k), f1 = *reinterpret_cast<const float4*>(fold + k + 4);
        const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __half2float(__float2half_rn(__fmul_rn(v[i], f[i])));
      }
    }
    float s, z;
    uint32_t c[8];
    if (ZERO) {
      // fmaxf drops a NaN, so it never sets a range
      float hi = 0.0f, lo = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) hi = fmaxf(hi, v[i]), lo = fmaxf(lo, -v[i]);
      hi = group_max<G / 8>(hi);
      lo = group_max<G / 8>(lo);
      // 7 significant bits: |q - z| <= 15 takes 4, so (q - z) * s fits fp16's 11
      s = __half2float(__float2half_rn(round_bits(__fdiv_rn(__fadd_rn(hi, lo), 15.0f), 7)));
      z = (s > 0.0f && !isinf(s)) ? fminf(rintf(__fdiv_rn(lo, s)), 15.0f) : 0.0f;
      codes_of(v, s, z, 0.0f, 15.0f, c);
    } else {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
      m = group_max<G / 8>(m);
      // 8 significant bits: |q| <= 7 takes 3, so q * s fits fp16's 11
      s = __half2float(__float2half_rn(round_bits(__fdiv_rn(m, 7.0f), 8)));
      z = 8.0f;
      codes_of(v, s, z, 1.0f, 15.0f, c);
    }
    *reinterpret_cast<uint32_t*>(rec + word_offset(r, l)) = pack_word(c);
    if ((l & (G / 8 - 1)) == 0) {
      const int g = l / (G / 8);
      *reinterpret_cast<__half*>(rec + kW4CodeBytes + (r * NG + g) * 2) = __float2half_rn(s);
      if (ZERO) rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + g] = static_cast<uint8_t>(z);
    }
  }
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_pack(const uint8_t* __restrict__ codes, const __half* __restrict__ scales,
              const uint8_t* __restrict__ zeros, uint8_t* __restrict__ out, int64_t N, int64_t K, int KT) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int l = threadIdx.x & 15;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 4);
  const int r = static_cast<int>(n & (kW4Rows - 1));
  const Span sp = k_span(KT);
  const int64_t groups = (K + G - 1) / G;
  griddep_wait();
  uint8_t* rec = out + ((n >> 7) * KT + sp.t0) * REC;
  for (int kt = sp.t0; kt < sp.t1; ++kt, rec += REC) {
    const int64_t k = static_cast<int64_t>(kt) * kW4K + 8 * l;
    const int64_t g = k / G;
    uint32_t z = ZERO ? 0u : 8u;
    __half s = __float2half_rn(0.0f);
    if (n < N && g < groups) {
      s = scales[n * groups + g];
      if (ZERO) z = zeros[n * groups + g] & 15u;
    }
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = z;
    if (n < N && k < K) {
      const uint2 raw = *reinterpret_cast<const uint2*>(codes + n * K + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = (raw.x >> (8 * i)) & 15u, c[4 + i] = (raw.y >> (8 * i)) & 15u;
    }
    *reinterpret_cast<uint32_t*>(rec + word_offset(r, l)) = pack_word(c);
    if ((l & (G / 8 - 1)) == 0) {
      const int gi = l / (G / 8);
      *reinterpret_cast<__half*>(rec + kW4CodeBytes + (r * NG + gi) * 2) = s;
      if (ZERO) rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + gi] = static_cast<uint8_t>(z);
    }
  }
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_dequantize(const uint8_t* __restrict__ in, __half* __restrict__ out, int64_t N, int64_t K, int KT) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  const int l = threadIdx.x & 15;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 4);
  const int r = static_cast<int>(n & (kW4Rows - 1));
  const Span sp = k_span(KT);
  griddep_wait();
  if (n >= N) return;
  const uint8_t* rec = in + ((n >> 7) * KT + sp.t0) * REC;
  const int g = l / (G / 8);
  struct Item {
    uint32_t word, z;
    __half s;
  };
  auto load = [&](const uint8_t* p, bool on) {
    Item it{};
    if (on) {
      it.word = *reinterpret_cast<const uint32_t*>(p + word_offset(r, l));
      it.s = *reinterpret_cast<const __half*>(p + kW4CodeBytes + (r * NG + g) * 2);
      it.z = ZERO ? p[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + g] : 8u;
    }
    return it;
  };
  Item next = load(rec, sp.t0 < sp.t1);
  for (int kt = sp.t0; kt < sp.t1; ++kt) {
    const Item it = next;
    rec += REC;
    next = load(rec, kt + 1 < sp.t1);
    const int64_t k = static_cast<int64_t>(kt) * kW4K + 8 * l;
    if (k >= K) continue;
    // (q - z) is exact in fp16, its product with s rounded once
    uint32_t h[4];
    dequant(it.word, 0x64006400u | it.z | it.z << 16, 0xD400D400u | it.z << 4 | it.z << 20, h);
    const __half2 s2 = __half2half2(it.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2_rn(*reinterpret_cast<const __half2*>(&h[i]), s2);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(out + n * K + k) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// Blocks of 16 channels; K is split until about 32 warps per SM exist (a
// narrow weight would otherwise walk K in too few warps).
dim3 grid_for(int64_t rows, int64_t kt, const Ctx& c) {
  const int64_t x = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
  int64_t y = (static_cast<int64_t>(c.num_sms) * 4 + x - 1) / x;
  if (y > kt) y = kt;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
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
  const dim3 grid = grid_for(w.nt() * kW4Rows, w.kt(), c);
#define SQ_CALL(G, Z)                                                                                              \
  launch_pdl(k_w4_pack<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, codes, scales, zeros, w.data, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_quantize(const __half* src, const float* s, const W4Weight& w, const Ctx& c) {
  const dim3 grid = grid_for(w.nt() * kW4Rows, w.kt(), c);
#define SQ_CALL(G, Z) \
  launch_pdl(k_w4_quantize<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, src, s, w.data, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_dequantize(const W4Weight& w, __half* out, const Ctx& c) {
  const dim3 grid = grid_for(w.N, w.kt(), c);
#define SQ_CALL(G, Z)                                                                                           \
  launch_pdl(k_w4_dequantize<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, static_cast<const uint8_t*>(w.data),   \
             out, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

}  // namespace sq
