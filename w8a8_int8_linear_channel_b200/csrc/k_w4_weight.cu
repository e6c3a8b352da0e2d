// k_w4_weight.cu -- making and reading packed 4-bit weights: quantization of
// an fp16 weight in groups, packing of codes a caller already has, and the
// fp16 values of a packed weight.  They come near the rate of HBM when they are
// written so that nothing but the eight values of a packed word is computed
// per thread: a warp takes two channels (the quantizer four), lane l the k =
// 8 l .. 8 l + 7 of a tile (one 16-byte load or store, one packed word), and
// walks along K with the next tile's load in flight.  16384 x 4096 with a fold:
// quantize 41 us (169 MB at 4.1 TB/s, 0.64 of the copy bandwidth; its schedulers
// are 78% busy), dequantize 32.5 us (5.2 TB/s, 0.81).
#include "sq_w4.cuh"

namespace sq {
namespace {

constexpr int kWarps = 8;

constexpr int kRowsPerBlock = 2 * kWarps;

// Byte offset in a record of the word with k = 8 l .. 8 l + 7 of channel r.
__device__ __forceinline__ int word_offset(int r, int l) { return r * 64 + (((l & 3) ^ ((r >> 1) & 3)) << 4) + 4 * (l >> 2); }

// Element 2 i of a word lies in bits 4 i .., element 2 i + 1 sixteen bits higher.
__host__ __device__ constexpr int nibble_shift(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

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

constexpr float kMagic = 12582912.0f;         // 1.5 * 2^23: a sum with it is an integer in the low mantissa bits
constexpr uint32_t kMagicBits = 0x4B400000u;

__device__ __forceinline__ float rcp_approx(float s) {
  float r;  // off by at most one step
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// The word of the codes clamp(rint(v / s) + z, lo, 15), the quotient as IEEE
// division gives it, ties to even; a NaN and every value of a group whose
// scale is 0 or Inf get z.
// t = v * inv is off by at most 2^-22 t; one correction by the remainder v - t s,
// which a fused multiply-add forms exactly (Markstein's method, IBM J. Res. Dev. 34, 1990),
// leaves 2^-44 t before its own rounding.  A quotient of k + 1/2 exactly (one
// weight in a few hundred: v has 11 bits, s 8) is an fp32 number and so comes out exactly, and any
// other is at least 2^-12 away from a half: both round as the quotient does.
// What is left to a slow path is a code out of range (clamped, or a NaN).
template <bool ZERO>
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float s, float z) {
  const float inv = rcp_approx(s);
  // The sum's bits are kMagicBits + code.  z = 8 is even, so adding it with the
  // magic number leaves ties to even what they are; an odd zero point is added
  // to the integer instead.
  const float base = ZERO ? kMagic : kMagic + 8.0f;
  const uint32_t off = ZERO ? kMagicBits - static_cast<uint32_t>(z) : 0u;
  uint32_t word = ZERO ? 0u : 0u - kMagicBits * 0x11111111u, range = ZERO ? 0u : kMagicBits;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t = __fmul_rn(v[i], inv);
    t = __fmaf_rn(__fmaf_rn(-t, s, v[i]), inv, t);
    const uint32_t c = __float_as_uint(__fadd_rn(t, base)) - off;
    range |= c;
    word += c << nibble_shift(i);
  }
  // (a scale below fp16's normal range is so coarse that -8 can come up, which
  // is in range but clamped)
  if ((ZERO ? range : range - kMagicBits) < 16u && s >= (ZERO ? 0x1p-24f : 0x1p-14f)) return word;
  const uint32_t zi = static_cast<uint32_t>(z);
  if (!(s > 0.0f) || isinf(s)) return zi * 0x11111111u;
  word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = isnan(v[i]) ? 0.0f : rintf(__fdiv_rn(v[i], s));
    const float c = fminf(fmaxf(__fadd_rn(q, z), ZERO ? 0.0f : 1.0f), 15.0f);
    word |= static_cast<uint32_t>(c) << nibble_shift(i);
  }
  return word;
}

// The quantizer is bound by instructions, so a lane takes two words (k = 8 l ..
// and 64 + 8 l ..) and a warp four channels: what a group costs is shared by
// more weights.
constexpr int kQuantRows = 4 * kWarps;

template <int G, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32)
    k_w4_quantize(const __half* __restrict__ src, const float* __restrict__ fold, uint8_t* __restrict__ out,
                  int64_t N, int64_t K, int KT) {
  constexpr int NG = kW4K / G;
  constexpr int REC = w4_record_bytes(G, ZERO);
  constexpr int LANES = G >= 64 ? 8 : 4;  // lanes of a group in each half of the tile
  const int l = threadIdx.x & 7;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kQuantRows + (threadIdx.x >> 3);
  const int r = static_cast<int>(n & (kW4Rows - 1));
  const Span sp = k_span(KT);
  griddep_wait();
  uint8_t* rec = out + ((n >> 7) * KT + sp.t0) * REC;
  const int k0 = sp.t0 * kW4K + 8 * l;
  const __half* row = src + n * K + k0;
  const float* frow = fold ? fold + k0 : nullptr;
  // k of this lane still to come: none for a channel past N
  int left = n < N ? static_cast<int>(K) - k0 : 0;
  auto load = [&](int k) {
    return left > k ? ld_stream(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
  };
  uint4 next[2] = {load(0), load(64)};
  const int word_at = word_offset(r, l);
  for (int kt = sp.t0; kt < sp.t1; ++kt) {
    uint4 raw[2] = {next[0], next[1]};
    next[0] = kt + 1 < sp.t1 ? load(kW4K) : make_uint4(0, 0, 0, 0);
    next[1] = kt + 1 < sp.t1 ? load(kW4K + 64) : make_uint4(0, 0, 0, 0);
    __half2* h[2] = {reinterpret_cast<__half2*>(&raw[0]), reinterpret_cast<__half2*>(&raw[1])};
    if (fold) {
      // the folded weight is an fp16 tensor, as in the INT8 quantizer
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (left > 64 * j) {
          const float4 f0 = *reinterpret_cast<const float4*>(frow + 64 * j), f1 = *reinterpret_cast<const float4*>(frow + 64 * j + 4);
          const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 w = __half22float2(h[j][i]);
            h[j][i] = __floats2half2_rn(__fmul_rn(w.x, f[2 * i]), __fmul_rn(w.y, f[2 * i + 1]));
          }
        }
      frow += kW4K;
    }
    // ranges, in fp16 (exact; the maximum drops a NaN, so it never sets a range)
    float hi[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2 zero = __float2half2_rn(0.0f);
      __half2 a = zero, b = zero;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a = __hmax2(a, ZERO ? h[j][i] : __habs2(h[j][i]));
        if (ZERO) b = __hmax2(b, __hneg2(h[j][i]));
      }
      hi[j] = __half2float(__hmax(__low2half(a), __high2half(a)));
      lo[j] = __half2float(__hmax(__low2half(b), __high2half(b)));
    }
    if (G == 128) {
      hi[0] = fmaxf(hi[0], hi[1]);
      lo[0] = fmaxf(lo[0], lo[1]);
    }
#pragma unroll
    for (int j = 0; j < (G == 128 ? 1 : 2); ++j) {
      hi[j] = group_max<LANES>(hi[j]);
      if (ZERO) lo[j] = group_max<LANES>(lo[j]);
    }
    float s = 0.0f, z = 8.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j == 0 || G != 128) {
        if (ZERO) {
          // 7 significant bits: |q - z| <= 15 takes 4, so (q - z) * s fits fp16's 11
          s = __half2float(__float2half_rn(round_bits(__fdiv_rn(__fadd_rn(hi[j], lo[j]), 15.0f), 7)));
          z = (s > 0.0f && !isinf(s)) ? fminf(rintf(__fdiv_rn(lo[j], s)), 15.0f) : 0.0f;
        } else {
          // 8 significant bits: |q| <= 7 takes 3, so q * s fits fp16's 11.  The
          // maximum has 11 bits, seven times the middle of two 8-bit numbers has
          // 12: a seventh is never halfway, nor nearer to it than 2^-14, and the
          // product rounds like it.
          s = __half2float(__float2half_rn(round_bits(__fmul_rn(hi[j], 1.0f / 7.0f), 8)));
        }
        const int g = G == 32 ? 2 * j + (l >> 2) : G == 64 ? j : 0;
        if ((l & (LANES - 1)) == 0) {
          *reinterpret_cast<__half*>(rec + kW4CodeBytes + (r * NG + g) * 2) = __float2half_rn(s);
          if (ZERO) rec[kW4CodeBytes + kW4Rows * NG * 2 + r * NG + g] = static_cast<uint8_t>(z);
        }
      }
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[j][i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
      *reinterpret_cast<uint32_t*>(rec + word_at + 8 * j) = codes_of<ZERO>(v, s, z);
    }
    rec += REC;
    row += kW4K;
    left -= kW4K;
  }
}

// 16384 x 4096, groups of 128: 28.6 us, 3.6 TB/s (0.56 of the copy bandwidth); groups of 32 with zero
// points 31.8 us.  An offline step; what it waits for is the latency of its loads.
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
    uint32_t word = z * 0x11111111u;
    if (n < N && k < K) {
      const uint2 raw = *reinterpret_cast<const uint2*>(codes + n * K + k);
      word = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) word |= (((i < 4 ? raw.x : raw.y) >> (8 * (i & 3))) & 15u) << nibble_shift(i);
    }
    *reinterpret_cast<uint32_t*>(rec + word_offset(r, l)) = word;
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

// Blocks of per_block channels; K is split until about 32 warps per SM exist (a
// narrow weight would otherwise walk K in too few warps).
dim3 grid_for(int64_t rows, int per_block, int64_t kt, const Ctx& c) {
  const int64_t x = (rows + per_block - 1) / per_block;
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
  const dim3 grid = grid_for(w.nt() * kW4Rows, kRowsPerBlock, w.kt(), c);
#define SQ_CALL(G, Z)                                                                                              \
  launch_pdl(k_w4_pack<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, codes, scales, zeros, w.data, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_quantize(const __half* src, const float* s, const W4Weight& w, const Ctx& c) {
  const dim3 grid = grid_for(w.nt() * kW4Rows, kQuantRows, w.kt(), c);
#define SQ_CALL(G, Z) \
  launch_pdl(k_w4_quantize<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, src, s, w.data, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

cudaError_t launch_w4_dequantize(const W4Weight& w, __half* out, const Ctx& c) {
  const dim3 grid = grid_for(w.N, kRowsPerBlock, w.kt(), c);
#define SQ_CALL(G, Z)                                                                                           \
  launch_pdl(k_w4_dequantize<G, Z>, grid, dim3(kWarps * 32), 0, c.stream, static_cast<const uint8_t*>(w.data),   \
             out, w.N, w.K, w.kt())
  SQ_W4_DISPATCH(w, SQ_CALL);
#undef SQ_CALL
}

}  // namespace sq
