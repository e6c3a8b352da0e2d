// k_w4_stream.cu -- y = x W^T with a packed 4-bit W for few tokens: the weight
// is streamed once, and everything else is arranged around that stream.
//
//   y[m, n] = fp16( sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[m, k] + bias[n] )
//
// The 4-bit codes become fp16 integers q - z, exact, and go into
// mma.m16n8k16 with the weight as the 16-row operand and the tokens as the
// 8-column one (fp32 accumulators); a group's sum is multiplied by its scale
// once, in fp32, so no weight is ever rounded.
//
// A CTA owns one 128-channel tile and a slice of K; the cluster's CTAs own
// the slices of the same tile and add their sums through distributed shared
// memory at the end (in slice order: no atomics, no workspace, the same bits
// on every run).  One warp streams records and token rows into a ring of
// stages with bulk copies; eight warps consume them, 16 channels each.
#include "sq_ptx.cuh"
#include "sq_w4.h"

namespace sq {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = (kConsumers + 1) * 32;
// Bytes between two tokens' 128 k in a stage: 256 + 64, so the eight lanes of
// a 16-byte read phase (two tokens x four chunks) hit different banks.
constexpr int kTokenPitch = 320;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2(float v) {
  const __half2 h = __float2half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
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

template <int NB, int G, bool ZERO>
struct Layout {
  static constexpr int BT = 8 * NB;
  static constexpr int REC = w4_record_bytes(G, ZERO);
  static constexpr int X = REC;
  static constexpr int STAGE = REC + BT * kTokenPitch;
  static constexpr int STAGES = NB == 1 ? 6 : NB == 2 ? 5 : 4;
  static constexpr int RED = STAGES * STAGE;               // fp32 [BT][kRedPitch]
  static constexpr int kRedPitch = kW4Rows + 4;
  static constexpr int BARS = RED + BT * kRedPitch * 4;    // full[STAGES], empty[STAGES]
  static constexpr int ROWS = BARS + 16 * STAGES;          // int32 pair index of every token of the block
  static constexpr int MISC = ROWS + BT * 4;               // abort flag, block's first pair, pair count, expert
  static constexpr int BYTES = MISC + 16;
};

template <int NB, int G, bool ZERO>
__global__ void __launch_bounds__(kThreads)
    k_w4_stream(const W4Product p, int slices, int blocks, int KT, uint32_t* status, uint64_t budget) {
  using L = Layout<NB, G, ZERO>;
  constexpr int NG = kW4K / G;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + L::MISC);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + L::MISC);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + L::ROWS);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // consecutive clusters take the token blocks of one weight tile (the tile
  // comes from L2 after the first)
  const int slice = blockIdx.x % slices;
  const int block = blockIdx.x / slices % blocks;
  const int tile = blockIdx.x / slices / blocks;
  const uint32_t full = sbase + L::BARS, empty = full + 8 * L::STAGES;

  if (tid == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kConsumers);
    }
    *abort = 0;
    fence_barrier_init();
  }
  griddep_wait();

  // which tokens this CTA's block holds
  int expert = 0, count = 0;
  if (p.offsets == nullptr) {
    const int64_t first = static_cast<int64_t>(block) * L::BT;
    count = static_cast<int>(p.M - first < L::BT ? p.M - first : L::BT);
    if (tid < L::BT) rows[tid] = static_cast<int32_t>(first + tid);
  } else {
    // block number `block` of the blocks of all experts in order: a scan of
    // ceil(n_e / BT) over the experts
    if (warp == 0) {
      int before = 0, found = -1, first = 0, n = 0;
      for (int e0 = 0; e0 < p.E && found < 0; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
          lo = p.offsets[e];
          hi = p.offsets[e + 1];
          // offsets that no plan wrote must not lead out of the order array
          lo = max(lo, 0);
          hi = static_cast<int>(min(static_cast<int64_t>(hi), p.M));
        }
        const int mine = hi > lo ? (hi - lo + L::BT - 1) / L::BT : 0;
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
          const int skip = (rel - __shfl_sync(0xffffffffu, inc - mine, src)) * L::BT;
          first = __shfl_sync(0xffffffffu, lo, src) + skip;
          n = min(__shfl_sync(0xffffffffu, hi, src) - first, L::BT);
          found = e0 + src;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        misc[1] = found;
        misc[2] = n;
      }
      if (found >= 0) {
        for (int i = lane; i < n; i += 32) {
          const int32_t pair = p.order[first + i];
          rows[i] = pair >= 0 && pair < p.M ? pair : -1;
        }
      }
    }
    __syncthreads();
    expert = misc[1];
    count = misc[2];
    if (expert < 0) return;  // the same for every CTA of the cluster
  }
  __syncthreads();

  const int kt0 = static_cast<int>(static_cast<int64_t>(KT) * slice / slices);
  const int kt1 = static_cast<int>(static_cast<int64_t>(KT) * (slice + 1) / slices);
  const int64_t nt = p.w.nt();
  const int64_t K = p.w.K;

  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;

  int issued = 0;  // stages the producer filled
  if (warp == kConsumers) {
    // ---- producer: one record and the block's token rows per stage
    const uint8_t* recs = p.w.data + ((static_cast<int64_t>(expert) * nt + tile) * KT) * L::REC;
    const __half* xrow = nullptr;
    if (lane < count && rows[lane] >= 0) xrow = p.x + static_cast<int64_t>(rows[lane] / p.div) * p.ldx;
    const int live = __popc(__ballot_sync(0xffffffffu, xrow != nullptr));
    for (int kt = kt0; kt < kt1; ++kt) {
      const int i = kt - kt0, s = i % L::STAGES;
      if (i >= L::STAGES && !mbar_wait(empty + 8 * s, ((i / L::STAGES) & 1) ^ 1, budget, status, abort)) break;
      const uint32_t stage = sbase + s * L::STAGE;
      const uint32_t xbytes = static_cast<uint32_t>(min(static_cast<int64_t>(kW4K), K - static_cast<int64_t>(kt) * kW4K)) * 2;
      if (lane == 0) {
        mbar_arrive_expect_tx(full + 8 * s, L::REC + live * xbytes);
        bulk_load(stage, recs + static_cast<int64_t>(kt) * L::REC, L::REC, full + 8 * s);
      }
      __syncwarp();
      if (xrow) bulk_load(stage + L::X + lane * kTokenPitch, xrow + static_cast<int64_t>(kt) * kW4K, xbytes, full + 8 * s);
      issued = i + 1;
    }
  } else {
    // ---- consumers: channels 16 * warp + (g, g + 8)
    const int g = lane >> 2, t = lane & 3;
    const int r0 = warp * 16 + g;
    const uint32_t off0 = r0 * 64 + ((t ^ ((r0 >> 1) & 3)) << 4);
    const uint32_t off1 = off0 + 8 * 64;  // (r0 + 8) >> 1 has the same low two bits
    bool tok[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) tok[b] = 8 * b + g < count && rows[8 * b + g] >= 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      const int i = kt - kt0, s = i % L::STAGES;
      if (!mbar_wait(full + 8 * s, (i / L::STAGES) & 1, budget, status, abort)) break;
      const uint32_t stage = sbase + s * L::STAGE;
      const uint4 c0 = lds128(stage + off0), c1 = lds128(stage + off1);
      const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
      const uint8_t* rec = smem + s * L::STAGE;
      const __half* sc = reinterpret_cast<const __half*>(rec + kW4CodeBytes);
      const uint8_t* zp = rec + kW4CodeBytes + kW4Rows * NG * 2;
      // k of this tile that exist: past them the stage's token bytes are stale
      const int klen = static_cast<int>(min(static_cast<int64_t>(kW4K), K - static_cast<int64_t>(kt) * kW4K));
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        const float s0 = __half2float(sc[r0 * NG + gi]), s1 = __half2float(sc[(r0 + 8) * NG + gi]);
        uint32_t lo0 = 0x64086408u, hi0 = 0xD480D480u, lo1 = lo0, hi1 = hi0;  // z = 8: 1032, -72
        if (ZERO) {
          const float z0 = zp[r0 * NG + gi], z1 = zp[(r0 + 8) * NG + gi];
          lo0 = h2(1024.0f + z0), hi0 = h2(-64.0f - z0);
          lo1 = h2(1024.0f + z1), hi1 = h2(-64.0f - z1);
        }
        float part[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[b][j] = 0.0f;
#pragma unroll
        for (int w = gi * (G / 32); w < (gi + 1) * (G / 32); ++w) {
          uint32_t a0[4], a1[4];
          dequant(w0[w], lo0, hi0, a0);
          dequant(w1[w], lo1, hi1, a1);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (tok[b] && 32 * w + 8 * t < klen)
              x = lds128(stage + L::X + (8 * b + g) * kTokenPitch + 64 * w + 16 * t);
            mma_f16(part[b], a0[0], a1[0], a0[1], a1[1], x.x, x.y);
            mma_f16(part[b], a0[2], a1[2], a0[3], a1[3], x.z, x.w);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          acc[b][0] = __fmaf_rn(s0, part[b][0], acc[b][0]);
          acc[b][1] = __fmaf_rn(s0, part[b][1], acc[b][1]);
          acc[b][2] = __fmaf_rn(s1, part[b][2], acc[b][2]);
          acc[b][3] = __fmaf_rn(s1, part[b][3], acc[b][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * s);
    }
    float* red = reinterpret_cast<float*>(smem + L::RED);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float* q = red + (8 * b + 2 * t) * L::kRedPitch + r0;
      q[0] = acc[b][0];
      q[L::kRedPitch] = acc[b][1];
      q[8] = acc[b][2];
      q[L::kRedPitch + 8] = acc[b][3];
    }
  }
  griddep_launch_dependents();
  if (slices > 1)
    cluster_sync_all();
  else
    __syncthreads();

  if (*abort && warp == kConsumers) {
    // a wait ran out: let the copies in flight land before the CTA leaves
    for (int i = max(0, issued - L::STAGES); i < issued; ++i)
      mbar_drain(full + 8 * (i % L::STAGES), (i / L::STAGES) & 1, budget);
  }

  // Each CTA of the cluster finishes its share of the tile's channels.
  const int n0 = kW4Rows * slice / slices, n1 = kW4Rows * (slice + 1) / slices;
  const int width = n1 - n0;
  const uint32_t red = sbase + L::RED;
  for (int i = tid; i < width * count; i += kThreads) {
    const int tk = i / width, r = n0 + (i - tk * width);
    const int64_t n = static_cast<int64_t>(tile) * kW4Rows + r;
    if (n >= p.w.N || rows[tk] < 0) continue;
    float v = 0.0f;
    const uint32_t off = red + (tk * L::kRedPitch + r) * 4;
    if (slices > 1) {
      for (int c = 0; c < slices; ++c) v = __fadd_rn(v, ld_cluster_f32(mapa_shared(off, c)));
    } else {
      v = *reinterpret_cast<const float*>(smem + (off - sbase));
    }
    if (p.bias) v = __fadd_rn(v, __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + n]));
    if (p.relu) v = v > 0.0f ? v : 0.0f;
    const int64_t o = static_cast<int64_t>(rows[tk]) * p.w.N + n;
    if (p.y)
      p.y[o] = __float2half_rn(v);
    else
      p.y32[o] = v;
  }
  if (slices > 1) cluster_sync_all();  // the others may still read this CTA's sums
}

template <int NB, int G, bool ZERO>
cudaError_t launch(const W4Product& p, const Ctx& c) {
  using L = Layout<NB, G, ZERO>;
  auto kernel = k_w4_stream<NB, G, ZERO>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t nt = p.w.nt(), kt = p.w.kt();
  // Blocks of BT tokens: exactly, or for experts the most that any routing
  // of p.M pairs can need (CTAs of blocks that do not exist leave at once).
  int64_t blocks = (p.M + L::BT - 1) / L::BT;
  if (p.offsets) blocks = p.M < blocks + p.E ? p.M : blocks + p.E;
  // K is split until about two CTAs per SM exist, four tiles each at least.
  int slices = 1;
  while (slices < 8 && nt * blocks * slices < 2 * c.num_sms && kt / (slices + 1) >= 4) ++slices;
  cudaLaunchConfig_t cfg = {};
  if (nt * blocks * slices > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(nt * blocks * slices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = slices;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, slices, static_cast<int>(blocks), static_cast<int>(kt), c.status, c.budget_ns);
}

template <int NB>
cudaError_t launch_g(const W4Product& p, const Ctx& c) {
  if (p.w.zero) {
    if (p.w.group == 32) return launch<NB, 32, true>(p, c);
    if (p.w.group == 64) return launch<NB, 64, true>(p, c);
    return launch<NB, 128, true>(p, c);
  }
  if (p.w.group == 32) return launch<NB, 32, false>(p, c);
  if (p.w.group == 64) return launch<NB, 64, false>(p, c);
  return launch<NB, 128, false>(p, c);
}

}  // namespace

cudaError_t launch_w4_product(const W4Product& p, const Ctx& c) {
  const int64_t per = p.offsets ? (p.M + p.E - 1) / p.E : p.M;
  if (per <= 8) return launch_g<1>(p, c);
  if (per <= 16) return launch_g<2>(p, c);
  return launch_g<4>(p, c);
}

}  // namespace sq
