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
// A CTA owns one 128-channel tile and a slice of K; the CTAs of a cluster own
// the slices of one tile.  One warp streams records and token rows into a ring
// of stages with bulk copies; eight warps consume them: four groups of 32
// channels, times two that take the even and the odd K tiles.  At the end
// every warp pushes its sums to the CTA of the cluster that finishes those
// channels (distributed shared memory), which adds them in a fixed order: no
// atomics, no workspace, the same bits on every run.
#include "sq_w4.cuh"

namespace sq {
namespace {

constexpr int kRowGroups = 4;   // warps along the channels, 32 each
constexpr int kKGroups = 2;     // warps along K: even and odd tiles
constexpr int kConsumers = kRowGroups * kKGroups;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kMaxSlices = 8;   // portable cluster size
// Bytes between two tokens' 128 k in a stage: 256 + 64, so the eight lanes of
// a 16-byte read phase (two tokens x four chunks) hit different banks.
constexpr int kTokenPitch = 320;

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NB, int G, bool ZERO>
struct Layout {
  static constexpr int BT = 8 * NB;
  static constexpr int REC = w4_record_bytes(G, ZERO);
  static constexpr int X = REC;
  static constexpr int STAGE = REC + BT * kTokenPitch;
  // even (a K group keeps to its half of the stages), and such that three CTAs fit an SM (two of 16 tokens)
  static constexpr int STAGES = NB == 1 && 6 * STAGE <= 67 * 1024 ? 6 : 4;
  // sums of every slice and K group for the channels this CTA finishes:
  // fp32 [slices * kKGroups][channels per CTA][BT]
  static constexpr int RED = STAGES * STAGE;
  static constexpr int RED_ROWS = kKGroups * (kW4Rows + kMaxSlices);
  static constexpr int BARS = RED + RED_ROWS * BT * 4;     // full[STAGES], empty[STAGES]
  static constexpr int ROWS = BARS + 16 * STAGES;          // int32 pair index of every token of the block
  static constexpr int MISC = ROWS + BT * 4;               // abort flag, expert, token count
  static constexpr int BYTES = MISC + 16;
};

// One K tile of 32 channels x BT tokens.  Channels r0 + 16 m + (0, 8); klen is
// how many of the tile's k exist (past them a stage holds stale token bytes).
template <int NB, int G, bool ZERO, bool TAIL>
__device__ __forceinline__ void consume(uint32_t stage, const uint8_t* rec, int r0, int lane, int klen,
                                        float (&acc)[2][NB][4]) {
  using L = Layout<NB, G, ZERO>;
  constexpr int NG = kW4K / G;
  const int g = lane >> 2, t = lane & 3;
  uint32_t w[2][2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    // (r >> 1) & 3 is the same for r0, r0 + 8, r0 + 16, r0 + 24
    const uint32_t off = stage + (r0 + 16 * m) * 64 + ((t ^ ((r0 >> 1) & 3)) << 4);
    const uint4 c0 = lds128(off), c1 = lds128(off + 8 * 64);
    w[m][0][0] = c0.x, w[m][0][1] = c0.y, w[m][0][2] = c0.z, w[m][0][3] = c0.w;
    w[m][1][0] = c1.x, w[m][1][1] = c1.y, w[m][1][2] = c1.z, w[m][1][3] = c1.w;
  }
  const __half* sc = reinterpret_cast<const __half*>(rec + kW4CodeBytes) + r0 * NG;
  const uint8_t* zp = rec + kW4CodeBytes + kW4Rows * NG * 2 + r0 * NG;
  const uint32_t xa = stage + L::X + g * kTokenPitch + 16 * t;
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    float part[2][NB][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[m][b][j] = 0.0f;
    uint32_t lo[2][2], hi[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lo[m][h] = 0x64086408u, hi[m][h] = 0xD480D480u;  // z = 8: 1032, -72
        if (ZERO) {
          // 0x6400 | z is 1024 + z; -(64 + z) is 0xD400 | 16 z
          const uint32_t z = zp[(16 * m + 8 * h) * NG + gi];
          lo[m][h] = 0x64006400u | z | z << 16;
          hi[m][h] = 0xD400D400u | z << 4 | z << 20;
        }
      }
#pragma unroll
    for (int q = gi * (G / 32); q < (gi + 1) * (G / 32); ++q) {
      uint4 x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        x[b] = make_uint4(0, 0, 0, 0);
        if (!TAIL || 32 * q + 8 * t < klen) x[b] = lds128(xa + 8 * b * kTokenPitch + 64 * q);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a0[4], a1[4];
        dequant(w[m][0][q], lo[m][0], hi[m][0], a0);
        dequant(w[m][1][q], lo[m][1], hi[m][1], a1);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          mma_f16(part[m][b], a0[0], a1[0], a0[1], a1[1], x[b].x, x[b].y);
          mma_f16(part[m][b], a0[2], a1[2], a0[3], a1[3], x[b].z, x[b].w);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float s0 = __half2float(sc[16 * m * NG + gi]), s1 = __half2float(sc[(16 * m + 8) * NG + gi]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        acc[m][b][0] = __fmaf_rn(s0, part[m][b][0], acc[m][b][0]);
        acc[m][b][1] = __fmaf_rn(s0, part[m][b][1], acc[m][b][1]);
        acc[m][b][2] = __fmaf_rn(s1, part[m][b][2], acc[m][b][2]);
        acc[m][b][3] = __fmaf_rn(s1, part[m][b][3], acc[m][b][3]);
      }
    }
  }
}

template <int NB, int G, bool ZERO>
__global__ void __launch_bounds__(kThreads)
    k_w4_stream(const W4Product p, int slices, int KT, int nt, uint32_t share_inv, uint32_t* status, uint64_t budget) {
  using L = Layout<NB, G, ZERO>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + L::MISC);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + L::MISC);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + L::ROWS);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // consecutive clusters take the token blocks of one weight tile (the tile
  // comes from L2 after the first)
  const int slice = static_cast<int>(cluster_ctarank());
  const int block = static_cast<int>(cluster_id_x());
  const int tile = static_cast<int>(blockIdx.y);
  const uint32_t full = sbase + L::BARS, empty = full + 8 * L::STAGES;

  if (tid == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kRowGroups);
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
    if (tid < L::BT) rows[tid] = tid < count ? static_cast<int32_t>(first + tid) : -1;
    __syncthreads();
  } else {
    if (warp == 0) {
      int start = 0;
      expert = w4_find_block(p, block, L::BT, lane, &start, &count);
      if (lane == 0) {
        misc[1] = expert;
        misc[2] = count;
      }
      if (expert >= 0)
        for (int i = lane; i < L::BT; i += 32) {
          const int32_t pair = i < count ? p.order[start + i] : -1;
          rows[i] = pair >= 0 && pair < p.M ? pair : -1;
        }
    }
    __syncthreads();
    expert = misc[1];
    count = misc[2];
    if (expert < 0) return;  // the same for every CTA of the cluster
  }

  const int each = KT / slices, more = KT - each * slices;  // K tiles per slice, slices with one more
  const int kt0 = each * slice + min(slice, more);
  const int n = each + (slice < more ? 1 : 0);
  const int tail = static_cast<int>(p.w.K & (kW4K - 1));  // k of the last tile when it is short
  const int share = (kW4Rows + slices - 1) / slices;       // channels each CTA of the cluster finishes

  int issued = 0;  // stages the producer filled
  if (warp == kConsumers) {
    // ---- producer: one record and the block's token rows per stage
    const uint8_t* rec = p.w.data + ((static_cast<int64_t>(expert) * nt + tile) * KT + kt0) * L::REC;
    const __half* xrow = nullptr;
    if (lane < count && rows[lane] >= 0)
      xrow = p.x + static_cast<int64_t>(rows[lane] / p.div) * p.ldx + static_cast<int64_t>(kt0) * kW4K;
    const int live = __popc(__ballot_sync(0xffffffffu, xrow != nullptr));
    uint32_t stage = sbase, bar = full, phase = 1;
    for (int i = 0; i < n; ++i) {
      if (i >= L::STAGES && !w4_wait_warp(bar + 8 * L::STAGES, phase, budget, status, abort)) break;
      const uint32_t xbytes = tail && kt0 + i == KT - 1 ? 2 * tail : 2 * kW4K;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, L::REC + live * xbytes);
        bulk_load(stage, rec, L::REC, bar);
      }
      __syncwarp();
      if (xrow) {
        bulk_load(stage + L::X + lane * kTokenPitch, xrow, xbytes, bar);
        xrow += kW4K;
      }
      rec += L::REC;
      issued = i + 1;
      stage += L::STAGE;
      bar += 8;
      if (bar == full + 8 * L::STAGES) {
        stage = sbase;
        bar = full;
        phase ^= 1;
      }
    }
    if (slices > 1) {
      cluster_arrive();  // every CTA of the cluster runs: its shared memory may be written
      cluster_wait();
    }
  } else {
    // ---- consumers
    const int g = lane >> 2, t = lane & 3;
    const int kg = warp / kRowGroups;
    const int r0 = (warp % kRowGroups) * 32 + g;
    if (slices > 1) cluster_arrive();
    float acc[2][NB][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][b][j] = 0.0f;
    uint32_t s = kg, phase = 0;
    for (int i = kg; i < n; i += kKGroups) {
      if (!w4_wait_warp(full + 8 * s, phase, budget, status, abort)) break;
      const uint32_t stage = sbase + s * L::STAGE;
      if (tail && kt0 + i == KT - 1)
        consume<NB, G, ZERO, true>(stage, smem + s * L::STAGE, r0, lane, tail, acc);
      else
        consume<NB, G, ZERO, false>(stage, smem + s * L::STAGE, r0, lane, kW4K, acc);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * s);
      s += kKGroups;
      if (s >= L::STAGES) {
        s -= L::STAGES;
        phase ^= 1;
      }
    }
    // push the sums to the CTAs that finish these channels
    if (slices > 1) cluster_wait();
    const uint32_t src = (slice * kKGroups + kg) * share;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 16 * m + 8 * h;
        const int owner = static_cast<int>(r * share_inv >> 16);  // r / share
        uint32_t at = sbase + L::RED + ((src + r - owner * share) * L::BT + 2 * t) * 4;
        if (slices > 1) at = mapa_shared(at, owner);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (slices > 1)
            st_cluster_v2(at + 32 * b, acc[m][b][2 * h], acc[m][b][2 * h + 1]);
          else
            *reinterpret_cast<float2*>(smem + (at - sbase) + 32 * b) = make_float2(acc[m][b][2 * h], acc[m][b][2 * h + 1]);
        }
      }
  }
  __syncwarp();
  griddep_launch_dependents();
  if (slices > 1)
    cluster_sync_all();  // releases the pushes; nothing of this CTA is touched from outside after it
  else
    __syncthreads();
  if (*abort && warp == kConsumers) {
    // a wait ran out: let the copies in flight land before the CTA leaves
    for (int i = max(0, issued - L::STAGES); i < issued; ++i)
      mbar_drain(full + 8 * (i % L::STAGES), (i / L::STAGES) & 1, budget);
  }

  // Each CTA of the cluster finishes its share of the tile's channels.
  const float* red = reinterpret_cast<const float*>(smem + L::RED);
  const int64_t n0 = static_cast<int64_t>(tile) * kW4Rows + slice * share;
  const int64_t left = min(p.w.N - n0, static_cast<int64_t>(kW4Rows - slice * share));
  const int width = static_cast<int>(left < share ? left : share);
  const int sums = slices * kKGroups;
  for (int tk = warp; tk < count; tk += kConsumers + 1) {
    const int row = rows[tk];
    if (row < 0) continue;
    for (int r = lane; r < width; r += 32) {
      float v = 0.0f;
#pragma unroll 4
      for (int c = 0; c < sums; ++c) v = __fadd_rn(v, red[(c * share + r) * L::BT + tk]);
      if (p.bias) v = __fadd_rn(v, __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + n0 + r]));
      if (p.relu) v = v > 0.0f ? v : 0.0f;
      const int64_t o = static_cast<int64_t>(row) * p.w.N + n0 + r;
      if (p.y)
        p.y[o] = __float2half_rn(v);
      else
        p.y32[o] = v;
    }
  }
}

template <int NB, int G, bool ZERO>
cudaError_t launch(const W4Product& p, const Ctx& c) {
  using L = Layout<NB, G, ZERO>;
  auto kernel = k_w4_stream<NB, G, ZERO>;
  static KernelSetup setup;
  int per_sm = 0;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(kernel), kThreads, L::BYTES, c.device, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t nt = p.w.nt(), kt = p.w.kt();
  const int64_t blocks = w4_blocks(p, L::BT);
  const int slices = w4_slices(nt * blocks, kt, static_cast<int64_t>(c.num_sms) * per_sm, 6);
  // ceil(2^16 / share): r * share_inv >> 16 is r / share for every channel r < 128
  const uint32_t share = (kW4Rows + slices - 1) / slices, share_inv = (65536 + share - 1) / share;
  cudaLaunchConfig_t cfg = {};
  if (nt > 65535 || blocks * slices > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * slices), static_cast<unsigned>(nt));
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
  return cudaLaunchKernelEx(&cfg, kernel, p, slices, static_cast<int>(kt), static_cast<int>(nt), share_inv, c.status, c.budget_ns);
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

cudaError_t launch_w4_stream(const W4Product& p, const Ctx& c, int64_t tokens) {
  if (tokens <= 8) return launch_g<1>(p, c);
  return launch_g<2>(p, c);
}

int64_t w4_blocks(const W4Product& p, int bt) {
  const int64_t blocks = (p.M + bt - 1) / bt;
  if (!p.offsets) return blocks;
  return p.M < blocks + p.E ? p.M : blocks + p.E;
}

int w4_slices(int64_t units, int64_t kt, int64_t slots, int start_tiles) {
  int slices = 1;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= kMaxSlices && (s == 1 || kt / s >= 4); ++s) {
    const int64_t cost = ((units * s + slots - 1) / slots) * ((kt + s - 1) / s + start_tiles);
    if (cost < best) {
      best = cost;
      slices = s;
    }
  }
  return slices;
}

cudaError_t launch_w4_product(const W4Product& p, const Ctx& c) {
  // the tokens that share a weight tile: for experts the average
  const int64_t tokens = p.offsets ? (p.M + p.E - 1) / p.E : p.M;
  return tokens <= 8 ? launch_w4_stream(p, c, tokens) : launch_w4_gemm(p, c, tokens);
}

}  // namespace sq
