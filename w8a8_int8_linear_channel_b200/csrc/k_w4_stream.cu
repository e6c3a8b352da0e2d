// k_w4_stream.cu -- y = x W^T with a packed 4-bit W for few tokens: the weight
// is streamed once per eight tokens, and everything else is arranged around
// that stream.
//
//   y[m, n] = fp16( sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[m, k] + bias[n] )
//
// The 4-bit codes become fp16 integers q - z, exact, and go into
// mma.m16n8k16 with the weight as the 16-row operand and the tokens as the
// 8-column one (fp32 accumulators); a group's sum is multiplied by its scale
// once, in fp32, so no weight is ever rounded.
//
// Every warp is a stream of its own: it owns 32 channels and every second or
// fourth K tile of its CTA's slice, copies a tile's codes (2 KB, contiguous) and
// scales into a ring of its own in shared memory two tiles ahead, and shares
// nothing with other warps until the end: a lane reads back the codes that it
// copied itself.  With the same arithmetic behind a ring of bulk copies for the
// whole CTA, 100 more instructions per tile went into barriers and the producer.
//
// What bounds it is the issue of instructions: 271 per 32 channels x 128 k with
// everything, 181 of them arithmetic.  49152 x 12288 at one token takes 64.6 us
// = 4.8 TB/s (0.74 of the copy bandwidth; 47.9 us without the arithmetic), its
// schedulers 68% busy; 4096 x 4096 takes 5.0 us, most of it start and finish.
//
// A CTA owns 64 or 128 channels and a slice of K; the CTAs of a cluster own the
// slices of the same channels.  At the end every warp pushes its sums to the CTA of
// the cluster that finishes those channels (distributed shared memory), which
// adds them in a fixed order: no atomics, no workspace, the same bits on every
// run.
#include "../../include/sq.h"
#include "sq_w4.cuh"

namespace sq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTokens = 8;
constexpr int kMaxSlices = 8;  // portable cluster size

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

// The first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint4 ld_x(const __half* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A warp's own ring in shared memory, kDepth tiles deep: of every tile the
// codes of its 32 channels (as four 16-byte chunks per lane: what a lane copies
// it reads back itself), their scales and their zero points.
constexpr int kDepth = 3;
template <int G, bool ZERO>
struct Ring {
  static constexpr int NG = kW4K / G;
  static constexpr int SCALES = 32 * 64;
  static constexpr int ZEROS = SCALES + 32 * NG * 2;
  static constexpr int STAGE = ZEROS + (ZERO ? 32 * NG : 0);
  static constexpr int WARP = kDepth * STAGE;

  // Starts the copy of one tile; rows points at the warp's first channel's codes.
  static __device__ __forceinline__ void copy(uint32_t stage, const uint8_t* rec, int first, int lane, uint32_t code_at) {
#pragma unroll
    for (int j = 0; j < 4; ++j) cp_async16(stage + lane * 16 + j * 512, rec + code_at + j * 512);
    const uint8_t* s = rec + kW4CodeBytes + first * (NG * 2);
    if (lane < 4 * NG) cp_async16(stage + SCALES + lane * 16, s + lane * 16);
    if (ZERO) {
      const uint8_t* z = rec + kW4CodeBytes + kW4Rows * NG * 2 + first * NG;
      if (lane < 2 * NG) cp_async16(stage + ZEROS + lane * 16, z + lane * 16);
    }
  }
};

// The k of a tile's four steps that a lane holds of its token: 32 q + 8 t ...
// With TAIL only klen of the tile's k exist; a step past them reads the row's
// first k of the tile instead (some address that exists).
template <bool TAIL>
__device__ __forceinline__ uint4 ld_step(const __half* x, int q, int t, int klen) {
  return ld_x(!TAIL || 32 * q + 8 * t < klen ? x + 32 * q : x - 8 * t);
}

// One K tile.  xv holds this lane's token (a lane whose token slot is empty has
// some other token: its column goes nowhere); every step's registers are
// loaded again, for the next tile (at xnext), as soon as they have been used.
template <int G, bool ZERO, bool TAIL, bool NEXT_TAIL>
__device__ __forceinline__ void consume(const uint8_t* stage, int lane, uint4 (&xv)[4], const __half* xnext, int klen,
                                        float (&acc)[2][4]) {
  using R = Ring<G, ZERO>;
  constexpr int NG = R::NG;
  const int g = lane >> 2, t = lane & 3;
  if (TAIL) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (32 * q + 8 * t >= klen) xv[q] = make_uint4(0, 0, 0, 0);
  }
  uint4 codes[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) codes[j] = *reinterpret_cast<const uint4*>(stage + lane * 16 + j * 512);
  // channel r0 + 8 j of the tile is channel g + 8 j of the warp
  const __half* scales = reinterpret_cast<const __half*>(stage + R::SCALES) + g * NG;
  const uint8_t* zeros = stage + R::ZEROS + g * NG;
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    float part[2][4];
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = 0x64086408u, hi[j] = 0xD480D480u;  // z = 8: 1032, -72
      if (ZERO) {
        // 0x6400 | z is 1024 + z, twice; 960 less that is -(64 + z)
        lo[j] = zeros[8 * j * NG + gi] * 0x10001u + 0x64006400u;
        hi[j] = hsub2(0x63806380u, lo[j]);
      }
    }
#pragma unroll
    for (int q = gi * (G / 32); q < (gi + 1) * (G / 32); ++q) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a0[4], a1[4];
        const uint4 &c0 = codes[2 * m], &c1 = codes[2 * m + 1];
        dequant(q == 0 ? c0.x : q == 1 ? c0.y : q == 2 ? c0.z : c0.w, lo[2 * m], hi[2 * m], a0);
        dequant(q == 0 ? c1.x : q == 1 ? c1.y : q == 2 ? c1.z : c1.w, lo[2 * m + 1], hi[2 * m + 1], a1);
        if (q == gi * (G / 32))
          mma_f16_first(part[m], a0[0], a1[0], a0[1], a1[1], xv[q].x, xv[q].y);
        else
          mma_f16(part[m], a0[0], a1[0], a0[1], a1[1], xv[q].x, xv[q].y);
        mma_f16(part[m], a0[2], a1[2], a0[3], a1[3], xv[q].z, xv[q].w);
      }
      xv[q] = ld_step<NEXT_TAIL>(xnext, q, t, klen);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float s0 = __half2float(scales[16 * m * NG + gi]), s1 = __half2float(scales[(16 * m + 8) * NG + gi]);
      acc[m][0] = __fmaf_rn(s0, part[m][0], acc[m][0]);
      acc[m][1] = __fmaf_rn(s0, part[m][1], acc[m][1]);
      acc[m][2] = __fmaf_rn(s1, part[m][2], acc[m][2]);
      acc[m][3] = __fmaf_rn(s1, part[m][3], acc[m][3]);
    }
  }
}

// kRowGroups warps along the channels, 32 each, and the others along K.
template <int kRowGroups, int G, bool ZERO>
__global__ void __launch_bounds__(kThreads, 3)
    k_w4_stream(const W4Product p, int slices, int KT, int nt, int share_shift) {
  constexpr int kKGroups = kWarps / kRowGroups;
  constexpr int kRows = kRowGroups * 32, kParts = kW4Rows / kRows;  // channels per CTA, CTAs per weight tile
  using R = Ring<G, ZERO>;
  constexpr int REC = w4_record_bytes(G, ZERO);
  // sums of every slice and K group for the channels this CTA finishes:
  // [slices * kKGroups][kRows / slices][kTokens]
  extern __shared__ __align__(128) uint8_t smem[];  // every warp's ring
  __shared__ __align__(16) float red[kKGroups * kRows * kTokens];
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int slice = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.y) / kParts, part0 = static_cast<int>(blockIdx.y) % kParts * kRows;
  const int g = lane >> 2, t = lane & 3;
  const int kg = warp / kRowGroups, r0 = (warp % kRowGroups) * 32 + g;  // channel of this CTA's
  const int each = KT / slices, more = KT - each * slices;  // K tiles per slice, slices with one more
  const int kt0 = each * slice + min(slice, more);
  const int n = each + (slice < more ? 1 : 0);
  if (slices > 1) cluster_arrive();  // waited for before the pushes: every CTA of the cluster runs by then
  griddep_wait();

  const int block = static_cast<int>(cluster_id_x());
  // this lane's token: slot g of the block
  int expert = 0, start = 0, count, row = -1;
  if (p.offsets == nullptr) {
    const int64_t first = static_cast<int64_t>(block) * kTokens;
    count = static_cast<int>(p.M - first < kTokens ? p.M - first : kTokens);
    if (g < count) row = static_cast<int>(first) + g;
  } else {
    expert = w4_find_block(p, block, kTokens, lane, &start, &count);
    if (expert < 0) {  // there is no such block; the same for every CTA of the cluster
      if (slices > 1) cluster_wait();
      return;
    }
  }
  float acc[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = 0.0f;
  {
    const uint8_t* rec =
        p.w.data + ((static_cast<int64_t>(expert) * nt + tile) * KT + kt0 + kg) * static_cast<int64_t>(REC);
    // the CTA's last tile when it is short (its length: tail)
    const int tail = static_cast<int>(p.w.K) & (kW4K - 1);
    const int last = tail && kt0 + n == KT ? n - 1 : -1;
    // (the chunk's place is the same for r0, r0 + 8, r0 + 16, r0 + 24)
    const uint32_t code_at = (part0 + r0) * 64 + ((t ^ ((r0 >> 1) & 3)) << 4);
    uint8_t* ring = smem + warp * R::WARP;
    const uint32_t ring_at = smem_u32(ring);
    const int first = part0 + (warp % kRowGroups) * 32;
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) {
      if (kg + d * kKGroups < n) R::copy(ring_at + d * R::STAGE, rec + d * (kKGroups * REC), first, lane, code_at);
      cp_async_commit();
    }
    rec += (kDepth - 1) * (kKGroups * REC);
    // (which token: only after the weight's first tiles are on their way)
    if (p.offsets != nullptr && g < count) {
      const int32_t pair = p.order[start + g];
      if (pair >= 0 && pair < p.M) row = pair;
    }
    const int some = row < 0 ? 0 : p.div == 1 ? row : row / p.div;
    const __half* x = p.x + some * p.ldx + static_cast<int64_t>(kt0 + kg) * kW4K + 8 * t;
    int now = 0, ahead = (kDepth - 1) * R::STAGE;  // byte offsets of this tile's stage and of the one to fill
    uint4 xv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      xv[q] = make_uint4(0, 0, 0, 0);
      if (kg < n) xv[q] = kg == last ? ld_step<true>(x, q, t, tail) : ld_step<false>(x, q, t, 0);
    }
    for (int i = kg; i < n; i += kKGroups) {
      cp_async_wait<kDepth - 2>();
      __syncwarp();  // the other lanes' scales have landed too, and the stage to fill has been read
      if (i + (kDepth - 1) * kKGroups < n) R::copy(ring_at + ahead, rec, first, lane, code_at);
      cp_async_commit();
      rec += kKGroups * REC;
      if (i + kKGroups < n) x += kKGroups * kW4K;  // (the last tile loads itself again)
      if (i == last)
        consume<G, ZERO, true, true>(ring + now, lane, xv, x, tail, acc);
      else if (i + kKGroups == last)
        consume<G, ZERO, false, true>(ring + now, lane, xv, x, tail, acc);
      else
        consume<G, ZERO, false, false>(ring + now, lane, xv, x, 0, acc);
      now = now == (kDepth - 1) * R::STAGE ? 0 : now + R::STAGE;
      ahead = ahead == (kDepth - 1) * R::STAGE ? 0 : ahead + R::STAGE;
    }
  }
  griddep_launch_dependents();

  // push the sums to the CTAs that finish these channels
  const int share = 1 << share_shift;  // channels each CTA of the cluster finishes: kRows / slices
  if (slices > 1) cluster_wait();
  const uint32_t src = (slice * kKGroups + kg) * share;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 8 * j;
    const int owner = r >> share_shift;
    const uint32_t at = (src + (r & (share - 1))) * kTokens + 2 * t;
    const float a = acc[j >> 1][2 * (j & 1)], b = acc[j >> 1][2 * (j & 1) + 1];
    if (slices > 1)
      st_cluster_v2(mapa_shared(smem_u32(red + at), owner), a, b);
    else
      *reinterpret_cast<float2*>(red + at) = make_float2(a, b);
  }
  __syncwarp();
  if (slices > 1)
    cluster_sync_all();  // releases the pushes; nothing of this CTA is touched from outside after it
  else
    __syncthreads();

  // Each CTA of the cluster finishes its share of the tile's channels, a warp per token.
  const int out = __shfl_sync(0xffffffffu, row, 4 * warp);
  if (out < 0) return;
  const int64_t n0 = static_cast<int64_t>(tile) * kW4Rows + part0 + slice * share;
  const int64_t left = min(p.w.N - n0, static_cast<int64_t>(kRows - slice * share));
  const int width = static_cast<int>(left < share ? left : share);
  const int sums = slices * kKGroups;
  for (int r = lane; r < width; r += 32) {
    float v = 0.0f;
#pragma unroll 4
    for (int c = 0; c < sums; ++c) v = __fadd_rn(v, red[(c * share + r) * kTokens + warp]);
    if (p.bias) v = __fadd_rn(v, __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + n0 + r]));
    if (p.relu) v = v > 0.0f ? v : 0.0f;
    const int64_t o = static_cast<int64_t>(out) * p.w.N + n0 + r;
    if (p.y)
      p.y[o] = __float2half_rn(v);
    else
      p.y32[o] = v;
  }
}

// Slices of K (the cluster size, a power of two, so that the CTAs finish as many
// channels each), a K tile per warp at least: the fewest that give the shortest
// busiest SM.  CTAs on one SM share its issue slots, so their tiles add up (one
// CTA alone cannot fill them: it takes the time of one and a half); each
// costs 16 tiles' worth besides.  Clusters of more than two do not pack every
// SM.  With 1 / 2 / 4 slices 4096 x 4096 at one token takes 6.5 / 5.0 / 6.0 us, 8192 x
// 8192 13.9 / 12.0 / 14.6, 16384 x 4096 11.8 / 13.4 / 17.1, 12288 x 49152 (192
// CTAs) 85.1 / 65.5 / 67.2.
int pick_slices(int64_t ctas, int64_t kt, int k_groups, int num_sms) {
  int slices = 1;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= kMaxSlices && (s == 1 || s <= kt / k_groups); s *= 2) {
    const int64_t sms = s <= 2 ? num_sms : num_sms - num_sms / 8;
    const int64_t n = (ctas * s + sms - 1) / sms, tiles = (kt + s - 1) / s;
    const int64_t cost = (n == 1 ? 3 : 2 * n) * tiles + 32 * n;
    if (cost < best) best = cost, slices = s;
  }
  return slices;
}

template <int kRowGroups, int G, bool ZERO>
cudaError_t launch(const W4Product& p, const Ctx& c) {
  auto kernel = k_w4_stream<kRowGroups, G, ZERO>;
  constexpr int kKGroups = kWarps / kRowGroups, kRows = kRowGroups * 32;
  constexpr size_t smem = kWarps * Ring<G, ZERO>::WARP;
  static KernelSetup setup;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(kernel), smem, c.device);
  if (e != cudaSuccess) return e;
  const int64_t nt = p.w.nt(), kt = p.w.kt();
  const int64_t blocks = w4_blocks(p, kTokens), units = (p.w.N + kRows - 1) / kRows;
  // (experts: about a block each, if there are that many pairs)
  const int64_t likely = !p.offsets ? blocks : p.M < p.E ? p.M : p.E;
  const int slices = pick_slices(units * likely, kt, kKGroups, c.num_sms);
  int share_shift = kRowGroups == 2 ? 6 : 7;
  for (int s = slices; s > 1; s >>= 1) --share_shift;
  static_assert(kRows == (kRowGroups == 2 ? 64 : 128), "channels per CTA");
  static_assert(kRowGroups < 4 || SQ_W4_MAX_N <= 65535LL * kRows, "grid.y");
  if (units > 65535 || blocks * slices > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * slices), static_cast<unsigned>(units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, slices, static_cast<int>(kt), static_cast<int>(nt), share_shift);
}

template <int kRowGroups>
cudaError_t launch_g(const W4Product& p, const Ctx& c) {
  if (p.w.zero) {
    if (p.w.group == 32) return launch<kRowGroups, 32, true>(p, c);
    if (p.w.group == 64) return launch<kRowGroups, 64, true>(p, c);
    return launch<kRowGroups, 128, true>(p, c);
  }
  if (p.w.group == 32) return launch<kRowGroups, 32, false>(p, c);
  if (p.w.group == 64) return launch<kRowGroups, 64, false>(p, c);
  return launch<kRowGroups, 128, false>(p, c);
}

}  // namespace

cudaError_t launch_w4_stream(const W4Product& p, const Ctx& c) {
  // Two warps along the channels and four along K where CTAs are few (4096 x
  // 4096 at one token 5.0 us against 6.9), four and two where they fill the GPU several
  // times over (an expert layer of 32 tokens 164 us against 172).
  const int64_t likely = !p.offsets ? w4_blocks(p, kTokens) : p.M < p.E ? p.M : p.E;
  return p.w.nt() * likely >= 3 * c.num_sms ? launch_g<4>(p, c) : launch_g<2>(p, c);
}

int64_t w4_blocks(const W4Product& p, int bt) {
  const int64_t blocks = (p.M + bt - 1) / bt;
  if (!p.offsets) return blocks;
  return p.M < blocks + p.E ? p.M : blocks + p.E;
}

// Which kernel.  Up to eight tokens per weight tile always this one.  With
// more it reads the weight once per eight tokens, which still pays where an SM
// has little to do altogether (starting the tensor cores' pipeline takes 3 us
// longer): 1024 x 1024 at 64 tokens 3.5 us here, 9.9 there; 4096 x 4096 at 16
// tokens 7.0 and 9.1, at 24 10.2 and 9.0; 4096 x 16384 at 16 29.4 and 18.4.
// Experts' tokens scatter around the average (most of them still need one
// block of eight): 64 experts with 10 tokens each 207 us a layer here and 222
// there, with 12 242 and 217; 256 small experts with 10 122 and 129, with 16
// 162 and 130.  The average is all the host knows.  Where the load is uneven this kernel
// still holds (64 experts, 640 pairs, half of them on one: a product of 2048 x 4096 91 us here,
// 99 there), until nearly all pairs meet one expert, whose weight it then reads once per eight (all of them on one:
// 73 and 37; 512 experts of 512 x 2048, 4096 pairs: evenly 115 and 118, all on one 82 and 52).
constexpr int kTilesPerSm = 32;    // 64 channels x 128 k x eight tokens
constexpr int kTokensExperts = 10;

cudaError_t launch_w4_product(const W4Product& p, const Ctx& c) {
  // the tokens that share a weight tile: for experts the average
  const int64_t tokens = p.offsets ? (p.M + p.E - 1) / p.E : p.M;
  const int64_t work = w4_blocks(p, kTokens) * 2 * p.w.nt() * p.w.kt();  // 64-channel K tiles
  const bool stream = tokens <= kTokens || (p.offsets ? tokens <= kTokensExperts : work <= kTilesPerSm * c.num_sms);
  return stream ? launch_w4_stream(p, c) : launch_w4_gemm(p, c, tokens);
}

}  // namespace sq
