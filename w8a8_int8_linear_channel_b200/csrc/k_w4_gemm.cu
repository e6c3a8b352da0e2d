// k_w4_gemm.cu -- y = x W^T with a packed 4-bit W on the 5th-generation tensor
// cores, for more tokens than k_w4_stream.cu takes.
//
// Swap-AB: the MMA's 128-row M slot takes 128 output channels, its N slot the
// tokens.  The weight operand is made on the fly: a thread per channel turns
// codes into fp16 numbers (q - z) * s in registers and stores them to tensor
// memory, from where tcgen05.mma reads its A operand; the tokens (B) are
// staged in shared memory.  A weight made by the library's quantizer is
// exactly an fp16 number, so nothing is rounded before the fp32 accumulators
// (a scale of more than 8 significant bits, 7 with zero points, costs one fp16
// rounding per weight, and (q - z) * s past 65504 is Inf).
//
// Why tensor memory: writing the 32 KB of a dequantized 128 x 128 tile to
// shared memory and reading it back as the MMA's operand would take twice the
// shared-memory bandwidth that a tile's time leaves.
//
// Roles: eight or sixteen dequantization warps (also the epilogue), one MMA
// issuer, one producer of records (bulk copies), and for the token rows one
// TMA producer, or four warps of cp.async where an expert's rows lie scattered.
// All waits are bounded.
//
// 16384 x 4096 at 2048 tokens: 211 us, 1.30 PFLOP/s (0.77 of the measured matrix
// product).  Of a CTA of 32 K tiles, about 49,000 cycles, some 4500 pass until its
// first MMA (which block, tensor memory, a record's latency, the first
// operand), 1240 per K tile (1024 for the MMAs at full rate; 1160 are left with 14
// tokens: the chain of record, operand, MMA and release) and 4700 from the last MMA to
// its end; with one CTA per SM nothing covers the two ends.  For few tokens
// the chain per K tile is all: 4096 x 16384 at 16 tokens 18.4 us.
//
// Tensor memory is not waited for among this kernel's CTAs: one takes 256 columns
// and its shared memory lets two of them share an SM, or 512 and one.  Beside the INT8
// products' CTAs (over 190 KB of shared memory) none of them fits.
#include "sq_tmap.h"
#include "sq_w4.cuh"

namespace sq {
namespace {

constexpr int kMaxSlices = 8;
constexpr int kACols = kW4K / 2;  // 32-bit TMEM columns of one 128 x 128 fp16 operand

// One lane of the warp (the same on every call).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands, fp32 accumulate, issued by
// the lane with `leader` set.  The whole warp runs the issuing code, so its
// operands stay in uniform registers: inside an `if (lane == 0)` an MMA of 16
// tokens took 44 cycles to issue, this way 9 (32 tokens 16, 64 tokens 32: the
// tensor core's own rate).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc,
                                           uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}

// kind::f16, fp16 A and B (both K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Thread i of the warp stores 16 registers to columns [col, col + 16) of TMEM
// lane (lane base + i).
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Of registers that a load from tensor memory is writing.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Columns [col, col + 16) of the warp's lanes, complete on return.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
  tmem_ld_32x32b_x16(taddr, r);
  tmem_ld_wait(r);
}

// 16 lanes x 32 columns; register 4 i + j of thread t: lane t / 4 (+ 8 for j = 2, 3), column 8 i + 2 (t % 4) + (j & 1).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Four 8 x 8 matrices of fp16, as mma fragments hold them, stored transposed:
// the lane's address is that of one row of eight.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2_rn(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 bytes global -> shared, or 16 zero bytes when `bytes` is 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrive on `bar` (one of its expected arrivals) when this thread's copies so
// far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// BT tokens and RT weight tiles (128 channels each) per CTA.
template <int BT, int RT, int G, bool ZERO>
struct Layout {
  static constexpr int DEQ = RT == 2 ? 16 : 8;  // dequantization warps: RT weight tiles x even / odd K tiles
  static constexpr int MMA_WARP = DEQ, REC_WARP = DEQ + 1, X_WARP = DEQ + 2;
  static constexpr int X_THREADS = 128;  // of the cp.async form
  static constexpr int THREADS = X_WARP * 32 + X_THREADS;
  static constexpr int REC = w4_record_bytes(G, ZERO);
  // boxes of [BT][64 k] per token stage, 128-byte swizzle (with 128 tokens and half
  // the memory two stages of two boxes took 29.3 us where four of one take 23.4, 16384 x 4096)
  static constexpr int XB = BT == 128 && RT == 1 ? 1 : 2;
  static constexpr int SPT = 2 / XB;                       // token stages per K tile
  static constexpr int XSTAGE = XB * BT * 128;
  static constexpr int XS = 4;                            // token stages
  static constexpr int RS = 4;                            // record stages, RT records each
  static constexpr int AS = RT == 2 || BT == 128 ? 2 : 3;  // operand buffers in tensor memory
  static constexpr int D_COLS = RT * BT;
  static constexpr int A0 = D_COLS;
  static constexpr int TMEM_COLS = RT == 2 ? 512 : 256;
  static constexpr int RED_PITCH = BT + 4;
  static constexpr int RED_BYTES = (kW4Rows + kMaxSlices) * RED_PITCH * 4;
  // the cluster's sums reuse the token stages: by then every MMA has read them
  static constexpr int X = 0;
  static constexpr int R = X + (XS * XSTAGE > RED_BYTES || RT == 2 ? XS * XSTAGE : (RED_BYTES + 1023) / 1024 * 1024);
  static constexpr int BARS = R + RS * RT * REC;
  static constexpr int NBARS = 2 * XS + 2 * RS + AS + 1;
  static constexpr int XROW = BARS + (NBARS * 8 + 15) / 16 * 16;  // int32 [BT]: x row of every token, -1 none
  static constexpr int YROW = XROW + BT * 4;                      // int32 [BT]: y row, -1 none
  static constexpr int MISC = YROW + BT * 4;                      // abort, TMEM address, expert, count
  static constexpr int BYTES = MISC + 16 + 1024;                  // alignment slack
  static_assert(D_COLS + AS * RT * kACols <= TMEM_COLS, "tensor memory");
  // The parity of a barrier's phase tells two successive uses of a stage
  // apart, not three.  A group of warps (K tiles of one parity) that asks for
  // tile j has seen the MMAs of tile j - 2 - AS done, so that tile had landed;
  // tile j - RS, the stage's use before, must not be a later one, unless it is
  // the same group's (RS even).
  static_assert(RS % 2 == 0 || RS >= AS + 2, "a wait could take the phase before the last for its own");
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static_assert(BT * (RT * kW4Rows * 4 + 16) <= BARS, "the staged output tile");
  static_assert(RT == 2 || (3 * (BYTES + 1024) > 233472 && 2 * (BYTES + 1024) <= 233472), "two CTAs per SM");
  static_assert(RT == 1 || 2 * (BYTES + 1024) > 233472, "one CTA per SM");
};

template <int BT, int RT, int G, bool ZERO>
__global__ void __launch_bounds__(Layout<BT, RT, G, ZERO>::THREADS, RT == 2 ? 1 : 2)
    k_w4_gemm(const __grid_constant__ CUtensorMap tmX, const W4Product p, int nslices, int blocks, int KT,
              uint32_t* status, uint64_t budget) {
  using L = Layout<BT, RT, G, ZERO>;
  constexpr int NG = kW4K / G;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + L::MISC);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + L::MISC);
  int32_t* xrow = reinterpret_cast<int32_t*>(smem + L::XROW);
  int32_t* yrow = reinterpret_cast<int32_t*>(smem + L::YROW);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const int slices = RT == 2 ? 1 : nslices;
  const int slice = blockIdx.x % slices;
  const int block = blockIdx.x / slices % blocks;
  const int tile = blockIdx.x / slices / blocks * RT;  // first weight tile
  // done: the MMAs of a token stage have run (the last one of a K tile frees the
  // operand buffer too: a buffer's tile is AS tiles back, and by then the stage
  // is at most one use further)
  const uint32_t x_full = sbase + L::BARS, done = x_full + 8 * L::XS;
  const uint32_t r_full = done + 8 * L::XS, r_empty = r_full + 8 * L::RS;
  const uint32_t a_full = r_empty + 8 * L::RS, d_full = a_full + 8 * L::AS;

  const int kt0 = KT * slice / slices, n = KT * (slice + 1) / slices - kt0;  // this CTA's K tiles
  const int64_t nt = p.w.nt();

  // Until the first MMA a CTA waits for three latencies in a row (which expert,
  // its records, the operand made of them); what can go beside them does:
  // one warp sets up the barriers, finds the block and sends for its first
  // records, while another takes tensor memory and the last ones look up the rows.
  // (the record of weight tile t and K tile i, to be counted on its stage's barrier)
  auto load_record = [&](int expert, int i, uint32_t rs, int t) {
    // the last weight tile may stand alone: its place is taken by itself
    // again, and nothing of the copy is written out
    const int64_t wt = tile + t < nt ? tile + t : nt - 1;
    bulk_load(sbase + L::R + (rs * RT + t) * L::REC,
              p.w.data + ((static_cast<int64_t>(expert) * nt + wt) * KT + kt0 + i) * L::REC, L::REC, r_full + 8 * rs);
  };
  const int early = n < L::RS ? n : L::RS;
  if (warp == L::REC_WARP) {
    for (int i = lane; i < L::NBARS; i += 32) {
      uint32_t arrivals = 1;
      if (i < L::XS) arrivals = p.offsets ? L::X_THREADS : 1;                             // x_full
      if (i >= 2 * L::XS + L::RS && i < L::NBARS - 1) arrivals = RT == 2 ? 8 : 4;       // r_empty, a_full
      mbar_init(sbase + L::BARS + 8 * i, arrivals);
    }
    if (lane == 0) *abort = 0;
    fence_barrier_init();
    __syncwarp();
  }
  if (warp == L::MMA_WARP) {
    tmem_alloc(smem_u32(misc + 1), L::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  if (warp == L::REC_WARP) {
    int expert = 0, start = block * BT, count = BT;
    if (p.offsets == nullptr)
      count = static_cast<int>(p.M - start < BT ? p.M - start : BT);
    else
      expert = w4_find_block(p, block, BT, lane, &start, &count);
    if (lane == 0) misc[2] = expert, misc[3] = count;
    if (lane < early && expert >= 0) mbar_arrive_expect_tx(r_full + 8 * lane, RT * L::REC);
    __syncwarp();
    if (lane < early * RT && expert >= 0) load_record(expert, lane / RT, lane / RT, lane % RT);
    __syncwarp();
  } else if (warp >= L::X_WARP) {
    // the block's rows (every warp finds the block for itself)
    int start = block * BT, count = BT;
    if (p.offsets == nullptr)
      count = static_cast<int>(p.M - start < BT ? p.M - start : BT);
    else if (w4_find_block(p, block, BT, lane, &start, &count) < 0)
      count = 0;
    for (int i = tid - L::X_WARP * 32; i < BT; i += L::X_THREADS) {
      int32_t row = i >= count ? -1 : p.offsets ? p.order[start + i] : start + i;
      if (row < 0 || row >= p.M) row = -1;
      yrow[i] = row;
      xrow[i] = row < 0 ? -1 : p.div == 1 ? row : row / p.div;
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  const int expert = misc[2], count = misc[3];
  if (expert < 0) {  // there is no such block; the same for every CTA of the cluster
    if (warp == L::MMA_WARP) tmem_dealloc(tmem, L::TMEM_COLS);
    return;
  }

  if (warp < L::DEQ) {
    // ---- dequantization: thread = channel; a group of four warps takes weight
    // tile t and the K tiles of one parity
    const int t = RT == 2 ? (warp >> 2) & 1 : 0;
    const int parity = warp >> (RT == 2 ? 3 : 2);
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    // stage and buffer counters in steps of two tiles
    uint32_t rs = parity, rp = 0, as = parity;
    for (int i = parity; i < n; i += 2) {
      if (!w4_wait_warp(r_full + 8 * rs, rp, budget, status, abort)) break;
      const int rec = L::R + (rs * RT + t) * L::REC;
      uint4 c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = lds128(sbase + rec + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
      uint32_t s2[NG], z[NG];
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const uint32_t s = *reinterpret_cast<const uint16_t*>(smem + rec + kW4CodeBytes + (r * NG + j) * 2);
        s2[j] = s | s << 16;
        z[j] = ZERO ? smem[rec + kW4CodeBytes + kW4Rows * NG * 2 + r * NG + j] : 8u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(r_empty + 8 * rs);
      const uint32_t col = tmem + L::A0 + (as * RT + t) * kACols + lanes;
      auto values = [&](int w, uint32_t (&v)[16]) {
        const int j = w / (G / 32);
        const uint32_t lo = 0x64006400u | z[j] | z[j] << 16, hi = 0xD400D400u | z[j] << 4 | z[j] << 20;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t h[4];
          dequant(w == 0 ? c[q].x : w == 1 ? c[q].y : w == 2 ? c[q].z : c[q].w, lo, hi, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = hmul2(h[e], s2[j]);
        }
      };
      // Half of the values are made before the buffer is free, so that the MMAs
      // of the tile before (1070 cycles with 128 tokens and two weight tiles) cover the other half.
      uint32_t v0[16], v1[16];
      values(0, v0);
      values(1, v1);
#pragma unroll
      for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(v0[e]), "+r"(v1[e]));  // (not sunk below the wait)
      // the tile that used this buffer before
      const int b = i - L::AS;
      const int bs = b * L::SPT + L::SPT - 1;  // its last stage
      if (b >= 0 && !w4_wait_warp(done + 8 * (bs % L::XS), (bs / L::XS) & 1, budget, status, abort)) break;
      tc_fence_after();
      tmem_st_x16(col, v0);
      tmem_st_x16(col + 16, v1);
      values(2, v0);
      tmem_st_x16(col + 32, v0);
      values(3, v1);
      tmem_st_x16(col + 48, v1);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full + 8 * as);
      if ((rs += 2) >= L::RS) rs -= L::RS, rp ^= 1;
      if ((as += 2) >= L::AS) as -= L::AS;
    }
  } else if (warp == L::MMA_WARP) {
    // ---- MMA issue (see mma_f16_ts: the whole warp, one lane elected)
    // (a block that is not full, the last one of an expert or of all tokens, takes
    // as many columns as it has tokens, in sixteens)
    const uint32_t idesc = idesc_f16(kW4Rows, (count + 15) & ~15);
    const uint32_t leader = elect_one();
    const uint64_t desc0 = sdesc_k_sw128(sbase + L::X);
    const bool short_tail = p.w.K - static_cast<int64_t>(kt0 + n - 1) * kW4K <= 64;  // one box in the last tile
    const int steps = 2 * n - (short_tail ? 1 : 0);  // boxes of 64 k
    uint32_t xs = 0, as = 0, xp = 0, ap = 0;
    bool ready = false;  // the stage's operands were seen to be there while the stage before was being issued
    for (int i = 0; i < steps; i += L::XB) {
      if (!ready) {
        if ((L::XB == 2 || !(i & 1)) && !w4_wait_warp(a_full + 8 * as, ap, budget, status, abort)) break;
        if (!w4_wait_warp(x_full + 8 * xs, xp, budget, status, abort)) break;
      }
      tc_fence_after();
      if (p.offsets) fence_proxy_async_smem();  // cp.async rows, visible to this thread, to the MMA's reads
      const uint64_t b0 = desc0 + xs * (L::XSTAGE >> 4);
      const uint32_t a0 = tmem + L::A0 + as * (RT * kACols) + (L::XB == 1 && (i & 1) ? 32 : 0), mine = done + 8 * xs;
      if (++xs == L::XS) xs = 0, xp ^= 1;
      const bool last = L::XB == 2 || (i & 1);  // of the K tile
      if (last && ++as == L::AS) as = 0, ap ^= 1;
#pragma unroll
      for (int j = 0; j < 4 * L::XB; ++j) {
        if (j == 4 && i + 1 >= steps) break;  // (the A columns past K are zero, the B rows were not copied)
        const uint64_t b = b0 + (((j >> 2) * BT * 128 + (j & 3) * 32) >> 4);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          mma_f16_ts(tmem + t * BT, a0 + t * kACols + 8 * j, b, idesc, i > 0 || j > 0, leader);
        if (j == 4 * L::XB - 2)
          ready = __all_sync(0xffffffffu, i + L::XB < steps && (!last || mbar_try_wait(a_full + 8 * as, ap)) &&
                                              mbar_try_wait(x_full + 8 * xs, xp));
      }
      if (leader) mma_commit(mine);
    }
    if (leader) mma_commit(d_full);  // also after a wait that ran out: nothing in flight is left behind
  } else if (warp == L::REC_WARP) {
    // ---- record producer
    int issued = lane == 0 ? early : 0;  // (the other lanes wait for nothing)
    for (int i = early; i < n && lane == 0; ++i) {
      const uint32_t rs = i % L::RS;
      if (!w4_wait(r_empty + 8 * rs, (i / L::RS & 1) ^ 1, budget, status, abort)) break;
      mbar_arrive_expect_tx(r_full + 8 * rs, RT * L::REC);
#pragma unroll
      for (int t = 0; t < RT; ++t) load_record(expert, i, rs, t);
      issued = i + 1;
    }
    // records in flight land before the CTA can leave (at once unless a wait ran out)
    for (int i = max(0, issued - L::RS); i < issued; ++i)
      mbar_drain(r_full + 8 * (i % L::RS), (i / L::RS) & 1, budget);
  } else if (p.offsets == nullptr) {
    // ---- token rows of one matrix: TMA; rows past M and k past K read as zero
    if (warp == L::X_WARP && lane == 0) {
      int issued = 0;
      uint32_t xs = 0, xp = 1;
      for (int i = 0; i < n * L::SPT; ++i) {
        const int32_t k = kt0 * kW4K + i * (64 * L::XB);
        // a box of a short last tile may lie past K altogether: it is left
        // out, and so are its MMAs
        const int64_t left = p.w.K - k;
        if (left <= 0) break;
        if (!w4_wait(done + 8 * xs, xp, budget, status, abort)) break;
        const uint32_t stage = sbase + L::X + xs * L::XSTAGE, bar = x_full + 8 * xs;
        const int boxes = L::XB == 2 && left > 64 ? 2 : 1;
        mbar_arrive_expect_tx(bar, boxes * (BT * 128));
        for (int b = 0; b < boxes; ++b) tma_load_2d(stage + b * (BT * 128), &tmX, bar, k + 64 * b, block * BT);
        issued = i + 1;
        if (++xs == L::XS) xs = 0, xp ^= 1;
      }
      // copies in flight land before the CTA can leave (at once unless a wait ran out)
      for (int i = max(0, issued - L::XS); i < issued; ++i)
        mbar_drain(x_full + 8 * (i % L::XS), (i / L::XS) & 1, budget);
    }
  } else {
    // ---- an expert's token rows: 16 (8) lanes copy a row's 128 (64) k of a stage; each
    // thread's arrival fires when its copies have landed, so the ring fills ahead
    constexpr int LANES = 8 * L::XB, ROWS = L::X_THREADS / LANES;
    const int lt = tid - L::X_WARP * 32;
    const int c = lt & (LANES - 1), r0 = lt / LANES;
    const uint32_t at = static_cast<uint32_t>(c >> 3) * (BT * 128) + r0 * 128 + (((c & 7) ^ (r0 & 7)) << 4);
    const __half* src[BT / ROWS];  // rows r0 + ROWS j: row & 7 does not depend on j
    uint32_t live = 0;
#pragma unroll
    for (int j = 0; j < BT / ROWS; ++j) {
      const int32_t xr = xrow[r0 + ROWS * j];
      if (xr >= 0) live |= 1u << j;
      src[j] = p.x + static_cast<int64_t>(xr >= 0 ? xr : 0) * p.ldx + static_cast<int64_t>(kt0) * kW4K + 8 * c;
    }
    int left = static_cast<int>(p.w.K) - kt0 * kW4K - 8 * c;
    uint32_t xs = 0, xp = 1;
    for (int i = 0; i < n * L::SPT && left + 8 * c > 0; ++i) {
      if (!w4_wait_warp(done + 8 * xs, xp, budget, status, abort)) break;
      const uint32_t dst = sbase + L::X + xs * L::XSTAGE + at;
      const uint32_t mask = left > 0 ? live : 0;  // past K: zeros, and no address is read
#pragma unroll
      for (int j = 0; j < BT / ROWS; ++j) {
        if (ROWS * j >= count) break;  // rows that no MMA reads but the last sixteen's rest, whose columns go nowhere
        const bool on = mask >> j & 1;
        cp_async16(dst + j * (ROWS * 128), on ? src[j] : p.x, on ? 16 : 0);
        src[j] += 64 * L::XB;
      }
      left -= 64 * L::XB;
      cp_async_arrive(x_full + 8 * xs);
      if (++xs == L::XS) xs = 0, xp ^= 1;
    }
    cp_async_wait_all();
  }
  __syncwarp();

  // ---- epilogue
  // The warps that read the sums wait for the last MMAs.  If that wait or one before
  // it ran out, the status word says so and this CTA stores nothing; the MMAs that
  // were issued are waited for all the same, since they still read shared memory.
  if (warp < L::DEQ && !w4_wait_warp(d_full, 0, budget, status, abort)) mbar_drain(d_full, 0, budget);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool ok = *abort == 0;  // the same in every warp: no wait follows
  griddep_launch_dependents();
  if (slices > 1) {
    cluster_sync_all();  // the token stages of every CTA are free
    // the cluster's sum needs every slice
    if (!ok && tid < slices) st_cluster_u32(mapa_shared(smem_u32(misc), tid), 1);
  }
  // Without slices a tile goes out through shared memory (every stage is free
  // by now), so that a warp writes 512 consecutive bytes of a row; written
  // from the accumulators' own layout, 32 channels of one token per store, a
  // 128 x 256 tile took 5.5 us.
  const int es = p.y ? 2 : 4;
  const bool staged = slices == 1 && (p.w.N * es) % 16 == 0;
  const uint32_t pitch = RT * kW4Rows * es + 16;
  if (ok && staged && p.y && warp < L::DEQ) {
    // fp16: fragments of 8 channels x 8 tokens, rounded and stored transposed
    // (2048 x 16384 x 4096: 212 us, one value at a time 219)
    const int t = RT == 2 ? (warp >> 2) & 1 : 0;
    const int c0 = (warp >> (RT == 2 ? 3 : 2)) * (BT / 2), c1 = c0 + BT / 2;
    const uint32_t d = tmem + t * BT + (static_cast<uint32_t>(warp & 3) << 21);
    float bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t ch = static_cast<int64_t>(tile + t) * kW4Rows + (warp & 3) * 32 + (lane >> 2) + 8 * j;
      bias[j] = p.bias && ch < p.w.N ? __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + ch]) : 0.0f;
    }
    // lane l's row: token l % 8 of the fragment, channels 8 (l / 8) ..
    const uint32_t at = sbase + (lane & 7) * pitch + (t * kW4Rows + (warp & 3) * 32 + (lane >> 3) * 8) * 2;
    for (int col = c0; col < c1; col += 32) {
      if (col >= count) break;
      __syncwarp();
      uint32_t v[2][16];
      tmem_ld_16x256b_x4(d + col, v[0]);
      tmem_ld_16x256b_x4(d + col + (16u << 16), v[1]);
      tmem_ld_wait(v[0]);
      tmem_ld_wait(v[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo = __uint_as_float(v[j >> 1][4 * i + 2 * (j & 1)]), hi = __uint_as_float(v[j >> 1][4 * i + 2 * (j & 1) + 1]);
          if (p.bias) lo = __fadd_rn(lo, bias[j]), hi = __fadd_rn(hi, bias[j]);
          if (p.relu) lo = lo > 0.0f ? lo : 0.0f, hi = hi > 0.0f ? hi : 0.0f;
          const __half2 h = __floats2half2_rn(lo, hi);
          m[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        stmatrix_x4_trans(at + (col + 8 * i) * pitch, m[0], m[1], m[2], m[3]);
      }
    }
  } else if (ok && warp < L::DEQ) {
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const int t = RT == 2 ? (warp >> 2) & 1 : 0;
    const int c0 = (warp >> (RT == 2 ? 3 : 2)) * (BT / 2), c1 = c0 + BT / 2;
    const int64_t ch = static_cast<int64_t>(tile + t) * kW4Rows + r;
    float bias = 0.0f;
    if (p.bias && ch < p.w.N) bias = __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + ch]);
    const int share = (kW4Rows + slices - 1) / slices;
    constexpr int STEP = 16;
    for (int col = c0; col < c1; col += STEP) {
      if (col >= count) break;  // no token of this block lies there
      __syncwarp();
      uint32_t v[STEP];
      tmem_ld_cols(tmem + t * BT + col + lanes, v);
      if (slices > 1) {
        const int owner = r / share;
        const uint32_t at =
            mapa_shared(sbase + ((slice * share + r - owner * share) * L::RED_PITCH + col) * 4, owner);
#pragma unroll
        for (int j = 0; j < STEP; j += 4) {
          st_cluster_v4(at + j * 4, __uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                        __uint_as_float(v[j + 3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
          float f = __uint_as_float(v[j]);
          if (p.bias) f = __fadd_rn(f, bias);
          if (p.relu) f = f > 0.0f ? f : 0.0f;
          if (staged) {
            *reinterpret_cast<float*>(smem + (col + j) * pitch + (t * kW4Rows + r) * 4) = f;
          } else {
            const int32_t row = yrow[col + j];
            if (row < 0 || ch >= p.w.N) continue;
            const int64_t o = static_cast<int64_t>(row) * p.w.N + ch;
            if (p.y)
              p.y[o] = __float2half_rn(f);
            else
              p.y32[o] = f;
          }
        }
      }
    }
  }
  if (ok && staged) {
    __syncthreads();
    // 16-byte pieces; a row's pieces go to consecutive lanes
    const int per = RT * kW4Rows * es / 16;  // a power of two
    const int shift = __ffs(per) - 1;
    uint8_t* out = p.y ? reinterpret_cast<uint8_t*>(p.y) : reinterpret_cast<uint8_t*>(p.y32);
    const int64_t row_bytes = p.w.N * es, first = static_cast<int64_t>(tile) * kW4Rows * es;
    for (int i = tid; i < count << shift; i += L::THREADS) {
      const int tk = i >> shift, c = (i & (per - 1)) * 16;
      const int32_t row = yrow[tk];
      if (row < 0 || first + c >= row_bytes) continue;
      *reinterpret_cast<uint4*>(out + row * row_bytes + first + c) = *reinterpret_cast<const uint4*>(smem + tk * pitch + c);
    }
  }
  __syncwarp();
  if (slices > 1) {
    cluster_sync_all();  // releases the pushes; nothing of this CTA is touched from outside after it
    const int share = (kW4Rows + slices - 1) / slices;
    const float* red = reinterpret_cast<const float*>(smem);
    const int64_t n0 = static_cast<int64_t>(tile) * kW4Rows + slice * share;
    const int64_t left = min(p.w.N - n0, static_cast<int64_t>(kW4Rows - slice * share));
    const int width = static_cast<int>(left < share ? left : share);
    const int todo = *abort == 0 ? width * count : 0;
    for (int i = tid; i < todo; i += L::THREADS) {
      const int tk = i / width, q = i - tk * width;
      const int32_t row = yrow[tk];
      if (row < 0) continue;
      float f = 0.0f;
#pragma unroll 4
      for (int s = 0; s < slices; ++s) f = __fadd_rn(f, red[(s * share + q) * L::RED_PITCH + tk]);
      if (p.bias) f = __fadd_rn(f, __half2float(p.bias[static_cast<int64_t>(expert) * p.w.N + n0 + q]));
      if (p.relu) f = f > 0.0f ? f : 0.0f;
      const int64_t o = static_cast<int64_t>(row) * p.w.N + n0 + q;
      if (p.y)
        p.y[o] = __float2half_rn(f);
      else
        p.y32[o] = f;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == L::MMA_WARP) tmem_dealloc(tmem, L::TMEM_COLS);
}

// Slices of K per weight tile (the cluster size).  A CTA's time is taken as
// 0.39 us per K tile (0.59 with 128 tokens), 4.5 for start and finish and 4 more
// for the cluster's sum (4096 x 4096 at 64 tokens: 15.7 us with one slice, 14.6 with
// two, 10.8 with four; 4096 x 16384 at 16: two 30.5, four 18.6, eight 17.8, four chosen).
// Two CTAs on an SM overlap their tiles, hardly the rest: 4096 x 4096 at 384 tokens
// takes 19.8 us with one slice, 29.0 with two.  Clusters of more than two do not
// pack every SM of a GPC; an eighth is taken off (4096 x 16384 at 384 tokens with
// one / two / three slices 67.8 / 64.4 / 75.3 us).
int pick_slices(int64_t units, int64_t kt, int bt, int num_sms) {
  int slices = 1;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= kMaxSlices && (s == 1 || kt / s >= 4); ++s) {
    const int64_t sms = s <= 2 ? num_sms : num_sms - num_sms / 8;
    const int64_t per_sm = (units * s + sms - 1) / sms;
    const int64_t cost = (per_sm + 1) / 2 * ((kt + s - 1) / s) * (bt == 64 ? 39 : 59) + per_sm * (s == 1 ? 450 : 850);
    if (cost < best) best = cost, slices = s;
  }
  return slices;
}

template <int BT, int RT, int G, bool ZERO>
cudaError_t launch(const W4Product& p, const Ctx& c) {
  using L = Layout<BT, RT, G, ZERO>;
  auto kernel = k_w4_gemm<BT, RT, G, ZERO>;
  static KernelSetup setup;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(kernel), L::BYTES, c.device);
  if (e != cudaSuccess) return e;
  CUtensorMap tm = {};
  if (!p.offsets && !make_tmap_f16_rows(&tm, p.x, p.M, p.w.K, p.ldx, BT)) return cudaErrorUnknown;
  const int64_t tiles = (p.w.nt() + RT - 1) / RT, kt = p.w.kt();
  const int64_t blocks = w4_blocks(p, BT);
  const int slices = RT == 1 ? pick_slices(tiles * blocks, kt, BT, c.num_sms) : 1;
  if (tiles * blocks * slices > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * blocks * slices));
  cfg.blockDim = dim3(L::THREADS);
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
  return cudaLaunchKernelEx(&cfg, kernel, tm, p, slices, static_cast<int>(blocks), static_cast<int>(kt), c.status,
                            c.budget_ns);
}

template <int BT, int RT>
cudaError_t launch_g(const W4Product& p, const Ctx& c) {
  if (p.w.zero) {
    if (p.w.group == 32) return launch<BT, RT, 32, true>(p, c);
    if (p.w.group == 64) return launch<BT, RT, 64, true>(p, c);
    return launch<BT, RT, 128, true>(p, c);
  }
  if (p.w.group == 32) return launch<BT, RT, 32, false>(p, c);
  if (p.w.group == 64) return launch<BT, RT, 64, false>(p, c);
  return launch<BT, RT, 128, false>(p, c);
}

}  // namespace

cudaError_t launch_w4_gemm(const W4Product& p, const Ctx& c, int64_t tokens) {
  // Blocks of 64 tokens or 128.  A block's MMAs are only as wide as it has
  // tokens, so narrower blocks would save nothing (16384 x 4096 at 16 tokens took
  // the same with blocks of 16, 32 or 64).  An expert's tokens scatter around the
  // average, and a second block makes its weight's operand once more: 64 experts
  // with 12 tokens each, blocks of 64 / 128: 217 / 219 us a layer, with 20 230 /
  // 227, with 32 249 / 236 (blocks of 16 with 12 tokens a fifth more than of 64).
  if (tokens <= (p.offsets ? 16 : 64)) return launch_g<64, 1>(p, c);
  // One weight tile per CTA and two CTAs per SM, or two tiles and one CTA, which
  // halves the token traffic: 16384 x 4096 at 2048 tokens 223 and 213 us (a large
  // CTA 0.95 of two small ones), for experts, whose rows come without TMA,
  // 506 and 419 us a layer of 1024 tokens.  But 384 tokens, 192 large CTAs, take 57.3
  // us and 384 small ones 47.8; and where large CTAs would not cover the SMs only
  // small ones can be sliced along K.
  const int64_t blocks = w4_blocks(p, 128), nt = p.w.nt();
  const int64_t pairs = blocks * ((nt + 1) / 2);
  const int64_t small = (blocks * nt + c.num_sms - 1) / c.num_sms, large = (pairs + c.num_sms - 1) / c.num_sms;
  if (pairs >= c.num_sms && (p.offsets || large * 100 <= small * 53)) return launch_g<128, 2>(p, c);
  return launch_g<128, 1>(p, c);
}

}  // namespace sq
