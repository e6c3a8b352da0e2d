// k_moe.cu -- routing of tokens to experts: scores and selection, the
// (token, expert) pairs sorted by expert, and the weighted sum of the
// experts' outputs.
#include "sq_ptx.cuh"
#include "sq_w4.h"

namespace sq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteWarps = 4;
constexpr int kMaxV = 16;  // scores a lane holds: up to 512 experts

__device__ __forceinline__ double neg_inf() { return __longlong_as_double(0xfff0000000000000ll); }

// The largest value of the warp and the lowest index among its holders; every
// lane gets both.
__device__ __forceinline__ void warp_argmax(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kAll, v, o);
    const int oi = __shfl_xor_sync(kAll, i, o);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// The whole definition in 64 bits, for any token; lane l holds experts 32 v + l.
// c: room for E choices, used for group scores.
template <int V>
__device__ __noinline__ void route_exactly(const RouteArgs& a, int64_t t, int lane, double* c) {
  const int E = a.E;

  double p[V], choice[V];
  float l[V];
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 32 * v + lane;
    l[v] = -INFINITY;
    if (e < E) {
      l[v] = a.half ? __half2float(static_cast<const __half*>(a.logits)[t * a.ld + e])
                    : static_cast<const float*>(a.logits)[t * a.ld + e];
      if (isnan(l[v])) l[v] = -INFINITY;  // masked, like -inf
    }
    top = fmaxf(top, l[v]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0 / (1.0 + exp(-static_cast<double>(l[v])));
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // equal to the maximum first: an infinite maximum has score one, not NaN
      p[v] = l[v] == -INFINITY ? 0.0 : l[v] == top ? 1.0 : exp(static_cast<double>(l[v]) - static_cast<double>(top));
      sum += p[v];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (sum > 0.0) {
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] /= sum;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 32 * v + lane;
    choice[v] = neg_inf();
    if (e < E && l[v] != -INFINITY) {
      choice[v] = a.bias ? p[v] + static_cast<double>(a.bias[e]) : p[v];
      if (isnan(choice[v])) choice[v] = neg_inf();
    }
  }

  if (a.topk_group < a.n_group) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (32 * v + lane < E) c[32 * v + lane] = choice[v];
    __syncwarp();
    const int per = E / a.n_group;
    double score = neg_inf();
    if (lane < a.n_group) {
      double first = neg_inf(), second = neg_inf();
      for (int i = 0; i < per; ++i) {
        const double x = c[lane * per + i];
        if (x > first) {
          second = first;
          first = x;
        } else if (x > second) {
          second = x;
        }
      }
      score = a.group_top == 2 && second > neg_inf() ? first + second : first;
      if (isnan(score)) score = neg_inf();
    }
    unsigned keep = 0;
    for (int j = 0; j < a.topk_group; ++j) {
      double best = score;
      int which = lane;
      warp_argmax(best, which);
      if (best == neg_inf()) break;
      keep |= 1u << which;
      if (lane == which) score = neg_inf();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 32 * v + lane;
      if (e < E && !(keep >> (e / per) & 1u)) choice[v] = neg_inf();
    }
  }

  // topk rounds of the warp's largest choice; lane j keeps the j-th expert
  int my_id = -1;
  double my_p = 0.0, chosen = 0.0;
  for (int j = 0; j < a.topk; ++j) {
    double best = neg_inf();
    int which = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (choice[v] > best) {
        best = choice[v];
        which = 32 * v + lane;
      }
    warp_argmax(best, which);
    if (best == neg_inf()) break;
    double score = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (32 * v + lane == which) {
        choice[v] = neg_inf();
        score = p[v];
      }
    score = __shfl_sync(kAll, score, which & 31);
    chosen += score;
    if (lane == j) {
      my_id = which;
      my_p = score;
    }
  }
  if (lane < a.topk) {
    double w = my_p;
    if (a.renormalize) w = chosen > 0.0 ? w / chosen : 0.0;
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = static_cast<float>(w * a.scale);
  }
}

// Sortable bits of a float (no NaN).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kNegInfKey = 0x007fffffu;  // order_key(-inf)

// Lane l holds experts V l .. V l + V - 1; logits masked as in route_exactly.
template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&l)[V]) {
  const int e0 = lane * V;
  const int bytes = a.half ? 2 : 4;
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * bytes;
  if (V * bytes % 16 == 0 && (a.ld * bytes) % 16 == 0 && a.E % V == 0) {
    // 16 bytes at a time: 8 (4) experts, all of them below E or none
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      if (e0 + v < a.E) {
        if (!a.half) {
          const float4 f = *reinterpret_cast<const float4*>(row + (e0 + v) * 4);
          l[v] = f.x, l[(v + 1) % V] = f.y, l[(v + 2) % V] = f.z, l[(v + 3) % V] = f.w;
        } else {
          const uint2 f = *reinterpret_cast<const uint2*>(row + (e0 + v) * 2);
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f.x));
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f.y));
          l[v] = x.x, l[(v + 1) % V] = x.y, l[(v + 2) % V] = y.x, l[(v + 3) % V] = y.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[(v + i) % V] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = -INFINITY;
      if (e0 + v < a.E)
        l[v] = a.half ? __half2float(reinterpret_cast<const __half*>(row)[e0 + v])
                      : reinterpret_cast<const float*>(row)[e0 + v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (isnan(l[v])) l[v] = -INFINITY;
}

// The same choice from 32-bit scores, whenever they are far enough apart to be
// sure of it; false otherwise, and nothing is written.
//
// Without a bias and groups the choices are in the order of the logits, which
// needs no score at all, as long as 64-bit scores of different logits differ.
// They do for sigmoids of logits from -600 to 20 and exponentials down to
// exp(-600), unless both logits are next to 0: two 32-bit numbers not both below
// 2^-12 are at least 2^-36 apart, which a score shows.  With them, a 32-bit choice is within
// 2^-18 + 2^-19 |c| of the exact one: the exponential is off by 2^-20 relatively
// (its argument up to 2^-19 where the score is then next to 0 or 1), a sum of up to 512 exponentials by
// 2^-19, and score and choice are rounded.  Two choices whose 32-bit values differ by
// more than four times that are in their exact order.  So are two groups' scores, but a score of
// two choices c + d is only within 2^-17 + 2^-18 (|c| + |d|): a bias may give them
// opposite signs, so their magnitudes count, not the sum's.  With
// 256 experts under a bias about one token in fifty is not sure.
template <int V>
__device__ __forceinline__ bool route_fast(const RouteArgs& a, int64_t t, int lane) {
  const int E = a.E;
  const bool groups = a.topk_group < a.n_group;
  const int per = E / a.n_group, lanes = per / V;  // lanes per group
  if (groups && (lanes * V != per || (lanes & (lanes - 1)))) return false;
  float l[V], c[V];
  load_logits<V>(a, t, lane, l);
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
  top = order_value(__reduce_max_sync(kAll, order_key(top)));
  if (a.sigmoid ? !(top <= 20.0f) : !(top < INFINITY)) return false;  // (all masked: -inf passes)
  const bool scores = groups || a.bias;
  if (scores) {
    if (top == -INFINITY) return false;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = a.sigmoid ? __fdividef(1.0f, __fadd_rn(1.0f, __expf(-l[v]))) : __expf(__fadd_rn(l[v], -top));
      sum = __fadd_rn(sum, c[v]);
    }
    float scale = 1.0f;
    if (!a.sigmoid) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, o));
      scale = __fdividef(1.0f, sum);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane * V + v;
      c[v] = __fmul_rn(c[v], scale);
      if (a.bias && e < E) c[v] = __fadd_rn(c[v], a.bias[e]);
      if (l[v] == -INFINITY || isnan(c[v])) c[v] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l[v];
  }
  auto apart_by = [](float larger, float smaller, float magnitude) {
    return __fadd_rn(larger, -smaller) > 0x1p-16f + 0x1p-17f * magnitude;
  };
  auto apart = [&](float larger, float smaller) {
    return apart_by(larger, smaller, fmaxf(fabsf(larger), fabsf(smaller)));
  };

  if (groups) {
    float first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      second = fmaxf(second, fminf(first, c[v]));
      first = fmaxf(first, c[v]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float f = __shfl_xor_sync(kAll, first, o), s2 = __shfl_xor_sync(kAll, second, o);
      second = fmaxf(fmaxf(second, s2), fminf(first, f));
      first = fmaxf(first, f);
    }
    const bool two = a.group_top == 2 && second > -INFINITY;
    float score = two ? __fadd_rn(first, second) : first;
    if (lane * V >= E) score = -INFINITY;
    // the largest magnitude that any group's score is made of (its bits are in its order)
    const float parts = two ? __fadd_rn(fabsf(first), fabsf(second)) : fabsf(first);
    const float magnitude =
        __uint_as_float(__reduce_max_sync(kAll, score == -INFINITY ? 0u : __float_as_uint(parts)));
    bool keep = false;
    float before = INFINITY;
    for (int j = 0; j <= a.topk_group; ++j) {
      const uint32_t key = order_key(score), best = __reduce_max_sync(kAll, key);
      const float value = order_value(best);
      if (best == kNegInfKey) break;
      if (j == a.topk_group) {
        if (!apart_by(before, value, magnitude)) return false;  // the last group kept and the first one left out
        break;
      }
      before = value;
      const int src = __ffs(__ballot_sync(kAll, key == best)) - 1;
      if ((lane & ~(lanes - 1)) == (src & ~(lanes - 1))) {
        keep = true;
        score = -INFINITY;
      }
    }
    if (!keep) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = -INFINITY;
    }
  }

  // topk rounds of the warp's largest choice (ties to the lowest lane and, in
  // it, the lowest expert); lane j keeps the j-th expert
  // (32-bit scores give up the bits of their keys that then say which of the
  // lane's experts it is; 2^-19 |c| at most, which `apart` allows for)
  uint32_t key[V], mine = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = order_key(c[v]);
    if (scores && key[v] != kNegInfKey) key[v] = (key[v] & ~static_cast<uint32_t>(V - 1)) | (V - 1 - v);
    mine = max(mine, key[v]);
  }
  int my_id = -1;
  float before = INFINITY;
  for (int j = 0; j < a.topk + (scores ? 1 : 0); ++j) {
    const uint32_t best = __reduce_max_sync(kAll, mine);
    if (best == kNegInfKey) break;
    if (scores) {
      const float value = order_value(best);
      if (j > 0 && !apart(before, value)) return false;
      before = value;
      if (j == a.topk) break;
    }
    const int src = __ffs(__ballot_sync(kAll, mine == best)) - 1;
    int at = V - 1 - static_cast<int>(best & (V - 1)), id = src * V + at;
    if (!scores) {
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) at = v;
      id = __shfl_sync(kAll, lane * V + at, src);
    }
    if (lane == j) my_id = id;
    if (lane == src) {
      mine = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v == at) key[v] = 0;
        mine = max(mine, key[v]);
      }
      mine = max(mine, kNegInfKey);
    }
  }
  float my_logit = 0.0f;
  if (my_id >= 0)
    my_logit = a.half ? __half2float(static_cast<const __half*>(a.logits)[t * a.ld + my_id])
                      : static_cast<const float*>(a.logits)[t * a.ld + my_id];
  // (one left out that might tie with a chosen one is as near to 0 as that)
  if (!scores &&
      __any_sync(kAll, my_id >= 0 && (my_logit < (a.sigmoid ? 0.0f : top) - 600.0f || fabsf(my_logit) < 0x1p-12f)))
    return false;

  // the chosen experts' weights, in 64 bits
  double p = 0.0;
  if (my_id >= 0)
    p = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(my_logit)))
                  : exp(static_cast<double>(my_logit) - static_cast<double>(top));
  double sum = 1.0;
  if (a.renormalize || !a.sigmoid) {
    sum = p;
    if (!a.renormalize) {
      sum = 0.0;  // the softmax's own sum
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l[v] != -INFINITY) sum += exp(static_cast<double>(l[v]) - static_cast<double>(top));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = static_cast<float>((sum > 0.0 ? p / sum : 0.0) * a.scale);
  }
  return true;
}

// One warp per token.  Scores count in 64 bits: which experts a token goes to
// must not hang on the last bits of a 32-bit exponential, and two choices may
// lie arbitrarily close.  Most tokens can be decided without forming them.
// 8192 tokens, 256 experts in 8 groups, under a bias: 21.9 us, and 28.9 all in
// 64 bits.  Groups whose experts do not fill a power of two of lanes are all decided in 64
// bits: 160 experts in 8 groups 32-34 us, 128 in 8 groups 17.
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_moe_route(const RouteArgs a) {
  extern __shared__ double sh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  // the next launch may start beside few tokens (an expert layer of one token 33.1 us ->
  // 32.4); beside many its waiting blocks cost 3% (8192 tokens 22.1 -> 22.8)
  if (gridDim.x <= 128) griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  if (!route_fast<V>(a, t, lane)) route_exactly<V>(a, t, lane, sh + warp * a.E);
}

// ------------------------------------------------------------------ plan ----
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanPart = 2048;  // pairs sorted at a time
constexpr int kPerWarp = kPlanPart / kPlanWarps;
constexpr int kPlanChunks = 512;  // CTAs at most

// Parts per CTA, and CTAs.
struct PlanShape {
  int parts, chunks;
};
PlanShape plan_shape(int64_t P) {
  const int64_t all = (P + kPlanPart - 1) / kPlanPart;
  const int64_t parts = (all + kPlanChunks - 1) / kPlanChunks;
  return {static_cast<int>(parts), static_cast<int>((all + parts - 1) / parts)};
}

__global__ void __launch_bounds__(kPlanThreads)
    k_plan_count(const int32_t* __restrict__ ids, int64_t P, int E, int64_t chunk, int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) hist[e] = 0;
  __syncthreads();
  const int64_t end = min(P, (blockIdx.x + 1) * chunk);
  for (int64_t q = blockIdx.x * chunk + threadIdx.x; q < end; q += kPlanThreads) {
    const int e = ids[q];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);  // integer counts: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

// A stable counting sort, 2048 pairs (a part) at a time: counts per warp and
// expert, their scan, then every warp places its pairs in their order.
//
// Up to 2048 pairs one CTA does it all (64 pairs in 3.1 us, 2048 in 5.7).  More are
// split into chunks of one or more parts, whose histograms `counts` holds: every CTA
// adds up all of them itself instead of a third launch (65536 pairs of 256 experts take 9.8 us in
// two launches, both latency).  That work grows with the square of the number of chunks, so
// there are 512 at most and a CTA takes its parts one after the other: 2^20 / 2^22 / 2^24 pairs
// take 58 / 88 / 253 us, with at most 256 chunks 44 / 104 / 373, with 1024 54 / 189 / 351, and 2^22
// with a chunk per part 370.
__global__ void __launch_bounds__(kPlanThreads)
    k_plan_place(const int32_t* __restrict__ ids, int64_t P, int E, const int32_t* __restrict__ counts, int chunks,
                 int parts, int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  extern __shared__ int32_t sh32[];
  int32_t* wcount = sh32;                  // [warps][E]
  int32_t* total = sh32 + kPlanWarps * E;  // [E + 1]: pairs of all chunks, then their exclusive scan
  int32_t* base = total + E + 1;           // [E]: pairs of the chunks before this one, then where the next part's go
  __shared__ int32_t carry[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  for (int part = 0; part < parts; ++part) {
    const int64_t start = (static_cast<int64_t>(blockIdx.x) * parts + part) * kPlanPart;
    if (start >= P) break;
    for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) wcount[i] = 0;
    __syncthreads();
    const int64_t first = start + warp * kPerWarp;
    int32_t mine[kPerWarp / 32];
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
      const int64_t q = first + 32 * i + lane;
      mine[i] = q < P ? ids[q] : -1;
      if (mine[i] >= E) mine[i] = -1;
      if (mine[i] >= 0) atomicAdd(&wcount[warp * E + mine[i]], 1);
    }
    __syncthreads();
    if (part == 0) {
      for (int e = tid; e < E; e += kPlanThreads) {
        int32_t before = 0, all = 0;
        if (chunks == 1) {
          for (int w = 0; w < kPlanWarps; ++w) all += wcount[w * E + e];
        } else {
#pragma unroll 8
          for (int c = 0; c < chunks; ++c) {
            const int32_t n = counts[static_cast<int64_t>(c) * E + e];
            if (c < static_cast<int>(blockIdx.x)) before += n;
            all += n;
          }
        }
        total[e] = all;
        base[e] = before;
      }
      __syncthreads();
      // exclusive scan of total[0 .. E) in place, E <= 2 * kPlanThreads
      int32_t a0 = 2 * tid < E ? total[2 * tid] : 0, a1 = 2 * tid + 1 < E ? total[2 * tid + 1] : 0;
      int32_t inc = a0 + a1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(kAll, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) carry[warp] = inc;
      __syncthreads();
      int32_t pre = 0;
      for (int w = 0; w < warp; ++w) pre += carry[w];
      const int32_t ex = pre + inc - a0 - a1;
      if (2 * tid < E) total[2 * tid] = ex;
      if (2 * tid + 1 < E) total[2 * tid + 1] = ex + a0;
      if (tid == kPlanThreads - 1) total[E] = pre + inc;
      __syncthreads();
      if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += kPlanThreads) offsets[e] = total[e];
    }
    // where each warp's pairs go, and where the next part's begin
    for (int e = tid; e < E; e += kPlanThreads) {
      int32_t at = base[e] + (part == 0 ? total[e] : 0);
      for (int w = 0; w < kPlanWarps; ++w) {
        const int32_t n = wcount[w * E + e];
        wcount[w * E + e] = at;
        at += n;
      }
      base[e] = at;
    }
    // entries past the last routed pair
    for (int64_t q = start + tid; q < P && q < start + kPlanPart; q += kPlanThreads)
      if (q >= total[E]) order[q] = -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
      const int e = mine[i];
      const unsigned same = __match_any_sync(kAll, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int32_t at = 0;
      if (e >= 0) at = wcount[warp * E + e];
      __syncwarp();
      if (e >= 0) {
        if (rank == 0) wcount[warp * E + e] = at + __popc(same);
        order[at + rank] = static_cast<int32_t>(first + 32 * i + lane);
      }
      __syncwarp();
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- combine ----
// y[t] = sum_j weights[t, j] * row (t, j), j ascending, fp32; VEC columns per thread.
// 1024 tokens x 8 fp32 rows of 4096: 27 us, 5.3 TB/s, 0.82 of the copy bandwidth.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    k_moe_combine(const T* __restrict__ rows, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                  int64_t T_, int topk, int64_t N, int E, __half* __restrict__ y) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t per = N / VEC;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= T_ * per) return;
  const int64_t t = i / per, n = (i - t * per) * VEC;
  float acc[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) acc[v] = 0.0f;
  for (int j = 0; j < topk; ++j) {
    const int e = ids[t * topk + j];
    if (e < 0 || e >= E) continue;  // no expert took this pair: its row was never written
    const float w = weights[t * topk + j];
    const T* row = rows + (t * topk + j) * N + n;
    T v[VEC];
    if constexpr (VEC == 4 && sizeof(T) == 4)
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(row);
    else if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(row);
    else
      v[0] = row[0];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = __fmaf_rn(w, static_cast<float>(v[k]), acc[k]);
  }
  __half out[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) out[v] = __float2half_rn(acc[v]);
  if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(y + t * N + n) = *reinterpret_cast<const uint2*>(out);
  else
    y[t * N + n] = out[0];
}

template <int V>
cudaError_t route(const RouteArgs& a, const Ctx& c) {
  const size_t smem = a.topk_group < a.n_group ? sizeof(double) * kRouteWarps * a.E : 0;
  const int64_t blocks = (a.T + kRouteWarps - 1) / kRouteWarps;
  return launch_pdl(k_moe_route<V>, dim3(static_cast<unsigned>(blocks)), dim3(kRouteWarps * 32), smem, c.stream, a);
}

template <typename T>
cudaError_t combine(const T* rows, const int32_t* ids, const float* weights, int64_t tokens, int topk, int64_t N,
                    int E, __half* y, const Ctx& c) {
  const int vec = N % 4 == 0 ? 4 : 1;
  const int64_t n = tokens * (N / vec);
  const unsigned blocks = static_cast<unsigned>((n + 255) / 256);
  if (vec == 4)
    return launch_pdl(k_moe_combine<T, 4>, dim3(blocks), dim3(256), 0, c.stream, rows, ids, weights, tokens, topk, N,
                      E, y);
  return launch_pdl(k_moe_combine<T, 1>, dim3(blocks), dim3(256), 0, c.stream, rows, ids, weights, tokens, topk, N,
                    E, y);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, const Ctx& c) {
  if (a.E <= 32) return route<1>(a, c);
  if (a.E <= 64) return route<2>(a, c);
  if (a.E <= 128) return route<4>(a, c);
  if (a.E <= 256) return route<8>(a, c);
  return route<kMaxV>(a, c);
}

size_t moe_plan_workspace_bytes(int64_t P, int E) {
  const int chunks = plan_shape(P).chunks;
  return chunks > 1 ? static_cast<size_t>(chunks) * E * sizeof(int32_t) : 0;
}

cudaError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* order, int32_t* ws,
                            const Ctx& c) {
  const PlanShape s = plan_shape(P);
  if (s.chunks > 1) {
    const cudaError_t e = launch_pdl(k_plan_count, dim3(s.chunks), dim3(kPlanThreads), sizeof(int32_t) * E, c.stream,
                                     ids, P, E, static_cast<int64_t>(s.parts) * kPlanPart, ws);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_plan_place, dim3(s.chunks), dim3(kPlanThreads), sizeof(int32_t) * ((kPlanWarps + 2) * E + 1),
                    c.stream, ids, P, E, static_cast<const int32_t*>(ws), s.chunks, s.parts, offsets, order);
}

cudaError_t launch_moe_combine(const __half* y16, const float* y32, const int32_t* ids, const float* weights,
                               int64_t T, int topk, int64_t N, int E, __half* y, const Ctx& c) {
  if (y16) return combine(y16, ids, weights, T, topk, N, E, y, c);
  return combine(y32, ids, weights, T, topk, N, E, y, c);
}

}  // namespace sq
