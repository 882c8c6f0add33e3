// moe_route_topk and moe_route_topk_backward: experts and weights from given router logits,
// and the logits' gradient.
//   s = softmax(z) or sigmoid(z); choice score c = z (softmax), s + bias (sigmoid); groups by
//   the sum of their two best c; the K best c of the kept groups; w = scale s_k [/ sum s].
// The choice is that of the real numbers: the candidates are compared in binary32, and where
// two that matter lie closer than the error of that, the token is decided again in binary64.
// Logits themselves (softmax, or sigmoid without a bias, which rises with the logit) are
// compared as they are, and sums of two logits by their rounded value and its exact error.
//
// A token is a warp's: lane l holds the experts [l NPL, (l + 1) NPL), so a reduction that
// takes the lower lane takes the lower expert.
#include <cuda_fp16.h>
#include <float.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kMaxN = 512;
constexpr unsigned kAll = 0xffffffffu;

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (std::is_same<T, float>::value)
    return v;
  else if constexpr (std::is_same<T, __half>::value)
    return __half2float(v);
  else
    return __bfloat162float(v);
}
template <class T>
__device__ __forceinline__ T from_f32(float f) {
  if constexpr (std::is_same<T, float>::value)
    return f;
  else if constexpr (std::is_same<T, __half>::value)
    return __float2half_rn(f);
  else
    return __float2bfloat16_rn(f);
}
// +inf counts as the largest finite number; NaN as -inf, a masked expert.
__device__ __forceinline__ float settle(float z) {
  return z != z ? -INFINITY : fminf(z, FLT_MAX);
}
// Biases beyond +-2^100 count as that, so that no sum of scores is infinite; NaN as -inf.
constexpr float kMostBias = 0x1p100f;
__device__ __forceinline__ float settle_bias(float b) {
  return b > -INFINITY ? fminf(fmaxf(b, -kMostBias), kMostBias) : -INFINITY;
}

struct RouteParams {
  int64_t B;
  int N, K, n_group, topk_group;
  int sigmoid, renorm, vec;
  float scale;
  const void *z;
  const float *bias;
  int32_t *idx;
  float *w;
  int32_t *counts;
  uint32_t inv_gs;  // 2^20 / (experts of a group), rounded up
  int npl;
};

// N values of one token, settled: this lane's NPL, -inf past the end.
template <class T, int NPL>
__device__ __forceinline__ void load_row(const T *row, int N, bool vec, int lane, float *z) {
  constexpr int kBytes = NPL * (int)sizeof(T);
  const int base = lane * NPL;
  if (vec) {  // whole lanes, aligned
    constexpr int kPart = kBytes < 16 ? kBytes : 16;
    alignas(16) T v[NPL];
    if (base < N) {
#pragma unroll
      for (int i = 0; i < kBytes / kPart; ++i) {
        char *to = reinterpret_cast<char *>(v) + i * kPart;
        const char *from = reinterpret_cast<const char *>(row + base) + i * kPart;
        if constexpr (kPart == 16)
          *reinterpret_cast<uint4 *>(to) = __ldg(reinterpret_cast<const uint4 *>(from));
        else if constexpr (kPart == 8)
          *reinterpret_cast<uint2 *>(to) = __ldg(reinterpret_cast<const uint2 *>(from));
        else if constexpr (kPart == 4)
          *reinterpret_cast<uint32_t *>(to) = __ldg(reinterpret_cast<const uint32_t *>(from));
        else
          *reinterpret_cast<uint16_t *>(to) = __ldg(reinterpret_cast<const uint16_t *>(from));
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) z[i] = base < N ? settle(to_f32(v[i])) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) z[i] = base + i < N ? settle(to_f32(row[base + i])) : -INFINITY;
  }
}

// A key that orders as the number does; 0 for what is not a candidate (-inf).
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);
  return c == -INFINITY ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Binary32 sigmoid whose result is off by less than 2^-21 (of its value from the quick
// exponential and quotient, both within 2^-22 of theirs for arguments that matter).
__device__ __forceinline__ float quick_sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(fminf(-z, 87.0f))); }
// Two choice scores that binary32 tells apart wrongly lie closer than this.
__device__ __forceinline__ float margin(float c) { return 0x1p-19f * fmaxf(1.0f, fabsf(c)); }
// How far a + b, the sum of a group's two best scores, may be off: by the errors of both (each a
// sigmoid's 2^-21 and a rounding, half its margin at most) and its own rounding.  The sum itself
// says nothing of that: of scores of either sign it may be next to 0 where they are large.
__device__ __forceinline__ float group_error(float a, float b) {
  const float sum = a + b;
  return sum > -INFINITY ? 0.5f * (margin(a) + margin(b)) : 0.0f;
}

__device__ __forceinline__ double sigmoid64(float z) {
  const double x = exp(-fabs((double)z));
  return (z >= 0.0f ? 1.0 : x) / (1.0 + x);
}

// What orders sums of two logits besides their rounded value s: its exact error (Knuth's
// two-sum), or of sums past binary32's range their half.
__device__ __forceinline__ float sum_error(float a, float b, float s) {
  const float bb = s - a;
  return fabsf(s) < INFINITY ? (a - (s - bb)) + (b - bb) : 0.5f * a + 0.5f * b;
}

// The choice in binary64, for tokens that binary32 leaves open.  kFromLogits: candidates of
// the kept groups are compared by their logits.
template <int NPL>
__device__ __noinline__ int choose64(const RouteParams &P, const float *z, int lane, double *scratch) {
  const int base = lane * NPL;
  double c[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    c[i] = (double)z[i];
    if (P.sigmoid && z[i] != -INFINITY) {
      c[i] = sigmoid64(z[i]);
      if (P.bias) c[i] += (double)settle_bias(P.bias[base + i]);
    }
  }
  if (P.n_group > 1) {
    // scratch[group]: the sum of its two best
    for (int g = 0; g < P.n_group; ++g) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = base + i;
        if (e >= P.N || (int)(((uint32_t)e * P.inv_gs) >> 20) != g) continue;
        b = fmax(b, fmin(a, c[i]));
        a = fmax(a, c[i]);
      }
      for (int d = 16; d; d >>= 1) {
        const double oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (lane == 0) scratch[g] = a + b;
    }
    __syncwarp();
    uint32_t keep = 0;
    if (lane < P.n_group) {
      int ahead = 0;
      for (int j = 0; j < P.n_group; ++j)
        ahead += scratch[j] > scratch[lane] || (scratch[j] == scratch[lane] && j < lane);
      keep = ahead < P.topk_group;
    }
    keep = __ballot_sync(kAll, keep);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = base + i;
      if (e < P.N && !(keep >> (((uint32_t)e * P.inv_gs) >> 20) & 1)) c[i] = -INFINITY;
    }
    __syncwarp();
  }
  if (P.sigmoid && !P.bias) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY) c[i] = (double)z[i];
  }
  int mine = -1;
  for (int r = 0; r < P.K; ++r) {
    double best = -INFINITY;
    int at = kMaxN;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] > best) best = c[i], at = base + i;
    for (int d = 16; d; d >>= 1) {
      const double o = __shfl_xor_sync(kAll, best, d);
      const int oa = __shfl_xor_sync(kAll, at, d);
      if (o > best || (o == best && oa < at)) best = o, at = oa;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (base + i == at) c[i] = -INFINITY;
    if (lane == r) mine = at == kMaxN ? -1 : at;
  }
  return mine;
}

// The score of expert e in binary64.
__device__ __forceinline__ double score64(const RouteParams &P, float z, int e) {
  if (!P.sigmoid) return (double)z;
  const double s = sigmoid64(z);
  return P.bias ? s + (double)settle_bias(P.bias[e]) : s;
}

// Experts that the lanes mark (bit i: base + i) into `list`, in order; their number.
__device__ __forceinline__ int collect(uint32_t marks, int base, int lane, int *list) {
  const int n = __popc(marks);
  int before = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, before, d);
    if (lane >= d) before += o;
  }
  const int total = __shfl_sync(kAll, before, 31);
  __syncwarp();
  if (total <= 32)
    for (before -= n; marks; marks &= marks - 1) list[before++] = base + __ffs(marks) - 1;
  __syncwarp();
  return total;
}

// The choice for one token by a warp: lane r's is the r-th.  Scores that lie closer than
// binary32 can tell are collected and compared in binary64, a lane each (all experts of the
// token in binary64 where they are more than 32: tens of microseconds).  `rows`: room for a
// token's values, 33 words apart every 32; `wide`: 32 doubles.
template <class T, int NPL>
__device__ __forceinline__ int choose(const RouteParams &P, int64_t t, const float *z, int lane, float *rows,
                                      double *wide) {
  const T *row = static_cast<const T *>(P.z) + t * P.N;
  const int base = lane * NPL, gs = P.N / P.n_group;
  auto pad = [](int e) { return e + (e >> 5); };
  auto group_of = [&](int e) { return (int)(((uint32_t)e * P.inv_gs) >> 20); };
  auto all64 = [&] {
    float copy[NPL];  // z itself stays in registers
#pragma unroll
    for (int i = 0; i < NPL; ++i) copy[i] = z[i];
    return choose64<NPL>(P, copy, lane, wide);
  };
  int *list = reinterpret_cast<int *>(rows);
  float c[NPL];
  // scores that groups and, with a bias, experts are compared by
  const bool scored = P.sigmoid && (P.bias || P.n_group > 1);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    c[i] = z[i];
    if (scored && z[i] != -INFINITY) {
      c[i] = quick_sigmoid(z[i]);
      if (P.bias) c[i] += settle_bias(__ldg(P.bias + base + i));
    }
  }
  if (P.n_group > 1) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (base + i < P.N) rows[pad(base + i)] = c[i];
    __syncwarp();
    // lanes of one group: each its part of the experts, then across
    int share = 32 / P.n_group;
    share = 1 << (31 - __clz(share));
    const int g = lane / share;
    float a = -INFINITY, b = -INFINITY;
    if (g < P.n_group)
      for (int i = lane % share; i < gs; i += share) {
        const float v = rows[pad(g * gs + i)];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    for (int d = 1; d < share; d <<= 1) {
      const float oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    const float s = a + b;
    const float low_bits = P.sigmoid ? 0.0f : sum_error(a, b, s);
    int ahead = 0;
    for (int j = 0; j < P.n_group; ++j) {
      const float os = __shfl_sync(kAll, s, j * share), oe = __shfl_sync(kAll, low_bits, j * share);
      ahead += os > s || (os == s && (oe > low_bits || (oe == low_bits && j < g)));
    }
    bool kept = g < P.n_group && ahead < P.topk_group;
    if (P.sigmoid && P.topk_group < P.n_group) {
      // the least that a kept group may have, and the most that one left out may
      const float err = group_error(a, b);
      const uint32_t in = __reduce_min_sync(kAll, kept ? key_of(s - err) : kAll);
      const uint32_t out = __reduce_max_sync(kAll, g < P.n_group && !kept ? key_of(s + err) : 0u);
      const float low = of_key(in), high = of_key(out);
      if (in != 0 && out != 0 && low <= high) {
        // groups on either side that may belong to the other, by the sums of their best in 64 bits
        const bool open = g < P.n_group && (kept ? s - err <= high : s + err >= low);
        const uint32_t open_lanes = __ballot_sync(kAll, open);
        uint32_t marks = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const int of = group_of(base + i) * share;
          const float second = __shfl_sync(kAll, b, of & 31);
          if (base + i < P.N && (open_lanes >> of & 1) && c[i] >= second - margin(second)) marks |= 1u << i;
        }
        const int n = collect(marks, base, lane, list);
        if (n > 32) return all64();
        if (lane < n) wide[lane] = score64(P, settle(to_f32(row[list[lane]])), list[lane]);
        __syncwarp();
        double first = -INFINITY, next = -INFINITY;
        if (open)
          for (int j = 0; j < n; ++j)
            if (group_of(list[j]) == g) {
              const double v = wide[j];
              next = v > first ? first : v > next ? v : next;
              first = v > first ? v : first;
            }
        const double both = first + next;
        const uint32_t places = __popc(__ballot_sync(kAll, open && kept && lane % share == 0));
        uint32_t before = 0;
        for (int j = 0; j < P.n_group; ++j) {
          const double other = __shfl_sync(kAll, both, j * share);
          before += (open_lanes >> (j * share) & 1) && (other > both || (other == both && j < g));
        }
        if (open) kept = before < places;
        __syncwarp();
      }
    }
    const uint32_t lanes = __ballot_sync(kAll, kept);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const bool in = base + i < P.N && (lanes >> (group_of(base + i) * share) & 1);
      if (P.sigmoid && !P.bias) c[i] = z[i];
      if (!in) c[i] = -INFINITY;
    }
  }
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = key_of(c[i]);
  // one more than K where neighbours are compared
  const bool compare = P.sigmoid && P.bias;
  const int rounds = compare ? P.K + 1 : P.K;
  int mine = -1, last_e = 0;
  uint32_t last = 0, lowest = 0;  // of the one before, of the K-th
  bool open = false, beyond = false;  // beyond: the K-th ties with the next, and so may others be near
  for (int r = 0; r < rounds; ++r) {
    uint32_t kb = 0;
    int ib = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i] > kb) kb = key[i], ib = i;  // strict: the lower index keeps a tie
    const uint32_t best = __reduce_max_sync(kAll, kb);
    if (best == 0) break;
    const int owner = __ffs(__ballot_sync(kAll, kb == best)) - 1;
    const int e = __shfl_sync(kAll, base + ib, owner);
    if (compare && last != 0 && of_key(last) - of_key(best) <= margin(of_key(last))) {
      const bool differ = to_f32(row[e]) != to_f32(row[last_e]) || P.bias[e] != P.bias[last_e];  // else they tie
      open = open || differ;
      beyond = r == P.K && !differ;
    }
    last = best;
    last_e = e;
    if (r < P.K) lowest = best;
    if (lane == owner)
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == ib) key[i] = 0u;
    if (lane == r && r < P.K) mine = e;
  }
  if (beyond && !open) {  // the same for all lanes
    const float c0 = of_key(lowest), z0 = settle(to_f32(row[last_e])), b0 = P.bias[last_e];
    bool near = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY && fabsf(c[i] - c0) <= margin(c0)) near = near || z[i] != z0 || P.bias[base + i] != b0;
    open = __any_sync(kAll, near);
  }
  if (open) {
    // all that may be among the K best
    const float least = of_key(lowest) - margin(of_key(lowest));
    uint32_t marks = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY && c[i] >= least) marks |= 1u << i;
    const int n = collect(marks, base, lane, list);
    if (n > 32) return all64();
    const int e = lane < n ? list[lane] : 0;
    const double v = lane < n ? score64(P, settle(to_f32(row[e])), e) : 0.0;
    wide[lane] = v;
    __syncwarp();
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += wide[j] > v || (wide[j] == v && j < lane);  // the list is in order
    __syncwarp();
    if (lane < n) list[32 + rank] = e;
    __syncwarp();
    if (lane < P.K && lane < n) mine = list[32 + lane];
    __syncwarp();
  }
  return mine;
}

// One token by a warp: its choice, weights and counts.
template <class T, int NPL>
__device__ __forceinline__ void one_token(const RouteParams &P, int64_t t, int lane, float *rows, double *wide,
                                          int *histogram) {
  float z[NPL];
  load_row<T, NPL>(static_cast<const T *>(P.z) + t * P.N, P.N, P.vec, lane, z);
  const int mine = choose<T, NPL>(P, t, z, lane, rows, wide);
  // the weights of the chosen, a lane each
  float top = 0.0f, total = 0.0f;
  const float zk = mine >= 0 ? settle(to_f32(static_cast<const T *>(P.z)[t * P.N + mine])) : -INFINITY;
  float sk;
  if (P.sigmoid) {
    const float x = expf(-fabsf(zk)), q = 1.0f / (1.0f + x);
    sk = mine < 0 ? 0.0f : zk >= 0.0f ? q : x * q;
  } else if (P.renorm) {
    top = zk;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    sk = mine >= 0 ? expf(zk - top) : 0.0f;
  } else {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = fmaxf(top, z[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) total += expf(z[i] - top);
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    sk = mine >= 0 ? expf(zk - top) / total : 0.0f;
  }
  if (P.renorm) {
    total = sk;
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    if (total > 0.0f) sk /= total;
  }
  if (lane < P.K) {
    P.idx[t * P.K + lane] = mine;
    P.w[t * P.K + lane] = sk * P.scale;
    if (mine >= 0) atomicAdd(histogram + mine, 1);
  }
}

// T: the logits' type.  Warps take every so many-th token.  kCluster: the grid is one cluster,
// whose blocks add up their counts in shared memory and write them, with nothing set to zero
// before.
template <class T, int NPL, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32) route_topk_kernel(const __grid_constant__ RouteParams P) {
  __shared__ float rows[kWarps][kMaxN + kMaxN / 32];
  __shared__ double wide[kWarps][32];
  __shared__ int histogram[kMaxN];
  for (int i = threadIdx.x; i < P.N; i += kWarps * 32) histogram[i] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < P.B; t += (int64_t)gridDim.x * kWarps)
    one_token<T, NPL>(P, t, lane, rows[warp], wide[warp], histogram);
  if (!P.counts) return;
  __syncthreads();
  if constexpr (kCluster) {
    cluster_sync();  // the blocks' counts
    const int rank = (int)cluster_ctarank();
    for (int i = rank * kWarps * 32 + threadIdx.x; i < P.N; i += (int)gridDim.x * kWarps * 32) {
      int n = 0;
      for (int b = 0; b < (int)gridDim.x; ++b) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(histogram + i), b)) : "memory");
        n += v;
      }
      P.counts[i] = n;
    }
    cluster_sync();  // no block ends while another reads its counts
  } else {
    for (int i = threadIdx.x; i < P.N; i += kWarps * 32)
      if (histogram[i]) atomicAdd(P.counts + i, histogram[i]);
  }
}

// --------------------------------------------------------------- many tokens
// Four lanes a token, each with 8 of every 32 experts: a token's K best are sorted lists of
// keys in registers, built 8 experts at a time and merged, instead of K reductions over a warp:
// 65536 tokens, 256 experts in 8 groups, biases, K = 8: 50 us, 140 a warp a token.  A key holds
// the upper 23 bits of the score's order and the expert; neighbours that it leaves open are put
// in order by their scores.  What bounds it: instructions (about 360 a token) at 44 % of the
// issue slots, waiting on one another; 24 warps an SM are what registers and shared memory hold.
// Steps that counted: the counts in shared memory (-65 us); scores that binary32 leaves open
// compared here, in 64 bits, instead of by calls (-10: 50 tokens of 65536, but a call's code is
// never in the instruction cache); of the kept groups only what may be among the best is sorted;
// loops over chunks and lanes are not unrolled, the code being longer than that cache (512
// experts, K = 16, binary32: 122 -> 115 us).
constexpr int kQuadWarps = 8, kMostGroups = 16;

__device__ __forceinline__ uint32_t expert_key(float c, int e) {
  const uint32_t k = key_of(c);
  return k == 0 ? 0u : (k & ~511u) | (uint32_t)(511 - e);
}

// Comparators of keys, the larger first.
__device__ __forceinline__ void order(uint32_t &a, uint32_t &b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Batcher's odd-even merge sort of 8.
__device__ __forceinline__ void sort8(uint32_t *k) {
  order(k[0], k[1]), order(k[2], k[3]), order(k[4], k[5]), order(k[6], k[7]);
  order(k[0], k[2]), order(k[1], k[3]), order(k[4], k[6]), order(k[5], k[7]);
  order(k[1], k[2]), order(k[5], k[6]);
  order(k[0], k[4]), order(k[1], k[5]), order(k[2], k[6]), order(k[3], k[7]);
  order(k[2], k[4]), order(k[3], k[5]);
  order(k[1], k[2]), order(k[3], k[4]), order(k[5], k[6]);
}
// A sequence that rises once and falls once, in order.
template <int M>
__device__ __forceinline__ void sort_bitonic(uint32_t *k) {
#pragma unroll
  for (int d = M / 2; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (!(i & d)) order(k[i], k[i + d]);
}
// The two largest of what is left out.
struct Rest {
  uint32_t first, second;
  __device__ __forceinline__ void add(uint32_t k) {
    second = max(second, min(first, k));
    first = max(first, k);
  }
};
// The largest M of a sorted list of M and one of n <= M, sorted.
template <int M, int n>
__device__ __forceinline__ void merge(uint32_t *list, const uint32_t *more, Rest &rest) {
#pragma unroll
  for (int i = 0; i < n; ++i) {
    uint32_t &l = list[M - n + i];
    rest.add(min(l, more[n - 1 - i]));
    l = max(l, more[n - 1 - i]);
  }
  sort_bitonic<M>(list);
}

// A token that the keys leave open.
template <class T>
__device__ __noinline__ void token_again(const RouteParams &P, int64_t t, int lane, float *rows, double *wide,
                                         int *histogram) {
  switch (P.npl) {
    case 1: return one_token<T, 1>(P, t, lane, rows, wide, histogram);
    case 2: return one_token<T, 2>(P, t, lane, rows, wide, histogram);
    case 4: return one_token<T, 4>(P, t, lane, rows, wide, histogram);
    case 8: return one_token<T, 8>(P, t, lane, rows, wide, histogram);
    default: return one_token<T, 16>(P, t, lane, rows, wide, histogram);
  }
}

// Words of shared memory a warp has.
__host__ __device__ __forceinline__ int quad_words(int N, int n_group) {
  const int keys = n_group == 1 ? 0 : 8 * (N + 4), values = kMaxN + kMaxN / 32;
  return keys > values ? keys : values;
}

// The hardware's 2^x and 1/x.  1 / (1 + 2^(-z log2 e)) of any finite z: 2^x may be infinite,
// whose reciprocal is 0.
__device__ __forceinline__ float sigmoid_of_finite(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
// Whether 8 logits are all finite: the largest of their magnitudes' bits.
template <class T>
__device__ __forceinline__ bool all_finite(const uint4 *v) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t m = 0x7fffffffu;
    const uint32_t a = max(max(v[0].x & m, v[0].y & m), max(v[0].z & m, v[0].w & m));
    return max(a, max(max(v[1].x & m, v[1].y & m), max(v[1].z & m, v[1].w & m))) < 0x7f800000u;
  } else {
    const uint32_t m = 0x7fff7fffu, w = __vmaxu2(__vmaxu2(v->x & m, v->y & m), __vmaxu2(v->z & m, v->w & m));
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (w >> 16) < kInf && (w & 0xffffu) < kInf;
  }
}

// KP: room of a list, K at most.  N a multiple of 8, groups of multiples of 32 experts.
template <class T, int KP>
__global__ void __launch_bounds__(kQuadWarps * 32, 3) route_topk_quad_kernel(const __grid_constant__ RouteParams P) {
  // of each warp: its tokens' scores; for a token's second choice, its own
  extern __shared__ uint4 dynamic[];
  // the groups' sums and their errors, or the sums in 64 bits; or 32 doubles
  __shared__ double group_sums[kQuadWarps][2 * 8 * kMostGroups / 2];
  __shared__ int histogram[kMaxN];  // 524288 additions to 256 words of global memory: 65 us
  for (int i = threadIdx.x; i < P.N; i += kQuadWarps * 32) histogram[i] = 0;
  bool fine = true;  // the biases are what they count as
  if (P.bias)
    for (int i = threadIdx.x; i < P.N; i += kQuadWarps * 32) fine = fine && fabsf(__ldg(P.bias + i)) <= kMostBias;
  fine = __syncthreads_and(fine);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, token = lane >> 2, q = lane & 3;
  const int chunks = (P.N + 31) / 32, pitch = chunks * 32 + 4;  // words: two tokens share no bank
  uint32_t *warp_words = reinterpret_cast<uint32_t *>(dynamic) + warp * quad_words(P.N, P.n_group);
  float *values = reinterpret_cast<float *>(warp_words) + token * pitch + q * 8;
  const int per_group = chunks / P.n_group;
  const bool biased = P.sigmoid && P.bias;
  const int64_t step = (int64_t)gridDim.x * kQuadWarps * 8;
  int64_t t0 = ((int64_t)blockIdx.x * kQuadWarps + warp) * 8;
  // The whole warp's tokens wait for a loop of their own: called from the midst of this one,
  // their choice took as long as all others together (its registers).
  int waiting = 0, pending = 0;  // lane l has the l-th
  while (t0 < P.B) {
    for (; t0 < P.B && waiting <= 24; t0 += step) {
      const int64_t t = t0 + token;
      const bool live = t < P.B;
      const T *row = static_cast<const T *>(P.z) + (live ? t : P.B - 1) * P.N;
      constexpr int kLoads = (int)sizeof(T) / 2;
      auto load8 = [&](int chunk, uint4 *v) {
        const int e = chunk * 32 + q * 8;
        if (e < P.N) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(row + e) + i);
          return true;
        }
        return false;
      };
      auto settled8 = [&](int chunk, float *z) {
        uint4 v[kLoads];
        const bool some = load8(chunk, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = some ? settle(to_f32(reinterpret_cast<T *>(v)[i])) : -INFINITY;
      };
      // the scores that experts are compared by
      auto scores = [&](int chunk, float *c) {
        uint4 v[kLoads];
        const int e = chunk * 32 + q * 8;
        if (load8(chunk, v) && fine && all_finite<T>(v)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = to_f32(reinterpret_cast<T *>(v)[i]);
          if (biased) {
            float b[8];
            *reinterpret_cast<float4 *>(b) = __ldg(reinterpret_cast<const float4 *>(P.bias + e));
            *reinterpret_cast<float4 *>(b + 4) = __ldg(reinterpret_cast<const float4 *>(P.bias + e) + 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = sigmoid_of_finite(c[i]) + b[i];
          }
          return;
        }
        settled8(chunk, c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (biased && e < P.N && c[i] != -INFINITY)
            c[i] = sigmoid_of_finite(c[i]) + settle_bias(__ldg(P.bias + e + i));
      };
      uint32_t list[KP + 1];  // and the largest left out
      Rest rest = {0, 0};
#pragma unroll
      for (int i = 0; i < KP; ++i) list[i] = 0;
      bool open = false;
      auto add = [&](uint32_t *k) {
        sort8(k);
        merge<KP, 8>(list, k, rest);
      };
      if (P.n_group == 1) {
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          float c[8];
          uint32_t k[8];
          scores(ch, c);
#pragma unroll
          for (int i = 0; i < 8; ++i) k[i] = expert_key(c[i], ch * 32 + q * 8 + i);
          add(k);
        }
      } else {
        float *sum = reinterpret_cast<float *>(group_sums[warp]) + token * 2 * kMostGroups, *err = sum + kMostGroups;
        float a = -INFINITY, b = -INFINITY;
        float seconds[kMostGroups / 4];  // the second best of the groups q, q + 4, ...
#pragma unroll
        for (int i = 0; i < kMostGroups / 4; ++i) seconds[i] = -INFINITY;
        int in_group = 0, g = 0;
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          float c[8];
          scores(ch, c);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            b = fmaxf(b, fminf(a, c[i]));
            a = fmaxf(a, c[i]);
          }
          reinterpret_cast<float4 *>(values + ch * 32)[0] = make_float4(c[0], c[1], c[2], c[3]);
          reinterpret_cast<float4 *>(values + ch * 32)[1] = make_float4(c[4], c[5], c[6], c[7]);
          if (++in_group == per_group) {
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
              const float oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
              b = fmaxf(fminf(a, oa), fmaxf(b, ob));
              a = fmaxf(a, oa);
            }
#pragma unroll
            for (int i = 0; i < kMostGroups / 4; ++i)
              if (g == 4 * i + q) seconds[i] = b;
            if (P.sigmoid && !P.bias) {  // of logits the two best have the two best scores
              a = a == -INFINITY ? a : quick_sigmoid(a);
              b = b == -INFINITY ? b : quick_sigmoid(b);
            }
            const float s = a + b;
            if (q == 0) sum[g] = s, err[g] = P.sigmoid ? group_error(a, b) : sum_error(a, b, s);
            a = b = -INFINITY;
            in_group = 0;
            ++g;
          }
        }
        __syncwarp();
        // kept: fewer than topk_group groups rank before it; four lanes, a group each in turn
        uint32_t kept;
        // the least that a kept group may have, the most of the others; least second best of the kept
        float lowest, highest, least;
        auto rank = [&](auto before) {  // before(j, g): group j ranks before group g
          kept = 0;
          lowest = least = INFINITY;
          highest = -INFINITY;
#pragma unroll
          for (int i = 0; i < kMostGroups / 4; ++i) {
            const int g = 4 * i + q;
            if (g >= P.n_group) break;
            int ahead = 0;
            for (int j = 0; j < P.n_group; ++j) ahead += before(j, g);
            if (ahead < P.topk_group) {
              kept |= 1u << g;
              lowest = fminf(lowest, sum[g] - err[g]);
              least = fminf(least, seconds[i]);
            } else {
              highest = fmaxf(highest, sum[g] + err[g]);
            }
          }
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            kept |= __shfl_xor_sync(kAll, kept, d);
            lowest = fminf(lowest, __shfl_xor_sync(kAll, lowest, d));
            highest = fmaxf(highest, __shfl_xor_sync(kAll, highest, d));
            least = fminf(least, __shfl_xor_sync(kAll, least, d));
          }
        };
        if (P.sigmoid)
          rank([&](int j, int g) { return sum[j] > sum[g] || (sum[j] == sum[g] && j < g); });
        else
          rank([&](int j, int g) {
            return sum[j] > sum[g] || (sum[j] == sum[g] && (err[j] > err[g] || (err[j] == err[g] && j < g)));
          });
        const bool border = P.sigmoid && lowest > -INFINITY && highest > -INFINITY && lowest <= highest;
        if (__any_sync(kAll, border)) {
          // The sums of the groups at the border in 64 bits, of the others as they are, where the
          // binary32 ones were.
          double exact[kMostGroups / 4], *sums = reinterpret_cast<double *>(sum);
#pragma unroll
          for (int i = 0; i < kMostGroups / 4; ++i) {
            const int g = 4 * i + q;
            if (g >= P.n_group) break;
            const float s = sum[g];
            exact[i] = (double)s;
            if (!border || s + err[g] < lowest || s - err[g] > highest) continue;
            const float from = seconds[i] - margin(seconds[i]);
            const float *all = values - q * 8 + g * per_group * 32;
            double best = -INFINITY, next = -INFINITY;
            for (int j = 0; j < per_group * 32; ++j)
              if (all[j] >= from) {
                const int x = g * per_group * 32 + j;
                const double v = score64(P, settle(to_f32(row[x])), x);
                next = v > best ? best : v > next ? v : next;
                best = v > best ? v : best;
              }
            exact[i] = best + next;
          }
          __syncwarp();  // the sums are read
#pragma unroll
          for (int i = 0; i < kMostGroups / 4; ++i)
            if (4 * i + q < P.n_group) sums[4 * i + q] = exact[i];
          __syncwarp();
          rank([&](int j, int g) { return sums[j] > sums[g] || (sums[j] == sums[g] && j < g); });
        }
        __syncwarp();  // the sums are read
        // The kept groups hold two experts each that score at least their least second best: the
        // K best, if they are no more than those, do too.  Few others do (256 experts: about 14
        // of 128), and only those are sorted.
        if (P.K <= 2 * P.topk_group && !__any_sync(kAll, least == -INFINITY)) {
          if (biased) least -= 2.0f * margin(least);  // what may tie with the last of them
          uint32_t *first = nullptr, *more = nullptr;  // lists: 8 words each of this lane's own, read before
          int count = 0;
          for (int done = 0; done < P.topk_group * per_group; done += 4) {
            uint32_t marks = 0, place = 0;  // 8 experts and the chunk of up to 4 steps
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              if (done + n >= P.topk_group * per_group) break;
              const int ch = (__ffs(kept) - 1) * per_group + in_group;
              if (++in_group == per_group) in_group = 0, kept &= kept - 1;
              const float4 lo = reinterpret_cast<const float4 *>(values + ch * 32)[0];
              const float4 hi = reinterpret_cast<const float4 *>(values + ch * 32)[1];
              const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) marks |= c[i] >= least ? 1u << (8 * n + i) : 0u;
              place |= (uint32_t)ch << (8 * n);
              if (done + n == 0) first = reinterpret_cast<uint32_t *>(values + ch * 32);
              if (done + n == 1) more = reinterpret_cast<uint32_t *>(values + ch * 32);
            }
            for (; marks; marks &= marks - 1, ++count) {
              const int bit = __ffs(marks) - 1, ch = (int)(place >> (bit & 24)) & 255, i = bit & 7;
              const uint32_t k = expert_key(values[ch * 32 + i], ch * 32 + q * 8 + i);
              if (count < 8)
                first[count] = k;
              else if (count < 16 && more)
                more[count - 8] = k;
            }
          }
          const uint32_t over = __ballot_sync(kAll, count > (more ? 16 : 8));  // of any of the four lanes
          if (over >> (lane & ~3) & 15u) open = true;
          const int most = __reduce_max_sync(kAll, min(count, more ? 16 : 8));
          for (int n = 0; n < most; n += 8) {
            uint32_t k[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = n + i < count && n + i < 16 ? (n ? more : first)[i] : 0u;
            add(k);
          }
        } else {
          for (int n = 0; n < P.topk_group; ++n, kept &= kept - 1)
            for (int i = 0; i < per_group; ++i) {
              const int ch = (__ffs(kept) - 1) * per_group + i;
              uint32_t k[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) k[j] = expert_key(values[ch * 32 + j], ch * 32 + q * 8 + j);
              add(k);
            }
        }
      }
      // the four lanes' lists
#pragma unroll 1
      for (int d = 1; d < 4; d <<= 1) {
        uint32_t other[KP];
#pragma unroll
        for (int i = 0; i < KP; ++i) other[i] = __shfl_xor_sync(kAll, list[i], d);
        const uint32_t other_first = __shfl_xor_sync(kAll, rest.first, d);
        rest.add(__shfl_xor_sync(kAll, rest.second, d));
        rest.add(other_first);
        merge<KP, KP>(list, other, rest);
      }
      // Neighbours that the keys' upper bits leave open, the largest left out among them, are put
      // in order by their scores; what binary32 leaves open, and what is nearer than that among
      // the others left out, is the whole warp's.
      list[KP] = rest.first;
      bool near = false;
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        const uint32_t hi = list[i], lo = list[i + 1];
        if (i < P.K && hi != 0 && lo != 0)
          near = near || (biased ? of_key(hi & ~511u) - of_key(lo | 511u) <= margin(of_key(hi))
                                 : sizeof(T) == 4 && (hi ^ lo) < 512u);
      }
      if (__any_sync(kAll, near)) {
        constexpr int kOwn = KP / 4 + 1;
        float own[kOwn], c[KP + 1];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          uint32_t k = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j == q && 4 * i + j <= KP) k = list[4 * i + j];
          const int e = 511 - (int)(k & 511u);
          own[i] = -INFINITY;
          if (k != 0) {
            own[i] = settle(to_f32(row[e]));
            if (biased) own[i] = sigmoid_of_finite(own[i]) + settle_bias(__ldg(P.bias + e));
          }
        }
#pragma unroll
        for (int i = 0; i <= KP; ++i) c[i] = __shfl_sync(kAll, own[i / 4], (lane & ~3) + (i & 3));
#pragma unroll
        for (int pass = 0; pass < 4; ++pass)
#pragma unroll
          for (int i = pass & 1; i < KP; i += 2) {
            const bool swap = c[i] < c[i + 1] || (c[i] == c[i + 1] && (list[i] & 511u) < (list[i + 1] & 511u));
            const float x = c[i];
            const uint32_t l = list[i];
            c[i] = swap ? c[i + 1] : x;
            list[i] = swap ? list[i + 1] : l;
            c[i + 1] = swap ? x : c[i + 1];
            list[i + 1] = swap ? l : list[i + 1];
          }
        // Places that binary32 does not tell from the one before, of those up to the K-th, or from
        // the K-th, of the others.  Where all of those are of one logit and one bias they do tie.
        uint32_t ties = 0;
        bool differ = false;
        float bound = INFINITY;  // the K-th's score
#pragma unroll
        for (int i = 0; i < KP; ++i) {
          if (list[i + 1] == 0) break;
          if (c[i] < c[i + 1]) open = true;  // further from its place than the passes go
          if (i < P.K) bound = c[i];
          if (biased && bound - c[i + 1] <= margin(bound)) {
            const int x = 511 - (int)(list[i] & 511u), y = 511 - (int)(list[i + 1] & 511u);
            ties |= 3u << i;
            differ = differ || to_f32(row[x]) != to_f32(row[y]) || P.bias[x] != P.bias[y];
          }
          if (i == P.K - 1 && rest.second != 0) {
            const float most = of_key(rest.second | 511u);
            if (biased ? c[i] - most <= margin(c[i]) : sizeof(T) == 4 && c[i] <= most) open = true;
          }
        }
        if (!differ) ties = 0;
        if (__any_sync(kAll, ties != 0)) {
          // their scores in 64 bits (of the others, which are further apart, binary32's): for each
          // place, those that come before it
          double d[kOwn];
          int before[kOwn] = {};
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            uint32_t k = 0;
            d[i] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j == q && 4 * i + j <= KP) k = list[4 * i + j], d[i] = (double)c[4 * i + j];
            const int e = 511 - (int)(k & 511u);
            if (k != 0 && (ties >> (4 * i + q) & 1)) d[i] = score64(P, settle(to_f32(row[e])), e);
            own[i] = __uint_as_float(k);
          }
          for (int j = 0; j <= KP; ++j) {
            const int from = (lane & ~3) + (j & 3);
            double other = d[0];
            uint32_t ok = __float_as_uint(own[0]);
#pragma unroll
            for (int i = 1; i < kOwn; ++i)
              if (j / 4 == i) other = d[i], ok = __float_as_uint(own[i]);
            other = __shfl_sync(kAll, other, from);
            ok = __shfl_sync(kAll, ok, from);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
              const uint32_t k = __float_as_uint(own[i]);
              before[i] += ok != 0 && (other > d[i] || (other == d[i] && (ok & 511u) > (k & 511u)));
            }
          }
          // the list by those numbers
          uint32_t sorted[KP + 1];
#pragma unroll
          for (int p = 0; p <= KP; ++p) sorted[p] = 0;
          for (int j = 0; j <= KP; ++j) {
            const int from = (lane & ~3) + (j & 3);
            int at = before[0];
            uint32_t k = __float_as_uint(own[0]);
#pragma unroll
            for (int i = 1; i < kOwn; ++i)
              if (j / 4 == i) at = before[i], k = __float_as_uint(own[i]);
            at = __shfl_sync(kAll, at, from);
            k = __shfl_sync(kAll, k, from);
#pragma unroll
            for (int p = 0; p <= KP; ++p)
              if (p == at && k != 0) sorted[p] = k;
          }
          if (ties)
#pragma unroll
            for (int p = 0; p <= KP; ++p) list[p] = sorted[p];
        }
      }
      // this lane's of the chosen: places q, q + 4, ...
      int mine[(KP + 3) / 4];
#pragma unroll
      for (int i = 0; i < (KP + 3) / 4; ++i) {
        uint32_t k = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j == q && 4 * i + j < KP) k = list[4 * i + j];
        mine[i] = k == 0 ? -1 : 511 - (int)(k & 511u);
      }
      for (uint32_t todo = __ballot_sync(kAll, open && live && q == 0); todo; todo &= todo - 1, ++waiting)
        if (lane == waiting) pending = (int)t0 + ((__ffs(todo) - 1) >> 2);
      // weights
      auto sum4 = [](float v) {  // in the order of a whole warp's sum, so that the weights are the same
        v += __shfl_xor_sync(kAll, v, 2);
        return v + __shfl_xor_sync(kAll, v, 1);
      };
      auto max4 = [](float v) {
        v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
        return fmaxf(v, __shfl_xor_sync(kAll, v, 2));
      };
      float s[(KP + 3) / 4], total = 0.0f, top = -INFINITY;
#pragma unroll
      for (int i = 0; i < (KP + 3) / 4; ++i) {
        if (4 * i + q >= P.K) mine[i] = -1;
        s[i] = mine[i] >= 0 ? settle(to_f32(row[mine[i]])) : -INFINITY;
        top = fmaxf(top, s[i]);
      }
      if (!P.sigmoid) {
        if (!P.renorm) {
          for (int ch = 0; ch < chunks; ++ch) {
            float z[8];
            settled8(ch, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, z[i]);
          }
        }
        top = max4(top);
        if (top == -INFINITY) top = 0.0f;
        if (!P.renorm) {
          for (int ch = 0; ch < chunks; ++ch) {
            float z[8];
            settled8(ch, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) total += expf(z[i] - top);
          }
          total = sum4(total);
        }
      }
#pragma unroll
      for (int i = 0; i < (KP + 3) / 4; ++i) {
        if (P.sigmoid) {
          const float x = expf(-fabsf(s[i])), w = 1.0f / (1.0f + x);
          s[i] = mine[i] < 0 ? 0.0f : s[i] >= 0.0f ? w : x * w;
        } else {
          s[i] = mine[i] < 0 ? 0.0f : expf(s[i] - top);
          if (!P.renorm) s[i] = mine[i] < 0 ? 0.0f : s[i] / total;
        }
      }
      if (P.renorm) {
        const float chosen = sum4(KP > 8 ? (s[0] + s[(KP > 8) * 2]) + (s[1] + s[(KP > 8) * 3]) : s[0] + s[1]);
#pragma unroll
        for (int i = 0; i < (KP + 3) / 4; ++i)
          if (chosen > 0.0f) s[i] /= chosen;
      }
      if (live && !open) {
#pragma unroll
        for (int i = 0; i < (KP + 3) / 4; ++i) {
          const int k = 4 * i + q;
          if (k < P.K) {
            P.idx[t * P.K + k] = mine[i];
            P.w[t * P.K + k] = s[i] * P.scale;
            if (mine[i] >= 0) atomicAdd(histogram + mine[i], 1);
          }
        }
      }
    }
    __syncwarp();
    for (; waiting > 0; --waiting)
      token_again<T>(P, __shfl_sync(kAll, pending, waiting - 1), lane, reinterpret_cast<float *>(warp_words),
                     group_sums[warp], histogram);
    __syncwarp();
  }
  if (!P.counts) return;
  __syncthreads();
  for (int i = threadIdx.x; i < P.N; i += kQuadWarps * 32)
    if (histogram[i]) atomicAdd(P.counts + i, histogram[i]);
}

struct RouteGradParams {
  int64_t B;
  int N, K;
  int sigmoid, renorm, vec;
  float scale;
  const void *z;
  const int32_t *idx;
  const float *dw;
  void *dz;
};

// What the chosen of a token have in common of the gradient, over the lanes that `sum` and
// `most` reduce; then each one's.  z, g: the logit and the gradient of the weight, -inf and 0
// where there is none.
template <int n, class Sum, class Most>
__device__ __forceinline__ void chosen_gradients(const RouteGradParams &P, const float *z, const float *g, float *d,
                                                 Sum sum, Most most) {
  if (P.sigmoid) {
    float s[n], slope[n], total = 0.0f, along = 0.0f;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float x = z[i] == -INFINITY ? 0.0f : expf(-fabsf(z[i])), q = 1.0f / (1.0f + x);
      s[i] = z[i] == -INFINITY ? 0.0f : z[i] >= 0.0f ? q : x * q;
      slope[i] = x * q * q;  // s (1 - s)
      total += s[i];
      along += g[i] * s[i];
    }
    float mean = 0.0f;
    total = P.renorm ? sum(total) : 1.0f;
    if (P.renorm) mean = sum(along) / total;
    // a slope is at most its score, and so at most the total, which may be next to nothing
#pragma unroll
    for (int i = 0; i < n; ++i) d[i] = total > 0.0f ? P.scale * (g[i] - mean) * (slope[i] / total) : 0.0f;
  } else {
    float top = -INFINITY, w[n], total = 0.0f, along = 0.0f;
#pragma unroll
    for (int i = 0; i < n; ++i) top = fmaxf(top, z[i]);
    top = most(top);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      w[i] = z[i] == -INFINITY ? 0.0f : expf(z[i] - top);
      total += w[i];
    }
    total = fmaxf(sum(total), FLT_MIN);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      w[i] /= total;
      along += g[i] * w[i];
    }
    along = sum(along);
#pragma unroll
    for (int i = 0; i < n; ++i) d[i] = P.scale * w[i] * (g[i] - along);
  }
}

// Only the chosen logits have a gradient: four lanes a token, lane q with the places q, q + 4,
// ...; the warp's eight rows are set to zero together and the values written over.
template <class T, class O, int KP>
__global__ void __launch_bounds__(kWarps * 32) route_topk_grad_quad_kernel(const __grid_constant__ RouteGradParams P) {
  constexpr int n = (KP + 3) / 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, token = lane >> 2, q = lane & 3;
  auto sum = [](float v) {
    v += __shfl_xor_sync(kAll, v, 1);
    return v + __shfl_xor_sync(kAll, v, 2);
  };
  auto most = [](float v) {
    v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
    v = fmaxf(v, __shfl_xor_sync(kAll, v, 2));
    return v == -INFINITY ? 0.0f : v;
  };
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * 8; t0 < P.B; t0 += (int64_t)gridDim.x * kWarps * 8) {
    const int64_t t = t0 + token;
    const T *row = static_cast<const T *>(P.z) + t * P.N;
    int e[n];
    float z[n], g[n], d[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int k = 4 * i + q;
      e[i] = t < P.B && k < P.K ? P.idx[t * P.K + k] : -1;
      if ((unsigned)e[i] >= (unsigned)P.N) e[i] = -1;
      g[i] = e[i] >= 0 ? P.dw[t * P.K + k] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      z[i] = e[i] >= 0 ? settle(to_f32(row[e[i]])) : -INFINITY;
      if (z[i] == -INFINITY) g[i] = 0.0f, e[i] = -1;
    }
    // zeros while those are on their way
    const int64_t values = (P.B - t0 < 8 ? P.B - t0 : 8) * P.N;
    O *out = static_cast<O *>(P.dz) + t0 * P.N;
    int64_t done = 0;
    if (P.vec & 2) {  // the buffer at 16 bytes, and so every eighth row
      constexpr int kEach = 16 / (int)sizeof(O);
      for (int64_t i = lane; i < values / kEach; i += 32) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
      done = values / kEach * kEach;
    }
    for (int64_t i = done + lane; i < values; i += 32) out[i] = from_f32<O>(0.0f);
    chosen_gradients<n>(P, z, g, d, sum, most);
    // the same expert twice: the first place takes the sum
    float all[n] = {};
    bool first[n];
#pragma unroll
    for (int i = 0; i < n; ++i) first[i] = e[i] >= 0;
#pragma unroll
    for (int k = 0; k < 4 * n; ++k) {
      const int oe = __shfl_sync(kAll, e[k / 4], (lane & ~3) + (k & 3));
      const float od = __shfl_sync(kAll, d[k / 4], (lane & ~3) + (k & 3));
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (oe == e[i]) {
          all[i] += od;
          if (k < 4 * i + q) first[i] = false;
        }
    }
    __syncwarp();  // the zeros first
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (first[i]) out[token * P.N + e[i]] = from_f32<O>(all[i]);
  }
}

// Softmax over all experts, whose every logit has a gradient: a warp a token, lane r with the
// r-th chosen expert besides its share of the row.
template <class T, class O, int NPL>
__global__ void __launch_bounds__(kWarps * 32) route_topk_grad_kernel(const __grid_constant__ RouteGradParams P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, base = lane * NPL;
  auto sum = [](float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
  };
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < P.B; t += (int64_t)gridDim.x * kWarps) {
    const T *row = static_cast<const T *>(P.z) + t * P.N;
    O *out = static_cast<O *>(P.dz) + t * P.N;
    float p[NPL], top = -INFINITY, total = 0.0f;
    load_row<T, NPL>(row, P.N, P.vec & 1, lane, p);
    int e = -1;
    float g = 0.0f, zk = -INFINITY;
    if (lane < P.K) {
      e = P.idx[t * P.K + lane];
      if ((unsigned)e >= (unsigned)P.N) e = -1;
      if (e >= 0) {
        g = P.dw[t * P.K + lane];
        zk = settle(to_f32(row[e]));
      }
      if (zk == -INFINITY) g = 0.0f, e = -1;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = fmaxf(top, p[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) total += p[i] = expf(p[i] - top);
    const float inv = 1.0f / fmaxf(sum(total), FLT_MIN);
    const float pk = e >= 0 ? expf(zk - top) * inv : 0.0f;
    float d = P.scale * g * pk;
    const float rest = -sum(d);
    // the same expert twice: the first of the lanes takes the sum
    const unsigned same = __match_any_sync(kAll, e);
    bool first = e >= 0;
    if (__any_sync(kAll, e >= 0 && (same & (same - 1)))) {
      float all = 0.0f;
      for (int r = 0; r < P.K; ++r) {
        const float o = __shfl_sync(kAll, d, r);
        if (same >> r & 1) all += o;
      }
      d = all;
      first = first && lane == __ffs(same) - 1;
    }
    if (P.vec & 2) {
      constexpr int kBytes = NPL * (int)sizeof(O), kPart = kBytes < 16 ? kBytes : 16;
      alignas(16) O v[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = from_f32<O>(p[i] * inv * rest);
      if (base < P.N) {
#pragma unroll
        for (int i = 0; i < kBytes / kPart; ++i) {
          const char *from = reinterpret_cast<const char *>(v) + i * kPart;
          char *to = reinterpret_cast<char *>(out + base) + i * kPart;
          if constexpr (kPart == 16)
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
          else if constexpr (kPart == 8)
            *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(from);
          else if constexpr (kPart == 4)
            *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
          else
            *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (base + i < P.N) out[base + i] = from_f32<O>(p[i] * inv * rest);
    }
    __syncwarp();  // the row first
    if (first) out[e] = from_f32<O>(pk * rest + d);
  }
}

// ----------------------------------------------------------------- host side
// Tokens from which four lanes take one: that many more instructions in a row take 4 to 20 us
// before there are warps enough to fill the SMs.  256 experts in groups, biases: 2048 tokens
// 22 us, 9 a warp a token; 8192: 20 and 22; 65536: 50 and 140.  64 experts, logits alone:
// 2048: 4.1 and 3.5; 8192: 4.7 and 6.7; 65536: 13 and 36.
constexpr int kQuadFrom = 8192, kClusterTokens = 128;

bool off(const void *p, int a) { return (uintptr_t)p % a != 0; }
int size_of(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }
bool known(int type) { return type == MOE_TYPE_BF16 || type == MOE_TYPE_F16 || type == MOE_TYPE_F32; }

int check_topk(const moe_route_cfg *c, int type) {
  if (!c || !known(type)) return MOE_ERR_INVALID;
  if (c->B < 0 || c->N <= 0 || c->K <= 0) return MOE_ERR_INVALID;
  if (c->score_fn != MOE_SCORE_SOFTMAX && c->score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID;
  if (c->N > kMaxN || c->K > 16 || c->K > c->N) return MOE_ERR_UNSUPPORTED;
  if (c->n_group > 1 && (c->n_group > 32 || c->N % c->n_group || c->N / c->n_group < 2 || c->topk_group < 1 ||
                         c->topk_group > c->n_group || c->K > c->topk_group * (c->N / c->n_group)))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// Experts a lane holds, and whether its share of a row is one aligned piece.
int per_lane(int N) {
  int npl = 1;
  while (npl * 32 < N) npl *= 2;
  return npl;
}
bool whole(const void *p, int N, int npl, int size) {
  const int bytes = npl * size, part = bytes < 16 ? bytes : 16;
  return N % npl == 0 && !off(p, part) && (int64_t)N * size % part == 0;
}
template <class F>
int with_npl(int npl, F f) {
  using std::integral_constant;
  switch (npl) {
    case 1: return f(integral_constant<int, 1>());
    case 2: return f(integral_constant<int, 2>());
    case 4: return f(integral_constant<int, 4>());
    case 8: return f(integral_constant<int, 8>());
    default: return f(integral_constant<int, 16>());
  }
}
template <class F>
int with_type(int type, F f) {
  if (type == MOE_TYPE_F32) return f(float());
  return type == MOE_TYPE_F16 ? f(__half()) : f(__nv_bfloat16());
}
cudaLaunchConfig_t one_cluster(int blocks, cudaLaunchAttribute *attr, cudaStream_t st) {
  cudaLaunchConfig_t launch = {};
  launch.gridDim = dim3((unsigned)blocks);
  launch.blockDim = dim3(kWarps * 32);
  launch.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)blocks;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  launch.attrs = attr;
  launch.numAttrs = 1;
  return launch;
}
// Blocks of the largest cluster of this kernel that the device runs: 16 where its processors come
// in groups of enough, else half of that and so on.  Asked once a device.
template <auto kernel>
int largest_cluster(int *most) {
  static int sizes[kMaxDevices] = {};
  static std::mutex asked;
  const int dev = device_slot();
  if (dev < 0) return dev;
  const std::lock_guard<std::mutex> lock(asked);
  if (sizes[dev] == 0) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return set_cuda_error(e);
    int size = kClusterTokens / kWarps;
    for (; size > 1; size /= 2) {
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t launch = one_cluster(size, &attr, nullptr);
      int fit = 0;
      if (cudaOccupancyMaxActiveClusters(&fit, kernel, &launch) == cudaSuccess && fit > 0) break;
      cudaGetLastError();  // a size that the device does not take
    }
    sizes[dev] = size;
  }
  *most = sizes[dev];
  return MOE_OK;
}
unsigned grid_of(int64_t B) {
  const int64_t need = (B + kWarps - 1) / kWarps, most = (int64_t)device_sm_count() * 32;
  return (unsigned)(need < most ? need : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_route_topk(const moe_route_cfg *cfg, int type, const void *logits, const float *bias,
                              int32_t *topk_idx, float *topk_w, int32_t *expert_counts, void *stream) {
  const int rc = check_topk(cfg, type);
  if (rc != MOE_OK) return rc;
  if (bias && cfg->score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID;
  if (off(bias, 4) || off(topk_idx, 4) || off(topk_w, 4) || off(expert_counts, 4)) return MOE_ERR_INVALID;
  cudaStream_t st = as_stream(stream);
  if (cfg->B > 0 && (!logits || !topk_idx || !topk_w || off(logits, size_of(type)))) return MOE_ERR_INVALID;
  auto zero = [&] {
    if (!expert_counts) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(expert_counts, 0, sizeof(int32_t) * cfg->N, st);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e);
  };
  if (cfg->B == 0) return zero();
  const int npl = per_lane(cfg->N), n_group = cfg->n_group > 1 ? cfg->n_group : 1, gs = cfg->N / n_group;
  RouteParams P = {cfg->B, cfg->N, cfg->K, n_group, n_group > 1 ? cfg->topk_group : 1,
                   cfg->score_fn == MOE_SCORE_SIGMOID, cfg->renorm != 0, whole(logits, cfg->N, npl, size_of(type)),
                   cfg->route_scale, logits, bias, topk_idx, topk_w, expert_counts,
                   (uint32_t)(((1u << 20) + gs - 1) / gs), npl};
  // Four lanes a token where rows come in aligned eights and groups in 32s, and there are
  // tokens for every SM's warps.
  const bool eights = cfg->N % 8 == 0 && !off(logits, 16) && !off(bias, 16) && (n_group == 1 || (gs % 32 == 0 && n_group <= kMostGroups));
  if (eights && cfg->B >= kQuadFrom) {
    const int cleared = zero();
    if (cleared != MOE_OK) return cleared;
    const uint32_t smem = (uint32_t)(kQuadWarps * quad_words(cfg->N, n_group) * 4);
    return with_type(type, [&](auto t) {
      auto run = [&](auto kernel) {
        const int64_t need = (cfg->B + kQuadWarps * 8 - 1) / (kQuadWarps * 8), most = (int64_t)device_sm_count() * 3;
        if (smem > 32 * 1024) {
          const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     kQuadWarps * quad_words(kMaxN, 2) * 4);
          if (e != cudaSuccess) return set_cuda_error(e);
        }
        kernel<<<(unsigned)(need < most ? need : most), kQuadWarps * 32, smem, st>>>(P);
        return check_launch();
      };
      return cfg->K <= 8 ? run(route_topk_quad_kernel<decltype(t), 8>) : run(route_topk_quad_kernel<decltype(t), 16>);
    });
  }
  // A cluster of up to 16 blocks needs no counts set to zero (3.5 us), as long as a warp has one
  // token (128 tokens on 8 blocks: 13 us; 11 with counts set to zero).
  const int64_t blocks = (cfg->B + kWarps - 1) / kWarps;
  return with_type(type, [&](auto t) {
    return with_npl(npl, [&](auto n) {
      if (expert_counts && blocks <= kClusterTokens / kWarps) {
        constexpr auto kernel = route_topk_kernel<decltype(t), decltype(n)::value, true>;
        int most = 0;
        const int found = largest_cluster<kernel>(&most);
        if (found != MOE_OK) return found;
        if (blocks <= most) {
          cudaLaunchAttribute attr;
          const cudaLaunchConfig_t launch = one_cluster((int)blocks, &attr, st);
          const cudaError_t e = cudaLaunchKernelEx(&launch, kernel, P);
          return e == cudaSuccess ? check_launch() : set_cuda_error(e);
        }
      }
      const int cleared = zero();
      if (cleared != MOE_OK) return cleared;
      route_topk_kernel<decltype(t), n.value, false><<<grid_of(cfg->B), kWarps * 32, 0, st>>>(P);
      return check_launch();
    });
  });
}

extern "C" int moe_route_topk_backward(const moe_route_cfg *cfg, int type, const void *logits,
                                       const int32_t *topk_idx, const float *dtopk_w, int out_type, void *dlogits,
                                       void *stream) {
  const int rc = check_topk(cfg, type);
  if (rc != MOE_OK) return rc;
  if (out_type != type && out_type != MOE_TYPE_F32 && (type != MOE_TYPE_F32 || !known(out_type))) return MOE_ERR_INVALID;
  if (cfg->B == 0) return MOE_OK;
  if (!logits || !topk_idx || !dtopk_w || !dlogits || off(logits, size_of(type)) || off(topk_idx, 4) ||
      off(dtopk_w, 4) || off(dlogits, size_of(out_type)))
    return MOE_ERR_INVALID;
  const int npl = per_lane(cfg->N);
  const bool every = cfg->score_fn == MOE_SCORE_SOFTMAX && !cfg->renorm;  // logits have a gradient
  RouteGradParams P = {cfg->B, cfg->N, cfg->K, cfg->score_fn == MOE_SCORE_SIGMOID, cfg->renorm != 0,
                       whole(logits, cfg->N, npl, size_of(type)) ? 1 : 0, cfg->route_scale, logits, topk_idx, dtopk_w, dlogits};
  if (every ? whole(dlogits, cfg->N, npl, size_of(out_type)) : !off(dlogits, 16)) P.vec |= 2;
  cudaStream_t st = as_stream(stream);
  auto run = [&](auto t, auto o) {
    if (!every) {
      const unsigned grid = grid_of((cfg->B + 7) / 8);
      if (cfg->K <= 8)
        route_topk_grad_quad_kernel<decltype(t), decltype(o), 8><<<grid, kWarps * 32, 0, st>>>(P);
      else
        route_topk_grad_quad_kernel<decltype(t), decltype(o), 16><<<grid, kWarps * 32, 0, st>>>(P);
      return check_launch();
    }
    return with_npl(npl, [&](auto n) {
      route_topk_grad_kernel<decltype(t), decltype(o), n.value><<<grid_of(cfg->B), kWarps * 32, 0, st>>>(P);
      return check_launch();
    });
  };
  return with_type(type, [&](auto t) {
    if (out_type == MOE_TYPE_F32) return run(t, float());
    if constexpr (std::is_same<decltype(t), float>::value)
      return out_type == MOE_TYPE_F16 ? run(t, __half()) : run(t, __nv_bfloat16());
    else
      return run(t, t);
  });
}
