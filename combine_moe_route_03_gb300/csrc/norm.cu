// moe_rms_norm and moe_rms_norm_backward: the root-mean-square norm in front of a layer,
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w,
// y in 16 bits and / or in 8 with the scales that the FP8 products take, and its gradients
//   g = dy w,  dx = r (g - h r^2 mean(g h)) + dres,  dw = sum over rows of dy h r.
//
// Bound by memory: a value is read and written once each way, against about 10 operations
// (25 with codes).  A row is held in the registers of one block from its loads to its stores
// (a warp, where rows are short), so each statistic is a reduction inside it, binary32, in a
// fixed order: lanes, then warps.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "columns.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
// Most threads of a row's block: 4 vectors a thread reach kMaxH with 512, and so keep 128
// registers a thread.
template <int V, int N, bool kBlock>
constexpr int kMost = !kBlock ? 256 : V * N >= 32 ? 512 : 1024;

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

// V consecutive values (8, or 1 where a row's start or length allows no vector).
template <class T, int V>
struct alignas(V * sizeof(T) >= 16 ? 16 : V * sizeof(T)) Pack {
  T t[V];
};
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_once(const T *p) {
  Pack<T, V> o;
  if constexpr (V * sizeof(T) >= 16) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4 *>(&o)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  } else {
    o = *reinterpret_cast<const Pack<T, V> *>(p);
  }
  return o;
}
template <class T, int V>
__device__ __forceinline__ void store(T *p, const float *f) {
  Pack<T, V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) o.t[i] = from_f32<T>(f[i]);
  if constexpr (V * sizeof(T) >= 16) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<uint4 *>(&o)[i];
  } else {
    *reinterpret_cast<Pack<T, V> *>(p) = o;
  }
}
template <int V>
__device__ __forceinline__ void load_w(const float *p, float *f) {
  if constexpr (V == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    f[0] = __ldg(p);
  }
}

// Sums of one or two values over the threads of a row, the same bits in all of them.  `part`
// is of the row alone; two calls in turn take two of them, so one barrier a call is enough.
template <int kSums>
__device__ __forceinline__ void row_sum(float *v, float (*part)[32], bool block) {
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int d = 16; d; d >>= 1) v[s] += __shfl_xor_sync(0xffffffffu, v[s], d);
  if (!block) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int s = 0; s < kSums; ++s)
    if (lane == 0) part[s][warp] = v[s];
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    v[s] = lane < warps ? part[s][lane] : 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1) v[s] += __shfl_xor_sync(0xffffffffu, v[s], d);
  }
}

struct NormParams {
  int64_t rows;
  int H;
  float eps, inv_h;
  int fmt;
  const void *x, *res;
  const float *w;
  void *sum, *y;
  uint8_t *A, *A_sf;
};

// Eight values of a row -> e4m3 codes.  The 16 lanes of a block of 128 columns are
// neighbours (8-bit outputs have columns in multiples of 128 and blocks of whole warps).
__device__ __forceinline__ void store_codes(const NormParams &P, int64_t row, int col, const float *f,
                                            unsigned mask) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
  for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, d));
  const int kb = col >> 7;
  uint32_t c[4];
  if (P.fmt == MOE_FMT_FP8) {
    const int e = ue8m0_exp(amax);
    const float inv = pow2i(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
    if ((col & 127) == 0) P.A_sf[sf_byte_off(row, kb, sf_groups(P.H))] = (uint8_t)(e + 127);
  } else {
    float s = __fdiv_rn(amax, 448.0f);
    if (s == 0.0f) s = 1.0f;
    if (s > 0x1p-100f && s < 0x1p100f) {
      // The quotient to the nearest from the reciprocal to the nearest, and one step with the
      // exact remainder (Markstein, Computation of elementary functions on the IBM RISC
      // System/6000 processor, 1990): 8192 x 7168, 94 us with a division a value.
      const float inv = __frcp_rn(s);
      auto over = [&](float x) {
        const float q = x * inv;
        return fmaf(fmaf(-q, s, x), inv, q);
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = e4m3x2(over(f[2 * i]), over(f[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s));
    }
    if ((col & 127) == 0) reinterpret_cast<float *>(P.A_sf)[row * (P.H >> 7) + kb] = s;
  }
  *reinterpret_cast<uint2 *>(P.A + row * P.H + col) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// T: x and y; R: residual and sum.  A thread holds N packs of V values of its row: columns
// (t + i * threads) * V.  kBlock: a row a block, else a row a warp.
template <class T, class R, int V, int N, bool kBlock>
__global__ void __launch_bounds__(kMost<V, N, kBlock>) norm_kernel(const NormParams P) {
  __shared__ float part[1][32];
  const int threads = kBlock ? blockDim.x : 32, t = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int64_t row = kBlock ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= P.rows) return;  // a whole warp (kBlock: never)
  const T *x = static_cast<const T *>(P.x) + row * P.H;
  const R *res = static_cast<const R *>(P.res) + row * P.H;
  float h[N][V];
  Pack<T, V> px[N];
  Pack<R, V> pr[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (t + i * threads) * V;
    if (c < P.H) px[i] = load_once<T, V>(x + c);
    if (P.res && c < P.H) pr[i] = load_once<R, V>(res + c);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (t + i * threads) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[i][j] = c < P.H ? to_f32(px[i].t[j]) : 0.0f;
      if (P.res && c < P.H) h[i][j] += to_f32(pr[i].t[j]);
      ss += h[i][j] * h[i][j];
    }
  }
  if (P.sum) {
    R *sum = static_cast<R *>(P.sum) + row * P.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (t + i * threads) * V;
      if (c < P.H) store<R, V>(sum + c, h[i]);
    }
  }
  row_sum<1>(&ss, part, kBlock);
  const float r = rsqrtf(ss * P.inv_h + P.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (t + i * threads) * V;
    const unsigned mask = __ballot_sync(0xffffffffu, c < P.H);  // whole blocks of 16 lanes
    if (c >= P.H) continue;
    float w[V];
    load_w<V>(P.w + c, w);
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] = h[i][j] * r * w[j];
    if (P.y) store<T, V>(static_cast<T *>(P.y) + row * P.H + c, h[i]);
    if constexpr (V == 8)
      if (P.A) store_codes(P, row, c, h[i], mask);
  }
}

// ------------------------------------------------------- many rows of a block each
// Persistent blocks whose threads copy their own packs of the rows to come into shared memory
// (asynchronously, kStages rows deep) and read them back themselves, so nothing waits for
// another thread but the row's sums: loads of the next rows run beside a row's statistics and
// stores.  8192 rows of 7168, residual, 16 bits and codes: 156 us a row a block without it.
__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last kBut of this thread's groups have landed.
template <int kBut>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kBut) : "memory");
}

// 16-byte pieces of this thread's N packs of 8 values, interleaved over the threads.
template <class T, int N>
struct Own {
  static constexpr int kPieces = sizeof(T) / 2;
  static __device__ __forceinline__ void fetch(uint4 *slot, const T *row, int t, int threads, int packs) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = t + i * threads;
      if (c < packs)
#pragma unroll
        for (int k = 0; k < kPieces; ++k) copy16(slot + k * packs + c, row + c * 8 + k * 8 / kPieces);
    }
  }
  static __device__ __forceinline__ Pack<T, 8> read(const uint4 *slot, int c, int packs) {
    Pack<T, 8> o;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) reinterpret_cast<uint4 *>(&o)[k] = slot[k * packs + c];
    return o;
  }
};

template <class T, class R, int N, int kStages>
__global__ void __launch_bounds__(512, N <= 2 ? 2 : 1) norm_rows_kernel(const NormParams P) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][1][32];
  const int threads = blockDim.x, t = threadIdx.x, packs = P.H >> 3;
  const int of_x = packs * Own<T, N>::kPieces, stage = of_x + (P.res ? packs * Own<R, N>::kPieces : 0);
  const T *x = static_cast<const T *>(P.x);
  const R *res = static_cast<const R *>(P.res);
  auto fetch = [&](int64_t row, int s) {
    if (row < P.rows) {
      Own<T, N>::fetch(ring + s * stage, x + row * P.H, t, threads, packs);
      if (P.res) Own<R, N>::fetch(ring + s * stage + of_x, res + row * P.H, t, threads, packs);
    }
    copies_done();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  int s = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < P.rows; row += gridDim.x, turn ^= 1) {
    wait_copies<kStages - 1>();
    const uint4 *slot = ring + s * stage;
    float h[N][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = t + i * threads;
      if (c < packs) {
        const Pack<T, 8> px = Own<T, N>::read(slot, c, packs);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = to_f32(px.t[j]);
        if (P.res) {
          const Pack<R, 8> pr = Own<R, N>::read(slot + of_x, c, packs);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += to_f32(pr.t[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
        if (P.sum) store<R, 8>(static_cast<R *>(P.sum) + row * P.H + c * 8, h[i]);
      }
    }
    row_sum<1>(&ss, part[turn], true);
    fetch(row + (int64_t)kStages * gridDim.x, s);  // what the slot held is in registers
    if (++s == kStages) s = 0;
    const float r = rsqrtf(ss * P.inv_h + P.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = t + i * threads;
      const unsigned mask = __ballot_sync(0xffffffffu, c < packs);  // whole blocks of 16 lanes
      if (c >= packs) continue;
      float w[8];
      load_w<8>(P.w + c * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * r * w[j];
      if (P.y) store<T, 8>(static_cast<T *>(P.y) + row * P.H + c * 8, h[i]);
      if (P.A) store_codes(P, row, c * 8, h[i], mask);
    }
  }
}

struct NormGradParams {
  int64_t rows;
  int H;
  float eps, inv_h;
  const void *h, *dy, *dres;
  const float *w;
  void *dx;
  float *part;  // [blocks][H] sums of dw, or NULL
  int dres_ahead;  // copied with the row
};

// T: dy; R: h, dres and dx.  Blocks (kBlock) or warps take every so many-th row, and keep the
// sums of dw of their rows in registers: a column has the same thread in every row.
template <class T, class R, int V, int N, bool kBlock>
__global__ void __launch_bounds__(kMost<V, N, kBlock>) norm_grad_kernel(const NormGradParams P) {
  __shared__ float part[2][2][32];
  const int threads = kBlock ? blockDim.x : 32, t = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int groups = kBlock ? 1 : blockDim.x >> 5, group = kBlock ? 0 : threadIdx.x >> 5;
  const int64_t first = (int64_t)blockIdx.x * groups + group, step = (int64_t)gridDim.x * groups;
  float dw[N][V] = {};
  int turn = 0;
  for (int64_t row = first; row < P.rows; row += step, turn ^= 1) {
    const R *h = static_cast<const R *>(P.h) + row * P.H;
    const T *dy = static_cast<const T *>(P.dy) + row * P.H;
    const R *dres = static_cast<const R *>(P.dres) + row * P.H;
    R *dx = static_cast<R *>(P.dx) + row * P.H;
    Pack<R, V> ph[N], pr[N];
    Pack<T, V> pd[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (t + i * threads) * V;
      if (c < P.H) {
        ph[i] = load_once<R, V>(h + c);
        pd[i] = load_once<T, V>(dy + c);
        if (P.dres) pr[i] = load_once<R, V>(dres + c);
      }
    }
    float s[2] = {0.0f, 0.0f};  // of h^2, and of g h
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (t + i * threads) * V;
      if (c >= P.H) continue;
      float w[V];
      load_w<V>(P.w + c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float hf = to_f32(ph[i].t[j]);
        s[0] += hf * hf;
        s[1] += to_f32(pd[i].t[j]) * w[j] * hf;
      }
    }
    row_sum<2>(s, part[turn], kBlock);
    const float r = rsqrtf(s[0] * P.inv_h + P.eps);
    const float along = s[1] * P.inv_h * r * r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (t + i * threads) * V;
      if (c >= P.H) continue;
      float w[V], o[V];
      load_w<V>(P.w + c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float hf = to_f32(ph[i].t[j]), d = to_f32(pd[i].t[j]);
        dw[i][j] += d * (hf * r);
        o[j] = r * (d * w[j] - hf * along);
        if (P.dres) o[j] += to_f32(pr[i].t[j]);
      }
      store<R, V>(dx + c, o);
    }
  }
  if (!P.part) return;
  if constexpr (!kBlock) {
    // the warps' sums meet in shared memory, one warp after the other
    extern __shared__ float all[];  // [H]
    for (int g = 0; g < groups; ++g) {
      if (g == group)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int c = (t + i * threads) * V + j;
            if (c < P.H) all[c] = (g ? all[c] : 0.0f) + dw[i][j];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < P.H; c += blockDim.x) P.part[(int64_t)blockIdx.x * P.H + c] = all[c];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (t + i * threads) * V;
      if (c < P.H) store<float, V>(P.part + (int64_t)blockIdx.x * P.H + c, dw[i]);
    }
  }
}

// The same with rows copied ahead, and the sums of the next row made beside this one's
// gradients, so that the one barrier a row is reached with its sums long written: 8192 rows of
// 7168, all in 16 bits, 276 us a row at a time, 124 with the barrier between a row's halves.
// Two packs a thread and 512 threads leave registers for both (8192 x 7168: 77 us; one pack,
// 896 threads: 86).
template <class T, class R, int N, int kStages, int kBound>
__global__ void __launch_bounds__(kBound, 1) norm_grad_rows_kernel(const NormGradParams P) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][2][32];
  const int threads = blockDim.x, t = threadIdx.x, packs = P.H >> 3;
  const int warp = t >> 5, lane = t & 31, warps = threads >> 5;
  const int of_h = packs * Own<R, N>::kPieces, of_dy = of_h + packs * Own<T, N>::kPieces;
  const int stage = of_dy + (P.dres_ahead ? of_h : 0);
  const R *h = static_cast<const R *>(P.h), *dres = static_cast<const R *>(P.dres);
  const T *dy = static_cast<const T *>(P.dy);
  auto fetch = [&](int64_t row, int s) {
    if (row < P.rows) {
      Own<R, N>::fetch(ring + s * stage, h + row * P.H, t, threads, packs);
      Own<T, N>::fetch(ring + s * stage + of_h, dy + row * P.H, t, threads, packs);
      if (P.dres_ahead) Own<R, N>::fetch(ring + s * stage + of_dy, dres + row * P.H, t, threads, packs);
    }
    copies_done();
  };
  float w[N][8], dw[N][8] = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (t + i * threads < packs) load_w<8>(P.w + (t + i * threads) * 8, w[i]);
  // this thread's part of the sums of h^2 and g h of the row in slot s, to `part`
  auto sums = [&](int s, int turn) {
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = t + i * threads;
      if (c >= packs) continue;
      const Pack<R, 8> ph = Own<R, N>::read(ring + s * stage, c, packs);
      const Pack<T, 8> pd = Own<T, N>::read(ring + s * stage + of_h, c, packs);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hf = to_f32(ph.t[j]);
        sum[0] += hf * hf;
        sum[1] += to_f32(pd.t[j]) * w[i][j] * hf;
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int d = 16; d; d >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], d);
      if (lane == 0) part[turn][k][warp] = sum[k];
    }
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  int s = 0, turn = 0;
  wait_copies<kStages - 1>();
  sums(0, 0);
  __syncthreads();
  for (int64_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
    float total[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      total[k] = lane < warps ? part[turn][k][lane] : 0.0f;
#pragma unroll
      for (int d = 16; d; d >>= 1) total[k] += __shfl_xor_sync(0xffffffffu, total[k], d);
    }
    const float r = rsqrtf(total[0] * P.inv_h + P.eps);
    const float along = total[1] * P.inv_h * r * r * r;
    const int next = s + 1 == kStages ? 0 : s + 1;
    turn ^= 1;
    wait_copies<kStages - 2>();
    if (row + gridDim.x < P.rows) sums(next, turn);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = t + i * threads;
      if (c >= packs) continue;
      const Pack<R, 8> ph = Own<R, N>::read(ring + s * stage, c, packs);
      const Pack<T, 8> pd = Own<T, N>::read(ring + s * stage + of_h, c, packs);
      float o[8];
      if (P.dres) {
        const Pack<R, 8> pr = P.dres_ahead ? Own<R, N>::read(ring + s * stage + of_dy, c, packs)
                                           : load_once<R, 8>(dres + row * P.H + c * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = to_f32(pr.t[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hf = to_f32(ph.t[j]), d = to_f32(pd.t[j]);
        dw[i][j] += d * (hf * r);
        o[j] = fmaf(d * w[i][j], r, o[j]) - hf * along;
      }
      store<R, 8>(static_cast<R *>(P.dx) + row * P.H + c * 8, o);
    }
    __syncthreads();  // the next row's sums are written, this one's slot is read
    fetch(row + (int64_t)kStages * gridDim.x, s);
    s = next;
  }
  if (!P.part) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = t + i * threads;
    if (c < packs) store<float, 8>(P.part + (int64_t)blockIdx.x * P.H + c * 8, dw[i]);
  }
}

// ----------------------------------------------------------------- host side
// How a row is spread: V values a load, n loads a thread, `threads` of a row (32: a warp a
// row).  A block a row from 64 loads of 32 lanes on; with few rows it takes more threads with
// fewer loads each.
struct Shape {
  int V, n, threads;
  bool block;
};
Shape shape_of(int H, bool vec, bool few) {
  Shape s;
  s.V = vec ? 8 : 1;
  const int packs = (H + s.V - 1) / s.V, most = vec ? 4 : 16;
  s.block = packs > 32 * most || (few && packs > 64);
  if (!s.block) {
    s.threads = 32;
    s.n = packs <= 32 ? 1 : packs <= 64 ? 2 : most;
    if (!vec) s.n = most;
    return s;
  }
  s.n = vec ? (few && packs <= 1024 ? 1 : few ? 2 : 4) : (packs <= 4096 ? 4 : 16);
  s.threads = ((packs + s.n - 1) / s.n + 31) / 32 * 32;  // kMaxH takes 1024 at most
  return s;
}

// Blocks an SM of the gradients: one kernel more adds up a part of dw each.
constexpr int kMostGradBlocks = 8;

// The kernels that copy rows ahead: threads with n packs of a row, up to 4 rows ahead, and as
// many blocks as the SMs hold.  They take over where each block has rows enough to copy ahead,
// and rows of several warps.
struct Ahead {
  int n, threads, stages, most;  // most: blocks of an SM by shared memory; 0: not to be used
  uint32_t smem;
};
Ahead ahead_of(int64_t rows, int H, bool vec, int row_bytes, bool grad) {
  Ahead a = {};
  const int packs = H / 8;
  if (!vec || H < (grad ? 256 : 1024)) return a;  // (forward, 512 columns: a warp a row is as fast)
  a.n = grad ? (packs > 256 ? 2 : 1) : packs > 1024 ? 4 : 2;
  a.threads = ((packs + a.n - 1) / a.n + 31) / 32 * 32;
  // 16 bits and a residual: two blocks of two rows an SM; the backward's one block of 4 or 3
  a.stages = grad ? (row_bytes > 54 * 1024 ? 3 : 4) : row_bytes > 24 * 1024 || a.n == 4 ? 2 : 4;
  a.smem = (uint32_t)(a.stages * row_bytes);
  a.most = std::min(2048 / a.threads, (int)(220u * 1024 / (a.smem + 1024)));
  if (!grad && rows < 4 * (int64_t)device_sm_count()) a.most = 0;
  if (grad) a.most = std::min(a.most, kMostGradBlocks);
  return a;
}
// Grid of such a kernel: the blocks that are resident, no more than rows.
template <auto kernel>
int resident(const Ahead &a, int64_t rows, int *grid) {
  static int regs[kMaxDevices] = {};
  static std::mutex asked;  // threads whose first calls come at once
  const int dev = device_slot();
  if (dev < 0) return dev;
  const std::lock_guard<std::mutex> lock(asked);
  if (regs[dev] == 0) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return set_cuda_error(e);
    regs[dev] = (at.numRegs + 7) / 8 * 8;
  }
  const int by_regs = 65536 / (regs[dev] * a.threads);
  const int64_t most = (int64_t)device_sm_count() * std::max(1, std::min(a.most, by_regs));
  *grid = (int)std::min(rows, most);
  return MOE_OK;
}

int check_norm(int64_t rows, int H, float eps, int type, int res_type) {
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_F16) return MOE_ERR_INVALID;
  if (res_type != type && res_type != MOE_TYPE_F32) return MOE_ERR_INVALID;
  if (rows < 0 || H < 1 || !(eps >= 0.0f)) return MOE_ERR_INVALID;
  if (H > kMaxH || rows > INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Calls f with the types and the shape as constants: of the gradients (kGrad) whole vectors only
// where no rows are copied ahead, rows below 256 columns and those of binary32 past 12456.
template <bool kGrad, class F>
int with_shape(int type, int res_type, const Shape &s, F f) {
  auto shaped = [&](auto t, auto r) {
    using std::integral_constant;
    const integral_constant<bool, true> block;
    const integral_constant<bool, false> warp;
    const integral_constant<int, 8> v8;
    const integral_constant<int, 1> v1;
    const integral_constant<int, 1> n1;
    [[maybe_unused]] const integral_constant<int, 2> n2;
    const integral_constant<int, 4> n4;
    const integral_constant<int, 16> n16;
    if (s.V == 1) {
      if (s.n == 4) return f(t, r, v1, n4, block);
      return s.block ? f(t, r, v1, n16, block) : f(t, r, v1, n16, warp);
    }
    if constexpr (kGrad) {
      if constexpr (std::is_same<decltype(r), float>::value)
        if (s.block) return f(t, r, v8, n4, block);
      return f(t, r, v8, n1, warp);
    } else {
      if (s.n == 1) return s.block ? f(t, r, v8, n1, block) : f(t, r, v8, n1, warp);
      if (s.n == 2) return s.block ? f(t, r, v8, n2, block) : f(t, r, v8, n2, warp);
      return s.block ? f(t, r, v8, n4, block) : f(t, r, v8, n4, warp);
    }
  };
  if (type == MOE_TYPE_BF16)
    return res_type == MOE_TYPE_F32 ? shaped(__nv_bfloat16(), float()) : shaped(__nv_bfloat16(), __nv_bfloat16());
  return res_type == MOE_TYPE_F32 ? shaped(__half(), float()) : shaped(__half(), __half());
}

template <bool kGrad, class F>
int with_ahead(int type, int res_type, const Ahead &a, F f) {
  auto shaped = [&](auto t, auto r) {
    using std::integral_constant;
    [[maybe_unused]] const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    [[maybe_unused]] const integral_constant<int, 3> three;
    const integral_constant<int, 4> four;
    const integral_constant<int, 512> b512;
    [[maybe_unused]] const integral_constant<int, 1024> b1024;
    if constexpr (kGrad) {
      if (a.n == 1) return f(t, r, one, four, b512);  // rows of up to 20 KB
      if (a.threads > 512) return a.stages == 4 ? f(t, r, two, four, b1024) : f(t, r, two, three, b1024);
      if constexpr (std::is_same<decltype(r), float>::value)  // 16-bit rows this short leave room for 4
        if (a.stages == 3) return f(t, r, two, three, b512);
      return f(t, r, two, four, b512);
    } else {
      if (a.n == 4) return f(t, r, four, two, b512);
      return a.stages == 4 ? f(t, r, two, four, b512) : f(t, r, two, two, b512);
    }
  };
  if (type == MOE_TYPE_BF16)
    return res_type == MOE_TYPE_F32 ? shaped(__nv_bfloat16(), float()) : shaped(__nv_bfloat16(), __nv_bfloat16());
  return res_type == MOE_TYPE_F32 ? shaped(__half(), float()) : shaped(__half(), __half());
}

bool off(const void *p, int a) { return (uintptr_t)p % a != 0; }

// Blocks of the backward: each holds the sums of dw of its rows, which a second kernel reads.
int grad_blocks(int64_t rows, const Shape &s) {
  const int groups = s.block ? 1 : 8;
  const int64_t need = (rows + groups - 1) / groups;
  const int64_t most = (int64_t)device_sm_count() * (!s.block ? 4 : std::max(2, std::min(kMostGradBlocks, 2048 / s.threads)));
  return (int)(need < most ? need : most);
}
// Rows copied ahead by the backward, with dres where three of a row's tensors fit, else without
// (dres_ahead: which).
Ahead grad_ahead(int64_t rows, int H, bool vec, int size, bool dres, int *dres_ahead) {
  Ahead a = ahead_of(rows, H, vec, H * (2 + size * (dres ? 2 : 1)), true);
  *dres_ahead = dres;
  if (a.most == 0 && dres) {  // rows too long for three: dres is loaded as it is needed
    *dres_ahead = 0;
    a = ahead_of(rows, H, vec, H * (2 + size), true);
  }
  return a;
}
Shape grad_shape(const moe_norm_grad_args &a) {
  bool vec = a.H % 8 == 0;
  for (const void *p : {a.h, a.dy, a.dres, (const void *)a.w, (const void *)a.dx})
    if (off(p, 16)) vec = false;
  return shape_of(a.H, vec, false);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_rms_norm(const moe_norm_args *a, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  const int rc = check_norm(a->rows, a->H, a->eps, a->type, a->res_type);
  if (rc != MOE_OK) return rc;
  const bool coded = a->fmt == MOE_FMT_FP8 || a->fmt == MOE_FMT_FP8_F32;
  if (!coded && a->fmt != MOE_FMT_BF16) return MOE_ERR_INVALID;
  if (coded && a->H % 128) return MOE_ERR_UNSUPPORTED;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->w || (a->sum && !a->residual) || (!coded && (!a->y || a->A || a->A_sf)) || (coded && (!a->A || !a->A_sf)))
    return MOE_ERR_INVALID;
  const int size = a->res_type == MOE_TYPE_F32 ? 4 : 2;
  if (off(a->x, 2) || off(a->y, 2) || off(a->residual, size) || off(a->sum, size) || off(a->w, 4)) return MOE_ERR_INVALID;
  bool vec = a->H % 8 == 0;
  for (const void *p : {a->x, a->residual, (const void *)a->w, (const void *)a->sum, (const void *)a->y})
    if (off(p, 16)) vec = false;
  if (coded && (!vec || off(a->A, 16) || off(a->A_sf, 16))) return MOE_ERR_INVALID;
  NormParams P = {a->rows, a->H, a->eps, 1.0f / a->H, a->fmt, a->x, a->residual, a->w, a->sum, a->y,
                  static_cast<uint8_t *>(a->A), static_cast<uint8_t *>(a->A_sf)};
  const Ahead ahead = ahead_of(a->rows, a->H, vec, a->H * (2 + (a->residual ? size : 0)), false);
  if (ahead.most > 0)
    return with_ahead<false>(a->type, a->res_type, ahead, [&](auto t, auto r, auto n, auto stages, auto) {
      constexpr auto kernel = norm_rows_kernel<decltype(t), decltype(r), decltype(n)::value, decltype(stages)::value>;
      int grid = 0;
      const int found = resident<kernel>(ahead, a->rows, &grid);
      if (found != MOE_OK) return found;
      kernel<<<grid, ahead.threads, ahead.smem, as_stream(stream)>>>(P);
      return check_launch();
    });
  const Shape s = shape_of(a->H, vec, a->rows <= 2 * device_sm_count());
  return with_shape<false>(a->type, a->res_type, s, [&](auto t, auto r, auto v, auto n, auto block) {
    const unsigned grid = (unsigned)(s.block ? a->rows : (a->rows + 7) / 8);
    norm_kernel<decltype(t), decltype(r), v.value, n.value, block.value>
        <<<grid, s.block ? s.threads : 256, 0, as_stream(stream)>>>(P);
    return check_launch();
  });
}

extern "C" size_t moe_rms_norm_workspace_size(const moe_norm_grad_args *a) {
  if (!a || check_norm(a->rows, a->H, a->eps, a->type, a->res_type) != MOE_OK || a->rows == 0) return 0;
  // the most blocks that any alignment of the tensors asks for, with dres or without
  int most = grad_blocks(a->rows, shape_of(a->H, false, false)), ahead;
  for (bool dres : {true, false}) {
    if (a->H % 8) break;
    const Ahead s = grad_ahead(a->rows, a->H, true, a->res_type == MOE_TYPE_F32 ? 4 : 2, dres, &ahead);
    most = std::max(most, s.most > 0 ? (int)std::min<int64_t>(a->rows, (int64_t)device_sm_count() * s.most)
                                     : grad_blocks(a->rows, shape_of(a->H, true, false)));
  }
  return (size_t)most * a->H * sizeof(float);
}

extern "C" int moe_rms_norm_backward(const moe_norm_grad_args *a, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  if (!a) return MOE_ERR_INVALID;
  const int rc = check_norm(a->rows, a->H, a->eps, a->type, a->res_type);
  if (rc != MOE_OK) return rc;
  const int size = a->res_type == MOE_TYPE_F32 ? 4 : 2;
  if (off(a->dw, 4)) return MOE_ERR_INVALID;
  cudaStream_t st = as_stream(stream);
  if (a->rows == 0) {
    if (!a->dw || a->accumulate) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(a->dw, 0, sizeof(float) * a->H, st);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e);
  }
  if (!a->h || !a->dy || !a->w || !a->dx) return MOE_ERR_INVALID;
  if (off(a->h, size) || off(a->dres, size) || off(a->dx, size) || off(a->dy, 2) || off(a->w, 4)) return MOE_ERR_INVALID;
  if (a->dw && (!workspace || off(workspace, 16) || workspace_bytes < moe_rms_norm_workspace_size(a))) return MOE_ERR_INVALID;
  const Shape s = grad_shape(*a);
  int blocks = grad_blocks(a->rows, s);
  NormGradParams P = {a->rows, a->H, a->eps, 1.0f / a->H, a->h, a->dy, a->dres, a->w, a->dx,
                      a->dw ? static_cast<float *>(workspace) : nullptr, 0};
  const Ahead ahead = grad_ahead(a->rows, a->H, s.V == 8, size, a->dres != nullptr, &P.dres_ahead);
  const int done = ahead.most > 0 ? with_ahead<true>(a->type, a->res_type, ahead, [&](auto t, auto r, auto n, auto stages, auto bound) {
    constexpr auto kernel = norm_grad_rows_kernel<decltype(t), decltype(r), decltype(n)::value, decltype(stages)::value,
                                            decltype(bound)::value>;
    const int found = resident<kernel>(ahead, a->rows, &blocks);
    if (found != MOE_OK) return found;
    kernel<<<blocks, ahead.threads, ahead.smem, st>>>(P);
    return check_launch();
  }) : with_shape<true>(a->type, a->res_type, s, [&](auto t, auto r, auto v, auto n, auto block) {
    const size_t smem = s.block || !a->dw ? 0 : sizeof(float) * a->H;
    norm_grad_kernel<decltype(t), decltype(r), v.value, n.value, block.value>
        <<<blocks, s.block ? s.threads : 256, smem, st>>>(P);
    return check_launch();
  });
  if (done != MOE_OK || !a->dw) return done;
  return column_sum(P.part, blocks, a->H, a->dw, a->accumulate != 0, st);
}
