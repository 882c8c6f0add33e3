// moe_swiglu and moe_swiglu_backward: the gated activation between an expert's two
// products, h = w a u with a = g s, s = sigmoid(g), and its gradients
//   dg = w dh u (s + a (1 - s)),  du = w dh a,  dw = sum_j dh_j a_j u_j.
//
// Bound by memory: 3 columns of I values move forward, 5 backward, against about 10 and
// 20 operations a value.  A row is taken by one warp or one block (the host picks by the
// number of rows), so dw is a reduction inside it: lanes in their order, then warps in
// theirs, the same bits every time.  The rows of the segments are numbered through (a
// table of the segments in shared memory maps the number to the row), so padding costs
// nothing and no row is tested.  65536 rows of I = 2048: forward 130 us (6.2 TB/s),
// backward with dw 212 us (6.3 TB/s), where a copy runs at 6.8.
#include <cuda_fp16.h>

#include <type_traits>

#include "segments.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32(__half v) {
  return __half2float(v);
}
template <class T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float f) {
  return __float2bfloat16_rn(f);
}
template <>
__device__ __forceinline__ __half from_f32(float f) {
  return __float2half_rn(f);
}

template <class T>
union Vec8 {
  uint4 q;
  T t[8];
};

struct SwigluParams {
  SegParams seg;
  int I;
  const void *gu, *dh;
  const float *row_w;
  void *out;
  float *drow_w;
};

// Gates below -87: 1 + e^-g passes the divisors that __fdividef takes (2^126), and soon
// binary32 itself; the sigmoid is e^g to the last bit there.  A large u or w brings the
// products back into range; what stays below 2^-100 counts as zero.  kLow: with such gates.
// Eight values are tested for them at once, as whole numbers, and computed one by one if there
// is one (65536 rows of 2048: 130 us; selected value by value 158).
constexpr float kLowGate = -87.0f;
template <bool kLow>
__device__ __forceinline__ float sigmoid(float g) {
  if (kLow && g < kLowGate) return __expf(g);
  return __fdividef(1.0f, 1.0f + __expf(-g));
}
template <bool kLow>
__device__ __forceinline__ float settled(float r, float g) {
  return kLow && g < kLowGate && fabsf(r) < 0x1p-100f ? 0.0f : r;
}
// Whether any of 8 gates is that low: its bits, a number without sign, are above -87's.
template <class T>
__device__ __forceinline__ bool any_low(const Vec8<T> &g) {
  constexpr unsigned kBits = std::is_same<T, __half>::value ? 0xd570u : 0xc2aeu;
  const unsigned m = __vmaxu2(__vmaxu2(g.q.x, g.q.y), __vmaxu2(g.q.z, g.q.w));
  return (m >> 16) > kBits || (m & 0xffffu) > kBits;
}

// One value: forward (h), or backward (dg, du and the term of dw).
template <bool kLow>
__device__ __forceinline__ float forward_one(float g, float u, float w) {
  return settled<kLow>(w * (g * sigmoid<kLow>(g)) * u, g);
}
template <bool kLow>
__device__ __forceinline__ float backward_one(float g, float u, float dh, float w, float &dg,
                                              float &du) {
  const float s = sigmoid<kLow>(g), a = g * s, wd = w * dh;
  dg = settled<kLow>(wd * u * (s + a * (1.0f - s)), g);
  du = settled<kLow>(wd * a, g);
  return dh * a * u;
}

// kRow: threads of one row (32 or the block).  kVec: 8 values a load (I % 8 == 0 and
// 16-byte aligned tensors), else one.
template <class T, bool kBackward, bool kVec, int kRow>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams P) {
  __shared__ SegTable table;
  __shared__ int part[64];
  __shared__ float warp_sum[kThreads / 32];
  int total = P.seg.rows;
  if (P.seg.counts) {
    build_segments(P.seg, table, part, [](int n) { return n; }, blockIdx.x == 0);
    total = table.before[P.seg.E];
  }
  constexpr int kGroups = kThreads / kRow, V = kVec ? 8 : 1;
  const int group = threadIdx.x / kRow, t = threadIdx.x % kRow;
  const T *gu = static_cast<const T *>(P.gu), *dhp = static_cast<const T *>(P.dh);
  T *outp = static_cast<T *>(P.out);
  const int I = P.I;
  // with kRow == kThreads the block meets at barriers: `v` is the same in all threads.  64
  // bits: rows may number nearly 2^31, and the last step passes them by up to a grid's.
  for (int64_t v = (int64_t)blockIdx.x * kGroups + group; v < total; v += (int64_t)gridDim.x * kGroups) {
    int r = (int)v;
    if (P.seg.counts) {
      const int e = find_segment(table, P.seg.E, (int)v);
      r = table.start[e] + ((int)v - table.before[e]);
    }
    const float w = P.row_w ? P.row_w[r] : 1.0f;
    const T *g_row = gu + (size_t)r * 2 * I, *dh_row = dhp + (size_t)r * I;
    T *o_row = outp + (size_t)r * (kBackward ? 2 * I : I);
    float sum = 0.0f;
    auto one = [&](int j) {
      const float gf = to_f32(g_row[j]), uf = to_f32(g_row[I + j]);
      if constexpr (kBackward) {
        float dg, du;
        sum += backward_one<true>(gf, uf, to_f32(dh_row[j]), w, dg, du);
        o_row[j] = from_f32<T>(dg);
        o_row[I + j] = from_f32<T>(du);
      } else {
        o_row[j] = from_f32<T>(forward_one<true>(gf, uf, w));
      }
    };
#pragma unroll 4
    for (int j = t * V; j < I; j += kRow * V) {
      if constexpr (kVec) {
        Vec8<T> g, u, d, o, o2;
        g.q = __ldcs(reinterpret_cast<const uint4 *>(g_row + j));
        u.q = __ldcs(reinterpret_cast<const uint4 *>(g_row + I + j));
        if constexpr (kBackward) d.q = __ldcs(reinterpret_cast<const uint4 *>(dh_row + j));
        if (any_low(g)) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) one(j + i);
          continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gf = to_f32(g.t[i]), uf = to_f32(u.t[i]);
          if constexpr (kBackward) {
            float dg, du;
            sum += backward_one<false>(gf, uf, to_f32(d.t[i]), w, dg, du);
            o.t[i] = from_f32<T>(dg);
            o2.t[i] = from_f32<T>(du);
          } else {
            o.t[i] = from_f32<T>(forward_one<false>(gf, uf, w));
          }
        }
        *reinterpret_cast<uint4 *>(o_row + j) = o.q;
        if constexpr (kBackward) *reinterpret_cast<uint4 *>(o_row + I + j) = o2.q;
      } else {
        one(j);
      }
    }
    if (kBackward && P.drow_w) {
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if constexpr (kRow == 32) {
        if (t == 0) P.drow_w[r] = sum;
      } else {
        if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i) s += warp_sum[i];
          P.drow_w[r] = s;
        }
        __syncthreads();
      }
    }
  }
}

template <class T, bool kBackward>
int launch(const SwigluParams &P, bool vec, cudaStream_t st) {
  // One warp a row moves 8 rows a block; with few rows a block a row spreads the work.
  const bool wide = P.seg.rows < 16 * device_sm_count() && P.I > 256;
  const int groups = wide ? 1 : kThreads / 32;
  const int64_t need = ((int64_t)P.seg.rows + groups - 1) / groups;
  // Eight blocks an SM are resident.  The forward over long rows gains from three times as
  // many blocks, handed out as others end (I = 2048: 131 us against 146; I = 520: 45 and
  // 46, left alone); each block builds the segments' table, which the backward does not repay
  // (I = 2048: 215 us against 211; 520: 78 against 75).
  const int64_t most = (int64_t)device_sm_count() * (!kBackward && P.I >= 1024 ? 24 : 8);
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (vec) {
    if (wide)
      swiglu_kernel<T, kBackward, true, kThreads><<<grid, kThreads, 0, st>>>(P);
    else
      swiglu_kernel<T, kBackward, true, 32><<<grid, kThreads, 0, st>>>(P);
  } else {
    if (wide)
      swiglu_kernel<T, kBackward, false, kThreads><<<grid, kThreads, 0, st>>>(P);
    else
      swiglu_kernel<T, kBackward, false, 32><<<grid, kThreads, 0, st>>>(P);
  }
  return check_launch();
}

int swiglu(const moe_swiglu_args *a, bool backward, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  if (a->type != MOE_TYPE_BF16 && a->type != MOE_TYPE_F16) return MOE_ERR_INVALID;
  if (a->I < 1) return MOE_ERR_INVALID;
  if (a->I > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  const int rc = check_segments(a->seg, true);
  if (rc != MOE_OK) return rc;
  if (a->seg.rows == 0) return MOE_OK;
  if (!a->gu || !a->out || (backward && !a->dh) || (!backward && (a->dh || a->drow_w)))
    return MOE_ERR_INVALID;
  bool vec = a->I % 8 == 0;
  for (const void *p : {a->gu, a->dh, (const void *)a->out}) {
    if ((uintptr_t)p % 2) return MOE_ERR_INVALID;
    if ((uintptr_t)p % 16) vec = false;
  }
  if ((uintptr_t)a->row_w % 4 || (uintptr_t)a->drow_w % 4) return MOE_ERR_INVALID;
  SwigluParams P;
  P.seg = seg_params(a->seg, a->status);
  P.I = a->I;
  P.gu = a->gu;
  P.dh = a->dh;
  P.row_w = a->row_w;
  P.out = a->out;
  P.drow_w = a->drow_w;
  cudaStream_t st = as_stream(stream);
  if (a->type == MOE_TYPE_BF16)
    return backward ? launch<__nv_bfloat16, true>(P, vec, st) : launch<__nv_bfloat16, false>(P, vec, st);
  return backward ? launch<__half, true>(P, vec, st) : launch<__half, false>(P, vec, st);
}

}  // namespace

cudaError_t swiglu_default_status(int32_t *bits, bool clear) { return take_default_status(bits, clear); }

}  // namespace moe

extern "C" int moe_swiglu(const moe_swiglu_args *args, void *stream) {
  return moe::swiglu(args, false, stream);
}
extern "C" int moe_swiglu_backward(const moe_swiglu_args *args, void *stream) {
  return moe::swiglu(args, true, stream);
}
