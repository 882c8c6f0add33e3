// moe_grouped_gemm and moe_grouped_wgrad: grouped products of 16-bit operands over
// ragged row segments,
//   forward   out[r][j] = sum_i x[r][i] w[e][j][i]
//   trans     out[r][i] = sum_j x[r][j] w[e][j][i]
//   gradient  out[e][j][i] = sum_{r in e} dy[r][j] x[r][i].
// All three are out[q][p] = sum_t Q(q, t) P(p, t) with p the output's contiguous index.
#include <cuda_fp16.h>

#include "segments.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, BQ = 64, BP = 64, BT = 16;

struct GroupedParams {
  SegParams seg;
  int64_t np, nt;  // extents of p and (forward, trans) t; the gradient's q extent is nq
  int64_t nq;
  const void *q, *p;
  int64_t q_stride, q_step;  // Q(q, t) = q[q * q_stride + t * q_step]
  int64_t p_stride, p_step, p_expert;
  void *out;
  bool accumulate;
};

template <class T>
__device__ __forceinline__ float load(const void *b, int64_t i);
template <>
__device__ __forceinline__ float load<__nv_bfloat16>(const void *b, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(b)[i]);
}
template <>
__device__ __forceinline__ float load<__half>(const void *b, int64_t i) {
  return __half2float(static_cast<const __half *>(b)[i]);
}
__device__ __forceinline__ void store(__nv_bfloat16 *o, float f, bool) { *o = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store(__half *o, float f, bool) { *o = __float2half_rn(f); }
__device__ __forceinline__ void store(float *o, float f, bool acc) { *o = acc ? *o + f : f; }

template <class T, class O, bool kGrad>
__global__ void __launch_bounds__(kThreads) grouped_kernel(const GroupedParams P) {
  __shared__ SegTable table;
  __shared__ long long part[33];
  __shared__ float sq[BT][BQ + 1], sp[BT][BP + 1];
  const int qt_fixed = (int)((P.nq + BQ - 1) / BQ);
  build_segments(P.seg, table, part, [&](int n) { return kGrad ? qt_fixed : (n + BQ - 1) / BQ; },
                 blockIdx.x == 0);
  const int64_t pt = (P.np + BP - 1) / BP, units = table.before[P.seg.E] * pt;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int band = (int)(unit / pt);
    const int e = find_segment(table, P.seg.E, band);
    const int64_t p0 = unit % pt * BP, q0 = (int64_t)(band - table.before[e]) * BQ;
    const int64_t r0 = table.start[e], rows = table.count[e];
    const int64_t nq = kGrad ? P.nq : rows, nt = kGrad ? rows : P.nt;
    const int64_t qb = kGrad ? r0 * P.q_step : r0 * P.q_stride;
    const int64_t pb = kGrad ? r0 * P.p_step : e * P.p_expert;
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < nt; t0 += BT) {
      for (int i = tid; i < BT * BQ; i += kThreads) {
        const int64_t t = t0 + i / BQ, q = q0 + i % BQ, p = p0 + i % BP;
        sq[i / BQ][i % BQ] = t < nt && q < nq ? load<T>(P.q, qb + q * P.q_stride + t * P.q_step) : 0.0f;
        sp[i / BP][i % BP] = t < nt && p < P.np ? load<T>(P.p, pb + p * P.p_stride + t * P.p_step) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sq[t][ty + 16 * a], sp[t][tx + 16 * b], acc[a][b]);
      __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t q = q0 + ty + 16 * a, p = p0 + tx + 16 * b;
        if (q < nq && p < P.np && !(kGrad && P.accumulate && rows == 0))
          store(static_cast<O *>(P.out) + ((kGrad ? e * P.nq : r0) + q) * P.np + p, acc[a][b],
                P.accumulate);
      }
  }
}

int check_common(const moe_segments &seg, int n, int k, int type) {
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_F16) return MOE_ERR_INVALID;
  if (n <= 0 || k <= 0) return MOE_ERR_INVALID;
  const int rc = check_segments(seg, false);
  if (rc != MOE_OK) return rc;
  if (n % 8 || k % 8) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }

template <class T, class O, bool kGrad>
int launch(const GroupedParams &P, int num_sms, void *stream) {
  const int sms = num_sms > 0 ? num_sms : device_sm_count();
  grouped_kernel<T, O, kGrad><<<sms * 4, kThreads, 0, as_stream(stream)>>>(P);
  return check_launch();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm(const moe_ggemm_args *a, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  const int rc = check_common(a->seg, a->n, a->k, a->type);
  if (rc != MOE_OK) return rc;
  if (a->trans != 0 && a->trans != 1) return MOE_ERR_INVALID;
  if (a->seg.rows == 0) return MOE_OK;
  if (!a->x || !a->w || !a->out || off16(a->x) || off16(a->w) || off16(a->out)) return MOE_ERR_INVALID;
  GroupedParams P = {};
  P.seg = seg_params(a->seg, a->status);
  P.np = a->trans ? a->k : a->n;
  P.nt = a->trans ? a->n : a->k;
  P.q = a->x;
  P.q_stride = P.nt;
  P.q_step = 1;
  P.p = a->w;
  P.p_stride = a->trans ? 1 : a->k;
  P.p_step = a->trans ? a->k : 1;
  P.p_expert = (int64_t)a->n * a->k;
  P.out = a->out;
  return a->type == MOE_TYPE_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, false>(P, a->num_sms, stream)
                                  : launch<__half, __half, false>(P, a->num_sms, stream);
}

extern "C" int moe_grouped_wgrad(const moe_wgrad_args *a, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  const int rc = check_common(a->seg, a->n, a->k, a->type);
  if (rc != MOE_OK) return rc;
  if ((a->out_type != a->type && a->out_type != MOE_TYPE_F32) ||
      (a->accumulate && a->out_type != MOE_TYPE_F32))
    return MOE_ERR_INVALID;
  if (!a->dy || !a->x || !a->out || off16(a->dy) || off16(a->x) || off16(a->out)) return MOE_ERR_INVALID;
  GroupedParams P = {};
  P.seg = seg_params(a->seg, a->status);
  P.np = a->k;
  P.nq = a->n;
  P.q = a->dy;
  P.q_stride = 1;
  P.q_step = a->n;
  P.p = a->x;
  P.p_stride = 1;
  P.p_step = a->k;
  P.out = a->out;
  P.accumulate = a->accumulate != 0;
  if (a->out_type == MOE_TYPE_F32)
    return a->type == MOE_TYPE_BF16 ? launch<__nv_bfloat16, float, true>(P, a->num_sms, stream)
                                    : launch<__half, float, true>(P, a->num_sms, stream);
  return a->type == MOE_TYPE_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, true>(P, a->num_sms, stream)
                                  : launch<__half, __half, true>(P, a->num_sms, stream);
}
