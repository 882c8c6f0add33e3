// moe_adamw: one AdamW step over many tensors, moments in binary32 or in 8-bit
// square-law codes with a scale per 256 values; moe_adamw_decode / _encode turn the codes
// into binary32 moments and back.
//
// A warp takes a block of 256 values, 8 per lane (values 4*lane..+3 of each half, so
// every load of the warp is contiguous); the block's largest magnitude is one warp
// reduction, and old codes are read and new ones written in the same pass.  The tensors'
// table travels as a kernel parameter: nothing is kept on the device between calls.
// Bound by memory with binary32 moments: 28 bytes a value with 16-bit gradients and a 16-bit
// copy, 7.0 TB/s over 201 M values (803 us).  With 8-bit moments 16 bytes a value and 97
// instructions: 6.1 TB/s (526 us), 85 % of the issue slots.
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;          // values of one 8-bit block
// Threads of a CTA: the step on codes is long arithmetic on loads made a block ahead, and
// runs best in small CTAs, each replaced as it ends (201 M values: 526 us in CTAs of 32, 582
// of 128, 654 of 256); the step on binary32 moments is memory alone (803 us in CTAs of 256;
// 854 against 827 in CTAs of 64 and 64 blocks a CTA).
constexpr int threads_of(bool bits8) { return bits8 ? 32 : 256; }
constexpr int kChunk = 16;  // blocks of a CTA, at most (64: 826 us and 551 us)
constexpr int kCodesThreads = 256;
constexpr float kInvM = (float)(1.0 / 127), kInvR = (float)(1.0 / 255);
constexpr float kSqM = 127.0f * 127.0f, kSqR = 255.0f * 255.0f;

struct Entry {
  int64_t n;
  float *p;
  const void *g;
  void *copy, *m, *v;
  float *m_scale, *r_scale;
  int16_t g_type, copy_type;
  int16_t aligned;  // every pointer allows 16-byte accesses of 4 values and more
};

template <int kMax>
struct Table {
  int n;
  int chunk_blocks;      // blocks of one CTA's chunk
  uint32_t chunk0[kMax + 1];
  Entry t[kMax];
};

struct Hyper {
  float decay, beta1, alpha1, beta2, alpha2, step, inv_bc2, eps;
  const float *grad_scale;
};

__device__ __forceinline__ float load_g(const void *g, int type, int64_t i) {
  if (type == MOE_TYPE_F32) return static_cast<const float *>(g)[i];
  if (type == MOE_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(g)[i]);
  return __half2float(static_cast<const __half *>(g)[i]);
}
__device__ __forceinline__ void store_copy(void *c, int type, int64_t i, float f) {
  if (type == MOE_TYPE_BF16)
    static_cast<__nv_bfloat16 *>(c)[i] = __float2bfloat16_rn(f);
  else if (type == MOE_TYPE_F16)
    static_cast<__half *>(c)[i] = __float2half_rn(f);
  else
    static_cast<float *>(c)[i] = f;
}
// Four values of 16 bits, two to a word, in binary32.
__device__ __forceinline__ void widen4(uint2 q, bool bf16, float *o) {
  if (bf16) {
    o[0] = __uint_as_float(q.x << 16), o[1] = __uint_as_float(q.x & 0xffff0000u);
    o[2] = __uint_as_float(q.y << 16), o[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&q.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&q.y));
    o[0] = a.x, o[1] = a.y, o[2] = b.x, o[3] = b.y;
  }
}
__device__ __forceinline__ uint32_t narrow2(float lo, float hi, bool bf16) {
  uint32_t r;
  if (bf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes: see moe_adamw in include/moe.h.
// Byte k of w, less `zero`, as a float, exactly: as the low bits of 2^23 + byte.
__device__ __forceinline__ float byte_f32(uint32_t w, int k, float zero) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 | k)) - (8388608.0f + zero);
}
// Code k of a word of four.  m: the sign bits flipped (w ^ 0x80808080) make a byte of c + 128.
__device__ __forceinline__ float decode_m(uint32_t flipped, int k, float s) {
  const float q = __fmul_rn(byte_f32(flipped, k, 128.0f), kInvM);
  return __fmul_rn(__fmul_rn(q, fabsf(q)), s);
}
__device__ __forceinline__ float decode_r(uint32_t w, int k, float s) {
  const float q = __fmul_rn(byte_f32(w, k, 0.0f), kInvR);
  return __fmul_rn(__fmul_rn(q, q), s);
}
// The whole number c with (c - 1/2)^2 <= z < (c + 1/2)^2, z = levels^2 x / s.  An
// approximate root, pulled down by more than its error and rounded to the nearest whole
// number, is c or c - 1; the bound between them, exact in binary32, says which.  Adding
// 1.5 * 2^23 rounds, and leaves the number in the low byte; the other bits mean nothing.
__device__ __forceinline__ uint32_t square_code(float x, float inv, float sq) {
  constexpr float kRound = 12582912.0f;
  const float z = __fmul_rn(__fmul_rn(x, inv), sq);
  float root;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(z));  // a subnormal z is code 0 either way
  const float y = __fmaf_rn(root, 1.0f - 0x1p-20f, kRound);
  const float h = __fadd_rn(__fadd_rn(y, -kRound), 0.5f);
  return __float_as_uint(y) + (z >= __fmul_rn(h, h) ? 1u : 0u);
}
// The low bytes of four words in one.
__device__ __forceinline__ uint32_t low_bytes(const uint32_t *c) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
__device__ __forceinline__ float block_inverse(float s) {
  return s >= 1.17549435e-38f ? __fdiv_rn(1.0f, s) : 0.0f;
}
// Largest magnitude of the warp's block; a NaN wins over every number.
__device__ __forceinline__ float block_max(const float *x) {
  float b = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(b), "f"(fabsf(x[j])));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b)));
}
__device__ __forceinline__ bool finite(float s) { return s <= 3.402823466e+38f; }

// Value j (0..7) of this lane sits at this place of its block.
__device__ __forceinline__ int place(int lane, int j) { return 128 * (j >> 2) + 4 * lane + (j & 3); }

// Loads of one lane's 8 values: `n` values are left in the tensor from the block's start.
template <class F>
__device__ __forceinline__ void each(int lane, int64_t n, F f) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (place(lane, j) < n) f(j, place(lane, j));
}

__device__ __forceinline__ void load_f32(const float *p, bool fast, int lane, int64_t n, float *o) {
  if (fast) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 q = __ldcs(reinterpret_cast<const float4 *>(p + place(lane, 4 * h)));
      o[4 * h] = q.x, o[4 * h + 1] = q.y, o[4 * h + 2] = q.z, o[4 * h + 3] = q.w;
    }
  } else {
    each(lane, n, [&](int j, int i) { o[j] = p[i]; });
  }
}
__device__ __forceinline__ void store_f32(float *p, bool fast, int lane, int64_t n, const float *o) {
  if (fast) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __stcs(reinterpret_cast<float4 *>(p + place(lane, 4 * h)),
             make_float4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]));
  } else {
    each(lane, n, [&](int j, int i) { p[i] = o[j]; });
  }
}
// Codes of one lane, four to a word: w[0] its values of the block's first half.
__device__ __forceinline__ void load_codes(const uint8_t *p, bool fast, int lane, int64_t n, uint32_t *w) {
  if (fast) {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = __ldcs(reinterpret_cast<const uint32_t *>(p + place(lane, 4 * h)));
  } else {
    w[0] = w[1] = 0;
    each(lane, n, [&](int j, int i) { w[j >> 2] |= (uint32_t)p[i] << (8 * (j & 3)); });
  }
}
__device__ __forceinline__ void store_codes(uint8_t *p, bool fast, int lane, int64_t n, const uint32_t *w) {
  if (fast) {
#pragma unroll
    for (int h = 0; h < 2; ++h) __stcs(reinterpret_cast<uint32_t *>(p + place(lane, 4 * h)), w[h]);
  } else {
    each(lane, n, [&](int j, int i) { p[i] = (uint8_t)(w[j >> 2] >> (8 * (j & 3))); });
  }
}
__device__ __forceinline__ void decode_block(const uint32_t *mc, const uint32_t *rc, float ms, float rs,
                                             float *m, float *v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = decode_m(mc[j >> 2] ^ 0x80808080u, j & 3, ms);
    const float x = decode_r(rc[j >> 2], j & 3, rs);
    v[j] = __fmul_rn(x, x);
  }
}
// Moments of a block (r = sqrt(v)) -> codes and scales.
__device__ __forceinline__ void encode_block(const float *m, const float *r, uint32_t *mc, uint32_t *rc,
                                             float &ms, float &rs) {
  ms = block_max(m);
  rs = block_max(r);
  uint32_t c[8] = {}, d[8] = {};
  if (finite(ms)) {  // else: code 0, which an infinite or NaN scale turns into NaN
    const float inv = block_inverse(ms);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = square_code(fabsf(m[j]), inv, kSqM);
      if (m[j] < 0.0f) c[j] = 0u - c[j];
    }
  }
  if (finite(rs)) {
    const float inv = block_inverse(rs);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = square_code(r[j], inv, kSqR) & 0xffu;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (r[j] > 0.0f) d[j] = max(d[j], 1u);
  mc[0] = low_bytes(c), mc[1] = low_bytes(c + 4);
  rc[0] = low_bytes(d), rc[1] = low_bytes(d + 4);
}

// A block of the fast path as it lies in memory, one lane's part.
template <bool k8Bit>
struct Raw {
  float4 p[2], g[2];      // g: 16-bit gradients in .x, .y
  float4 m[2], v[2];      // 32 bits
  uint32_t mc[2], rc[2];  // 8 bits
  float ms, rs;
};
template <bool k8Bit>
__device__ __forceinline__ void load_raw(const Entry &T, int64_t b, int lane, Raw<k8Bit> &R) {
  const int64_t i0 = b * kBlock;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = i0 + place(lane, 4 * h);
    R.p[h] = __ldcs(reinterpret_cast<const float4 *>(T.p + i));
    if (T.g_type == MOE_TYPE_F32) {
      R.g[h] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(T.g) + i));
    } else {
      const float2 q = __ldcs(reinterpret_cast<const float2 *>(static_cast<const uint16_t *>(T.g) + i));
      R.g[h].x = q.x, R.g[h].y = q.y;
    }
    if constexpr (k8Bit) {
      R.mc[h] = __ldcs(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(T.m) + i));
      R.rc[h] = __ldcs(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(T.v) + i));
    } else {
      R.m[h] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(T.m) + i));
      R.v[h] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(T.v) + i));
    }
  }
  if constexpr (k8Bit) {
    R.ms = T.m_scale[b];
    R.rs = T.r_scale[b];
  }
}
__device__ __forceinline__ void spread(const float4 *q, float *o) {
#pragma unroll
  for (int h = 0; h < 2; ++h) o[4 * h] = q[h].x, o[4 * h + 1] = q[h].y, o[4 * h + 2] = q[h].z, o[4 * h + 3] = q[h].w;
}

// The step of 8 values; r: the new sqrt(v).
__device__ __forceinline__ void update(const Hyper &H, float gs, float *g, float *p, float *m,
                                       float *v, float *r) {
  if (H.grad_scale) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], gs);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = g[j];
    m[j] = __fadd_rn(__fmul_rn(m[j], H.beta1), __fmul_rn(x, H.alpha1));
    v[j] = __fadd_rn(__fmul_rn(v[j], H.beta2), __fmul_rn(__fmul_rn(x, x), H.alpha2));
    r[j] = __fsqrt_rn(v[j]);
    float inv;  // of the denominator, within an ulp: p is not promised to the bit
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(r[j], H.inv_bc2, H.eps)));
    p[j] = fmaf(p[j], H.decay, -(m[j] * inv) * H.step);
  }
}

template <int kMax, bool k8Bit>
__global__ void __launch_bounds__(threads_of(k8Bit), 768 / threads_of(k8Bit))
    adamw_kernel(const __grid_constant__ Table<kMax> tab, const Hyper H) {
  constexpr int kWarps = threads_of(k8Bit) / 32;
  // the tensor of this CTA's chunk
  int lo = 0, hi = tab.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.chunk0[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid;
  }
  const Entry &T = tab.t[lo];
  const int64_t n_all = T.n;
  const int64_t blocks = (n_all + kBlock - 1) / kBlock;
  const int64_t first = (int64_t)(blockIdx.x - tab.chunk0[lo]) * tab.chunk_blocks;
  const int64_t last = min(first + tab.chunk_blocks, blocks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float gs = H.grad_scale ? *H.grad_scale : 1.0f;
  // whole blocks of aligned tensors; with codes, whose arithmetic is long, the next block's
  // loads are under way while one is worked on
  const int64_t whole = T.aligned ? min(last, n_all / kBlock) : first;
  int64_t b = first + warp;
  Raw<k8Bit> next;
  if (k8Bit && b < whole) load_raw<k8Bit>(T, b, lane, next);
  for (; b < whole; b += kWarps) {
    if (!k8Bit) load_raw<k8Bit>(T, b, lane, next);
    const Raw<k8Bit> R = next;
    if (k8Bit && b + kWarps < whole) load_raw<k8Bit>(T, b + kWarps, lane, next);
    const int64_t i0 = b * kBlock;
    float p[8], g[8], m[8], v[8], r[8];
    spread(R.p, p);
    if (T.g_type == MOE_TYPE_F32) {
      spread(R.g, g);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        widen4(make_uint2(__float_as_uint(R.g[h].x), __float_as_uint(R.g[h].y)),
               T.g_type == MOE_TYPE_BF16, g + 4 * h);
    }
    if constexpr (k8Bit) {
      decode_block(R.mc, R.rc, R.ms, R.rs, m, v);
    } else {
      spread(R.m, m);
      spread(R.v, v);
    }
    update(H, gs, g, p, m, v, r);
    store_f32(T.p + i0, true, lane, kBlock, p);
    if (T.copy) {
      if (T.copy_type == MOE_TYPE_F32) {
        store_f32(static_cast<float *>(T.copy) + i0, true, lane, kBlock, p);
      } else {
        const bool bf16 = T.copy_type == MOE_TYPE_BF16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(T.copy) + i0 + place(lane, 4 * h)),
                 make_uint2(narrow2(p[4 * h], p[4 * h + 1], bf16), narrow2(p[4 * h + 2], p[4 * h + 3], bf16)));
      }
    }
    if constexpr (k8Bit) {
      uint32_t mc[2], rc[2];
      float ms, rs;
      encode_block(m, r, mc, rc, ms, rs);
      store_codes(static_cast<uint8_t *>(T.m) + i0, true, lane, kBlock, mc);
      store_codes(static_cast<uint8_t *>(T.v) + i0, true, lane, kBlock, rc);
      if (lane == 0) {
        T.m_scale[b] = ms;
        T.r_scale[b] = rs;
      }
    } else {
      store_f32(static_cast<float *>(T.m) + i0, true, lane, kBlock, m);
      store_f32(static_cast<float *>(T.v) + i0, true, lane, kBlock, v);
    }
  }
  // the others, value by value
  for (; b < last; b += kWarps) {
    const int64_t i0 = b * kBlock, n = n_all - i0;
    float p[8] = {}, g[8] = {}, m[8] = {}, v[8] = {}, r[8];
    load_f32(T.p + i0, false, lane, n, p);
    each(lane, n, [&](int j, int i) { g[j] = load_g(T.g, T.g_type, i0 + i); });
    if constexpr (k8Bit) {
      uint32_t mc[2], rc[2];
      load_codes(static_cast<const uint8_t *>(T.m) + i0, false, lane, n, mc);
      load_codes(static_cast<const uint8_t *>(T.v) + i0, false, lane, n, rc);
      decode_block(mc, rc, T.m_scale[b], T.r_scale[b], m, v);
    } else {
      load_f32(static_cast<const float *>(T.m) + i0, false, lane, n, m);
      load_f32(static_cast<const float *>(T.v) + i0, false, lane, n, v);
    }
    update(H, gs, g, p, m, v, r);
    store_f32(T.p + i0, false, lane, n, p);
    if (T.copy) each(lane, n, [&](int j, int i) { store_copy(T.copy, T.copy_type, i0 + i, p[j]); });
    if constexpr (k8Bit) {
#pragma unroll
      for (int j = 0; j < 8; ++j)  // places past the tensor's end count for nothing
        if (place(lane, j) >= n) m[j] = r[j] = 0.0f;
      uint32_t mc[2], rc[2];
      float ms, rs;
      encode_block(m, r, mc, rc, ms, rs);
      store_codes(static_cast<uint8_t *>(T.m) + i0, false, lane, n, mc);
      store_codes(static_cast<uint8_t *>(T.v) + i0, false, lane, n, rc);
      if (lane == 0) {
        T.m_scale[b] = ms;
        T.r_scale[b] = rs;
      }
    } else {
      store_f32(static_cast<float *>(T.m) + i0, false, lane, n, m);
      store_f32(static_cast<float *>(T.v) + i0, false, lane, n, v);
    }
  }
}

template <bool kEncode>
__global__ void __launch_bounds__(kCodesThreads)
    codes_kernel(int64_t n_all, uint8_t *m_code, float *m_scale, uint8_t *r_code, float *r_scale,
                 float *mp, float *vp) {
  constexpr int kWarps = kCodesThreads / 32;
  const int64_t blocks = (n_all + kBlock - 1) / kBlock;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t b = (int64_t)blockIdx.x * kWarps + warp; b < blocks; b += (int64_t)gridDim.x * kWarps) {
    const int64_t i0 = b * kBlock, n = n_all - i0;
    const bool fast = n >= kBlock;
    float m[8] = {}, v[8] = {};
    uint32_t mc[2], rc[2];
    if constexpr (kEncode) {
      load_f32(mp + i0, fast, lane, n, m);
      load_f32(vp + i0, fast, lane, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fsqrt_rn(v[j]);
      float ms, rs;
      encode_block(m, v, mc, rc, ms, rs);
      store_codes(m_code + i0, fast, lane, n, mc);
      store_codes(r_code + i0, fast, lane, n, rc);
      if (lane == 0) {
        m_scale[b] = ms;
        r_scale[b] = rs;
      }
    } else {
      load_codes(m_code + i0, fast, lane, n, mc);
      load_codes(r_code + i0, fast, lane, n, rc);
      decode_block(mc, rc, m_scale[b], r_scale[b], m, v);
      store_f32(mp + i0, fast, lane, n, m);
      store_f32(vp + i0, fast, lane, n, v);
    }
  }
}

bool type_ok(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F16 || t == MOE_TYPE_F32; }
int type_size(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }
bool off(const void *p, size_t a) { return (uintptr_t)p % a != 0; }

template <int kMax>
int launch(const moe_adamw_tensor *t, int n, bool bits8, const Hyper &H, cudaStream_t st) {
  Table<kMax> tab;
  memset(&tab, 0, sizeof tab);
  tab.n = n;
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) blocks += (t[i].n + kBlock - 1) / kBlock;
  // fewer blocks a CTA, down to one a warp, where the step is small
  int chunk = kChunk;
  const int warps = threads_of(bits8) / 32;
  while (chunk > warps && blocks / chunk < 8 * device_sm_count()) chunk >>= 1;
  tab.chunk_blocks = chunk;
  uint64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor &a = t[i];
    Entry &e = tab.t[i];
    tab.chunk0[i] = (uint32_t)chunks;
    chunks += (uint64_t)((a.n + kBlock - 1) / kBlock + chunk - 1) / chunk;
    if (chunks > 0x7fffffffull) return MOE_ERR_UNSUPPORTED;
    e.n = a.n;
    e.p = a.p;
    e.g = a.g;
    e.copy = a.copy;
    e.m = a.m;
    e.v = a.v;
    e.m_scale = a.m_scale;
    e.r_scale = a.r_scale;
    e.g_type = (int16_t)a.g_type;
    e.copy_type = (int16_t)a.copy_type;
    e.aligned = !(off(a.p, 16) || off(a.g, 4 * type_size(a.g_type)) ||
                  (a.copy && off(a.copy, 4 * type_size(a.copy_type))) || off(a.m, bits8 ? 4 : 16) ||
                  off(a.v, bits8 ? 4 : 16));
  }
  tab.chunk0[n] = (uint32_t)chunks;
  if (chunks == 0) return MOE_OK;
  if (bits8)
    adamw_kernel<kMax, true><<<(unsigned)chunks, threads_of(true), 0, st>>>(tab, H);
  else
    adamw_kernel<kMax, false><<<(unsigned)chunks, threads_of(false), 0, st>>>(tab, H);
  return check_launch();
}

int check_codes(int64_t n, const void *mc, const void *ms, const void *rc, const void *rs,
                const void *m, const void *v) {
  if (n < 0) return MOE_ERR_INVALID;
  if (n > (1ll << 40)) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!mc || !ms || !rc || !rs || !m || !v) return MOE_ERR_INVALID;
  if (off(mc, 4) || off(rc, 4) || off(ms, 4) || off(rs, 4) || off(m, 16) || off(v, 16))
    return MOE_ERR_INVALID;
  return MOE_OK;
}
unsigned codes_grid(int64_t n) {
  const int64_t need = ((n + kBlock - 1) / kBlock + kCodesThreads / 32 - 1) / (kCodesThreads / 32);
  const int64_t most = (int64_t)device_sm_count() * 8;
  return (unsigned)(need < most ? need : most);
}

constexpr int kSmallTable = 32, kTable = 256;

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_adamw(const moe_adamw_cfg *cfg, const moe_adamw_tensor *tensors, int n_tensors,
                         void *stream) {
  if (!cfg || n_tensors < 0 || (n_tensors > 0 && !tensors)) return MOE_ERR_INVALID;
  if (cfg->state_bits != 8 && cfg->state_bits != 32) return MOE_ERR_INVALID;
  if (cfg->step < 1 || !(cfg->beta1 >= 0 && cfg->beta1 < 1) || !(cfg->beta2 >= 0 && cfg->beta2 < 1) ||
      !(cfg->eps >= 0) || off(cfg->grad_scale, 4))
    return MOE_ERR_INVALID;
  const bool bits8 = cfg->state_bits == 8;
  for (int i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor &t = tensors[i];
    if (t.n < 0) return MOE_ERR_INVALID;
    if (t.n > (1ll << 40)) return MOE_ERR_UNSUPPORTED;
    if (!type_ok(t.g_type) || (t.copy && !type_ok(t.copy_type))) return MOE_ERR_INVALID;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (bits8 && (!t.m_scale || !t.r_scale))) return MOE_ERR_INVALID;
    if (off(t.p, 4) || off(t.g, type_size(t.g_type)) ||
        (t.copy && off(t.copy, type_size(t.copy_type))) ||
        (!bits8 && (off(t.m, 4) || off(t.v, 4))) || off(t.m_scale, 4) || off(t.r_scale, 4))
      return MOE_ERR_INVALID;
  }
  Hyper H;
  const double bc1 = 1.0 - pow(cfg->beta1, (double)cfg->step);
  const double bc2 = 1.0 - pow(cfg->beta2, (double)cfg->step);
  H.decay = (float)(1.0 - cfg->lr * cfg->weight_decay);
  H.beta1 = (float)cfg->beta1;
  H.alpha1 = (float)(1.0 - cfg->beta1);
  H.beta2 = (float)cfg->beta2;
  H.alpha2 = (float)(1.0 - cfg->beta2);
  H.step = (float)(cfg->lr / bc1);
  H.inv_bc2 = (float)(1.0 / sqrt(bc2));
  H.eps = (float)cfg->eps;
  H.grad_scale = cfg->grad_scale;
  for (int i = 0; i < n_tensors; i += kTable) {
    const int n = n_tensors - i < kTable ? n_tensors - i : kTable;
    const int rc = n <= kSmallTable ? launch<kSmallTable>(tensors + i, n, bits8, H, as_stream(stream))
                                    : launch<kTable>(tensors + i, n, bits8, H, as_stream(stream));
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

extern "C" int moe_adamw_decode(int64_t n, const void *m_code, const float *m_scale,
                                const void *r_code, const float *r_scale, float *m, float *v,
                                void *stream) {
  const int rc = check_codes(n, m_code, m_scale, r_code, r_scale, m, v);
  if (rc != MOE_OK || n == 0) return rc;
  codes_kernel<false><<<codes_grid(n), kCodesThreads, 0, as_stream(stream)>>>(
      n, static_cast<uint8_t *>(const_cast<void *>(m_code)), const_cast<float *>(m_scale),
      static_cast<uint8_t *>(const_cast<void *>(r_code)), const_cast<float *>(r_scale), m, v);
  return check_launch();
}

extern "C" int moe_adamw_encode(int64_t n, const float *m, const float *v, void *m_code,
                                float *m_scale, void *r_code, float *r_scale, void *stream) {
  const int rc = check_codes(n, m_code, m_scale, r_code, r_scale, m, v);
  if (rc != MOE_OK || n == 0) return rc;
  codes_kernel<true><<<codes_grid(n), kCodesThreads, 0, as_stream(stream)>>>(
      n, static_cast<uint8_t *>(m_code), m_scale, static_cast<uint8_t *>(r_code), r_scale,
      const_cast<float *>(m), const_cast<float *>(v));
  return check_launch();
}
