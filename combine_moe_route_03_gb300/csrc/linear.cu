// moe_linear: a dense product of 16-bit operands on tcgen05 tensor cores with bias,
// activation and residual in its epilogue,
//   forward   z[r][j] = sum_i x[r][i] w[j][i]
//   trans     z[r][i] = sum_j x[r][j] w[j][i],    out = act(z + bias) + residual.
//
// Written z[q][p] = sum_t Q(q, t) P(p, t) with p the output's contiguous index, P the
// weights on the MMA's M side and the rows Q on its N side, which takes any multiple of 32 of
// them.  CTA pairs: cta_group::2 MMAs of 256 x N x 16, binary32 accumulators in tensor memory,
// each CTA with 128 of the tile's p and half of its q.  A unit of work is 256 p and up to 256 q,
// one accumulator; the other takes the next unit's MMAs while this one's is stored.  (Units of
// 512 q on both read the P tile once for the two, but nothing runs beside their stores: 8192 x
// 7168 x 2048 took 156 us so, 131 now; 8192 x 4096 x 7168 306 and 262.)
//   warp 0  producer: TMA tiles into a ring in shared memory
//   warp 1  MMA issuer (of the even CTA) and TMEM owner
//   warps 4-19  epilogue: TMEM -> registers -> global (with 8 warps it took longer than the
//           MMAs of a tile)
// With few rows there are fewer units than pairs, and the weights' bytes bound the call: a
// cluster of S pairs splits t.  The partial sums meet in shared memory: each CTA adds up its
// share of the tile's q's over the cluster in the pairs' order, so no workspace, no atomics,
// and the same bits every time.
// The tensor core's binary32 accumulation truncates; where that would show (binary32
// outputs, and sums past the lengths below) partial sums are added in the epilogue's
// registers with rounding to nearest.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "act.cuh"
#include "entry.cuh"
#include "pair16.cuh"
#include "segments.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 16, kThreads = 128 + 32 * kEpiWarps;
constexpr int BP = 256, BQ = 256;
constexpr int kDepth = 10;                  // most stages of the ring
constexpr uint32_t kRing = 222 * 1024;
constexpr uint32_t kPBytes = 128 * BT * 2;  // a CTA's half of a P tile
constexpr uint32_t kTmemCols = 512;
constexpr int kMostSplits = 8;              // clusters of 16 CTAs
constexpr int kSumBlocks = 8;               // blocks of a partial sum of binary32 outputs: 512 terms
constexpr int kJoinBlocks = 64;             // and of long 16-bit ones
constexpr int kLongestF16 = 16384, kLongestBf16 = 131072;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct Shared {
  uint64_t full[kDepth], empty[kDepth];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
};
constexpr uint32_t kSmem = kRing + sizeof(Shared) + 1024;
static_assert(kSmem <= 232448 && BQ * 128 * 4 <= kRing, "shared memory");

struct Maps {
  CUtensorMap p, q;  // q: boxes of half a unit's rows
};

struct LinearParams {
  int rows, np, nt;
  int nq;                 // q's of a unit, a multiple of 32
  int q_tiles, p_tiles, units;
  int band;               // q tiles of a band of units
  int blocks, chunk;      // 64-deep blocks of t; of one partial sum
  int splits;
  int stages;
  int p_blocked, bf16, act;
  const float *bias;
  const void *residual;
  void *pre, *out;
  int32_t *status;
};

template <class T>
__device__ __forceinline__ float low(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value)
    return __half2float(__ushort_as_half((unsigned short)(v & 0xffff)));
  else
    return __uint_as_float(v << 16);
}
template <class T>
__device__ __forceinline__ float high(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value)
    return __half2float(__ushort_as_half((unsigned short)(v >> 16)));
  else
    return __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2f(float a, float b, __half) {
  return pack2<__half>(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ uint32_t pack2f(float a, float b, __nv_bfloat16) {
  return pack2<__nv_bfloat16>(__float_as_uint(a), __float_as_uint(b));
}

// 32 sums (q) of this warp's 32 lanes (p) through the epilogue; `at`: the first q's and the
// lane's p's place in the output.  For 16-bit tensors neighbouring lanes swap one of each two
// q's, so that a lane has two consecutive p of one row: 4 bytes a lane, 64 contiguous a row,
// straight from registers; the swap is its own inverse, which brings the residual back.  The
// extent of p is a multiple of 8, so a pair is inside or outside as one.
// What is read or written once is marked so, and leaves the L2 to the operands (8192 x 7168 x
// 2048 with residual: 139 -> 138 us, 140 in later runs; the residual asked for a unit ahead: 144).
// kAhead q's of the residual are asked for at a time: all, or fewer where the registers hold
// sums besides.
template <class T, class O, int kAhead>
__device__ __forceinline__ void finish(const LinearParams &P, float *v, int64_t at, int nq, bool inside,
                                       float bias, int lane) {
  const int odd = lane & 1;
  const uint32_t pick = odd ? 0x3276u : 0x5410u;
  const int64_t np = P.np, pair = at - odd + odd * np;
  if (!inside) nq = 0;
  auto swap = [&](uint32_t mine) { return __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick); };
#pragma unroll
  for (int h = 0; h < 32; h += kAhead) {
    uint32_t res[kAhead];
    if (P.residual) {
      if constexpr (sizeof(O) == 4) {
        const float *r = static_cast<const float *>(P.residual) + at;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) res[j] = h + j < nq ? __float_as_uint(r[(h + j) * np]) : 0u;
      } else {
        const uint16_t *r = static_cast<const uint16_t *>(P.residual) + pair;
#pragma unroll
        for (int j = 0; j < kAhead; j += 2)
          res[j] = h + j + odd < nq ? __ldcs(reinterpret_cast<const uint32_t *>(r + (h + j) * np)) : 0u;
      }
    }
#pragma unroll
    for (int j = h; j < h + kAhead; ++j) v[j] += bias;
    if (P.pre) {
      uint16_t *o = static_cast<uint16_t *>(P.pre) + pair;
#pragma unroll
      for (int j = h; j < h + kAhead; j += 2) {
        const uint32_t w = swap(pack2f(v[j], v[j + 1], T()));
        if (j + odd < nq) __stcs(reinterpret_cast<uint32_t *>(o + j * np), w);
      }
    }
    if (P.act != MOE_ACT_NONE) {
#pragma unroll
      for (int j = h; j < h + kAhead; ++j) v[j] = activate(v[j], P.act);
    }
    if constexpr (sizeof(O) == 4) {
      float *o = static_cast<float *>(P.out) + at;
#pragma unroll
      for (int j = h; j < h + kAhead; ++j)
        if (j < nq) o[j * np] = P.residual ? v[j] + __uint_as_float(res[j - h]) : v[j];
    } else {
      uint16_t *o = static_cast<uint16_t *>(P.out) + pair;
#pragma unroll
      for (int j = h; j < h + kAhead; j += 2) {
        if (P.residual) {
          const uint32_t r = swap(res[j - h]);
          v[j] += low<O>(r);
          v[j + 1] += high<O>(r);
        }
        const uint32_t w = swap(pack2f(v[j], v[j + 1], O()));
        if (j + odd < nq) __stcs(reinterpret_cast<uint32_t *>(o + j * np), w);
      }
    }
  }
}

// Two neighbouring p of one row, in the split form.
template <class T, class O>
__device__ __forceinline__ void finish_two(const LinearParams &P, float a, float b, int64_t at, int p) {
  if (P.bias) a += __ldg(P.bias + p), b += __ldg(P.bias + p + 1);
  if (P.pre) *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(P.pre) + at) = pack2f(a, b, T());
  a = activate(a, P.act);
  b = activate(b, P.act);
  if constexpr (sizeof(O) == 4) {
    if (P.residual) {
      const float2 r = *reinterpret_cast<const float2 *>(static_cast<const float *>(P.residual) + at);
      a += r.x, b += r.y;
    }
    *reinterpret_cast<float2 *>(static_cast<float *>(P.out) + at) = make_float2(a, b);
  } else {
    if (P.residual) {
      const uint32_t r = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(P.residual) + at);
      a += low<O>(r), b += high<O>(r);
    }
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(P.out) + at) = pack2f(a, b, O());
  }
}

__device__ __forceinline__ float2 ld_cluster(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// Unit u: bands of q tiles, in one the p tiles, in one of those the band's q tiles, so that the
// units side by side on the GPU read few different tiles of either operand.
__device__ __forceinline__ void unit_tiles(const LinearParams &P, int u, int &pt, int &qt) {
  const int each = P.band * P.p_tiles, b = u / each, rest = u - b * each;
  const int wide = min(P.band, P.q_tiles - b * P.band);
  pt = rest / wide;
  qt = b * P.band + rest - pt * wide;
}

// T: operands; O: out and residual.  kJoin: partial sums are joined in registers (units of one
// accumulator), and over the cluster where t is split.
template <bool kTrans, class T, class O, bool kJoin>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ Maps M, const LinearParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared &S = *reinterpret_cast<Shared *>(smem + kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s_ring = smem_u32(smem);
  const uint32_t bar_full = smem_u32(S.full), bar_empty = smem_u32(S.empty);
  const uint32_t bar_acc_full = smem_u32(S.acc_full), bar_acc_empty = smem_u32(S.acc_empty);
  volatile int *abort = &S.abort;
  const int in_cluster = (int)cluster_ctarank(), rank = in_cluster & 1, split = in_cluster >> 1;
  const uint32_t lead = (uint32_t)(in_cluster & ~1);
  const uint16_t both = (uint16_t)(3u << lead);

  if (warp == 0) {
    if (lane < P.stages) {
      mbar_init(bar_full + 8 * lane, 1);
      mbar_init(bar_empty + 8 * lane, 1);
    }
    if (lane < 2) {
      mbar_init(bar_acc_full + 8 * lane, 1);
      mbar_init(bar_acc_empty + 8 * lane, 2 * kEpiWarps);  // both CTAs' epilogue warps
    }
    if (lane == 0) {
      S.abort = 0;
      tma_prefetch_desc(&M.p);
      tma_prefetch_desc(&M.q);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S.tmem), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // every CTA's barriers exist before anything targets them
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  auto fail = [&] {
    *abort = 1;
    segments_status(P.status, MOE_STATUS_TIMEOUT);
  };
  // Waits for what takes a whole unit last longer the deeper the unit.
  const uint64_t unit_limit = kWaitLimitNs + 2000ull * P.blocks;
  auto wait = [&](uint32_t bar, uint32_t parity, uint64_t limit) {
    const bool ok = mbar_wait(bar, parity, abort, limit);
    if (!ok) fail();
    return ok;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity, uint64_t limit) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit));
    if (!ok) fail();
    return ok;
  };
  const int clusters = (int)cluster_count_x();
  const int nq_unit = P.nq;
  // this pair's blocks of t
  const int first = kJoin ? (int)((int64_t)P.blocks * split / P.splits) : 0;
  const int last = kJoin ? (int)((int64_t)P.blocks * (split + 1) / P.splits) : P.blocks;
  const uint32_t stage_bytes = kPBytes + (uint32_t)nq_unit / 2 * (BT * 2);

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      const uint64_t pol_keep = policy_evict_normal(), pol_p = P.q_tiles == 1 ? policy_evict_first() : pol_keep;
      const uint32_t lead_full = mapa_shared(bar_full, lead);
      int slot = 0, filled = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = (int)cluster_id_x(); ok && u < P.units; u += clusters) {
        int pt, qt;
        unit_tiles(P, u, pt, qt);
        const int p0 = pt * BP + 128 * rank, q0 = qt * nq_unit + nq_unit / 2 * rank;
        for (int b = first; b < last; ++b) {
          const int t = b * BT;
          ok = wait(bar_empty + 8 * slot, phase ^ 1u, kWaitLimitNs);
          if (!ok) break;
          const uint32_t dst = s_ring + slot * stage_bytes, bar = lead_full + 8 * slot;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * slot, 2 * stage_bytes);
          if constexpr (!kTrans) {
            tma_load<true>(dst, &M.p, bar, t, p0, 0, 0, pol_p);
          } else if (P.p_blocked) {
            tma_load<true>(dst, &M.p, bar, 0, t, p0 >> 6, 0, pol_p);
          } else {
            tma_load<true>(dst, &M.p, bar, p0, t, 0, 0, pol_p);
            tma_load<true>(dst + 8192, &M.p, bar, p0 + 64, t, 0, 0, pol_p);
          }
          tma_load<true>(dst + kPBytes, &M.q, bar, t, q0, 0, 0, pol_keep);
          if (filled < P.stages) ++filled;
          if (++slot == P.stages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      // what the MMAs' commits still have to say to this CTA's barriers comes before its end
      ok = ok && !*abort;
      if (filled < P.stages) slot = 0, phase = 1;  // the slots in use, in their order
      for (int i = 0; ok && i < filled; ++i) {
        ok = wait(bar_empty + 8 * slot, phase ^ 1u, kWaitLimitNs);
        if (++slot == P.stages) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (*abort) {  // let the copies in flight land before the CTA can exit
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      // binary32 sums; A = P (bit 15: MN-major), B = Q
      const uint32_t idesc = (1u << 4) | ((uint32_t)P.bf16 << 7) | ((uint32_t)P.bf16 << 10) |
                             ((kTrans ? 1u : 0u) << 15) | ((uint32_t)(P.nq >> 3) << 17) | ((uint32_t)(BP >> 4) << 24);
      const int rem = P.nt - (P.blocks - 1) * BT;
      int acc = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      // accumulator number a has been read: the one before it in the same place (flip), or itself
      auto wait_acc = [&](int a, uint32_t flip) {
        const bool read = mbar_wait_relaxed(bar_acc_empty + 8 * (a & 1), ((uint32_t)(a >> 1) & 1u) ^ flip,
                                            abort, unit_limit);
        if (!read) fail();
        return read;
      };
      auto multiply = [&](uint32_t d, uint64_t dp, uint64_t dq, int steps, bool more) {
        mma_pair_f16(d, dp, dq, idesc, more);
        if (steps == BT / 16) {
#pragma unroll
          for (int j = 1; j < BT / 16; ++j)
            mma_pair_f16(d, dp + j * kStep<kTrans>, dq + j * kStep<false>, idesc, 1);
        } else {
          for (int j = 1; j < steps; ++j)
            mma_pair_f16(d, dp + j * kStep<kTrans>, dq + j * kStep<false>, idesc, 1);
        }
      };
      for (int u = (int)cluster_id_x(); ok && u < P.units; u += clusters) {
        for (int b0 = first; ok && b0 < last; b0 += P.chunk) {
          const int b1 = min(last, b0 + P.chunk);
          ok = wait_acc(acc, 1u);
          if (!ok) break;
          tc_fence_after();
          for (int b = b0; b < b1; ++b) {
            ok = wait(bar_full + 8 * slot, phase, kWaitLimitNs);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sp = s_ring + slot * stage_bytes;
            const uint64_t dp = operand_desc<kTrans>(sp), dq = operand_desc<false>(sp + kPBytes);
            const int steps = b == P.blocks - 1 ? (rem + 15) >> 4 : BT / 16;
            multiply(tmem + 256 * (acc & 1), dp, dq, steps, b != b0);
            tc_commit_pair_mc(bar_empty + 8 * slot, both);
            if (++slot == P.stages) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          tc_commit_pair_mc(bar_acc_full + 8 * (acc & 1), both);
          ++acc;
        }
      }
      // the odd CTA's last releases come before this one's end
      for (int a = max(0, acc - 2); ok && a < acc; ++a) ok = wait_acc(a, 0u);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    // A warp reads the TMEM lanes 32 * (warp % 4)..+31; the warps of a lane quarter take the
    // 32-column groups in turn.
    constexpr int kTurns = kEpiWarps / 4, kEach = BQ / (32 * kTurns);
    const int quarter = warp & 3, turn = (warp - 4) >> 2;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t lead_acc_empty = mapa_shared(bar_acc_empty, lead);
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lead_acc_empty + 8 * buf);
    };
    int acc = 0;
    bool ok = true;
    for (int u = (int)cluster_id_x(); ok && u < P.units; u += clusters) {
      int pt, qt;
      unit_tiles(P, u, pt, qt);
      const int p = pt * BP + 128 * rank + 32 * quarter + lane, q0 = qt * nq_unit;
      const int rows = min(nq_unit, P.rows - q0);
      const bool inside = p < P.np;
      const float bias = P.bias && inside ? __ldg(P.bias + p) : 0.0f;
      const int64_t at = (int64_t)q0 * P.np + p;
      if constexpr (kJoin) {
        float sum[kEach][32];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        for (int b0 = first; b0 < last; b0 += P.chunk, ++acc) {
          const int buf = acc & 1;
          if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int c = 32 * (turn + kTurns * i);
            if (c < rows) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {  // parts that leave the sums in registers
                uint32_t v[16];
                tmem_ld_x16(t_lane + 256 * buf + c + h, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[i][h + j] += __uint_as_float(v[j]);
              }
            }
          }
          release(buf);
        }
        if (!ok) break;
        if (P.splits == 1) {
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int c = 32 * (turn + kTurns * i);
            if (c < rows) finish<T, O, 8>(P, sum[i], at + (int64_t)c * P.np, rows - c, inside, bias, lane);
          }
        } else {
          // The ring is free: this pair's MMAs are done with it, and there is one unit.
          float *stage = reinterpret_cast<float *>(smem) + 32 * quarter + lane;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int c = 32 * (turn + kTurns * i);
            if (c < rows)
#pragma unroll
              for (int j = 0; j < 32; ++j) stage[(c + j) * 128] = sum[i][j];
          }
        }
      } else {
        const int buf = acc & 1;
        if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) break;
        ++acc;
        tc_fence_after();
#pragma unroll 1
        for (int c = 32 * turn; c < rows; c += 32 * kTurns) {
          uint32_t v[32];
          MOE_TMEM_LD_32x32b_X32(t_lane + 256 * buf + c, v);
          tc_wait_ld();
          if (c + 32 * kTurns >= rows) release(buf);
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
          finish<T, O, 32>(P, f, at + (int64_t)c * P.np, rows - c, inside, bias, lane);
        }
        if (32 * turn >= rows) release(buf);
      }
    }
  }

  if (kJoin && P.splits > 1) {
    __syncthreads();
    cluster_sync();  // the partial sums of all pairs
    int pt, qt;
    unit_tiles(P, (int)cluster_id_x(), pt, qt);
    const int p0 = pt * BP + 128 * rank, q0 = qt * nq_unit, rows = min(nq_unit, P.rows - q0);
    // this CTA's share of the q's, two p's a thread
    const int from = rows * split / P.splits, to = rows * (split + 1) / P.splits;
    const int lane2 = threadIdx.x & 63;
    if (p0 + 2 * lane2 < P.np) {
      for (int q = from + (int)(threadIdx.x >> 6); q < to; q += kThreads / 64) {
        const uint32_t addr = s_ring + (uint32_t)(q * 128 + 2 * lane2) * 4;
        float2 part[kMostSplits];
#pragma unroll
        for (int s = 0; s < kMostSplits; ++s)
          if (s < P.splits) part[s] = ld_cluster(mapa_shared(addr, (uint32_t)(2 * s + rank)));
        float a = part[0].x, b = part[0].y;
#pragma unroll
        for (int s = 1; s < kMostSplits; ++s)
          if (s < P.splits) a += part[s].x, b += part[s].y;
        const int p = p0 + 2 * lane2;
        finish_two<T, O>(P, a, b, (int64_t)(q0 + q) * P.np + p, p);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // no CTA ends while another reads its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// ----------------------------------------------------------------- host side
struct Plan {
  int nq, q_tiles, p_tiles, splits;
};
// Tile and split with the least time by a plain model in SM cycles, fitted to sweeps over both.
// A block of 64 t's takes the MMAs' 2 cycles a row or its bytes at 55 a cycle (and 60 more
// with the 6 stages that 256 rows leave); a split, the exchange and a larger cluster's launch.
Plan plan_of(int64_t rows, int np, int blocks, int pairs, const int *clusters) {
  Plan best = {};
  double least = 0;
  const int p_tiles = (np + BP - 1) / BP;
  for (int nq = 32; nq <= BQ; nq += 32) {
    const int64_t tiles = (rows + nq - 1) / nq;
    const int even = (int)(((rows + tiles - 1) / tiles + 31) / 32 * 32);
    if (even != nq) continue;
    const int64_t units = tiles * p_tiles;
    const double block = std::max(2.0 * nq, (16384 + 64.0 * nq) / 55) + (nq > 224 ? 60 : 0);
    for (int s = 1; s <= kMostSplits; ++s) {
      // one unit a cluster, and blocks for everyone
      if (s > 1 && (units > clusters[s] || units * s > pairs || s * 2 > blocks)) continue;
      const double waves = s > 1 ? 1 : (double)((units + pairs - 1) / pairs);
      const double time = waves * ((blocks + s - 1) / s * block + 300) + 6.0 * nq + (s > 1 ? 3800 + 22.0 * nq : 0);
      if (best.nq == 0 || time < least) {
        least = time;
        best = {nq, (int)tiles, p_tiles, s};
      }
    }
  }
  return best;
}

cudaLaunchConfig_t config(int ctas, int splits, cudaLaunchAttribute *attr, void *stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = as_stream(stream);
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 2 * splits;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Shared memory and cluster size of an instance, raised once a device.
template <auto kernel>
int prepare() {
  static bool done[kMaxDevices] = {};
  static std::mutex setting;  // threads whose first calls come at once
  const int dev = device_slot();
  if (dev < 0) return dev;
  const std::lock_guard<std::mutex> lock(setting);
  if (!done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return set_cuda_error(e);
    done[dev] = true;
  }
  return MOE_OK;
}

// Clusters of s pairs that the device runs at once, s = 1..kMostSplits: every instance takes an
// SM a CTA, so one answers for all.  Asked once a device.
int cluster_counts(const int **counts) {
  static int most[kMaxDevices][kMostSplits + 1] = {};
  static std::mutex asked;
  constexpr auto kernel = linear_kernel<false, __half, float, true>;
  const int dev = device_slot();
  if (dev < 0) return dev;
  const std::lock_guard<std::mutex> lock(asked);
  if (most[dev][1] == 0) {
    const int rc = prepare<kernel>();
    if (rc != MOE_OK) return rc;
    for (int s = kMostSplits; s >= 1; --s) {
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t cfg = config(2 * s, s, &attr, nullptr);
      int n = 0;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (s == 1 && (e != cudaSuccess || n <= 0))
        return set_cuda_error(e != cudaSuccess ? e : cudaErrorInvalidConfiguration);
      if (e != cudaSuccess) cudaGetLastError();  // a size that the device does not take
      most[dev][s] = e == cudaSuccess ? n : 0;
    }
  }
  *counts = most[dev];
  return MOE_OK;
}

template <bool kTrans, class T, class O, bool kJoin>
int launch(const Maps &maps, const LinearParams &P, int pairs, void *stream) {
  constexpr auto kernel = linear_kernel<kTrans, T, O, kJoin>;
  const int rc = prepare<kernel>();
  if (rc != MOE_OK) return rc;
  const int clusters = P.splits == 1 ? std::min(P.units, pairs) : P.units;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(2 * P.splits * clusters, P.splits, &attr, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, maps, P);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace

cudaError_t linear_default_status(int32_t *bits, bool clear) { return take_default_status(bits, clear); }

}  // namespace moe

using namespace moe;

extern "C" int moe_linear(const moe_linear_args *a, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  if (a->type != MOE_TYPE_BF16 && a->type != MOE_TYPE_F16) return MOE_ERR_INVALID;
  if (a->out_type != a->type && a->out_type != MOE_TYPE_F32) return MOE_ERR_INVALID;
  if (a->rows < 0 || a->n <= 0 || a->k <= 0 || (a->trans != 0 && a->trans != 1)) return MOE_ERR_INVALID;
  if (a->act < MOE_ACT_NONE || a->act > MOE_ACT_SILU) return MOE_ERR_INVALID;
  if (a->rows > INT32_MAX - 1024 || a->n % 8 || a->k % 8 || a->n > (1 << 24) || a->k > (1 << 24) ||
      (int64_t)a->n * a->k >= (1ll << 38))
    return MOE_ERR_UNSUPPORTED;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->w || !a->out || off16(a->x) || off16(a->w) || off16(a->out) || off16(a->residual) ||
      off16(a->pre) || (uintptr_t)a->bias % 4)
    return MOE_ERR_INVALID;
  LinearParams P = {};
  P.rows = (int)a->rows;
  P.np = a->trans ? a->k : a->n;
  P.nt = a->trans ? a->n : a->k;
  P.blocks = (P.nt + BT - 1) / BT;
  P.bf16 = a->type == MOE_TYPE_BF16;
  P.act = a->act;
  P.bias = a->bias;
  P.residual = a->residual;
  P.pre = a->pre;
  P.out = a->out;
  P.status = a->status;
  P.p_blocked = a->k % BT == 0;
  const bool f32 = a->out_type == MOE_TYPE_F32, longer = P.nt > (P.bf16 ? kLongestBf16 : kLongestF16);
  const int sms = a->num_sms > 0 ? a->num_sms : device_sm_count();
  const int *clusters = nullptr;
  const int found = cluster_counts(&clusters);
  if (found != MOE_OK) return found;
  const int pairs = std::max(1, std::min(sms / 2, clusters[1]));
  const Plan plan = plan_of(a->rows, P.np, P.blocks, pairs, clusters);
  const int64_t units = (int64_t)plan.p_tiles * plan.q_tiles;
  if (units > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  P.nq = plan.nq;
  P.q_tiles = plan.q_tiles;
  P.p_tiles = plan.p_tiles;
  // as many rows of x as columns of w in the units side by side
  P.band = std::max(1, (int)std::lround(std::sqrt((double)pairs * BP / plan.nq)));
  P.units = (int)units;
  P.splits = plan.splits;
  P.chunk = f32 ? kSumBlocks : longer ? kJoinBlocks : P.blocks;
  P.stages = (int)std::min<uint32_t>(kDepth, kRing / (kPBytes + plan.nq / 2 * (BT * 2)));
  const bool join = f32 || longer || P.splits > 1;
  Maps maps = {};
  const uint64_t n = a->n, k = a->k, rows = a->rows;
  bool ok = a->trans ? map_mn_major(&maps.p, a->w, 1, n, k, 2) : map_k_major(&maps.p, a->w, 1, n, k, 128);
  ok = ok && map_k_major(&maps.q, a->x, 1, rows, P.nt, plan.nq / 2);
  if (!ok) return MOE_ERR_CUDA;
  auto run = [&](auto trans, auto t) {
    constexpr bool kTrans = decltype(trans)::value;
    using T = decltype(t);
    if (f32) return launch<kTrans, T, float, true>(maps, P, pairs, stream);
    return join ? launch<kTrans, T, T, true>(maps, P, pairs, stream) : launch<kTrans, T, T, false>(maps, P, pairs, stream);
  };
  auto typed = [&](auto trans) { return P.bf16 ? run(trans, __nv_bfloat16()) : run(trans, __half()); };
  return a->trans ? typed(std::true_type()) : typed(std::false_type());
}
