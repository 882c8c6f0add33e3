// moe_grouped_gemm and moe_grouped_wgrad: grouped products of 16-bit operands over
// ragged row segments, on tcgen05 tensor cores,
//   forward   out[r][j] = sum_i x[r][i] w[e][j][i]
//   trans     out[r][i] = sum_j x[r][j] w[e][j][i]
//   gradient  out[e][j][i] = sum_{r in e} dy[r][j] x[r][i].
//
// All three are out[q][p] = sum_t Q(q, t) P(p, t) with p the output's contiguous index:
// P is the weights (forward, trans) or x (gradient), Q the rows of a segment or dy.  The
// MMA's M side (lanes of the accumulator) is p and its N side (columns) is q, because the
// ragged extent belongs on N: a segment's rows are cut to multiples of 32 there, against
// 128 or 256 on M, and an expert of 270 rows would else pay for 384 or 512.
//
// CTA pairs (two SMs of a TPC): cta_group::2 MMAs of 256 x N x 16, N <= 256, binary32
// accumulators in tensor memory.  Each CTA holds 128 of the tile's p and half of its q, so
// a 64-deep block of t moves 32 KB into each SM for 512 tensor cycles at N = 256.
//   warp 0  producer: TMA tiles into a ring of 6 stages (64 deep in t, 128-byte swizzle).
//           An operand whose contiguous index is t (forward: both; trans: Q) is K-major,
//           the others are MN-major in 64-wide column blocks: no operand is transposed by
//           anyone.  The weights' map has the expert as a dimension, so tiles that pass
//           an expert's edge in p or t read zeros, not the next expert.
//   warp 1  MMA issuer (of the even CTA) and TMEM owner.
//   warp 2  scheduler: decodes units from the table of segments, ahead of the others.
//   warp 3  gradient only: t runs over rows, and the block after a segment's last row
//           holds the next segment's (or padding: anything, NaN too).  MMAs take 16 rows
//           at a time, so at most 15 rows must not count; this warp writes zeros over them
//           in both operands before the MMA sees the stage.
//   warps 4-11  epilogue: TMEM -> registers -> global, two accumulators in turn, so a
//           unit's MMAs run beside the previous unit's stores.
// The tensor core's binary32 accumulation truncates: the relative error grows with the
// number of additions (measured 1e-6 at t = 1024 and 1.9e-5 at 16384).  16-bit outputs
// round far above that; binary32 gradients take partial sums of 512 rows and add them in
// the epilogue's registers with rounding to nearest.
#include <cuda_fp16.h>

#include "segments.cuh"

namespace moe {
namespace {

constexpr int kFwd = 0, kTrans = 1, kGrad = 2;
constexpr int kThreads = 384, kEpiWarps = 8;
constexpr int BP = 256, BQ = 256, BT = 64;  // tile of a CTA pair, depth of a stage
constexpr int kStages = 6, kUnitQ = 8;
constexpr uint32_t kPBytes = 128 * BT * 2, kQBytes = 128 * BT * 2;  // a CTA's halves
constexpr uint32_t kBoxRows = 32;                                   // rows of one Q box
constexpr int kSumBlocks = 8;  // blocks of one partial sum (binary32 output): 512 rows
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct Unit {
  int z;      // expert
  int p0;     // first p of the pair's tile
  int q0;     // first q: a row of the buffer (forward, trans), a column of dy (gradient)
  int nq;     // q's that exist, at most 256
  int n;      // N of the MMAs
  int t0;     // first t: 0, or the segment's first row (gradient)
  int blocks; // 64-deep blocks of t
  int rem;    // t's of the last block, 1..64
  int once;   // no other unit reads this P tile
  int end;
};

struct Shared {
  uint64_t full[kStages], empty[kStages], tail[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t unit_full[kUnitQ], unit_empty[kUnitQ];
  Unit unit[kUnitQ];
  uint32_t tmem;
  int abort;
  long long part[33];
  SegTable table;
};
constexpr uint32_t kOffShared = kStages * (kPBytes + kQBytes);
constexpr uint32_t kSmemBytes = kOffShared + sizeof(Shared) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

struct GroupedParams {
  SegParams seg;
  int np, nq, nt;  // extents of p; of q (gradient: n); of t (forward, trans)
  int bf16;
  int accumulate;
  void *out;
};

// ----------------------------------------------------------------------- PTX
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *map, uint32_t bar,
                                                 int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, uint32_t bar, int x,
                                            int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
// D (+)= A B^T over the pair: 256 rows of A (128 per CTA), N of B (half per CTA).
__device__ __forceinline__ void mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 16 t's of a stage: K-major rows of 128 bytes (step 32 bytes), or MN-major blocks of 64
// columns, 128 bytes per t (step 16 t's; column blocks 8 KB apart).
template <bool kMnMajor>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int step) {
  return kMnMajor ? smem_desc(base + 2048 * step, BT * 128, 1024, 2)
                  : smem_desc(base + 32 * step, 16, 1024, 2);
}

// ------------------------------------------------------------------- schedule
// Rows of a segment's row tiles: the fewest tiles of at most 256, evened out.
__device__ __forceinline__ int tile_rows(int count) {
  const int tiles = (count + BQ - 1) / BQ;
  return ((count + tiles - 1) / tiles + 31) / 32 * 32;
}
__device__ __forceinline__ int row_tiles(int count) {
  if (count <= 0) return 0;
  const int rows = tile_rows(count);
  return (count + rows - 1) / rows;
}

// Unit u: the segments in order, within one the p tiles, within one the row tiles (or, for
// the gradient, the q tiles), so units that share a weight tile run side by side.
template <int kMode>
__device__ __forceinline__ Unit get_unit(const GroupedParams &P, const SegTable &T, int64_t u,
                                         int p_tiles) {
  Unit U = {};
  if constexpr (kMode == kGrad) {
    const int q_tiles = (P.nq + BQ - 1) / BQ, per = p_tiles * q_tiles;
    const int e = find_segment(T, P.seg.E, (int)(u / per));
    const int local = (int)(u % per);
    U.z = e;
    U.p0 = local / q_tiles * BP;
    U.q0 = local % q_tiles * BQ;
    U.nq = min(BQ, P.nq - U.q0);
    U.n = U.nq > 128 ? 256 : 128;  // whole 64-wide column blocks in each CTA
    U.t0 = T.start[e];
    U.blocks = (T.count[e] + BT - 1) / BT;
    U.rem = T.count[e] - (U.blocks - 1) * BT;
  } else {
    const int e = find_segment(T, P.seg.E, (int)(u / p_tiles));
    const int tiles = T.before[e + 1] - T.before[e], rows = tile_rows(T.count[e]);
    const int64_t local = u - (int64_t)T.before[e] * p_tiles;
    const int qt = (int)(local % tiles);
    U.z = e;
    U.p0 = (int)(local / tiles) * BP;
    U.q0 = T.start[e] + qt * rows;
    U.nq = min(rows, T.count[e] - qt * rows);
    U.n = (U.nq + 31) / 32 * 32;
    U.blocks = (P.nt + BT - 1) / BT;
    U.rem = P.nt - (U.blocks - 1) * BT;
    U.once = tiles == 1;
  }
  return U;
}

// ------------------------------------------------------------------- epilogue
template <class O>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  return f32_to_bf16_bits(a) | (f32_to_bf16_bits(b) << 16);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return (uint32_t)__half_as_ushort(__float2half_rn(a)) |
         ((uint32_t)__half_as_ushort(__float2half_rn(b)) << 16);
}

// 32 columns (q0 + 0..31) of this warp's 32 lanes (p0 + lane) to the rows of a 16-bit
// output.  Neighbouring lanes swap one of each two columns, so that a lane holds two
// consecutive p of one row: 4-byte stores, 64 contiguous bytes a row.  np is even and p0 a
// multiple of 32, so a pair is inside or outside as one.
template <class O>
__device__ __forceinline__ void store_columns(const uint32_t *v, uint16_t *out, int64_t pitch,
                                              int p, int np, int nq, int lane) {
  const int odd = lane & 1;
  uint16_t *o = out + (p - odd) + odd * pitch;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float a = __uint_as_float(v[j]), b = __uint_as_float(v[j + 1]);
    const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    const uint32_t w = odd ? pack2<O>(got, b) : pack2<O>(a, got);
    if (p < np && j + odd < nq) *reinterpret_cast<uint32_t *>(o + (int64_t)j * pitch) = w;
  }
}

template <int kMode, class O>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const GroupedParams P) {
  constexpr bool kF32 = sizeof(O) == 4;
  constexpr bool kPMn = kMode != kFwd, kQMn = kMode == kGrad;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared &S = *reinterpret_cast<Shared *>(smem + kOffShared);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s_p = smem_u32(smem), s_q = s_p + kStages * kPBytes;
  const uint32_t bar_full = smem_u32(S.full), bar_empty = smem_u32(S.empty);
  const uint32_t bar_tail = smem_u32(S.tail);
  const uint32_t bar_acc_full = smem_u32(S.acc_full), bar_acc_empty = smem_u32(S.acc_empty);
  const uint32_t bar_unit_full = smem_u32(S.unit_full), bar_unit_empty = smem_u32(S.unit_empty);
  volatile int *abort = &S.abort;
  constexpr uint16_t kBoth = 3;
  const int rank = (int)cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full + 8 * s, kMode == kGrad ? 2 : 1);  // gradient: each CTA arrives
      mbar_init(bar_empty + 8 * s, 1);
      mbar_init(bar_tail + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full + 8 * b, 1);
      mbar_init(bar_acc_empty + 8 * b, 2 * kEpiWarps);  // both CTAs' epilogue warps
    }
    for (int q = 0; q < kUnitQ; ++q) {
      mbar_init(bar_unit_full + 8 * q, 1);
      // producer, MMA, epilogue warps, and the gradient's tail warp
      mbar_init(bar_unit_empty + 8 * q, 2 + kEpiWarps + (kMode == kGrad ? 1 : 0));
    }
    S.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S.tmem), kTmemCols);
    tmem_relinquish_pair();
  }
  build_segments(
      P.seg, S.table, S.part,
      [&](int n) {
        if constexpr (kMode == kGrad) return P.accumulate && n == 0 ? 0 : 1;
        return row_tiles(n);
      },
      cluster_id_x() == 0 && rank == 0);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before anything targets them
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int p_tiles = (P.np + BP - 1) / BP;
  const int64_t units = (int64_t)S.table.before[P.seg.E] * p_tiles *
                        (kMode == kGrad ? (P.nq + BQ - 1) / BQ : 1);

  auto fail = [&] {
    *abort = 1;
    status_or(P.seg.status, MOE_STATUS_TIMEOUT);
  };
  // Waits for what takes a whole unit last longer the deeper the unit.
  const uint64_t unit_limit = kWaitLimitNs + 2000ull * ((kMode == kGrad ? P.seg.rows : P.nt) / BT);
  // A wait of one thread, and one of all lanes of a warp that go on together or not at all.
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
  auto take = [&](int seq, Unit &U) {
    const int slot = seq % kUnitQ;
    if (!wait(bar_unit_full + 8 * slot, (uint32_t)(seq / kUnitQ) & 1u, unit_limit)) return false;
    U = S.unit[slot];
    return true;
  };
  auto take_warp = [&](int seq, Unit &U) {
    const int slot = seq % kUnitQ;
    if (!wait_warp(bar_unit_full + 8 * slot, (uint32_t)(seq / kUnitQ) & 1u, unit_limit)) return false;
    U = S.unit[slot];
    return true;
  };
  auto release_unit = [&](int seq) { mbar_arrive(bar_unit_empty + 8 * (seq % kUnitQ)); };
  // Blocks of one accumulation: all of the unit's, or (binary32 output) kSumBlocks.
  auto sums_of = [](const Unit &U) {
    return kF32 ? max(1, (U.blocks + kSumBlocks - 1) / kSumBlocks) : 1;
  };

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_normal();
      const uint32_t lead_full = mapa_shared(bar_full, 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int seq = 0; ok; ++seq) {
        Unit U;
        if (!take(seq, U)) break;
        release_unit(seq);
        if (U.end) break;
        const uint64_t pol_p = U.once ? pol_stream : pol_keep;
        const int half = U.n / 2;
        const int boxes = kQMn ? half / 64 : (half + (int)kBoxRows - 1) / (int)kBoxRows;
        const uint32_t bytes = kPBytes + boxes * (kQMn ? 8192u : kBoxRows * 128u);
        const int p0 = U.p0 + 128 * rank, q0 = U.q0 + half * rank;
        for (int b = 0; b < U.blocks; ++b) {
          if (!wait(bar_empty + 8 * stage, phase ^ 1, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const uint32_t dp = s_p + stage * kPBytes, dq = s_q + stage * kQBytes;
          const int t = U.t0 + b * BT;
          const bool tail = kMode == kGrad && b == U.blocks - 1 && (U.rem & 15);
          if (tail) {
            // completes here, for the tail warp
            const uint32_t bar = bar_tail + 8 * stage;
            mbar_arrive_expect_tx(bar, bytes);
            for (int j = 0; j < 2; ++j) tma_load_3d(dp + 8192 * j, &tmP, bar, p0 + 64 * j, t, 0, pol_keep);
            for (int j = 0; j < boxes; ++j)
              tma_load_3d(dq + 8192 * j, &tmQ, bar, q0 + 64 * j, t, 0, pol_keep);
          } else {
            const uint32_t bar = lead_full + 8 * stage;
            if (rank == 0)
              mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * bytes);
            else if (kMode == kGrad)
              mbar_arrive_cluster(bar);
            if constexpr (kMode == kFwd) {
              tma_load_3d_pair(dp, &tmP, bar, t, p0, U.z, pol_p);
            } else {
              for (int j = 0; j < 2; ++j)
                tma_load_3d_pair(dp + 8192 * j, &tmP, bar, p0 + 64 * j, t, kMode == kGrad ? 0 : U.z, pol_p);
            }
            for (int j = 0; j < boxes; ++j) {
              if constexpr (kQMn)
                tma_load_3d_pair(dq + 8192 * j, &tmQ, bar, q0 + 64 * j, t, 0, pol_keep);
              else
                tma_load_3d_pair(dq + kBoxRows * 128 * j, &tmQ, bar, t, q0 + (int)kBoxRows * j, 0, pol_keep);
            }
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort) {  // let the copies in flight land before the CTA can exit
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------- MMA issuer
      // binary32 sums; A = P, B = Q, bits 15 / 16: MN-major
      const uint32_t idesc0 = (1u << 4) | ((uint32_t)P.bf16 << 7) | ((uint32_t)P.bf16 << 10) |
                              ((kPMn ? 1u : 0u) << 15) | ((kQMn ? 1u : 0u) << 16) |
                              ((uint32_t)(BP >> 4) << 24);
      int stage = 0, acc = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int seq = 0; ok; ++seq) {
        Unit U;
        if (!take(seq, U)) break;
        release_unit(seq);
        if (U.end) break;
        if (rank != 0) continue;  // the odd CTA only follows the unit stream
        const uint32_t idesc = idesc0 | ((uint32_t)(U.n >> 3) << 17);
        const int sums = sums_of(U);
        for (int s = 0; s < sums && ok; ++s) {
          const int buf = acc & 1;
          const uint32_t d = tmem + 256 * buf;
          if (!mbar_wait_cluster(bar_acc_empty + 8 * buf, ((uint32_t)(acc >> 1) & 1u) ^ 1u, abort,
                                 kWaitLimitNs)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const int b0 = kF32 ? s * kSumBlocks : 0;
          const int b1 = kF32 ? min(U.blocks, b0 + kSumBlocks) : U.blocks;
          for (int b = b0; b < b1; ++b) {
            if (!mbar_wait_cluster(bar_full + 8 * stage, phase, abort, kWaitLimitNs)) {
              fail();
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sp = s_p + stage * kPBytes, sq = s_q + stage * kQBytes;
            const int steps = b == U.blocks - 1 ? (U.rem + 15) >> 4 : BT / 16;
#pragma unroll
            for (int j = 0; j < BT / 16; ++j)
              if (j < steps)
                mma_pair_f16(d, operand_desc<kPMn>(sp, j), operand_desc<kQMn>(sq, j), idesc,
                             (b != b0) | (j != 0));
            tc_commit_pair_mc(bar_empty + 8 * stage, kBoth);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          tc_commit_pair_mc(bar_acc_full + 8 * buf, kBoth);
          ++acc;
        }
      }
    } else if (warp == 2 && lane == 0) {
      // --------------------------------------------------------- scheduler
      int seq = 0;
      auto push = [&](const Unit &U) {
        const int slot = seq % kUnitQ;
        if (!wait(bar_unit_empty + 8 * slot, ((uint32_t)(seq / kUnitQ) & 1u) ^ 1u, unit_limit))
          return false;
        S.unit[slot] = U;
        mbar_arrive(bar_unit_full + 8 * slot);
        ++seq;
        return true;
      };
      bool ok = true;
      for (int64_t u = cluster_id_x(); ok && u < units; u += cluster_count_x())
        ok = push(get_unit<kMode>(P, S.table, u, p_tiles));
      if (ok) {
        Unit end = {};
        end.end = 1;
        push(end);
      }
    } else if (kMode == kGrad && warp == 3) {
      // -------------------------------------- rows past the segment's last
      const uint32_t lead_full = mapa_shared(bar_full, 0);
      int stage = 0;
      uint32_t parity = 0;  // of each stage's tail barrier
      for (int seq = 0;; ++seq) {
        Unit U;
        if (!take_warp(seq, U)) break;
        __syncwarp();
        if (lane == 0) release_unit(seq);
        if (U.end) break;
        if (U.blocks > 0 && (U.rem & 15)) {
          const int s = (stage + U.blocks - 1) % kStages;
          if (!wait_warp(bar_tail + 8 * s, (parity >> s) & 1u, unit_limit)) break;
          parity ^= 1u << s;
          // 8 pieces of 16 bytes a row, in P's two column blocks and Q's (one or) two
          const int lines = 16 - (U.rem & 15);
          for (int i = lane; i < lines * 32; i += 32) {
            const int row = U.rem + (i >> 5), block = (i >> 3) & 3, piece = i & 7;
            uint8_t *base = smem + (block < 2 ? s * kPBytes : kStages * kPBytes + s * kQBytes);
            *reinterpret_cast<uint4 *>(base + (block & 1) * 8192 + row * 128 + piece * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead_full + 8 * s);
        }
        stage = (stage + U.blocks) % kStages;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // A warp reads the TMEM lanes 32 * (warp % 4)..+31; the two warps of a lane quarter
    // take the 32-column groups in turn.
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t lead_acc_empty = mapa_shared(bar_acc_empty, 0);
    int acc = 0;
    bool ok = true;
    for (int seq = 0; ok; ++seq) {
      Unit U;
      if (!take_warp(seq, U)) break;
      __syncwarp();
      if (lane == 0) release_unit(seq);
      if (U.end) break;
      const int p = U.p0 + 128 * rank + 32 * quarter + lane;
      const int64_t pitch = P.np;
      const int64_t row0 = kMode == kGrad ? (int64_t)U.z * P.nq + U.q0 : U.q0;
      O *out = static_cast<O *>(P.out) + row0 * pitch;
      auto release = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_acc_empty + 8 * buf);
      };
      if constexpr (kF32) {
        float sum[4][32];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[g][j] = 0.0f;
        const int sums = sums_of(U);
        for (int s = 0; s < sums; ++s, ++acc) {
          const int buf = acc & 1;
          if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (U.blocks > 0) {  // a segment without rows: nothing was accumulated
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int c = 32 * (half + 2 * g);
              if (c < U.nq) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t v[16];
                  tmem_ld_x16(t_lane + 256 * buf + c + 16 * h, v);
                  tc_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) sum[g][16 * h + j] += __uint_as_float(v[j]);
                }
              }
            }
          }
          release(buf);
        }
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = 32 * (half + 2 * g);
          if (c >= U.nq || p >= P.np) continue;
          float *o = reinterpret_cast<float *>(out) + (int64_t)c * pitch + p;
          if (P.accumulate) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < U.nq) sum[g][j] += o[(int64_t)j * pitch];
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < U.nq) o[(int64_t)j * pitch] = sum[g][j];
        }
      } else {
        const int buf = acc & 1;
        if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) break;
        ++acc;
        tc_fence_after();
        for (int c = 32 * half; c < U.nq; c += 64) {
          uint32_t v[32];
          MOE_TMEM_LD_32x32b_X32(t_lane + 256 * buf + c, v);
          tc_wait_ld();
          if (U.blocks == 0) {  // a segment without rows: nothing was accumulated
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0;
          }
          store_columns<O>(v, reinterpret_cast<uint16_t *>(out) + (int64_t)c * pitch, pitch, p, P.np,
                           U.nq - c, lane);
        }
        release(buf);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the even CTA's MMAs read the odd CTA's shared memory to the end
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// ----------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// 16-bit tensor [mats][rows][cols] (cols contiguous), boxes of box_rows x 64 columns.
bool make_map(CUtensorMap *m, const void *base, uint64_t mats, uint64_t rows, uint64_t cols,
              uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, mats};
  cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  cuuint32_t box[3] = {BT, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_common(const moe_segments &seg, int n, int k, int type) {
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_F16) return MOE_ERR_INVALID;
  if (n <= 0 || k <= 0) return MOE_ERR_INVALID;
  const int rc = check_segments(seg, false);
  if (rc != MOE_OK) return rc;
  if (n % 8 || k % 8) return MOE_ERR_UNSUPPORTED;
  // the tensor maps' strides, in bytes, and the unit numbers stay in range
  if ((int64_t)n * k >= (1ll << 38) || n > (1 << 24) || k > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }

// max_units: no more units than this (the grid need not be larger).
template <int kMode, class O>
int launch(const CUtensorMap &mp, const CUtensorMap &mq, const GroupedParams &P, int64_t max_units,
           int num_sms, void *stream) {
  static int max_clusters[kMaxDevices] = {};
  const int dev = device_slot();
  if (dev < 0) return dev;
  auto kernel = grouped_kernel<kMode, O>;
  const int sms = num_sms > 0 ? num_sms : device_sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms / 2 > 0 ? sms / 2 * 2 : 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (max_clusters[dev] == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    int n = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess || n <= 0)
      return set_cuda_error(e != cudaSuccess ? e : cudaErrorInvalidConfiguration);
    max_clusters[dev] = n;
  }
  int64_t clusters = cfg.gridDim.x / 2;
  if (clusters > max_clusters[dev]) clusters = max_clusters[dev];
  if (clusters > max_units) clusters = max_units;
  if (clusters < 1) return MOE_OK;
  cfg.gridDim = dim3((unsigned)(2 * clusters));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mp, mq, P);
  if (e != cudaSuccess) return set_cuda_error(e);
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
  P.bf16 = a->type == MOE_TYPE_BF16;
  P.out = a->out;
  CUtensorMap mp, mq;
  if (!make_map(&mp, a->w, (uint64_t)a->seg.E, (uint64_t)a->n, (uint64_t)a->k, a->trans ? BT : 128) ||
      !make_map(&mq, a->x, 1, (uint64_t)a->seg.rows, (uint64_t)P.nt, kBoxRows))
    return MOE_ERR_CUDA;
  // row tiles: a full one per 256 rows, and one started in every segment that has rows
  const int64_t started = a->seg.E < a->seg.rows ? a->seg.E : a->seg.rows;
  const int64_t max_units = (a->seg.rows / BQ + started) * ((P.np + BP - 1) / BP);
  const bool bf = P.bf16;
  if (a->trans)
    return bf ? launch<kTrans, __nv_bfloat16>(mp, mq, P, max_units, a->num_sms, stream)
              : launch<kTrans, __half>(mp, mq, P, max_units, a->num_sms, stream);
  return bf ? launch<kFwd, __nv_bfloat16>(mp, mq, P, max_units, a->num_sms, stream)
            : launch<kFwd, __half>(mp, mq, P, max_units, a->num_sms, stream);
}

extern "C" int moe_grouped_wgrad(const moe_wgrad_args *a, void *stream) {
  if (!a) return MOE_ERR_INVALID;
  const int rc = check_common(a->seg, a->n, a->k, a->type);
  if (rc != MOE_OK) return rc;
  if ((a->out_type != a->type && a->out_type != MOE_TYPE_F32) ||
      (a->accumulate && a->out_type != MOE_TYPE_F32))
    return MOE_ERR_INVALID;
  if (!a->out || off16(a->out)) return MOE_ERR_INVALID;
  if (a->seg.rows > 0 && (!a->dy || !a->x || off16(a->dy) || off16(a->x))) return MOE_ERR_INVALID;
  GroupedParams P = {};
  P.seg = seg_params(a->seg, a->status);
  P.np = a->k;
  P.nq = a->n;
  P.bf16 = a->type == MOE_TYPE_BF16;
  P.out = a->out;
  P.accumulate = a->accumulate != 0;
  // without rows every segment is empty: the maps are not used, and need only be valid
  const uint64_t rows = a->seg.rows > 0 ? (uint64_t)a->seg.rows : 1;
  CUtensorMap mp, mq;
  if (!make_map(&mp, a->seg.rows > 0 ? a->x : a->out, 1, rows, (uint64_t)a->k, BT) ||
      !make_map(&mq, a->seg.rows > 0 ? a->dy : a->out, 1, rows, (uint64_t)a->n, BT))
    return MOE_ERR_CUDA;
  const int64_t max_units =
      (int64_t)a->seg.E * ((a->k + BP - 1) / BP) * ((a->n + BQ - 1) / BQ);
  if (a->out_type == MOE_TYPE_F32)
    return launch<kGrad, float>(mp, mq, P, max_units, a->num_sms, stream);
  return P.bf16 ? launch<kGrad, __nv_bfloat16>(mp, mq, P, max_units, a->num_sms, stream)
                : launch<kGrad, __half>(mp, mq, P, max_units, a->num_sms, stream);
}
