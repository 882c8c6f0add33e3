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
// accumulators in tensor memory.  Each CTA holds 128 of the tile's p and half of its q: a
// 64-deep block of t moves 32 KB into each SM for 512 tensor cycles at N = 256.  A unit of
// work is one expert, 256 p and up to 256 q (one accumulator; the other takes the next
// unit's MMAs while this one's is stored) or 512 (both: the P tile is read once for the two,
// 48 KB a block for 1024 cycles).  Units that share weights run side by side on the 76 pairs.
// The gradient's t is short, its output large: a unit there is 256 p and several Q tiles, one
// after the other, and the P tiles of the whole segment stay in shared memory meanwhile (of a
// longer one, chunk by chunk for two Q tiles).  Reading P once a Q tile instead bound it by
// L2 reads (12 TB/s): 16 experts of ~512 rows 346 us, now 307; of 2048, 1026 and 961.
//   warp 0  producer: TMA tiles into a ring in shared memory (128-byte swizzle).  An operand
//           whose contiguous index is t (forward: both; trans: Q) is K-major, the others are
//           MN-major in 64-wide column blocks: nothing is transposed by anyone.  The
//           weights' map has the expert as a dimension, so tiles that pass an expert's edge
//           in p or t read zeros, not the next expert.
//   warp 1  MMA issuer (of the even CTA) and TMEM owner.
//   warp 2  scheduler: decodes units from the table of segments, ahead of the others.
//   warp 3  gradient only: t runs over rows, and the block after a segment's last row
//           holds the next segment's (or padding: anything, NaN too).  MMAs take 16 rows
//           at a time, so at most 15 rows must not count; this warp writes zeros over them
//           in both operands before the MMAs may read the block.
//   warps 4-11  epilogue: TMEM -> registers -> global.  Forward and trans store the rows
//           from registers, which leaves the ring 212 KB; the gradient, whose units are
//           short and bound by their stores, hands blocks of 32 x 32 to bulk copies.
// The tensor core's binary32 accumulation truncates: the relative error grows with the
// number of additions (measured 1e-6 at t = 1024 and 1.9e-5 at 16384).  So long sums are
// joined: partial sums are added in the epilogue's registers with rounding to nearest.
// Binary32 gradients take 512 rows a partial sum.  16-bit outputs round far above the error
// of a sum of up to 16384 terms (fp16: 1/25 of its rounding) or 131072 (bf16, whose rounding
// is 8 times as coarse); what is longer is joined from partial sums of 4096 (t = 20000, fp16,
// 4096 x 2048 a product: forward 231 us against 210 in one sum, trans 223 and 210; gradient of
// 160000 rows, 4096 x 2048: as fast as two Q tiles that share P).
//
// What bounds it, and what it measured (64 experts, n = 4096, k = 7168; 6.76 TB/s and 1864
// TFLOP/s are a copy's and a dense library product's rates):
//   few rows an expert: the weights, once, from HBM (16 rows: 545 us, 6.9 TB/s).  By
//     Little's law that takes the 130 KB and more of weights that the ring keeps under way
//     in each SM; 64 KB gave 4.6 TB/s.
//   about 256 rows, ragged: weights, rows and output from and to HBM, 676 us (6.1 TB/s).
//   many rows: the tensor cores under the power cap, 1560 to 1960 TFLOP/s.
//   gradient, 16 experts of about 256 rows: 194 us, 4.8 TB/s of writes, shared memory 77 %
//     busy (copies in, MMAs, staging); zeros alone are written at 6.9 TB/s, the MMAs alone
//     would take 110 us.  2048 rows: 961 us, 2000 TFLOP/s.
// Tried and not kept: requests into L2 ahead of the ring (560 -> 667 us, they queue before
// the ring's own copies), Q multicast over clusters of two pairs (152 SMs hold 36 of them:
// 5 % slower), 128-deep blocks for the gradient, fewer slots for its Q (5: 197 us, 4: 213).
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "segments.cuh"

namespace moe {
namespace {

constexpr int kFwd = 0, kTrans = 1, kGrad = 2;
constexpr int kThreads = 384, kEpiWarps = 8;
constexpr int BP = 256, BQ = 256, BT = 64;  // tile of a CTA pair, depth of a block of t
constexpr int kWide = 2 * BQ;               // q's of a unit with both accumulators
constexpr int kUnitQ = 8;
constexpr uint32_t kPBytes = 128 * BT * 2;  // a CTA's half of a P tile
// Bytes of the operand ring, and of an epilogue warp's staging (gradient): a block of 32 x
// 32 16-bit values, or three in turn of 16 x 32 binary32 ones.
constexpr uint32_t kStage = 2048;
constexpr int kStages = 3;  // (two and six P slots: 464 against 434 us, 16 x ~512 rows)
constexpr uint32_t ring_bytes(int mode, bool f32) { return (mode != kGrad ? 212 : f32 ? 160 : 192) * 1024; }
constexpr uint32_t stage_bytes(int mode, bool f32) { return mode != kGrad ? 0 : f32 ? kStages * kStage : kStage; }
constexpr int kSumBlocks = 8;    // blocks of one partial sum (binary32 output): 512 rows
constexpr int kJoinBlocks = 64;  // of a joined sum with 16-bit output
constexpr int kLongestF16 = 16384, kLongestBf16 = 131072;  // terms of a sum that is not joined
// Slots of the gradient's operands, 16 KB each: P tiles stay while several Q tiles pass.  A Q
// slot's barriers serve a P tile too where one comes along.  Every use of a P tile has a Q tile
// of its own, so by the time that the Q slot of a block is free again, so is a P slot loaded
// as many P tiles ago as there are Q slots, or more.
constexpr int p_slots(bool f32) { return f32 ? 5 : 6; }
constexpr int q_slots(bool f32) { return (int)(ring_bytes(2, f32) / (16 * 1024)) - p_slots(f32); }
static_assert(q_slots(false) <= p_slots(false) && q_slots(true) <= p_slots(true), "P slots are reused by Q's barriers");
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__host__ __device__ constexpr uint32_t block_bytes(int n0, int n1) {  // of one CTA
  return kPBytes + (uint32_t)(n0 + n1) / 2 * (BT * 2);
}

struct Unit {
  int z;      // expert
  int p0;     // first p of the pair's tile
  int q0;     // first q: a row of the buffer (forward, trans), a column of dy (gradient)
  int nq;     // q's that exist, at most 512 (gradient: of all its Q tiles)
  int n[2];   // N of the MMAs of each accumulator (n[1] 0: one accumulator)
  int tiles, chunk; // gradient: Q tiles, and the blocks of t that each takes at a time
  int t0;     // first t: 0, or the segment's first row (gradient)
  int blocks; // 64-deep blocks of t
  int rem;    // t's of the last block, 1..64
  int once;   // no other unit reads this P tile
  int join;   // gradient: partial sums are joined by the epilogue (one Q tile a unit)
  int end;
};

// The operand ring.  Block i of the CTA's stream takes the barriers i % kDepth and room for
// its P tile and the Q tile of each accumulator, no more than they need: the fewer rows,
// the more blocks (and bytes of weights) are in flight.  A block that does not fit before
// the end starts at 0.  Every role that follows the stream keeps such a place and finds
// the same one.
constexpr int kDepth = 10;
template <uint32_t kBytes>
struct Ring {
  uint32_t pos = 0, end = 0;  // of the last block: its first byte after; the same, counted through
  uint32_t phase = 0;
  int bar = 0;
  // The place of the next block of `bytes`.
  __device__ __forceinline__ uint32_t place(uint32_t bytes) {
    if (pos + bytes > kBytes) {
      end += kBytes - pos;
      pos = 0;
    }
    const uint32_t at = pos;
    pos += bytes;
    end += bytes;
    return at;
  }
  __device__ __forceinline__ void next_block() {
    if (++bar == kDepth) {
      bar = 0;
      phase ^= 1;
    }
  }
};

// The gradient's slots of one operand, in turn.
template <int kSlots>
struct Slots {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kSlots) {
      at = 0;
      phase ^= 1;
    }
  }
};

struct Shared {
  uint64_t full[kDepth], empty[kDepth], tail[kDepth];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t unit_full[kUnitQ], unit_empty[kUnitQ];
  Unit unit[kUnitQ];
  uint32_t end[kDepth];  // Ring::end of the block that each barrier pair serves
  uint32_t tmem;
  int abort;
  int part[64];
  SegTable table;
};
constexpr uint32_t off_shared(int mode, bool f32) {
  return ring_bytes(mode, f32) + kEpiWarps * stage_bytes(mode, f32);
}
constexpr uint32_t smem_bytes(int mode, bool f32) { return off_shared(mode, f32) + sizeof(Shared) + 1024; }
static_assert(smem_bytes(kFwd, false) <= 232448 && smem_bytes(kGrad, false) <= 232448 &&
                  smem_bytes(kGrad, true) <= 232448,
              "shared memory");

// An MN-major operand's column blocks of 64 are a dimension of its map where the columns
// are a multiple of 64 (`blocked`: one copy brings two blocks), else one copy each.
struct Maps {
  CUtensorMap p;
  CUtensorMap q[8];  // K-major: boxes of 16, 32, ..., 128 rows; MN-major: of 1, 2 blocks
  CUtensorMap out;  // gradient
};

struct GroupedParams {
  SegParams seg;
  int np, nq, nt;  // extents of p; of q (gradient: n); of t (forward, trans)
  int p_blocked, q_blocked;
  int group;  // gradient: most Q tiles of a unit
  int longest; // most terms of a sum that is not joined (16-bit outputs)
  int bf16;
  int accumulate;
  void *out;
};

// ----------------------------------------------------------------------- PTX
// Copies of one box: counted on the even CTA's barrier, or (kPair false) on this CTA's.
template <bool kPair>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                         int y, int c, int z, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(c), "r"(z), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(c), "r"(z), "l"(policy)
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
// 32 columns of 16 TMEM lanes, as 16 x 8 blocks: r[4i], r[4i+1] hold lane t/4, columns
// 8i + 2(t%4) and +1 of thread t, r[4i+2], r[4i+3] lane t/4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 columns, the same way.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}
// Four 8x8 blocks of 16-bit values, each stored transposed; lane 8m + j gives the address
// of row j of block m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b,
                                                  uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// Arrive on an mbarrier of either CTA of the pair where no writes of this CTA's threads have
// to be ordered: operands land by TMA, and reads of an accumulator are ordered by the tcgen05
// fences before the arrival and after the (cluster-wide, relaxed) wait.  A release would first
// wait for the warp's global stores.  Writes take mbar_arrive_pair.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
// Where the pair's MMAs read what threads of the other CTA wrote to its shared memory: an
// arrival that releases those writes (the thread's, and those it has synchronised with) at
// cluster scope, and a wait that acquires them.  The fences are restricted to shared memory: an
// arrival with plain release also waits for whatever the SM is storing (16 experts of ~256
// rows, 4096 x 7168: 219 us, this 194).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_relaxed(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_relaxed(uint32_t bar, uint32_t parity, volatile int *abort,
                                                  uint64_t limit_ns) {
  if (mbar_try_wait_relaxed(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
#pragma unroll 1
  while (!mbar_try_wait_relaxed(bar, parity))
    if (*abort || globaltimer() - t0 > limit_ns) return false;
  return true;
}
__device__ __forceinline__ bool mbar_wait_pair(uint32_t bar, uint32_t parity, volatile int *abort,
                                               uint64_t limit_ns) {
  if (!mbar_wait_relaxed(bar, parity, abort, limit_ns)) return false;
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return true;
}
// The cluster's threads meet; nothing of their memory is ordered by it (a release would
// first wait for every store).  What one CTA sends to the other's barriers has been waited
// for there by then.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// One lane of a converged warp, chosen so that the compiler knows it is one: the
// descriptors of MMAs and copies sit in uniform registers, and behind `lane == 0` each
// would be issued through a loop over the lanes (80 cycles an MMA instead of 45).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tma_store(const void *map, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %5, %4}], [%1];" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z), "r"(0)
      : "memory");
}
__device__ __forceinline__ void tma_add(const void *map, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.4d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %5, %4}], "
      "[%1];" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z), "r"(0)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All of the thread's bulk stores but the last kBut have read their shared memory.
template <int kBut>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBut) : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Operand descriptors without their address, and what 16 t's add to it: K-major rows of
// 128 bytes (32 bytes a step), or MN-major blocks of 64 columns, 128 bytes per t (16 t's a
// step; column blocks 8 KB apart).  Addresses count 16 bytes.
template <bool kMnMajor>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (kMnMajor ? smem_desc(0, BT * 128, 1024, 2) : smem_desc(0, 16, 1024, 2)) + (addr >> 4);
}
template <bool kMnMajor>
constexpr uint64_t kStep = kMnMajor ? 2048 / 16 : 32 / 16;

// ------------------------------------------------------------------- schedule
// Rows of a segment's row tiles: one tile of up to 256 (one accumulator, the other one
// takes the next unit's MMAs meanwhile), else the fewest of up to `wide` (512: both; 256 where
// sums are joined, whose registers hold one), evened out.  (Unsigned: count and tiles may
// together pass 2^31.)
__device__ __forceinline__ int tile_rows(int count, int wide) {
  if (count <= wide) return (count + 31) / 32 * 32;
  const unsigned tiles = ((unsigned)count + wide - 1) / wide;
  return (int)((((unsigned)count + tiles - 1) / tiles + 31) / 32 * 32);
}
__device__ __forceinline__ int row_tiles(int count, int wide) {
  if (count <= wide) return count > 0;
  const int rows = tile_rows(count, wide);
  return (count + rows - 1) / rows;
}
// N of each accumulator for nq q's.
__device__ __forceinline__ void split_n(Unit &U) {
  if (U.nq <= BQ) {
    U.n[0] = (U.nq + 31) / 32 * 32;
    U.n[1] = 0;
  } else {
    U.n[0] = ((U.nq + 1) / 2 + 31) / 32 * 32;
    U.n[1] = (U.nq - U.n[0] + 31) / 32 * 32;
  }
}
// The gradient's Q tiles of a unit.  A short segment's P tiles all stay in their slots: one
// Q tile after the other passes over them (chunk: every block), as many as the host allows.  A
// long segment's pass in chunks, each Q tile in its own accumulator, so two.  Either way each P
// tile is read once for all of them, and an accumulator is stored beside the MMAs of the other.
// Binary32 outputs, where twice the stores bound a tile, take one (16 experts, 4096 x 7168,
// ~256 rows: 332 us against 352 in eights; 32 experts, 2048 x 2048, ~128 rows: 102 and 112),
// and joined sums in registers leave no room for more.
template <bool kF32, bool kLong>
__device__ __forceinline__ int grad_tiles(const GroupedParams &P, int count) {
  if (kF32 || (kLong && count > P.longest)) return 1;
  return count <= p_slots(false) * BT ? P.group : min(P.group, 2);
}
// Blocks of t that a Q tile takes at a time: of joined sums, those of one partial sum.
template <bool kF32>
__device__ __forceinline__ int grad_chunk(int blocks, bool join) {
  if (kF32) return kSumBlocks;
  if (join) return kJoinBlocks;
  const int chunks = (blocks + p_slots(false) - 1) / p_slots(false);
  return (blocks + chunks - 1) / max(chunks, 1);
}
// N of the MMAs of Q tile g: whole 64-wide column blocks in each CTA.
__device__ __forceinline__ int grad_n(int nq, int g) { return nq - BQ * g > BQ / 2 ? BQ : BQ / 2; }

// Unit u: the segments in order, within one the p tiles, within one the row tiles, so units
// that share a weight tile run side by side; for the gradient the groups of q tiles, within
// one the p tiles, so whole rows of the output are stored at a time (binary32, ~512 rows: 460
// us the other way, 434 this).  e: the segment of the caller's last unit, or -1.
template <int kMode, bool kF32, bool kLong>
__device__ __forceinline__ Unit get_unit(const GroupedParams &P, const SegTable &T, int u,
                                         int p_tiles, int &e) {
  Unit U = {};
  if (e < 0 || u >= T.before[e + 1] * p_tiles) e = find_segment(T, P.seg.E, u, p_tiles);
  const int tiles = T.before[e + 1] - T.before[e];  // q tiles of the segment
  const int local = u - T.before[e] * p_tiles, count = T.count[e];
  int pt, qt;
  if constexpr (kMode == kGrad) {
    qt = local / p_tiles;
    pt = local - qt * p_tiles;
  } else {
    pt = tiles == 1 ? local : local / tiles;
    qt = local - pt * tiles;
  }
  U.z = e;
  U.p0 = pt * BP;
  if constexpr (kMode == kGrad) {
    const int q = grad_tiles<kF32, kLong>(P, count) * BQ;
    U.q0 = qt * q;
    U.nq = min(q, P.nq - U.q0);
    U.tiles = (U.nq + BQ - 1) / BQ;
    U.t0 = T.start[e];
    U.blocks = (count + BT - 1) / BT;
    U.rem = count - (U.blocks - 1) * BT;
    U.join = kF32 || (kLong && count > P.longest);
    U.chunk = grad_chunk<kF32>(U.blocks, U.join);
  } else {
    const int rows = tile_rows(count, kLong ? BQ : kWide);
    U.q0 = T.start[e] + qt * rows;
    U.nq = min(rows, count - qt * rows);
    split_n(U);
    U.blocks = (P.nt + BT - 1) / BT;
    U.rem = P.nt - (U.blocks - 1) * BT;
    U.once = tiles == 1;
  }
  return U;
}

// ------------------------------------------------------------------- epilogue
template <class O>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
  uint32_t r;
  if constexpr (std::is_same<O, __half>::value)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return r;
}

// 32 accumulator columns (q) of this warp's 32 lanes (p) -> the rows of a 16-bit output;
// `out` at the first q and the warp's first p.  Neighbouring lanes swap one of each two
// q's, so that a lane holds two consecutive p of one row: 4-byte stores, 64 contiguous
// bytes a row, from registers.  (Staged in shared memory for wider stores or bulk copies,
// each block cost more in waits and proxy fences than these stores do.)  The extent of p
// is even and the first p a multiple of 32, so a pair is inside or outside as one.
template <class O>
__device__ __forceinline__ void store_columns(const uint32_t *v, uint16_t *out, int64_t pitch,
                                              int nq, bool inside, int lane) {
  const int odd = lane & 1;
  const uint32_t pick = odd ? 0x3276u : 0x5410u;
  uint16_t *o = out + (lane - odd) + odd * pitch;
  if (!inside) nq = 0;
#pragma unroll
  for (int j = 0; j < 32; j += 2, o += 2 * pitch) {
    const uint32_t mine = pack2<O>(v[j], v[j + 1]);
    const uint32_t w = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
    if (j + odd < nq) *reinterpret_cast<uint32_t *>(o) = w;
  }
}

// 32 accumulator columns (q) of this warp's 32 lanes (p), rounded: w[8h + 2i + (0, 1)] holds
// lanes 16h + (0, 8) + t/4, columns 8i + 2(t%4) and +1 of thread t.
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t *v) {
  tmem_ld_16x256b_x4(taddr, v);
  tmem_ld_16x256b_x4(taddr + (16u << 16), v + 16);
}
template <class O>
__device__ __forceinline__ void round_columns(const uint32_t *v, bool zero, uint32_t *w) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = zero ? 0u : pack2<O>(v[2 * i], v[2 * i + 1]);
}
// The block transposed into the warp's staging: rows [q][p] of 64 bytes, 16-byte pieces
// swizzled by row (the 64-byte TMA swizzle: neither these writes nor the copies out
// conflict on banks).
__device__ __forceinline__ uint32_t stage_offset(int q, int piece) {
  return 64 * q + 16 * (piece ^ ((q >> 1) & 3));
}
__device__ __forceinline__ void stage_rows(const uint32_t *w, uint32_t stage, int lane) {
  const int m = lane >> 3;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t *x = w + 8 * h + 4 * i;
      stmatrix_x4_trans(stage + stage_offset(16 * i + 8 * (m >> 1) + (lane & 7), 2 * h + (m & 1)),
                        x[0], x[1], x[2], x[3]);
    }
}

// kLong: 16-bit outputs with sums that may be longer than P.longest (forward and trans: that
// are).  An instance of its own, so that the others keep their registers.
template <int kMode, class O, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ Maps M, const GroupedParams P) {
  constexpr bool kF32 = sizeof(O) == 4;
  constexpr uint32_t kRing = ring_bytes(kMode, kF32);
  constexpr bool kPMn = kMode != kFwd, kQMn = kMode == kGrad;
  constexpr int kPSlots = p_slots(kF32), kQSlots = q_slots(kF32);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared &S = *reinterpret_cast<Shared *>(smem + off_shared(kMode, kF32));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s_ring = smem_u32(smem);
  const uint32_t bar_full = smem_u32(S.full), bar_empty = smem_u32(S.empty);
  const uint32_t bar_tail = smem_u32(S.tail);
  const uint32_t bar_acc_full = smem_u32(S.acc_full), bar_acc_empty = smem_u32(S.acc_empty);
  const uint32_t bar_unit_full = smem_u32(S.unit_full), bar_unit_empty = smem_u32(S.unit_empty);
  volatile int *abort = &S.abort;
  constexpr uint16_t kBoth = 3;
  const int rank = (int)cluster_ctarank();

  if (warp == 0) {  // a lane a barrier
    if (lane < kDepth) {
      mbar_init(bar_full + 8 * lane, kMode == kGrad ? 2 : 1);  // gradient: each CTA arrives
      mbar_init(bar_empty + 8 * lane, 1);
      mbar_init(bar_tail + 8 * lane, 1);
    }
    if (lane < 2) {
      mbar_init(bar_acc_full + 8 * lane, 1);
      mbar_init(bar_acc_empty + 8 * lane, 2 * kEpiWarps);  // both CTAs' epilogue warps
    }
    if (lane < kUnitQ) {
      mbar_init(bar_unit_full + 8 * lane, 1);
      // producer, MMA, epilogue warps, and the gradient's tail warp
      mbar_init(bar_unit_empty + 8 * lane, 2 + kEpiWarps + (kMode == kGrad ? 1 : 0));
    }
    if (lane == 0) {
      S.abort = 0;
      tma_prefetch_desc(&M.p);
      if (kMode == kGrad) tma_prefetch_desc(&M.out);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S.tmem), kTmemCols);
    tmem_relinquish_pair();
  }
  build_segments(
      P.seg, S.table, S.part,
      [&](int n) {
        if constexpr (kMode == kGrad) {
          const int q = grad_tiles<kF32, kLong>(P, n) * BQ;
          return P.accumulate && n == 0 ? 0 : (P.nq + q - 1) / q;
        }
        return row_tiles(n, kLong ? BQ : kWide);
      },
      cluster_id_x() == 0 && rank == 0);
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // both CTAs' barriers exist before anything targets them
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int p_tiles = (P.np + BP - 1) / BP;
  const int units = S.table.before[P.seg.E] * p_tiles;

  auto fail = [&] {
    *abort = 1;
    segments_status(P.seg.status, MOE_STATUS_TIMEOUT);
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

  if (warp < 4) {
    if (warp == 0) {
      if (elect_one()) {
        // ---------------------------------------------------------- producer
        const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_normal();
        const uint32_t lead_full = mapa_shared(bar_full, 0);
        if constexpr (kMode == kGrad) {
          int ps = 0;
          Slots<kQSlots> qs;
          bool ok = true;
          for (int seq = 0; ok; ++seq) {
            Unit U;
            if (!take(seq, U)) break;
            release_unit(seq);
            if (U.end) break;
            const int p0 = U.p0 + 128 * rank;
            const int tail = (U.rem & 15) ? U.blocks - 1 : -1;
            for (int b0 = 0; ok && b0 < U.blocks; b0 += U.chunk) {
              const int b1 = min(U.blocks, b0 + U.chunk);
              for (int g = 0; ok && g < U.tiles; ++g) {
                const int half = grad_n(U.nq, g) / 2, q0 = U.q0 + BQ * g + half * rank;
                const uint32_t bytes = half * (BT * 2) + (g == 0 ? kPBytes : 0);
                int t = U.t0 + b0 * BT;
                for (int b = b0; b < b1; ++b, t += BT, qs.next()) {
                  ok = wait(bar_empty + 8 * qs.at, qs.phase ^ 1u, kWaitLimitNs);
                  if (!ok) break;
                  const uint32_t to_p = s_ring + ps * kPBytes, to_q = s_ring + (kPSlots + qs.at) * kPBytes;
                  auto load = [&](auto counted_by_pair, uint32_t bar) {
                    constexpr bool kPair = decltype(counted_by_pair)::value;
                    if (g == 0) {
                      if (P.p_blocked) {
                        tma_load<kPair>(to_p, &M.p, bar, 0, t, p0 >> 6, 0, pol_keep);
                      } else {
                        tma_load<kPair>(to_p, &M.p, bar, p0, t, 0, 0, pol_keep);
                        tma_load<kPair>(to_p + 8192, &M.p, bar, p0 + 64, t, 0, 0, pol_keep);
                      }
                    }
                    if (P.q_blocked) {
                      tma_load<kPair>(to_q, &M.q[half / 64 - 1], bar, 0, t, q0 >> 6, 0, pol_keep);
                    } else {
                      for (int j = 0; j < half; j += 64)
                        tma_load<kPair>(to_q + 128 * j, &M.q[0], bar, q0 + j, t, 0, 0, pol_keep);
                    }
                  };
                  if (b == tail) {
                    // completes in this CTA, for its tail warp
                    mbar_arrive_expect_tx(bar_tail + 8 * qs.at, bytes);
                    load(std::false_type{}, bar_tail + 8 * qs.at);
                  } else {
                    if (rank == 0)
                      mbar_arrive_expect_tx(bar_full + 8 * qs.at, 2 * bytes);
                    else
                      mbar_arrive_remote(lead_full + 8 * qs.at);
                    load(std::true_type{}, lead_full + 8 * qs.at);
                  }
                  if (g == 0 && ++ps == kPSlots) ps = 0;
                }
              }
            }
          }
          // what the MMAs' commits still have to say to this CTA's barriers comes before its end
          ok = ok && !*abort;
          for (int i = 0; ok && i < kQSlots; ++i, qs.next())
            ok = wait(bar_empty + 8 * qs.at, qs.phase ^ 1u, kWaitLimitNs);
        } else {
          Ring<kRing> ring;
          uint32_t freed = 0;           // Ring::end of the last block that is known to be consumed,
          int old_bar = 0, blocks = 0;  // the barriers of the next, and the blocks not known to be
          uint32_t old_phase = 0;
          for (int seq = 0;; ++seq) {
            Unit U;
            if (!take(seq, U)) break;
            release_unit(seq);
            if (U.end) break;
            const uint64_t pol_p = U.once ? pol_stream : pol_keep;
            const int half0 = U.n[0] / 2, half1 = U.n[1] / 2;
            const int p0 = U.p0 + 128 * rank, qa = U.q0 + half0 * rank, qb = U.q0 + U.n[0] + half1 * rank;
            const CUtensorMap *map_a = &M.q[half0 / 16 - 1], *map_b = &M.q[half1 ? half1 / 16 - 1 : 0];
            const uint32_t bytes = block_bytes(U.n[0], U.n[1]), to_b = kPBytes + half0 * (BT * 2);
            int t = 0;
            bool ok = true;
            for (int b = 0; b < U.blocks; ++b, t += BT) {
              const uint32_t dst = s_ring + ring.place(bytes);
              while (ring.end - freed > kRing || blocks == kDepth) {
                ok = wait(bar_empty + 8 * old_bar, old_phase, kWaitLimitNs);
                if (!ok) break;
                freed = *(volatile uint32_t *)&S.end[old_bar];
                --blocks;
                if (++old_bar == kDepth) {
                  old_bar = 0;
                  old_phase ^= 1;
                }
              }
              if (!ok) break;
              *(volatile uint32_t *)&S.end[ring.bar] = ring.end;
              const uint32_t bar = lead_full + 8 * ring.bar;
              if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * ring.bar, 2 * bytes);
              if constexpr (kMode == kFwd) {
                tma_load<true>(dst, &M.p, bar, t, p0, 0, U.z, pol_p);
              } else if (P.p_blocked) {
                tma_load<true>(dst, &M.p, bar, 0, t, p0 >> 6, U.z, pol_p);
              } else {
                tma_load<true>(dst, &M.p, bar, p0, t, 0, U.z, pol_p);
                tma_load<true>(dst + 8192, &M.p, bar, p0 + 64, t, 0, U.z, pol_p);
              }
              tma_load<true>(dst + kPBytes, map_a, bar, t, qa, 0, 0, pol_keep);
              if (half1) tma_load<true>(dst + to_b, map_b, bar, t, qb, 0, 0, pol_keep);
              ++blocks;
              ring.next_block();
            }
            if (!ok) break;
          }
          // what the MMAs' commits still have to say to this CTA's barriers comes before its end
          for (bool ok = !*abort; ok && blocks > 0; --blocks) {
            ok = wait(bar_empty + 8 * old_bar, old_phase, kWaitLimitNs);
            if (++old_bar == kDepth) {
              old_bar = 0;
              old_phase ^= 1;
            }
          }
        }
        if (*abort) {  // let the copies in flight land before the CTA can exit
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 1000000ull) {
          }
        }
      }
    } else if (warp == 1) {
      if (elect_one()) {
        // -------------------------------------------------------- MMA issuer
        // binary32 sums; A = P, B = Q, bits 15 / 16: MN-major
        const uint32_t idesc0 = (1u << 4) | ((uint32_t)P.bf16 << 7) | ((uint32_t)P.bf16 << 10) |
                                ((kPMn ? 1u : 0u) << 15) | ((kQMn ? 1u : 0u) << 16) |
                                ((uint32_t)(BP >> 4) << 24);
        int acc = 0;
        bool ok = true;
        // accumulator number a has been read: the one before it in the same place (flip), or itself
        auto wait_acc = [&](int a, uint32_t flip) {
          const bool read = mbar_wait_relaxed(bar_acc_empty + 8 * (a & 1), ((uint32_t)(a >> 1) & 1u) ^ flip,
                                              abort, kWaitLimitNs);
          if (!read) fail();
          return read;
        };
        // 64-deep blocks, the last one in steps of 16; the accumulator d starts anew at the first
        auto multiply = [&](uint32_t d, uint64_t dp, uint64_t dq, uint32_t idesc, int steps, bool more) {
          mma_pair_f16(d, dp, dq, idesc, more);
          if (steps == BT / 16) {
#pragma unroll
            for (int j = 1; j < BT / 16; ++j)
              mma_pair_f16(d, dp + j * kStep<kPMn>, dq + j * kStep<kQMn>, idesc, 1);
          } else {
            for (int j = 1; j < steps; ++j)
              mma_pair_f16(d, dp + j * kStep<kPMn>, dq + j * kStep<kQMn>, idesc, 1);
          }
        };
        if constexpr (kMode == kGrad) {
          int ps = 0;
          Slots<kQSlots> qs;
          for (int seq = 0; ok; ++seq) {
            Unit U;
            if (!take(seq, U)) break;
            release_unit(seq);
            if (U.end) break;
            if (rank != 0) continue;  // the odd CTA only follows the unit stream
            const bool join = kF32 || (kLong && U.join);
            for (int b0 = 0; ok && b0 < U.blocks; b0 += U.chunk) {
              const int b1 = min(U.blocks, b0 + U.chunk), first = ps;
              ps = (ps + b1 - b0) % kPSlots;
              for (int g = 0; ok && g < U.tiles; ++g) {
                const int a = join ? acc : acc + g;
                const bool fresh = join || b0 == 0;
                if (fresh) {
                  ok = wait_acc(a, 1u);
                  if (!ok) break;
                  tc_fence_after();
                }
                const uint32_t idesc = idesc0 | ((uint32_t)(grad_n(U.nq, g) >> 3) << 17);
                int at = first;
                for (int b = b0; b < b1; ++b) {
                  // the odd CTA's tail warp wrote zeros into its part of a block with a tail
                  const bool tail = b == U.blocks - 1 && (U.rem & 15);
                  if (tail) {
                    ok = mbar_wait_pair(bar_full + 8 * qs.at, qs.phase, abort, kWaitLimitNs);
                    if (!ok) fail();
                  } else {
                    ok = wait(bar_full + 8 * qs.at, qs.phase, kWaitLimitNs);
                  }
                  if (!ok) break;
                  tc_fence_after();
                  multiply(tmem + 256 * (a & 1), operand_desc<kPMn>(s_ring + at * kPBytes),
                           operand_desc<kQMn>(s_ring + (kPSlots + qs.at) * kPBytes), idesc,
                           b == U.blocks - 1 ? (U.rem + 15) >> 4 : BT / 16, !fresh || b != b0);
                  tc_commit_pair_mc(bar_empty + 8 * qs.at, kBoth);
                  qs.next();
                  if (++at == kPSlots) at = 0;
                }
                if (ok && (join || b1 == U.blocks)) tc_commit_pair_mc(bar_acc_full + 8 * (a & 1), kBoth);
                if (join) ++acc;
              }
            }
            if (!join && U.blocks > 0) acc += U.tiles;
          }
        } else {
          Ring<kRing> ring;
          Unit N;  // the next unit, taken while this one's last block is awaited
          bool next = take(0, N);
          for (int seq = 0; ok && next; ++seq) {
            const Unit U = N;
            release_unit(seq);
            if (U.end) break;
            if (rank != 0) {  // the odd CTA only follows the unit stream
              next = take(seq + 1, N);
              continue;
            }
            const int accs = U.n[1] ? 2 : 1;
            const uint32_t bytes = block_bytes(U.n[0], U.n[1]);
            const uint32_t idesc_a = idesc0 | ((uint32_t)(U.n[0] >> 3) << 17);
            const uint32_t idesc_b = idesc0 | ((uint32_t)(U.n[1] >> 3) << 17);
            const uint64_t to_b = U.n[0] / 2 * (BT * 2) / 16;  // from one Q tile to the other
            const int piece = kLong ? kJoinBlocks : U.blocks;  // of one sum
            for (int b0 = 0; ok && b0 < U.blocks; b0 += piece) {
              const int b1 = min(U.blocks, b0 + piece);
              for (int a = 0; a < accs && ok; ++a)
                ok = wait_acc(acc + a, 1u);
              if (!ok) break;
              tc_fence_after();
              for (int b = b0; b < b1; ++b) {
                if (b == U.blocks - 1) next = take(seq + 1, N);
                ok = wait(bar_full + 8 * ring.bar, ring.phase, kWaitLimitNs);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sp = s_ring + ring.place(bytes);
                const uint64_t dp = operand_desc<kPMn>(sp), dq = operand_desc<kQMn>(sp + kPBytes);
                const int steps = b == U.blocks - 1 ? (U.rem + 15) >> 4 : BT / 16;
                multiply(tmem + 256 * (acc & 1), dp, dq, idesc_a, steps, b != b0);
                if (accs == 2)
                  multiply(tmem + 256 * ((acc + 1) & 1), dp, dq + to_b, idesc_b, steps, b != b0);
                tc_commit_pair_mc(bar_empty + 8 * ring.bar, kBoth);
                ring.next_block();
              }
              if (!ok) break;
              for (int a = 0; a < accs; ++a, ++acc) tc_commit_pair_mc(bar_acc_full + 8 * (acc & 1), kBoth);
            }
          }
        }
        // so do the odd CTA's last releases
        if (rank == 0)
          for (int a = max(0, acc - 2); ok && a < acc; ++a)
            ok = wait_acc(a, 0u);
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
      int segment = -1;
      for (int u = cluster_id_x(); ok && u < units; u += cluster_count_x())
        ok = push(get_unit<kMode, kF32, kLong>(P, S.table, u, p_tiles, segment));
      if (ok) {
        Unit end = {};
        end.end = 1;
        push(end);
      }
    } else if (kMode == kGrad && warp == 3) {
      // -------------------------------------- rows past the segment's last
      const uint32_t lead_full = mapa_shared(bar_full, 0);
      int ps = 0, qs = 0;   // slots of the unit's first blocks
      uint32_t parity = 0;  // of each tail barrier
      bool ok = true;
      for (int seq = 0; ok; ++seq) {
        Unit U;
        if (!take_warp(seq, U)) break;
        __syncwarp();
        if (lane == 0) release_unit(seq);
        if (U.end) break;
        if (U.blocks == 0) continue;
        // a row: 8 pieces of 16 bytes in each column block
        auto zero = [&](int slot, uint32_t bytes) {
          const int first = U.rem + (lane >> 3), last = (U.rem + 15) & ~15;
          for (uint32_t block = 0; block < bytes; block += 8192) {
            uint8_t *base = smem + slot * kPBytes + block + (lane & 7) * 16;
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              if (first + i < last) *reinterpret_cast<uint4 *>(base + (first + i) * 128) = make_uint4(0, 0, 0, 0);
          }
        };
        if (U.rem & 15) {
          const int b0 = (U.blocks - 1) / U.chunk * U.chunk, n = U.blocks - b0;  // the last chunk
          for (int g = 0; g < U.tiles; ++g) {
            const int q = (qs + U.tiles * b0 + (g + 1) * n - 1) % kQSlots;
            ok = wait_warp(bar_tail + 8 * q, (parity >> q) & 1u, unit_limit);
            if (!ok) break;
            parity ^= 1u << q;
            if (g == 0) zero((ps + U.blocks - 1) % kPSlots, kPBytes);
            zero(kPSlots + q, grad_n(U.nq, g) / 2 * (BT * 2));
            // zeros before the pair's MMAs, which the even CTA issues
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead_full + 8 * q);
          }
        }
        ps = (ps + U.blocks) % kPSlots;
        qs = (qs + U.tiles * U.blocks) % kQSlots;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // A warp reads the TMEM lanes 32 * (warp % 4)..+31; the two warps of a lane quarter
    // take the 32-column groups in turn.
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t lead_acc_empty = mapa_shared(bar_acc_empty, 0);
    uint8_t *stage0_ptr = smem + kRing + (warp - 4) * stage_bytes(kMode, kF32);
    const uint32_t stage0 = smem_u32(stage0_ptr);
    // A rounded block of 32 x 32 to the gradient's q.. x p..; what passes the extents is left out.
    auto stage_out = [&](const uint32_t *w, int q, int p, int z) {
      if (elect_one()) bulk_wait_read<0>();  // the block's last copy has left it
      __syncwarp();
      stage_rows(w, stage0, lane);
      fence_async_shared();
      __syncwarp();
      if (p < P.np && elect_one()) {
        tma_store(&M.out, stage0, p, q, z);
        bulk_commit();
      }
    };
    int turn = 0;
    int acc = 0;
    bool ok = true;
    for (int seq = 0; ok; ++seq) {
      Unit U;
      if (!take_warp(seq, U)) break;
      __syncwarp();
      if (lane == 0) release_unit(seq);
      if (U.end) break;
      const int pw = U.p0 + 128 * rank + 32 * quarter;  // the warp's first p
      auto release = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_acc_empty + 8 * buf);
      };
      if constexpr (kF32) {
        const int sums = (U.blocks + kSumBlocks - 1) / kSumBlocks;
        for (int g = 0; ok && g < U.tiles; ++g) {
          const int q0 = U.q0 + BQ * g, nq = min(BQ, U.nq - BQ * g);
          // Piece i of the warp's eight: 16 q's x 32 p, through its staging blocks in turn.
          auto piece_q = [&](int i) { return 32 * (half + 2 * (i >> 1)) + 16 * (i & 1); };
          auto block = [&](int i) { return (turn + i) % kStages; };
          float sum[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
          for (int s = 0; s < sums; ++s, ++acc) {
            const int buf = acc & 1;
            if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 32 * (half + 2 * i);
              if (c < nq) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t v[16];
                  tmem_ld_x16(t_lane + 256 * buf + c + 16 * h, v);
                  tc_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) sum[i][16 * h + j] += __uint_as_float(v[j]);
                }
              }
            }
            release(buf);
          }
          // With accumulate the copy adds to the output in L2 (each value once, so in no
          // particular order): 4.95 TB/s read and written.  Loads of the output beside the
          // MMAs and stores of the sums: 774 us against 760 (16 x ~256 rows); by each lane for
          // itself, 823; stores by lane instead of copies, 620 us against 362 (binary32,
          // nothing added).  A block is written only if its copy follows: the wait counts copies.
          if (!ok || pw >= P.np) continue;
          int done = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (piece_q(i) < nq) {
              const int k = block(i);
              done = i + 1;
              float *row = reinterpret_cast<float *>(stage0_ptr + k * kStage) + lane;
              if (elect_one()) bulk_wait_read<kStages - 1>();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 16; ++j) row[32 * j] = sum[i >> 1][16 * (i & 1) + j];
              fence_async_shared();
              __syncwarp();
              if (elect_one()) {
                if (P.accumulate)
                  tma_add(&M.out, stage0 + k * kStage, pw, q0 + piece_q(i), U.z);
                else
                  tma_store(&M.out, stage0 + k * kStage, pw, q0 + piece_q(i), U.z);
                bulk_commit();
              }
            }
          }
          turn = block(done);
        }
      } else if (kLong && (kMode != kGrad || U.join)) {
        // Partial sums of one accumulator's columns, joined in the registers that load_columns
        // (gradient) or a lane's 32 columns (forward, trans) give.
        constexpr int kPart = kMode == kGrad ? 8 : 16;
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        const int sums = (U.blocks + kJoinBlocks - 1) / kJoinBlocks, nq = U.nq;
        for (int s = 0; s < sums; ++s, ++acc) {
          const int buf = acc & 1;
          if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 32 * (half + 2 * i);
            if (c < nq) {
#pragma unroll
              for (int h = 0; h < 32; h += kPart) {  // parts that leave the sums in registers
                uint32_t v[kPart];
                if constexpr (kMode == kGrad)
                  tmem_ld_16x256b_x2(t_lane + 256 * buf + c + (h & 8 ? 16 : 0) + ((uint32_t)(h & 16) << 16), v);
                else
                  tmem_ld_x16(t_lane + 256 * buf + c + h, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < kPart; ++j) sum[i][h + j] += __uint_as_float(v[j]);
              }
            }
          }
          release(buf);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 32 * (half + 2 * i);
          if (c >= nq) continue;
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[i][j]);
          if constexpr (kMode == kGrad) {
            uint32_t w[16];
            round_columns<O>(v, false, w);
            stage_out(w, U.q0 + c, pw, U.z);
          } else {
            store_columns<O>(v, static_cast<uint16_t *>(P.out) + pw + (int64_t)(U.q0 + c) * P.np, P.np,
                             nq - c, pw + lane < P.np, lane);
          }
        }
      } else if constexpr (kMode == kGrad) {
        for (int g = 0; g < U.tiles; ++g) {
          const int buf = acc & 1, q0 = U.q0 + BQ * g, nq = min(BQ, U.nq - BQ * g);
          const bool some = U.blocks > 0;  // else nothing was accumulated
          if (some) {
            if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
              ok = false;
              break;
            }
            ++acc;
            tc_fence_after();
          }
          uint32_t v[32], w[16];
          if (32 * half < nq)
            load_columns(t_lane + 256 * buf + 32 * half, v);
          else if (some)
            release(buf);
#pragma unroll 1
          for (int c = 32 * half; c < nq; c += 64) {
            tc_wait_ld();
            round_columns<O>(v, !some, w);
            if (c + 64 < nq)
              load_columns(t_lane + 256 * buf + c + 64, v);  // on their way during the stores
            else if (some)
              release(buf);
            stage_out(w, q0 + c, pw, U.z);
          }
        }
      } else {
        const int accs = U.n[1] ? 2 : 1;
        for (int a = 0; a < accs; ++a, ++acc) {
          const int buf = acc & 1;
          if (!wait_warp(bar_acc_full + 8 * buf, (uint32_t)(acc >> 1) & 1u, unit_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int q0 = a ? U.n[0] : 0, nq = a ? U.nq - U.n[0] : min(U.nq, U.n[0]);
          uint16_t *out = static_cast<uint16_t *>(P.out) + pw + (int64_t)(U.q0 + q0) * P.np;
#pragma unroll 1
          for (int c = 32 * half; c < nq; c += 64) {
            uint32_t v[32];
            MOE_TMEM_LD_32x32b_X32(t_lane + 256 * buf + c, v);
            tc_wait_ld();
            if (c + 64 >= nq) release(buf);
            store_columns<O>(v, out + (int64_t)c * P.np, P.np, nq - c, pw + lane < P.np, lane);
          }
          if (32 * half >= nq) release(buf);
        }
      }
    }
    if (kMode == kGrad && elect_one()) bulk_wait_read<0>();
  }

  tc_fence_before();
  __syncthreads();
  cluster_meet();  // the even CTA's MMAs read the odd CTA's shared memory to the end
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

// Tensor [mats][rows][cols] (cols contiguous) of 2- or 4-byte values, boxes of box_rows x
// box_cols (of `blocks` column blocks where the columns are split into blocks of 64), the
// rows of a 16-bit box swizzled by their length (128, 64 bytes).
bool make_map(CUtensorMap *m, const void *base, uint64_t mats, uint64_t rows, uint64_t cols,
              uint32_t box_rows, uint32_t box_cols, bool f32, uint32_t blocks = 0) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t size = f32 ? 4 : 2;
  cuuint64_t dims[4] = {blocks ? BT : cols, rows, blocks ? cols / BT : 1, mats};
  cuuint64_t strides[3] = {cols * size, BT * size, rows * cols * size};
  cuuint32_t box[4] = {box_cols, box_rows, blocks ? blocks : 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
            const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            f32              ? CU_TENSOR_MAP_SWIZZLE_NONE
            : box_cols == BT ? CU_TENSOR_MAP_SWIZZLE_128B
                             : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// K-major operand: boxes of 64 columns.  MN-major: 64 rows of `blocks` column blocks.
bool map_k_major(CUtensorMap *m, const void *base, uint64_t mats, uint64_t rows, uint64_t cols,
                 uint32_t box_rows) {
  return make_map(m, base, mats, rows, cols, box_rows, BT, false);
}
bool map_mn_major(CUtensorMap *m, const void *base, uint64_t mats, uint64_t rows, uint64_t cols,
                  uint32_t blocks) {
  return make_map(m, base, mats, rows, cols, BT, BT, false, cols % BT == 0 ? blocks : 0);
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
template <int kMode, class O, bool kLong = false>
int launch(const Maps &maps, const GroupedParams &P, int64_t max_units, int num_sms, void *stream) {
  static int max_clusters[kMaxDevices] = {};
  const int dev = device_slot();
  if (dev < 0) return dev;
  auto kernel = grouped_kernel<kMode, O, kLong>;
  const int sms = num_sms > 0 ? num_sms : device_sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms / 2 > 0 ? sms / 2 * 2 : 2));
  cfg.blockDim = dim3(kThreads);
  constexpr uint32_t kSmem = smem_bytes(kMode, sizeof(O) == 4);
  cfg.dynamicSmemBytes = kSmem;
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
                                         (int)kSmem);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, maps, P);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace

cudaError_t grouped_default_status(int32_t *bits, bool clear) { return take_default_status(bits, clear); }

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
  P.longest = P.bf16 ? kLongestBf16 : kLongestF16;
  P.out = a->out;
  P.p_blocked = a->k % BT == 0;
  Maps maps = {};
  const uint64_t E = a->seg.E, n = a->n, k = a->k, rows = a->seg.rows;
  bool ok = a->trans ? map_mn_major(&maps.p, a->w, E, n, k, 2) : map_k_major(&maps.p, a->w, E, n, k, 128);
  for (int i = 0; i < 8; ++i) ok = ok && map_k_major(&maps.q[i], a->x, 1, rows, P.nt, 16 * (i + 1));
  if (!ok) return MOE_ERR_CUDA;
  // row tiles: a full one per 512 rows (256), and one started in every segment that has rows
  const bool longer = P.nt > P.longest;
  const int64_t started = a->seg.E < a->seg.rows ? a->seg.E : a->seg.rows;
  const int64_t max_units = (a->seg.rows / (longer ? BQ : kWide) + started) * ((P.np + BP - 1) / BP);
  if (max_units > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  auto run = [&](auto mode, auto value) {
    constexpr int kMode = decltype(mode)::value;
    using O = decltype(value);
    return longer ? launch<kMode, O, true>(maps, P, max_units, a->num_sms, stream)
                  : launch<kMode, O>(maps, P, max_units, a->num_sms, stream);
  };
  const std::integral_constant<int, kFwd> fwd;
  const std::integral_constant<int, kTrans> trans;
  if (a->trans) return P.bf16 ? run(trans, __nv_bfloat16()) : run(trans, __half());
  return P.bf16 ? run(fwd, __nv_bfloat16()) : run(fwd, __half());
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
  P.longest = P.bf16 ? kLongestBf16 : kLongestF16;
  P.out = a->out;
  P.accumulate = a->accumulate != 0;
  P.p_blocked = a->k % BT == 0;
  P.q_blocked = a->n % BT == 0;
  // More Q tiles a unit read P less often, fewer keep the pairs even: four where each pair
  // still has 16 units and more (16 experts, 4096 x 7168, ~256 rows: 206 us in ones, 196 in
  // twos, 194 in fours, 203 in sixteens; 32 experts, 2048 x 2048: 57.9 in ones, 60.0 in threes).
  const int64_t tiles = (int64_t)a->seg.E * ((a->k + BP - 1) / BP) * ((a->n + BQ - 1) / BQ);
  const int64_t pairs = std::max(1, (a->num_sms > 0 ? a->num_sms : device_sm_count()) / 2);
  P.group = (int)std::min<int64_t>(4, std::max<int64_t>(1, tiles / (16 * pairs)));
  // without rows every segment is empty: the maps are not used, and need only be valid
  const bool f32 = a->out_type == MOE_TYPE_F32, none = a->seg.rows == 0;
  const uint64_t E = a->seg.E, n = a->n, k = a->k, rows = none ? 1 : a->seg.rows;
  Maps maps = {};
  bool ok = map_mn_major(&maps.p, none ? a->out : a->x, 1, rows, k, 2);
  for (int i = 0; i < 2; ++i) ok = ok && map_mn_major(&maps.q[i], none ? a->out : a->dy, 1, rows, n, i + 1);
  ok = ok && make_map(&maps.out, a->out, E, n, k, f32 ? 16 : 32, 32, f32);
  if (!ok) return MOE_ERR_CUDA;
  const int64_t max_units = tiles;
  if (max_units > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (f32)
    return launch<kGrad, float>(maps, P, max_units, a->num_sms, stream);
  if (a->seg.rows > P.longest)  // some segment may be
    return P.bf16 ? launch<kGrad, __nv_bfloat16, true>(maps, P, max_units, a->num_sms, stream)
                  : launch<kGrad, __half, true>(maps, P, max_units, a->num_sms, stream);
  return P.bf16 ? launch<kGrad, __nv_bfloat16>(maps, P, max_units, a->num_sms, stream)
                : launch<kGrad, __half>(maps, P, max_units, a->num_sms, stream);
}
