// What the kernels of 16-bit products share: PTX of the CTA pair's copies, MMAs and barriers,
// operand descriptors, and the host's tensor maps.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int BT = 64;  // depth of a block of the sum: 128 bytes of a row

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
// Arrive on an mbarrier of either CTA of the pair where no writes of this CTA's threads have
// to be ordered: operands land by TMA, and reads of an accumulator are ordered by the tcgen05
// fences before the arrival and after the (cluster-wide, relaxed) wait.  A release would first
// wait for the warp's global stores.  Writes take mbar_arrive_pair.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
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
// Operand descriptors without their address, and what 16 t's add to it: K-major rows of
// 128 bytes (32 bytes a step), or MN-major blocks of 64 columns, 128 bytes per t (16 t's a
// step; column blocks 8 KB apart).  Addresses count 16 bytes;
// above their 18 bits a CTA's own shared addresses hold its rank in the cluster.
template <bool kMnMajor>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (kMnMajor ? smem_desc(0, BT * 128, 1024, 2) : smem_desc(0, 16, 1024, 2)) + ((addr & 0x3ffffu) >> 4);
}
template <bool kMnMajor>
constexpr uint64_t kStep = kMnMajor ? 2048 / 16 : 32 / 16;

template <class O>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
  uint32_t r;
  if constexpr (std::is_same<O, __half>::value)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return r;
}

// ----------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> known{nullptr};  // threads may ask at once
  EncodeTiledFn fn = known.load();
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      known.store(fn = reinterpret_cast<EncodeTiledFn>(p));
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

bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }

}  // namespace
}  // namespace moe
