// The ragged segments of moe_segments on the device: every kernel that walks them builds
// the same small table in shared memory from the counts.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxSegments = 1024;

// What a call without a status word finds wrong goes into a word of the library: one for the
// kernels of each source file, read by moe_read_default_status.
namespace {
__device__ int32_t default_status;
}
__device__ __forceinline__ void segments_status(int32_t *status, int bits) {
  status_or(status ? status : &default_status, bits);
}
// Bits of this source file's word; `clear`: and zero in it.
static inline cudaError_t take_default_status(int32_t *bits, bool clear) {
  const cudaError_t e = cudaMemcpyFromSymbol(bits, default_status, sizeof *bits);
  if (e != cudaSuccess || !clear || *bits == 0) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(default_status, &zero, sizeof zero);
}

// Host-side check of a segment description (counts may be NULL where `all_rows`).
inline int check_segments(const moe_segments &s, bool all_rows) {
  if (s.rows < 0) return MOE_ERR_INVALID;
  if (s.rows > INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (all_rows && !s.counts) return MOE_OK;
  if (!s.counts || s.E < 1 || s.align < 1 || s.cap < 0) return MOE_ERR_INVALID;
  if (s.E > kMaxSegments) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What the kernels take.
struct SegParams {
  const int32_t *counts;
  int E, align, cap, rows;
  int32_t *status;
};
inline SegParams seg_params(const moe_segments &s, int32_t *status) {
  return SegParams{s.counts, s.E, s.align, s.cap, (int)s.rows, status};
}

struct SegTable {
  int start[kMaxSegments];      // first row
  int count[kMaxSegments];      // rows, cut to the buffer
  int before[kMaxSegments + 1]; // rows (or units) of the segments before this one
};

// Inclusive sums over a warp, held at INT32_MAX: counts are the caller's and may be
// anything, and a sum that large lies past every buffer.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = (int)min((unsigned)v + (unsigned)o, (unsigned)INT32_MAX);
  }
  return v;
}

// The sum before this lane's, of an inclusive scan (held sums cannot be subtracted).
__device__ __forceinline__ int before_lane(int s, int lane) {
  const int o = __shfl_up_sync(0xffffffffu, s, 1);
  return lane ? o : 0;
}

// Fills start and count, and before with the exclusive sums of weight(count).  All
// threads of the block call it (a multiple of 32, at least 32); `part` is scratch of
// 2 x 32 entries.  The weights are first summed for the counts as they are, together with
// the starts; only if a count is found wrong (negative, above cap, or past the buffer) are
// they summed again for what is left of it.
template <class Weight>
__device__ void build_segments(const SegParams &P, SegTable &T, int *part, Weight weight,
                               bool report) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (P.E + 31) >> 5;
  auto size_of = [&](int n) {  // rows of the segment with its padding
    if (P.align == 1) return n;
    const long long s = ((long long)n + P.align - 1) / P.align * P.align;
    return (int)min(s, (long long)INT32_MAX);
  };
  int bad = 0;
  // One entry: its first row is known; counts what is kept of it.
  auto settle = [&](int e, int n, int start) {
    const long long first = P.cap > 0 ? (long long)e * P.cap : start;
    long long kept = max(n, 0);
    if (P.cap > 0) kept = min(kept, (long long)P.cap);
    kept = max(0ll, min(kept, P.rows - first));
    if (n < 0) bad |= MOE_STATUS_BAD_INDEX;
    if (kept < n) bad |= MOE_STATUS_CAPACITY;
    T.start[e] = (int)min(first, (long long)P.rows);
    T.count[e] = (int)kept;
  };
  for (int c = warp; c < chunks; c += warps) {
    const int e = 32 * c + lane;
    const int n = e < P.E ? P.counts[e] : 0;
    const int size = size_of(max(n, 0));
    const int w = e < P.E ? weight(min(max(n, 0), P.rows)) : 0;
    const int s = warp_scan(size, lane), sw = warp_scan(w, lane), start = before_lane(s, lane);
    if (e < P.E) {
      T.before[e] = sw - w;
      if (chunks == 1) {
        settle(e, n, start);
      } else {
        T.count[e] = n;
        T.start[e] = start;
      }
    }
    if (lane == 31) {
      part[c] = s, part[32 + c] = sw;
      if (chunks == 1) T.before[P.E] = sw;
    }
  }
  if (chunks > 1) {
    __syncthreads();
    const int size = lane < chunks ? part[lane] : 0, w = lane < chunks ? part[32 + lane] : 0;
    const int sizes = before_lane(warp_scan(size, lane), lane), weights = warp_scan(w, lane);
    const int total = __shfl_sync(0xffffffffu, weights, 31);
    for (int c = warp; c < chunks; c += warps) {
      const int e = 32 * c + lane;
      const int base = __shfl_sync(0xffffffffu, sizes, c);
      const int base_w = __shfl_sync(0xffffffffu, weights - w, c);
      if (e >= P.E) continue;
      settle(e, T.count[e], (int)min((unsigned)T.start[e] + (unsigned)base, (unsigned)INT32_MAX));
      T.before[e] += base_w;
    }
    if (threadIdx.x == 0) T.before[P.E] = total;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      int sum = 0;
      for (int e = 0; e < P.E; ++e) {
        T.before[e] = sum;
        sum += weight(T.count[e]);
      }
      T.before[P.E] = sum;
    }
    __syncthreads();
  }
  if (report && bad) segments_status(P.status, bad);
}

// The segment that holds item i where each of the `before` sums counts `scale` items: the
// last e with before[e] * scale <= i.
__device__ __forceinline__ int find_segment(const SegTable &T, int E, int i, int scale = 1) {
  int lo = 0, hi = E;  // before[lo] * scale <= i < before[hi] * scale
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (T.before[mid] * scale <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace moe
