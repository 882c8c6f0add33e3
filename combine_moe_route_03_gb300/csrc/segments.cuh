// The ragged segments of moe_segments on the device: every kernel that walks them builds
// the same small table in shared memory from the counts.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxSegments = 1024;

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

// Inclusive scan over a warp.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Fills start and count, and before with the exclusive sums of weight(count).  All
// threads of the block call it (a multiple of 32, at least 32); `part` is scratch of
// 2 x 32 entries.  Scans run in 64 bits: counts are the caller's and may be anything.
// The weights are first summed for the counts as they are, together with the starts; only
// if a count is found wrong (negative, above cap, or past the buffer) are they summed again
// for what is left of it.
template <class Weight>
__device__ void build_segments(const SegParams &P, SegTable &T, long long *part, Weight weight,
                               bool report) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (P.E + 31) >> 5;
  long long *part_size = part, *part_weight = part + 32;
  for (int c = warp; c < chunks; c += warps) {
    const int e = 32 * c + lane;
    const int n = e < P.E ? P.counts[e] : 0;
    const int kept = min(max(n, 0), P.rows);  // weight() takes counts of the buffer
    const long long size = e < P.E ? ((long long)max(n, 0) + P.align - 1) / P.align * P.align : 0;
    const long long w = e < P.E ? weight(kept) : 0;
    const long long s = warp_scan(size, lane), sw = warp_scan(w, lane);
    if (lane == 31) part_size[c] = s, part_weight[c] = sw;
    if (e < P.E) {
      T.count[e] = n;
      T.start[e] = (int)min(s - size, (long long)INT32_MAX);  // passes the buffer: cut below
      T.before[e] = (int)(sw - w);
    }
  }
  __syncthreads();
  const long long size = lane < chunks ? part_size[lane] : 0, w = lane < chunks ? part_weight[lane] : 0;
  const long long sizes = warp_scan(size, lane), weights = warp_scan(w, lane);
  int bad = 0;
  for (int c = warp; c < chunks; c += warps) {
    const int e = 32 * c + lane;
    const long long base = __shfl_sync(0xffffffffu, sizes - size, c);
    const int base_w = (int)__shfl_sync(0xffffffffu, weights - w, c);
    if (e >= P.E) continue;
    const int n = T.count[e];
    const long long first = P.cap > 0 ? (long long)e * P.cap : T.start[e] + base;
    long long kept = max(n, 0);
    if (P.cap > 0) kept = min(kept, (long long)P.cap);
    kept = max(0ll, min(kept, P.rows - first));
    if (n < 0) bad |= MOE_STATUS_BAD_INDEX;
    if (kept < n) bad |= MOE_STATUS_CAPACITY;
    T.start[e] = (int)min(first, (long long)P.rows);
    T.count[e] = (int)kept;
    T.before[e] += base_w;
  }
  const int total = (int)__shfl_sync(0xffffffffu, weights, 31);
  if (threadIdx.x == 0) T.before[P.E] = total;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      long long sum = 0;
      for (int e = 0; e < P.E; ++e) {
        T.before[e] = (int)sum;
        sum += weight(T.count[e]);
      }
      T.before[P.E] = (int)sum;
    }
    __syncthreads();
  }
  if (report && bad) status_or(P.status, bad);
}

// The segment that holds item i of the `before` sums: the last e with before[e] <= i.
__device__ __forceinline__ int find_segment(const SegTable &T, int E, int i) {
  int lo = 0, hi = E;  // before[lo] <= i < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (T.before[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace moe
