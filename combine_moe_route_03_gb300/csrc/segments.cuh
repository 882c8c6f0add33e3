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
// 33 entries.  Scans run in 64 bits: counts are the caller's and may be anything.
template <class Weight>
__device__ void build_segments(const SegParams &P, SegTable &T, long long *part, Weight weight,
                               bool report) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (P.E + 31) >> 5;
  int bad = 0;
  for (int pass = 0; pass < 2; ++pass) {  // 0: rows before each segment; 1: weights
    for (int c = warp; c < chunks; c += warps) {
      const int e = 32 * c + lane;
      long long v = 0;
      if (e < P.E) {
        if (pass == 0) {
          int n = P.counts[e];
          if (n < 0) {
            bad |= MOE_STATUS_BAD_INDEX;
            n = 0;
          }
          T.count[e] = n;
          v = ((long long)n + P.align - 1) / P.align * P.align;
        } else {
          v = weight(T.count[e]);
        }
      }
      const long long s = warp_scan(v, lane);
      if (lane == 31) part[c] = s;
      if (e < P.E) {
        if (pass == 0)  // kept as a 31-bit value: what passes the buffer is cut there
          T.start[e] = (int)min(s - v, (long long)INT32_MAX);
        else
          T.before[e] = (int)(s - v);
      }
    }
    __syncthreads();
    if (warp == 0) {
      const long long v = lane < chunks ? part[lane] : 0;
      const long long s = warp_scan(v, lane);
      part[lane] = s - v;
      if (lane == 31) part[32] = s;
    }
    __syncthreads();
    for (int c = warp; c < chunks; c += warps) {
      const int e = 32 * c + lane;
      if (e >= P.E) continue;
      if (pass == 0) {
        const long long first = P.cap > 0 ? (long long)e * P.cap : T.start[e] + part[c];
        const int want = T.count[e];
        long long n = P.cap > 0 ? min(want, P.cap) : want;
        n = max(0ll, min(n, P.rows - first));
        if (n < want) bad |= MOE_STATUS_CAPACITY;
        T.start[e] = (int)min(first, (long long)P.rows);
        T.count[e] = (int)n;
      } else {
        T.before[e] += (int)part[c];
      }
    }
    if (pass == 1 && threadIdx.x == 0) T.before[P.E] = (int)part[32];
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
