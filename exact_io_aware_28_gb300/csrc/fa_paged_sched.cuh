// How the decode kernels over a paged cache share out the work.
//
// Sequence b has ceil(L_b / KEYS) granules of KEYS keys for each of its `heads` key/value
// heads; all granules lie on one line (sequence by sequence, head by head) and worker w of W
// takes the granules [total w / W, total (w + 1) / W), W being the smaller of the grid's workers
// and the granules, so that no range is empty.  Every worker so gets the same share
// whatever the lengths are, and a (sequence, head) pair is cut only where a worker's range
// ends.  A segment is the part of one pair that lies in one worker's range; a worker has at
// most two segments that are not whole pairs, its first and its last, so the partial results
// need two slots a worker, however many sequences there are.  The cut depends on the lengths
// and on W alone: the same call gives the same bits.
#pragma once

#include "fa_internal.cuh"

namespace fa {
namespace sched {

__device__ __forceinline__ int clamp_len(const int32_t* cache_len, int b, int cap) {
  const int L = cache_len[b];
  return L < 0 ? 0 : (L > cap ? cap : L);
}

template <int KEYS>
__device__ __forceinline__ int granules(int L) {
  return (L + KEYS - 1) / KEYS;
}

// W: the workers that have a range.
__device__ __forceinline__ int active(long long total, int workers) {
  return total < workers ? static_cast<int>(total) : workers;
}

// First granule of worker w (of W, as below).
__device__ __forceinline__ long long range_start(long long total, int w, int workers) {
  return total * w / workers;
}

// The worker whose range holds granule x (total > 0).
__device__ __forceinline__ int owner(long long x, long long total, int workers) {
  return static_cast<int>(((x + 1) * workers - 1) / total);
}

// Slot of the partial result of the segment of a pair, first granule `pair_start`, in worker
// w's range: the second of the worker's two when the pair starts inside the range.
__device__ __forceinline__ int slot(long long pair_start, long long range_start_w, int w) {
  return 2 * w + (pair_start > range_start_w ? 1 : 0);
}

struct Start {
  long long first, last;  // the worker's range of granules
  int b;                  // the sequence the first granule belongs to
  long long before;       // granules of the sequences before b
};

// The worker's range and where it begins; called by all THREADS threads of the block.  With
// `prefix` (one block of the grid) the exclusive sums over the sequences, B + 1 of them, are
// written there for the combine kernel.  scratch: shared, THREADS / 32 + 1 long longs.
template <int KEYS, int THREADS>
__device__ __forceinline__ void find_start(Start* out, long long* scratch,
                                           const int32_t* cache_len, int B, int heads, int cap,
                                           int w, int workers, long long* prefix) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long sum = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b)
    sum += static_cast<long long>(granules<KEYS>(clamp_len(cache_len, b, cap))) * heads;
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long before = incl - sum, total = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    const long long v = scratch[i];
    if (i < warp) before += v;
    total += v;
  }
  const int W = active(total, workers);
  const long long first = w < W ? range_start(total, w, W) : total;
  if (tid == 0) {
    out->first = first;
    out->last = w < W ? range_start(total, w + 1, W) : total;
    out->b = 0;
    out->before = 0;
  }
  __syncthreads();
  const bool mine = first >= before && first < before + sum;
  if (mine || prefix) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long n =
          static_cast<long long>(granules<KEYS>(clamp_len(cache_len, b, cap))) * heads;
      if (prefix) prefix[b] = at;
      if (mine && first >= at && first < at + n) {
        out->b = b;
        out->before = at;
      }
      at += n;
    }
  }
  if (prefix && tid == 0) prefix[B] = total;
  __syncthreads();
}

// One segment: keys [k0, k1) of pair (b, head).
struct Segment {
  int b, head;
  int k0, k1;
  int len;                 // the sequence's length
  bool whole;              // the segment is the whole pair
  long long pair_start;    // first granule of the pair
};

// Walks a worker's segments in order; every warp role runs its own copy.
template <int KEYS>
struct Walk {
  const int32_t* cache_len;
  int heads, cap, b;
  long long at, last, before;

  __device__ __forceinline__ Walk(const Start& s, const int32_t* cl, int heads_, int cap_)
      : cache_len(cl), heads(heads_), cap(cap_), b(s.b), at(s.first), last(s.last),
        before(s.before) {}

  __device__ __forceinline__ bool next(Segment& sg) {
    if (at >= last) return false;
    for (;;) {
      const int L = clamp_len(cache_len, b, cap);
      const int n = granules<KEYS>(L);
      const long long all = static_cast<long long>(n) * heads;
      if (at < before + all) {
        sg.b = b;
        sg.head = static_cast<int>((at - before) / n);
        sg.len = L;
        sg.pair_start = before + static_cast<long long>(sg.head) * n;
        const int g0 = static_cast<int>(at - sg.pair_start);
        const int g1 = static_cast<int>(min(static_cast<long long>(n), last - sg.pair_start));
        sg.k0 = g0 * KEYS;
        sg.k1 = min(g1 * KEYS, L);
        sg.whole = g0 == 0 && g1 == n;
        at = sg.pair_start + g1;
        return true;
      }
      before += all;
      ++b;
    }
  }
};

}  // namespace sched
}  // namespace fa
