// The pages of a paged cache: requests forked, pages freed and moved together, and the copies of
// pages that forks and moves ask for.  The tables are everything there is to keep: how often a page
// is used and which are free is counted from the block tables and lengths at every call, so that
// nothing else can get out of step with them.
//
//  * fork: a new request takes over the entries of the pages that its source has filled, and for
//    the page that it has not a page from the front of the free list, in the order of the pairs:
//    entry sum_{j < i} [pair j takes one].  Every block forms that sum itself, then takes its share
//    of the rows.
//  * free: the entries of the requests that are done become -1 and their lengths 0; refs[p] counts
//    the entries that the requests left have of page p, and the pages without one are listed in
//    ascending order.
//  * compact: with U pages in use, the pages in use at or behind U, ascending, go to the pages free
//    before U, ascending; the tables follow.  No page is both source and destination, so that the
//    copies can run in any order.
//  * copy: pages, or their first rows, from page to page, bound by HBM.
//
// Free and compact need the whole count before the first rank and the whole renumbering before the
// first entry: one cluster does all of it, its barrier (some 0.3 us) in place of further launches.
// Latency bounds all three.  Measured: a fork of 3 requests 4 us, of 240 of up to 8192 tokens with the
// copy of their last pages 31; freeing 16 of 64 requests of 4096 tokens in pages of 64 10 us, the
// compaction after it 14, the copies of the pages that it moves (1 GB read and written in all) at 6.5
// TB/s, 0.96 of a plain copy's rate.  Every kernel launches as a dependent kernel (it waits for the
// previous kernel in the stream before touching global memory).
#include <limits.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kForkThreads = 256;
constexpr int kForkWarps = kForkThreads / 32;
constexpr int kCluster = 8;
constexpr int kPageThreads = 512;
constexpr int kWarps = kPageThreads / 32;
constexpr int kSweep = 8;                       // ballots of a warp and turn
constexpr int kSegment = 256;                   // table entries of a warp's unit of work
constexpr int kMaxRows = 8192;

__device__ __forceinline__ int clamped(int len, int cap) { return min(max(len, 0), cap); }

// ------------------------------------------------------------------ fork

struct ForkArgs {
  int32_t* cache_len;
  int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* free_pages;
  int n_free;
  const int32_t *src, *dst;
  int n;
  int32_t *copy_src, *copy_dst, *copy_rows, *pages_taken;
  int B, shift, num_pages;
};

__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkArgs a) {
  extern __shared__ int sh[];
  int* first = sh;              // [B] the first pair that names the row as its destination
  int* list = sh + a.B;         // [n] the pair's place in the free list, -1: none, -2: skipped
  int* warp_sum = list + a.n;   // [kForkWarps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = a.max_pages << a.shift, round = (1 << a.shift) - 1;
  for (int b = tid; b < a.B; b += kForkThreads) first[b] = INT_MAX;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  auto named = [&](int i, int* s, int* t) {
    *s = a.src[i];
    *t = a.dst[i];
    return *s >= 0 && *s < a.B && *t >= 0 && *t < a.B;
  };
  for (int i = tid; i < a.n; i += kForkThreads) {
    int s, t;
    if (named(i, &s, &t)) atomicMin(first + t, i);
  }
  __syncthreads();
  const int per = (a.n + kForkThreads - 1) / kForkThreads;
  const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    int s, t, kind = -2;
    if (named(i, &s, &t) && first[t] == i && first[s] == INT_MAX) {
      kind = -1;
      const int L = clamped(a.cache_len[s], cap);
      if (L & round) {
        const int p = a.table[s * a.table_stride + (L >> a.shift)];
        if (p >= 0 && p < a.num_pages) kind = sum++;
      }
    }
    list[i] = kind;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  for (int i = i0; i < i1; ++i)
    if (list[i] >= 0) list[i] += before;
  if (blockIdx.x == 0 && tid == kForkThreads - 1) *a.pages_taken = before + sum;
  __syncthreads();
  // A source is nobody's destination, so that no row read here is written.
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int e = list[i];
    if (e == -2) {
      if (tid == 0) a.copy_src[i] = a.copy_dst[i] = -1, a.copy_rows[i] = 0;
      continue;
    }
    const int s = a.src[i], t = a.dst[i];
    const int L = clamped(a.cache_len[s], cap), full = L >> a.shift;
    const int32_t* from = a.table + s * a.table_stride;
    int32_t* to = a.table + t * a.table_stride;
    for (int c = tid; c < full; c += kForkThreads) to[c] = from[c];
    if (tid == 0) {
      const int page = e >= 0 && e < a.n_free ? a.free_pages[e] : -1;
      const bool moved = page >= 0 && page < a.num_pages;
      if (L & round) to[full] = page;
      a.copy_src[i] = moved ? from[full] : -1;
      a.copy_dst[i] = moved ? page : -1;
      a.copy_rows[i] = moved ? L & round : 0;
      a.cache_len[t] = L;
    }
  }
}

// ------------------------------------------------------------------ free and compact

struct PagesArgs {
  int32_t* cache_len;
  int32_t* table;
  long long table_stride;
  int max_pages;
  int B, shift, num_pages;
};

// Every thread of the cluster; what was written before it, to global and to shared memory, is seen
// behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// `value` to the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void cluster_store(int* place, int rank, int value) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(ptx::smem_u32(place)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(value) : "memory");
}

struct Sweep {
  int warp_sum[kWarps];
  int sums[4][kCluster];        // every CTA's count, one row an exchange
};

// Pages of [c0, c1) for which pred holds, counted by the block.
template <class Pred>
__device__ __forceinline__ int count_pages(Sweep* w, int c0, int c1, Pred pred) {
  int n = 0;
  for (int p = c0 + threadIdx.x; p < c1; p += kPageThreads) n += pred(p) ? 1 : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) w->warp_sum[threadIdx.x >> 5] = n;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) all += w->warp_sum[i];
  return all;
}

// The block's count to every CTA of the cluster; seen after cluster_sync().
__device__ __forceinline__ void tell(Sweep* w, int row, int rank, int n) {
  if (threadIdx.x < kCluster) cluster_store(&w->sums[row][rank], threadIdx.x, n);
}
// Counts of the CTAs before this one, and of all.
__device__ __forceinline__ int2 told(const Sweep* w, int row, int rank) {
  int2 r = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kCluster; ++i) {
    if (i < rank) r.x += w->sums[row][i];
    r.y += w->sums[row][i];
  }
  return r;
}

// put(page, rank) for the pages of [c0, c1) for which pred holds, in ascending order, ranks from
// `base`: a warp has 256 neighbouring pages a turn and finds the ranks from its ballots.
template <class Pred, class Put>
__device__ __forceinline__ void rank_pages(Sweep* w, int c0, int c1, int base, Pred pred, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t below = (1u << lane) - 1u;
  for (int t = c0; t < c1; t += 32 * kSweep * kWarps) {
    const int p0 = t + warp * 32 * kSweep + lane;
    uint32_t hit[kSweep];
    int n = 0;
#pragma unroll
    for (int j = 0; j < kSweep; ++j) {
      const int p = p0 + 32 * j;
      hit[j] = __ballot_sync(0xffffffffu, p < c1 && pred(p));
      n += __popc(hit[j]);
    }
    __syncthreads();
    if (lane == 0) w->warp_sum[warp] = n;
    __syncthreads();
    int at = base;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int x = w->warp_sum[i];
      if (i < warp) at += x;
      base += x;
    }
#pragma unroll
    for (int j = 0; j < kSweep; ++j) {
      if (hit[j] >> lane & 1u) put(p0 + 32 * j, at + __popc(hit[j] & below));
      at += __popc(hit[j]);
    }
  }
}

// use(row, column, entry's address) for every table entry of a request's pages; the warps of the
// cluster take segments of rows in turn.  gone(b): the row is not read but cleared.
template <class Gone, class Use>
__device__ __forceinline__ void each_entry(const PagesArgs& a, int rank, Gone gone, Use use) {
  const int lane = threadIdx.x & 31;
  const int cap = a.max_pages << a.shift, round = (1 << a.shift) - 1;
  const int segs = (a.max_pages + kSegment - 1) / kSegment;
  for (int u = rank * kWarps + (threadIdx.x >> 5); u < a.B * segs; u += kCluster * kWarps) {
    const int b = u / segs, c0 = (u - b * segs) * kSegment;
    int32_t* row = a.table + b * a.table_stride;
    if (gone(b)) {
      const int c1 = min(a.max_pages, c0 + kSegment);
      for (int c = c0 + lane; c < c1; c += 32) row[c] = -1;
      if (c0 == 0 && lane == 0) a.cache_len[b] = 0;
      continue;
    }
    const int n = (clamped(a.cache_len[b], cap) + round) >> a.shift;
    const int c1 = min(n, c0 + kSegment);
#pragma unroll 4
    for (int c = c0 + lane; c < c1; c += 32) use(row + c);
  }
}

__global__ void __launch_bounds__(kPageThreads)
free_kernel(PagesArgs a, const int32_t* rows, int n, int32_t* refs, int32_t* free_pages,
            int32_t* n_free) {
  __shared__ Sweep w;
  __shared__ uint32_t gone[kMaxRows / 32];
  const int tid = threadIdx.x, rank = cluster_rank(), P = a.num_pages;
  const int c0 = static_cast<int>(static_cast<long long>(P) * rank / kCluster);
  const int c1 = static_cast<int>(static_cast<long long>(P) * (rank + 1) / kCluster);
  for (int i = tid; i < kMaxRows / 32; i += kPageThreads) gone[i] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  for (int i = tid; i < n; i += kPageThreads) {
    const int b = rows[i];
    if (b >= 0 && b < a.B) atomicOr(gone + (b >> 5), 1u << (b & 31));
  }
  for (int p = c0 + tid; p < c1; p += kPageThreads) refs[p] = 0;
  cluster_sync();
  each_entry(a, rank, [&](int b) { return (gone[b >> 5] >> (b & 31) & 1u) != 0; },
             [&](int32_t* e) {
               const int p = *e;
               if (p >= 0 && p < P) atomicAdd(refs + p, 1);
             });
  cluster_sync();
  auto free_page = [&](int p) { return __ldcg(refs + p) == 0; };
  tell(&w, 0, rank, count_pages(&w, c0, c1, free_page));
  cluster_sync();
  const int2 f = told(&w, 0, rank);
  rank_pages(&w, c0, c1, f.x, free_page, [&](int p, int r) { free_pages[r] = p; });
  for (int i = f.y + rank * kPageThreads + tid; i < P; i += kCluster * kPageThreads)
    free_pages[i] = -1;
  if (rank == 0 && tid == 0) *n_free = f.y;
}

__global__ void __launch_bounds__(kPageThreads)
compact_kernel(PagesArgs a, int32_t* moved, int32_t* copy_src, int32_t* copy_dst, int n_copies,
               int32_t* n_used) {
  __shared__ Sweep w;
  const int tid = threadIdx.x, rank = cluster_rank(), P = a.num_pages;
  const int c0 = static_cast<int>(static_cast<long long>(P) * rank / kCluster);
  const int c1 = static_cast<int>(static_cast<long long>(P) * (rank + 1) / kCluster);
  auto none = [](int) { return false; };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  for (int p = c0 + tid; p < c1; p += kPageThreads) moved[p] = 0;
  cluster_sync();
  each_entry(a, rank, none, [&](int32_t* e) {
    const int p = *e;
    if (p >= 0 && p < P) moved[p] = 1;       // in use; the same value from everybody
  });
  cluster_sync();
  tell(&w, 0, rank, count_pages(&w, c0, c1, [&](int p) { return __ldcg(moved + p) != 0; }));
  cluster_sync();
  const int U = told(&w, 0, rank).y;
  auto place = [&](int p) { return p < U && __ldcg(moved + p) == 0; };    // free, to be filled
  auto mover = [&](int p) { return p >= U && __ldcg(moved + p) == 1; };
  tell(&w, 1, rank, count_pages(&w, c0, c1, place));
  tell(&w, 2, rank, count_pages(&w, c0, c1, mover));
  cluster_sync();
  const int2 lo = told(&w, 1, rank), hi = told(&w, 2, rank);              // lo.y = hi.y
  rank_pages(&w, c0, c1, lo.x, place, [&](int p, int r) {
    if (r < n_copies) copy_dst[r] = p;
  });
  rank_pages(&w, c0, c1, hi.x, mover, [&](int p, int r) {
    if (r < n_copies) copy_src[r] = p;
    moved[p] = -2 - r;                       // its place is entry r of copy_dst
  });
  for (int i = hi.y + rank * kPageThreads + tid; i < n_copies; i += kCluster * kPageThreads)
    copy_src[i] = copy_dst[i] = -1;
  if (rank == 0 && tid == 0) *n_used = U;
  __syncthreads();
  for (int p = c0 + tid; p < c1; p += kPageThreads) {
    const int v = __ldcg(moved + p);
    if (v == 0) moved[p] = -1;
    else if (v == 1) moved[p] = p;
  }
  cluster_sync();
  // While the movers' places are written the entries follow: either form of moved says the same.
  auto where = [&](int v) { return v < -1 ? __ldcg(copy_dst + (-2 - v)) : v; };
  for (int p = max(c0, U) + tid; p < c1; p += kPageThreads) {
    const int v = __ldcg(moved + p);
    if (v < -1) moved[p] = where(v);
  }
  each_entry(a, rank, none, [&](int32_t* e) {
    const int p = *e;
    if (p >= U && p < P) *e = where(__ldcg(moved + p));
  });
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kPageThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ------------------------------------------------------------------ copies of pages

constexpr int kCopyThreads = 256;
constexpr int kPiece = 4 * kCopyThreads;     // 16-byte units of a page that a block copies at once

struct CopyArgs {
  uint4* pool[2];                 // the second may be null
  long long page_stride;          // 16-byte units
  int page_units, row_units, shift;
  const int32_t *src, *dst, *rows;
  int n, num_pages, pieces;
};

template <int POOLS>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const long long total = static_cast<long long>(a.n) * a.pieces;
  const int page = 1 << a.shift;
  // Lane i finds out about the block's i-th next piece.
  for (long long base = blockIdx.x; base < total; base += 32ll * gridDim.x) {
    const long long u = base + static_cast<long long>(lane) * gridDim.x;
    int s = -1, t = -1, first = 0, rows = page;
    if (u < total) {
      const int e = static_cast<int>(u / a.pieces);
      first = static_cast<int>(u - static_cast<long long>(e) * a.pieces) * kPiece;
      s = a.src[e];
      t = a.dst[e];
      if (a.rows) rows = min(max(a.rows[e], 0), page);
    }
    const bool ok = s >= 0 && s < a.num_pages && t >= 0 && t < a.num_pages && s != t && rows > 0;
    uint32_t todo = __ballot_sync(0xffffffffu, ok);
    while (todo) {
      const int j = __ffs(todo) - 1;
      todo &= todo - 1;
      const int js = __shfl_sync(0xffffffffu, s, j), jt = __shfl_sync(0xffffffffu, t, j);
      const int jf = __shfl_sync(0xffffffffu, first, j), jr = __shfl_sync(0xffffffffu, rows, j);
      uint4 x[POOLS][4];
      bool live[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = jf + i * kCopyThreads + tid;
        live[i] = at < a.page_units && (jr == page || ((at / a.row_units) & (page - 1)) < jr);
#pragma unroll
        for (int p = 0; p < POOLS; ++p)
          if (live[i]) x[p][i] = a.pool[p][js * a.page_stride + at];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = jf + i * kCopyThreads + tid;
#pragma unroll
        for (int p = 0; p < POOLS; ++p)
          if (live[i]) a.pool[p][jt * a.page_stride + at] = x[p][i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_fork(int32_t* cache_len, int32_t* table, long long table_stride,
                              int max_pages, const int32_t* free_pages, int n_free,
                              const int32_t* src, const int32_t* dst, int n, int32_t* copy_src,
                              int32_t* copy_dst, int32_t* copy_rows, int32_t* pages_taken, int B,
                              int page_shift, int num_pages, cudaStream_t s) {
  ForkArgs a{cache_len, table, table_stride, max_pages, free_pages, n_free, src, dst, n, copy_src,
             copy_dst, copy_rows, pages_taken, B, page_shift, num_pages};
  // All of the kernel's shared memory: what is declared in it would count beside this.
  const size_t smem = sizeof(int) * (static_cast<size_t>(B) + n + kForkWarps);
  if (smem > 48 * 1024) {       // to the most that a call takes: calls at once set the same
    cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (2 * kMaxRows + kForkWarps) *
                                             static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  const int blocks = n < 1 ? 1 : n < 2 * sm_count() ? n : 2 * sm_count();
  return launch_dependent(fork_kernel, dim3(blocks), dim3(kForkThreads), smem, s, a);
}

cudaError_t launch_paged_free(int32_t* cache_len, int32_t* table, long long table_stride,
                              int max_pages, const int32_t* rows, int n, int32_t* refs,
                              int32_t* free_pages, int32_t* n_free, int B, int page_shift,
                              int num_pages, cudaStream_t s) {
  const PagesArgs a{cache_len, table, table_stride, max_pages, B, page_shift, num_pages};
  return launch_cluster(free_kernel, s, a, rows, n, refs, free_pages, n_free);
}

cudaError_t launch_paged_compact(const int32_t* cache_len, int32_t* table, long long table_stride,
                                 int max_pages, int32_t* moved, int32_t* copy_src,
                                 int32_t* copy_dst, int n_copies, int32_t* n_used, int B,
                                 int page_shift, int num_pages, cudaStream_t s) {
  const PagesArgs a{const_cast<int32_t*>(cache_len), table, table_stride, max_pages, B, page_shift,
                    num_pages};   // only free_kernel writes the lengths
  return launch_cluster(compact_kernel, s, a, moved, copy_src, copy_dst, n_copies, n_used);
}

cudaError_t launch_paged_copy(void* k_cache, void* v_cache, long long page_stride,
                              const int32_t* src, const int32_t* dst, const int32_t* rows, int n,
                              int num_pages, int heads, int page_shift, int d, cudaStream_t s) {
  const int units = (heads << page_shift) * (d / 8);
  CopyArgs a{{static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache)}, page_stride / 8, units,
             d / 8, page_shift, src, dst, rows, n, num_pages, (units + kPiece - 1) / kPiece};
  const long long total = static_cast<long long>(n) * a.pieces, most = 8ll * sm_count();
  const dim3 grid(static_cast<unsigned>(total < most ? total : most));
  return v_cache ? launch_dependent(copy_kernel<2>, grid, dim3(kCopyThreads), 0, s, a)
                 : launch_dependent(copy_kernel<1>, grid, dim3(kCopyThreads), 0, s, a);
}

}  // namespace fa
