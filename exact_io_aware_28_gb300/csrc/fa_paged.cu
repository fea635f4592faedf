// The bookkeeping of a paged key/value cache: block tables and slot maps from the requests'
// lengths, and the write of new rows into their slots.
//
//  * tables: with o_b cached tokens and n_b new ones, request b holds ceil(o_b / p) pages of p
//    tokens and needs ceil((o_b + n_b) / p); the pages it lacks come off the free list in the
//    order of the requests, so page i of request b is entry off_b + i - ceil(o_b / p) of the
//    list, off being the exclusive sums of the pages lacking.  Token t of the packed new tokens
//    sits in the request whose range of the exclusive sums of n holds t.  Every block forms
//    both sums itself (8 B bytes from L2), which costs less than a second launch, and then
//    takes its share of the list entries and of the tokens.  Latency bounds it: 2.4 us for a step
//    of 64 requests, 6.5 us for 1024 requests and tables of 512 pages (2.3 MB).
//  * append: a copy of rows, 16 bytes a thread and access, bound by HBM: 1.5 us for 64 rows,
//    21.7 us for 16384 rows of 8 x 128 keys and values (134 MB, 6.2 TB/s).
//
// Both launch as dependent kernels (they wait for the previous kernel in the stream before
// touching global memory).
#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kTableThreads = 256;

// Index of the last of sums[0..n) that is <= x (sums[0] = 0 <= x; equal entries are empty
// ranges, of which the last one holds x).
__device__ __forceinline__ int find_range(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads)
tables_kernel(const int32_t* __restrict__ cache_len, const int32_t* __restrict__ new_len,
              const int32_t* __restrict__ free_pages, int n_free, int32_t* table,
              long long table_stride, int max_pages, int32_t* __restrict__ total_len,
              int32_t* __restrict__ token_start, int32_t* __restrict__ slots, int n_slots,
              int32_t* __restrict__ pages_taken, int B, int shift, int num_pages) {
  extern __shared__ int sums[];            // [B + 1] token starts, then [B + 1] list offsets
  __shared__ int2 warp_sum[kTableThreads / 32];
  int* start = sums;
  int* off = sums + B + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = max_pages << shift, round = (1 << shift) - 1;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const int per = (B + kTableThreads - 1) / kTableThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  auto lengths = [&](int b, int* o, int* n) {
    *o = min(max(cache_len[b], 0), cap);
    *n = min(max(new_len[b], 0), cap - *o);
  };
  int2 sum = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    int o, n;
    lengths(b, &o, &n);
    sum.x += n;
    sum.y += ((o + n + round) >> shift) - ((o + round) >> shift);
  }
  int2 incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, d);
    const int y = __shfl_up_sync(0xffffffffu, incl.y, d);
    if (lane >= d) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int2 at = make_int2(incl.x - sum.x, incl.y - sum.y);
  for (int i = 0; i < warp; ++i) {
    at.x += warp_sum[i].x;
    at.y += warp_sum[i].y;
  }
  const bool writer = blockIdx.x == 0;     // of the per-request outputs
  for (int b = b0; b < b1; ++b) {
    int o, n;
    lengths(b, &o, &n);
    start[b] = at.x;
    off[b] = at.y;
    if (writer) {
      total_len[b] = o + n;
      token_start[b] = at.x;
    }
    at.x += n;
    at.y += ((o + n + round) >> shift) - ((o + round) >> shift);
  }
  if (tid == kTableThreads - 1) {          // the last thread's sums are the totals
    start[B] = at.x;
    off[B] = at.y;
    if (writer) {
      token_start[B] = at.x;
      *pages_taken = at.y;
    }
  }
  __syncthreads();

  const int stride = gridDim.x * kTableThreads, first = blockIdx.x * kTableThreads + tid;
  const int lacking = off[B], tokens = start[B];
  for (int e = first; e < lacking; e += stride) {
    const int b = find_range(off, B, e);
    const int have = (min(max(cache_len[b], 0), cap) + round) >> shift;
    table[b * table_stride + have + (e - off[b])] = e < n_free ? free_pages[e] : -1;
  }
  // A token in a page taken just now finds it in the list, not in the table that another
  // block may be writing; one in a page held before finds it in the table.
  for (int t = first; t < n_slots; t += stride) {
    int slot = -1;
    if (t < tokens) {
      const int b = find_range(start, B, t);
      const int o = min(max(cache_len[b], 0), cap);
      const int have = (o + round) >> shift;
      const int x = o + (t - start[b]);
      const int col = x >> shift;
      int p;
      if (col < have) {
        p = table[b * table_stride + col];
      } else {
        const int e = off[b] + col - have;
        p = e < n_free ? free_pages[e] : -1;
      }
      if (p >= 0 && p < num_pages) slot = (p << shift) + (x & round);
    }
    slots[t] = slot;
  }
}

// Rows of two sources into their slots.  Source s has `chunks_s` 16-byte pieces a row; piece
// c of it goes to the slot's row at head c / per_head of the page (KV: both caches alike) or,
// for the latent cache (one destination), behind the pieces of source 0.
struct AppendArgs {
  const uint4* src[2];
  long long src_stride[2];   // 16-byte pieces between rows
  uint4* dst[2];
  long long page_stride;     // 16-byte pieces between pages
  const int32_t* slots;
  int T, num_slots, shift;
};

// PER: pieces of a row of one head (8 or 16); `heads` of them per token in each source.
template <int PER>
__global__ void __launch_bounds__(256) append_kv_kernel(AppendArgs a, int heads) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int row = heads * PER;
  const long long n = static_cast<long long>(a.T) * row;
  const long long stride = static_cast<long long>(gridDim.x) * 256;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += stride) {
    const int t = static_cast<int>(i / row), c = static_cast<int>(i - static_cast<long long>(t) * row);
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) continue;
    const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
    const int h = c / PER, cc = c % PER;
    const long long to = page * a.page_stride + ((static_cast<long long>(h) << a.shift) + r) * PER + cc;
    const uint4 k = a.src[0][t * a.src_stride[0] + c];
    const uint4 v = a.src[1][t * a.src_stride[1] + c];
    a.dst[0][to] = k;
    a.dst[1][to] = v;
  }
}

constexpr int kLatentPieces = FA_LATENT_RANK / 8, kRopePieces = FA_LATENT_ROPE / 8;
constexpr int kRowPieces = kLatentPieces + kRopePieces;

__global__ void __launch_bounds__(256) append_latent_kernel(AppendArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long n = static_cast<long long>(a.T) * kRowPieces;
  const long long stride = static_cast<long long>(gridDim.x) * 256;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += stride) {
    const int t = static_cast<int>(i / kRowPieces), c = static_cast<int>(i % kRowPieces);
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) continue;
    const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
    const uint4 x = c < kLatentPieces ? a.src[0][t * a.src_stride[0] + c]
                                      : a.src[1][t * a.src_stride[1] + c - kLatentPieces];
    a.dst[0][page * a.page_stride + static_cast<long long>(r) * kRowPieces + c] = x;
  }
}

int append_grid(long long pieces) {
  const long long blocks = (pieces + 255) / 256, most = 8ll * sm_count();
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_paged_tables(const int32_t* cache_len, const int32_t* new_len,
                                const int32_t* free_pages, int n_free, int32_t* table,
                                long long table_stride, int max_pages, int32_t* total_len,
                                int32_t* token_start, int32_t* slots, int n_slots,
                                int32_t* pages_taken, int B, int page_shift, int num_pages,
                                cudaStream_t s) {
  const size_t smem = 2 * sizeof(int) * (static_cast<size_t>(B) + 1);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  long long work = n_slots > B ? n_slots : B;
  long long blocks = (work + kTableThreads - 1) / kTableThreads;
  if (blocks > 2 * sm_count()) blocks = 2 * sm_count();
  return launch_dependent(tables_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kTableThreads),
                          smem, s, cache_len, new_len, free_pages, n_free, table, table_stride,
                          max_pages, total_len, token_start, slots, n_slots, pages_taken, B,
                          page_shift, num_pages);
}

cudaError_t launch_paged_append(const void* k, const void* v, long long k_stride,
                                long long v_stride, void* k_cache, void* v_cache,
                                long long page_stride, const int32_t* slots, int T, int num_pages,
                                int Hkv, int page_shift, int d, cudaStream_t s) {
  AppendArgs a{{static_cast<const uint4*>(k), static_cast<const uint4*>(v)},
               {k_stride / 8, v_stride / 8},
               {static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache)},
               page_stride / 8, slots, T, num_pages << page_shift, page_shift};
  const dim3 grid(append_grid(static_cast<long long>(T) * Hkv * (d / 8)));
  return d == 64 ? launch_dependent(append_kv_kernel<8>, grid, dim3(256), 0, s, a, Hkv)
                 : launch_dependent(append_kv_kernel<16>, grid, dim3(256), 0, s, a, Hkv);
}

cudaError_t launch_latent_append(const void* c, const void* k_rope, long long c_stride,
                                 long long rope_stride, void* cache, long long page_stride,
                                 const int32_t* slots, int T, int num_pages, int page_shift,
                                 cudaStream_t s) {
  AppendArgs a{{static_cast<const uint4*>(c), static_cast<const uint4*>(k_rope)},
               {c_stride / 8, rope_stride / 8},
               {static_cast<uint4*>(cache), nullptr},
               page_stride / 8, slots, T, num_pages << page_shift, page_shift};
  return launch_dependent(append_latent_kernel,
                          dim3(append_grid(static_cast<long long>(T) * kRowPieces)), dim3(256), 0,
                          s, a);
}

}  // namespace fa
