// Decode attention over a paged key/value cache, d = 64 or 128: one new query token per
// sequence, up to 16 query heads per key/value head, keys and values found through the
// sequence's block table.
//
// Mathematics.  o = softmax(scale q K^T) V over the keys j < L of the sequence whose pages are
// in the pool, in one pass with a running maximum m and sum l per head (log2 domain, c = scale
// log2 e); parts of a sequence computed by different CTAs join as o = sum 2^(m_i - M) o_i /
// sum 2^(m_i - M) l_i.  m, l, the scores and o are fp32; P is rounded once to bf16 as an
// operand of P V: each weight is off by half a step, 2^-8 of its value, as the output itself is.
//
// What bounds it: every key and value row is read once, 4 d bytes for 4 G d operations, so HBM
// does.  The two products go to the tensor cores with the keys as M, so that the G heads cost
// N = 16 columns and the CUDA cores only see the 128 x G scores of a tile:
//   S^T = K Q^T    A = K tile [128 keys][d] (K-major),  B = the group's query rows [16][d]
//   O^T += V^T P^T A = V tile read MN-major,            B = P^T [16][128 keys] (bf16)
// A tile is 128 keys, in boxes of a page's rows or 32 of them; the lanes of the producer warp each
// take a box: its table entry and its loads.  A page that lies outside the pool is not loaded, and
// its rows, like those past the length, are hidden: their scores are replaced, never computed with,
// and their V rows are zeroed in shared memory.
//
// A tile's way (scores, maximum, P, P V) is a chain of about 2.5k cycles, at d = 64 twice what HBM
// takes for its 32 KB, and an issuing thread spends some 1.8k cycles on a tile's twelve MMAs,
// commits and waits (traced).  So two groups of four softmax warps take the tiles in turn, each
// with its own maximum, sum and O^T, joined at the end like parts of different CTAs; and one
// thread issues the scores of every tile that has landed, another the P V products.  Score and P
// buffers go with the stages: a tile's stage is filled only after the P V of the tile before in
// it, so they are free by then.
//
// Work: fa_paged_sched.cuh cuts the line of all tiles into one range per CTA, one CTA per SM.
// A pair inside one range is finished there; only pairs that a range's end cuts go through the
// workspace and the combine kernel, at most two partial results a CTA.
//   warps 0, 2 producers (a lane per page);     warps 1, 3  MMA issuers (one thread each);
//   warps 4-11 softmax, thread = key row.
// Measured: d = 128, 32 query and 8 key/value heads, 64 sequences of 8192: 309 us, 6.95 TB/s, the
// rate of a plain copy.  d = 64, 24 and 8 heads, 48 ragged sequences to 5001: 60 us for 37 us of
// bytes, of which some 12 us do not grow with the lengths; pages of 16 tokens cost 12% more than
// pages of 256 at d = 64 and 4% at d = 128 (boxes of 2 KB and 4 KB).
// Every wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and leaves.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "fa_decode_units.cuh"
#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace decode;

// The segments of a worker's range of the line of all tiles.
struct RangeWalk {
  sched::Walk<kKeys> walk;
  long long first;
  int w;
  __device__ __forceinline__ RangeWalk(const sched::Start& s, const int32_t* cache_len, int heads,
                                       int cap, int w_)
      : walk(s, cache_len, heads, cap), first(s.first), w(w_) {}
  __device__ __forceinline__ bool next(Segment& sg) {
    if (!walk.next(sg)) return false;
    sg.slot = sched::slot(sg.pair_start, first, w);
    return true;
  }
};

template <int D, int GP>
__global__ void __launch_bounds__(kThreads, 1)
decode_paged_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mq, PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const Smem<D> sh(reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023)));
  Bars* bars = sh.bars;
  __shared__ sched::Start start;
  __shared__ long long scan[kThreads / 32 + 1];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int cap = a.max_pages << a.page_shift;

  if (tid == 0) init_bars<D>(bars);
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, kDecodeColumns);
    tmem_relinquish();
  }
  if (tid == 0) {
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mq);
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  sched::find_start<kKeys, kThreads>(&start, scan, a.cache_len, a.B, a.Hkv, cap, blockIdx.x,
                                     gridDim.x, blockIdx.x == 0 ? a.prefix : nullptr);
  const uint32_t tb = bars->tmem_base;
  segments<D, GP>(mk, mv, mq, a, sh, tb,
                  RangeWalk(start, a.cache_len, a.Hkv, cap, blockIdx.x));

  tc_fence_before();
  __syncthreads();
  if (bars->abort && tid == 0) {
    // Let any copy still in flight land before the CTA's shared memory is released.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tb, kDecodeColumns);
  }
}

// Joins the partial results of a pair that more than one CTA worked on; writes o = 0, lse = -inf
// for an empty sequence.  W warps (1 or 8) per (b, query head), each with every W-th part.
template <int D, int W>
__global__ void __launch_bounds__(256) decode_paged_combine_kernel(PagedArgs a, int workers) {
  constexpr int PS = TC<D>::PSTRIDE, PER = D / 32;
  __shared__ float red[8][D + 2];          // a warp's columns, maximum and sum
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % W;
  const long long row = blockIdx.x * static_cast<long long>(8 / W) + warp / W;
  if (row >= static_cast<long long>(a.B) * a.Hq) return;   // W = 8: the whole block
  const int b = static_cast<int>(row / a.Hq), hq = static_cast<int>(row % a.Hq);
  const int G = a.Hq / a.Hkv, g = hq / G, h = hq % G;
  const long long p0 = a.prefix[b], p1 = a.prefix[b + 1], total = a.prefix[a.B];
  const long long n = (p1 - p0) / a.Hkv;
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  float M = -INFINITY, lsum = 0.f;
  if (n > 0) {
    const long long first = p0 + g * n;
    workers = sched::active(total, workers);
    const int w0 = sched::owner(first, total, workers);
    const int parts = sched::owner(first + n - 1, total, workers) - w0 + 1;
    if (parts == 1) return;   // finished by its CTA
    // Only the first part can sit in the second of its worker's slots.
    const int slot0 = sched::slot(first, sched::range_start(total, w0, workers), w0);
    const float* part = a.part + static_cast<size_t>(h) * PS;
    const size_t stride = static_cast<size_t>(G) * PS;
    auto at = [&](int i) { return part + (i == 0 ? slot0 : 2 * (w0 + i)) * stride; };
    // The warp's parts are sub, sub + W, ...: lane j has the statistics of the j-th of a batch.
    for (int base = sub; base < parts; base += 32 * W) {
      const int mine = base + lane * W;
      const float* p = at(mine < parts ? mine : base);
      const float m = mine < parts ? p[D] : -INFINITY, l = mine < parts ? p[D + 1] : 0.f;
      const float mb = fmaxf(M, warp_max(m));
      const float use = mb == -INFINITY ? 0.f : mb;
      const float keep = ex2(M - use);           // M = -inf gives 0
      const float wt = ex2(m - use);             // a part without a visible key weighs 0
      M = mb;
      lsum = lsum * keep + l * wt;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= keep;
      const int cnt = min(32, (parts - base + W - 1) / W);
#pragma unroll 8
      for (int j = 0; j < cnt; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wt, j);
        const float* pj = at(base + j * W) + lane * PER;
        if constexpr (PER == 4) {
          const float4 v = *reinterpret_cast<const float4*>(pj);
          acc[0] = fmaf(wj, v.x, acc[0]);
          acc[1] = fmaf(wj, v.y, acc[1]);
          acc[2] = fmaf(wj, v.z, acc[2]);
          acc[3] = fmaf(wj, v.w, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(pj);
          acc[0] = fmaf(wj, v.x, acc[0]);
          acc[1] = fmaf(wj, v.y, acc[1]);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) red[warp][lane * PER + i] = acc[i];
    if (lane == 0) {
      red[warp][D] = M;
      red[warp][D + 1] = lsum;
    }
    __syncthreads();
    if (sub > 0) return;
    float mw[W];
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, mw[w] = red[w][D]);
    const float use = M == -INFINITY ? 0.f : M;
    lsum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float wt = ex2(mw[w] - use);
      lsum += red[w][D + 1] * wt;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(red[w][lane * PER + i], wt, acc[i]);
    }
  }
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;   // a NaN sum stays one
  __nv_bfloat16* orow = a.o + static_cast<size_t>(row) * D + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<uint32_t*>(orow + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0) a.lse[row] = lsum == 0.f ? -INFINITY : (M + __log2f(lsum)) * kLn2;
}

template <int D, int GP>
cudaError_t launch_g(const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
                     const PagedArgs& a, int workers, cudaStream_t s) {
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(decode_paged_kernel<D, GP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, TC<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  cudaError_t e = launch_dependent(decode_paged_kernel<D, GP>, dim3(workers), dim3(kThreads),
                                   TC<D>::SMEM, s, mk, mv, mq, a);
  if (e != cudaSuccess) return e;
  // Few pairs, many parts each: eight warps to a row, else one (d = 128, Hq = 32, Hkv = 8: 1 sequence
  // of 8192, 19 parts a pair, 11.8 against 15.0 us; 4 to 8000, 5 parts, 24.0 against 25.2; from 16
  // sequences on, 1.2 parts, no difference, and d = 64, 48 sequences, 61 against 59).
  const long long rows = static_cast<long long>(a.B) * a.Hq;
  if (workers > 4ll * a.B * a.Hkv)
    return launch_dependent(decode_paged_combine_kernel<D, 8>, dim3(static_cast<unsigned>(rows)),
                            dim3(256), 0, s, a, workers);
  return launch_dependent(decode_paged_combine_kernel<D, 1>,
                          dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s, a,
                          workers);
}

template <int D>
cudaError_t launch_d(const void* q, const void* k, const void* v, long long page_stride,
                     const PagedArgs& a, int workers, cudaStream_t s) {
  CUtensorMap mk, mv, mq;
  const int page = 1 << a.page_shift, rows = page < kBox ? page : kBox;
  if (!make_page_map(&mk, k, a.num_pages, a.Hkv, page, D, page_stride, rows) ||
      !make_page_map(&mv, v, a.num_pages, a.Hkv, page, D, page_stride, rows) ||
      !make_head_map_rows(&mq, q, 1, a.B * a.Hq, D, kN))
    return cudaErrorInvalidValue;
  const int G = a.Hq / a.Hkv;
  if (G > 8) return launch_g<D, 16>(mk, mv, mq, a, workers, s);
  if (G > 4) return launch_g<D, 8>(mk, mv, mq, a, workers, s);
  if (G > 2) return launch_g<D, 4>(mk, mv, mq, a, workers, s);
  if (G > 1) return launch_g<D, 2>(mk, mv, mq, a, workers, s);
  return launch_g<D, 1>(mk, mv, mq, a, workers, s);
}

}  // namespace

// Partial results (two a CTA), then the tile sums of the sequences.
size_t decode_paged_part_bytes(int G, int d) {
  return round_up(2 * static_cast<size_t>(sm_count()) * G * (d + 4) * sizeof(float), 256);
}

cudaError_t launch_decode_paged(const void* q, const void* k, const void* v,
                                long long page_stride, const int32_t* table,
                                long long table_stride, int max_pages, int page_shift,
                                int num_pages, const int32_t* cache_len, void* o, float* lse,
                                int B, int Hq, int Hkv, int d, float scale, void* workspace,
                                int* err, unsigned long long wait_ns, cudaStream_t s) {
  const size_t part = decode_paged_part_bytes(Hq / Hkv, d);
  PagedArgs a{table, table_stride, max_pages, page_shift, num_pages, cache_len, B, Hq, Hkv,
              scale * kLog2e, static_cast<__nv_bfloat16*>(o), lse,
              static_cast<float*>(workspace),
              reinterpret_cast<long long*>(static_cast<char*>(workspace) + part), err, wait_ns};
  // No more CTAs than there can be tiles.
  const long long tiles = static_cast<long long>(B) * Hkv *
                          (((static_cast<long long>(max_pages) << page_shift) + kKeys - 1) / kKeys);
  const int workers = tiles < sm_count() ? static_cast<int>(tiles) : sm_count();
  return d == 64 ? launch_d<64>(q, k, v, page_stride, a, workers, s)
                 : launch_d<128>(q, k, v, page_stride, a, workers, s);
}

}  // namespace fa
