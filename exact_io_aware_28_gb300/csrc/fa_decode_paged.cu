// Decode attention over a paged key/value cache, d = 64 or 128: one new query token per
// sequence, up to 16 query heads per key/value head, keys and values found through the
// sequence's block table.
//
// Mathematics.  o = softmax(scale q K^T) V over the keys j < L of the sequence whose pages are
// in the pool, in one pass with a running maximum m and sum l per head (log2 domain, c = scale
// log2 e); parts of a sequence computed by different CTAs join as o = sum 2^(m_i - M) o_i /
// sum 2^(m_i - M) l_i.  m, l, the scores and o are fp32; P is rounded once to bf16 as an
// operand of P V (half a step, 2^-9 of each weight's magnitude class, as the output's own).
//
// What bounds it: every key and value row is read once, 4 d bytes for 4 G d operations, so HBM
// does.  The two products go to the tensor cores with the keys as M, so that the G heads cost
// N = 16 columns and the CUDA cores only see the 128 x G scores of a tile:
//   S^T = K Q^T    A = K tile [128 keys][d] (K-major),  B = the group's query rows [16][d]
//   O^T += V^T P^T A = V tile read MN-major,            B = P^T [16][128 keys] (bf16)
// A tile is 128 keys = 128 / page boxes of page rows (one box when pages are larger); the lanes
// of the producer warp each take a page: its table entry and its boxes.  A page that lies
// outside the pool is not loaded, and its rows, like those past the length, are hidden: their
// scores are replaced, never computed with, and their V rows are zeroed in shared memory.
//
// Work: fa_paged_sched.cuh cuts the line of all tiles into one range per CTA, one CTA per SM.
// A pair inside one range is finished there; only pairs that a range's end cuts go through the
// workspace and the combine kernel, at most two partial results a CTA.
//   warp 0     producer (a lane per page);      warp 1  MMA issuer (one thread);
//   warp 2     tensor memory (S^T x 2, O^T x 2); warps 4-7 softmax, thread = key row.
// Every wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and leaves.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;
using sched::Segment;

constexpr int kKeys = 128;                    // keys per tile
constexpr int kN = 16;                        // query heads padded to the MMA's N
constexpr int kMaxStages = 4;
constexpr int kSub = kKeys * 128;             // [128 rows][64 bf16] swizzled subtile, 16 KB
constexpr int kPBytes = 2 * kN * 128;         // [16][128 keys] bf16
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units; exact, see fa_fwd_sm103.cu

struct Bars {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t p_free[2];
  uint64_t o_full[2];
  uint64_t xmax[2];
  uint64_t xsum[2];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t seen[kMaxStages];  // bit i: rows 16 i ... 16 i + 15 of the stage are in the pool
  int abort;
  int never;  // stays 0: the drain wait must not be cut short by an abort
};

template <int D>
struct TC {
  static constexpr int NSUB = D / 64;                  // 64-column subtiles of a K or V tile
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int STAGE = 2 * NSUB * kSub;        // K tile then V tile
  static constexpr int PAD = D == 128 ? 0 : kSub;      // zero rows d = 64..127 of V^T
  static constexpr int QBYTES = NSUB * kN * 128;       // [16][d] bf16
  static constexpr int PSTRIDE = D + 4;                // floats per (slot, head) partial row
  static constexpr int SMEM = 1024 + STAGES * STAGE + PAD + 2 * QBYTES + 2 * kPBytes +
                              2 * 4 * kN * 4 * 2 + static_cast<int>(sizeof(Bars));
  static_assert(STAGES <= kMaxStages && SMEM <= 227 * 1024, "shared memory");
};

struct PagedArgs {
  const int32_t* table;
  long long table_stride;
  int max_pages, page_shift, num_pages;
  const int32_t* cache_len;
  int B, Hq, Hkv;
  float c;                 // scale log2 e
  __nv_bfloat16* o;
  float* lse;
  float* part;             // [2 CTAs][G][D + 4]
  long long* prefix;       // [B + 1] tiles before each sequence
  int* err;
  unsigned long long wait_ns;
};

// Byte offset of element (row h, column r) in a [16][128] bf16 K-major operand tile stored as
// two 128B-swizzled [16][64] subtiles.
__device__ __forceinline__ uint32_t nk_offset(int h, int r) {
  return static_cast<uint32_t>((r >> 6) * (kN * 128) + (h >> 3) * 1024 + (h & 7) * 128 +
                               ((((r & 63) >> 3) ^ (h & 7)) << 4) + (r & 7) * 2);
}

// GP: query heads per key/value head rounded up to a power of two; G the actual number.
template <int D, int GP>
__global__ void __launch_bounds__(kThreads, 1)
decode_paged_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mq, PagedArgs a) {
  using C = TC<D>;
  constexpr int kStages = C::STAGES, kStage = C::STAGE, kQBytes = C::QBYTES;
  constexpr int kPStride = C::PSTRIDE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sKV = base;                                   // [kStages][K subtiles, V subtiles]
  uint8_t* sPad = sKV + kStages * kStage;                // d = 64: [128 keys][64] zeros
  uint8_t* sQ = sPad + C::PAD;                           // [2][kQBytes]
  uint8_t* sP = sQ + 2 * kQBytes;                        // [2][kPBytes]
  float* red_m = reinterpret_cast<float*>(sP + 2 * kPBytes);   // [2][4 warps][16 heads]
  float* red_l = red_m + 2 * 4 * kN;                           // [2][4 warps][16 heads]
  Bars* bars = reinterpret_cast<Bars*>(red_l + 2 * 4 * kN);
  __shared__ sched::Start start;
  __shared__ long long scan[kThreads / 32 + 1];
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv, cap = a.max_pages << a.page_shift;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 128);
      mbar_init(&bars->p_free[i], 1);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->xmax[i], 128);
      mbar_init(&bars->xsum[i], 128);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->never = 0;
    fence_mbar_init();
  }
  if constexpr (C::PAD > 0) {
    for (int i = tid; i < C::PAD / 16; i += kThreads)
      reinterpret_cast<uint4*>(sPad)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();   // read by the tensor cores
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 64);
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
  sched::Walk<kKeys> walk(start, a.cache_len, a.Hkv, cap);
  Segment sg;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // Lane i < boxes takes the i-th page of every tile (all of a tile's rows when pages hold
    // 128 tokens or more).
    const int shift = a.page_shift;
    const int rows = min(kKeys, 1 << shift);        // rows of a box
    const int boxes = kKeys / rows;
    const uint32_t bits = (1u << (rows / 16)) - 1u; // of a box in the stage's row mask
    bool ok = true;
    int n = 0, nu = 0;
    while (ok && walk.next(sg)) {
      const int qb = nu & 1;
      if (nu >= 2) {
        ok = mbar_wait_warp(&bars->q_empty[qb], ((nu >> 1) - 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full[qb], kQBytes);
        for (int s = 0; s < C::NSUB; ++s)
          tma_load_3d(sQ + qb * kQBytes + s * (kN * 128), &mq, &bars->q_full[qb], 64 * s,
                      sg.b * a.Hq + sg.head * G, 0);
      }
      const int32_t* row = a.table + sg.b * a.table_stride;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        const int st = n % kStages;
        const int x = k0 + lane * rows;             // first token of this lane's box
        int p = -1;
        if (lane < boxes && x < sg.len) p = row[x >> shift];
        const bool in = p >= 0 && p < a.num_pages;
        const uint32_t pages = __ballot_sync(0xffffffffu, in);
        if (n >= kStages) {
          ok = mbar_wait_warp(&bars->empty[st], ((n / kStages) - 1) & 1, abort_flag, a.err,
                              a.wait_ns);
          if (!ok) break;
        }
        if (lane == 0) {
          uint32_t seen = 0;
          for (int i = 0; i < boxes; ++i)
            if (pages >> i & 1u) seen |= bits << (i * (rows / 16));
          bars->seen[st] = seen;
          mbar_arrive_expect_tx(&bars->full[st],
                                static_cast<uint32_t>(__popc(pages)) * rows * D * 4);
        }
        __syncwarp();
        if (in) {
          uint8_t* dst = sKV + st * kStage + lane * rows * 128;
          const int y = x & ((1 << shift) - 1);     // its first row within the page
          for (int s = 0; s < C::NSUB; ++s) {
            tma_load_4d(dst + s * kSub, &mk, &bars->full[st], 64 * s, y, sg.head, p);
            tma_load_4d(dst + (C::NSUB + s) * kSub, &mv, &bars->full[st], 64 * s, y, sg.head, p);
          }
        }
      }
      ++nu;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, kN, false, false);
      constexpr uint32_t idO = idesc_bf16(128, kN, true, false);
      bool ok = true;
      // The flattened tile sequence: tile t of nt of the segment with ordinal nu.
      struct Cur { int t, nt, nu; } cur = {0, 0, -1}, nxt;
      auto next_tile = [&](Cur& c) -> bool {
        if (c.nu >= 0 && c.t + 1 < c.nt) {
          ++c.t;
          return true;
        }
        if (!walk.next(sg)) return false;
        c.t = 0;
        c.nt = (sg.k1 - sg.k0 + kKeys - 1) / kKeys;
        ++c.nu;
        return true;
      };
      auto issue_s = [&](const Cur& c, int m) -> bool {
        const int st = m % kStages;
        if (c.t == 0) {
          if (!mbar_wait(&bars->q_full[c.nu & 1], (c.nu >> 1) & 1, abort_flag, a.err, a.wait_ns))
            return false;
        }
        if (!mbar_wait(&bars->full[st], (m / kStages) & 1, abort_flag, a.err, a.wait_ns))
          return false;
        tc_fence_after();
        const uint64_t dK = sw128_desc(smem_u32(sKV + st * kStage), 16, 1024);
        const uint64_t dQ = sw128_desc(smem_u32(sQ + (c.nu & 1) * kQBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t offA = static_cast<uint64_t>(((kk >> 2) * kSub + (kk & 3) * 32) >> 4);
          const uint64_t offB = static_cast<uint64_t>(((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4);
          mma_ss(tb + (m & 1) * kN, dK + offA, dQ + offB, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit(&bars->s_full[m & 1]);
        if (c.t == c.nt - 1) mma_commit(&bars->q_empty[c.nu & 1]);
        return true;
      };
      int n = 0;
      bool have = next_tile(cur);
      if (have) ok = issue_s(cur, 0);
      while (ok && have) {
        nxt = cur;
        const bool have_next = next_tile(nxt);
        if (have_next) {
          ok = issue_s(nxt, n + 1);
          if (!ok) break;
        }
        ok = mbar_wait(&bars->p_full[n & 1], (n >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const int st = n % kStages;
        // A = V^T, M = 128: the second group of 64 rows is the next 64 columns of V (d =
        // 128) or the zero block (d = 64), LBO bytes further on.
        const uint32_t aV = smem_u32(sKV + st * kStage + C::NSUB * kSub);
        const uint32_t lbo = C::PAD > 0 ? smem_u32(sPad) - aV : static_cast<uint32_t>(kSub);
        const uint64_t dV = sw128_desc(aV, lbo, 1024);
        const uint64_t dP = sw128_desc(smem_u32(sP + (n & 1) * kPBytes), 16, 1024);
        const uint32_t tO = tb + 32 + (cur.nu & 1) * kN;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
          const uint64_t offA = static_cast<uint64_t>((2048 * kk) >> 4);
          const uint64_t offB = static_cast<uint64_t>(((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4);
          mma_ss(tO, dV + offA, dP + offB, idO, (cur.t > 0 || kk > 0) ? 1u : 0u);
        }
        mma_commit(&bars->p_free[n & 1]);
        mma_commit(&bars->empty[st]);
        if (cur.t == cur.nt - 1) mma_commit(&bars->o_full[cur.nu & 1]);
        cur = nxt;
        have = have_next;
        ++n;
      }
      // Every MMA issued has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, a.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax (thread = key row)
    const int w4 = warp & 3;
    const int r = 32 * w4 + lane;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * w4) << 16);
    bool ok = true;
    int n = 0, nu = 0;
    while (ok && walk.next(sg)) {
      float m_run[GP], l_run[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        m_run[h] = -INFINITY;
        l_run[h] = 0.f;
      }
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        const int st = n % kStages;
        // The stage has landed (its MMAs wait for it too); the wait orders the row mask.
        ok = mbar_wait_warp(&bars->full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        const bool vis = k0 + r < sg.k1 && ((bars->seen[st] >> (r >> 4)) & 1u);
        ok = mbar_wait_warp(&bars->s_full[n & 1], (n >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[16];
        tmem_ld16(lane_base + (n & 1) * kN, sv);
        tmem_wait_ld();
        float x[GP];
#pragma unroll
        for (int h = 0; h < GP; ++h) x[h] = vis ? __uint_as_float(sv[h]) * a.c : -INFINITY;
        // CTA-wide maximum per head: warp maxima through shared memory and an mbarrier.
        float* rm = red_m + (n & 1) * 4 * kN;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float v = warp_max(x[h]);
          if (lane == 0) rm[w4 * kN + h] = v;
        }
        mbar_arrive(&bars->xmax[n & 1]);
        ok = mbar_wait_warp(&bars->xmax[n & 1], (n >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        float alpha[GP], muse[GP];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float mt = fmaxf(fmaxf(rm[h], rm[kN + h]), fmaxf(rm[2 * kN + h], rm[3 * kN + h]));
          const float mn = mt > m_run[h] + kRescaleThreshold ? mt : m_run[h];
          const bool ch = mn != m_run[h];
          alpha[h] = ch ? ex2(m_run[h] - mn) : 1.f;   // m_run = -inf gives 0
          grow |= ch;
          m_run[h] = mn;
          muse[h] = mn == -INFINITY ? 0.f : mn;
        }
        // P^T into this tile's P buffer once the product two tiles back has read it.
        if (n >= 2) {
          ok = mbar_wait_warp(&bars->p_free[n & 1], ((n >> 1) - 1) & 1, abort_flag, a.err,
                              a.wait_ns);
          if (!ok) break;
        }
        uint8_t* pt = sP + (n & 1) * kPBytes;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float p = ex2(x[h] - muse[h]);   // x = -inf gives 0
          l_run[h] = l_run[h] * alpha[h] + p;
          *reinterpret_cast<__nv_bfloat16*>(pt + nk_offset(h, r)) = __float2bfloat16_rn(p);
        }
        if (!vis) {  // a hidden row: zero its V so that 0 x (anything) stays 0
          uint8_t* vt = sKV + st * kStage + C::NSUB * kSub;
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<uint4*>(vt + s * kSub + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
        }
        // Rescale the running O^T (lane = d) when a maximum moved after the first tile; the
        // product of the previous tile must have completed.
        if (grow && k0 > sg.k0) {
          ok = mbar_wait_warp(&bars->p_free[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.err,
                              a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          uint32_t ov[16];
          const uint32_t oaddr = lane_base + 32 + (nu & 1) * kN;
          tmem_ld16(oaddr, ov);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < GP; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * alpha[h]);
          tmem_st16(oaddr, ov);
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_full[n & 1]);
      }
      if (!ok) break;
      // ---- the segment's result: row sums over the CTA, then O^T columns (lane = d)
      float* rl = red_l + (nu & 1) * 4 * kN;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        float v = l_run[h];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) rl[w4 * kN + h] = v;
      }
      mbar_arrive(&bars->xsum[nu & 1]);
      ok = mbar_wait_warp(&bars->xsum[nu & 1], (nu >> 1) & 1, abort_flag, a.err, a.wait_ns);
      if (!ok) break;
      ok = mbar_wait_warp(&bars->o_full[nu & 1], (nu >> 1) & 1, abort_flag, a.err, a.wait_ns);
      if (!ok) break;
      tc_fence_after();
      uint32_t ov[16];
      tmem_ld16(lane_base + 32 + (nu & 1) * kN, ov);
      tmem_wait_ld();
      tc_fence_before();
      const int slot = sched::slot(sg.pair_start, start.first, blockIdx.x);
      float* out = a.part + static_cast<size_t>(slot) * G * kPStride;
      const size_t head0 = static_cast<size_t>(sg.b) * a.Hq + sg.head * G;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        if (h >= G) break;
        const float l = rl[h] + rl[kN + h] + rl[2 * kN + h] + rl[3 * kN + h];
        const float ovh = __uint_as_float(ov[h]);
        if (sg.whole) {
          if (r < D)
            a.o[(head0 + h) * D + r] = __float2bfloat16_rn(l == 0.f ? 0.f : ovh / l);
          if (r == 0) a.lse[head0 + h] = l == 0.f ? -INFINITY : (m_run[h] + __log2f(l)) * kLn2;
        } else {
          if (r < D) out[h * kPStride + r] = ovh;
          if (r == 0) {
            out[h * kPStride + D] = m_run[h];
            out[h * kPStride + D + 1] = l;
          }
        }
      }
      ++nu;
    }
  }

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
    tmem_dealloc(tb, 64);
  }
}

// One warp per (b, query head): joins the partial results of a pair that more than one CTA
// worked on; writes o = 0, lse = -inf for an empty sequence.
template <int D>
__global__ void __launch_bounds__(256) decode_paged_combine_kernel(PagedArgs a, int workers) {
  constexpr int PS = TC<D>::PSTRIDE, PER = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const long long row = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(a.B) * a.Hq) return;
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
    const int w1 = sched::owner(first + n - 1, total, workers);
    if (w0 == w1) return;   // finished by its CTA
    const float* part = a.part + static_cast<size_t>(h) * PS;
    const size_t stride = static_cast<size_t>(G) * PS;
    auto at = [&](int w) {
      return part + sched::slot(first, sched::range_start(total, w, workers), w) * stride;
    };
    for (int w = w0 + lane; w <= w1; w += 32) M = fmaxf(M, at(w)[D]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (M == -INFINITY) M = 0.f;
    for (int base = w0; base <= w1; base += 32) {
      const int w = base + lane;
      float wt = 0.f;
      if (w <= w1) {
        const float* p = at(w);
        wt = ex2(p[D] - M);     // a part without a visible key (-inf) weighs 0
        lsum += p[D + 1] * wt;
      }
      const int cnt = min(32, w1 - base + 1);
#pragma unroll 4
      for (int j = 0; j < cnt; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wt, j);
        const float* p = at(base + j) + lane * PER;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = fmaf(wj, p[i], acc[i]);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
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
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.B) * a.Hq + 7) / 8);
  return launch_dependent(decode_paged_combine_kernel<D>, dim3(blocks), dim3(256), 0, s, a,
                          workers);
}

template <int D>
cudaError_t launch_d(const void* q, const void* k, const void* v, long long page_stride,
                     const PagedArgs& a, int workers, cudaStream_t s) {
  CUtensorMap mk, mv, mq;
  const int page = 1 << a.page_shift, rows = page < kKeys ? page : kKeys;
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
