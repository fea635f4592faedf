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
// A tile is 128 keys = 128 / page boxes of page rows (one box when pages are larger); the lanes
// of the producer warp each take a page: its table entry and its boxes.  A page that lies
// outside the pool is not loaded, and its rows, like those past the length, are hidden: their
// scores are replaced, never computed with, and their V rows are zeroed in shared memory.
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

#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;
using sched::Segment;

constexpr int kKeys = 128;                    // keys per tile
constexpr int kN = 16;                        // query heads padded to the MMA's N
constexpr int kMaxStages = 6;
constexpr int kSub = kKeys * 128;             // [128 rows][64 bf16] swizzled subtile, 16 KB
constexpr int kPBytes = 2 * kN * 128;         // [16][128 keys] bf16
constexpr int kThreads = 384;
constexpr uint32_t kO = kMaxStages * kN;      // first column of O^T: 2 segments x 2 groups
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units; exact, see fa_fwd_sm103.cu

struct Bars {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];  // P V of the stage's tile has completed
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t s_full[kMaxStages];
  uint64_t p_full[kMaxStages];
  uint64_t o_full[2];
  uint64_t xmax[2];    // of each softmax group
  uint64_t xsum[2];    // of both, for a segment
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t seen[kMaxStages];  // bit i: rows 16 i ... 16 i + 15 of the stage are in the pool
  int abort;
  int never;  // stays 0: the drain wait must not be cut short by an abort
};

template <int D>
struct TC {
  static constexpr int NSUB = D / 64;                  // 64-column subtiles of a K or V tile
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int STAGE = 2 * NSUB * kSub;        // K tile then V tile
  static constexpr int QBYTES = NSUB * kN * 128;       // [16][d] bf16
  static constexpr int PSTRIDE = D + 4;                // floats per (slot, head) partial row
  static constexpr int SMEM = 1024 + STAGES * STAGE + 2 * QBYTES + STAGES * kPBytes +
                              (2 * 2 + 2 * 2 * 2) * 4 * kN * 4 + static_cast<int>(sizeof(Bars));
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
  uint8_t* sQ = sKV + kStages * kStage;                  // [2][kQBytes]
  uint8_t* sP = sQ + 2 * kQBytes;                        // [kStages][kPBytes]
  // A group's exchange of maxima: [2 groups][2][4 warps][16 heads]; a segment's statistics:
  // [2 segments][2 groups][4 warps: sums][16 heads], then the same of maxima (one row used).
  float* red_m = reinterpret_cast<float*>(sP + kStages * kPBytes);
  float* red_l = red_m + 2 * 2 * 4 * kN;
  float* seg_m = red_l + 2 * 2 * 4 * kN;
  Bars* bars = reinterpret_cast<Bars*>(seg_m + 2 * 2 * 4 * kN);
  __shared__ sched::Start start;
  __shared__ long long scan[kThreads / 32 + 1];
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv, cap = a.max_pages << a.page_shift;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 2);
      mbar_init(&bars->empty[s], 1);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_full[s], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->xmax[i], 128);
      mbar_init(&bars->xsum[i], 256);
    }
    mbar_init(&bars->drain, 2);
    bars->abort = 0;
    bars->never = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 256);
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

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    // Warp 0 has the queries and the keys, warp 2 the values: one warp issues a box in some 70
    // cycles, and small pages make many.  Lane i < boxes takes the i-th page of every tile (all of
    // a tile's rows when pages hold 128 tokens or more).
    const bool keys = warp == 0;
    const CUtensorMap* map = keys ? &mk : &mv;
    const int shift = a.page_shift;
    const int rows = min(kKeys, 1 << shift);        // rows of a box
    const int boxes = kKeys / rows;
    const uint32_t bits = (1u << (rows / 16)) - 1u; // of a box in the stage's row mask
    bool ok = true;
    int n = 0, nu = 0;
    while (ok && walk.next(sg)) {
      const int qb = nu & 1;
      if (keys && nu >= 2) {
        ok = mbar_wait_warp(&bars->q_empty[qb], ((nu >> 1) - 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
      }
      if (keys && lane == 0) {
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
          if (keys) {
            uint32_t seen = 0;
            for (int i = 0; i < boxes; ++i)
              if (pages >> i & 1u) seen |= bits << (i * (rows / 16));
            bars->seen[st] = seen;
          }
          mbar_arrive_expect_tx(&bars->full[st],
                                static_cast<uint32_t>(__popc(pages)) * rows * D * 2);
        }
        __syncwarp();
        if (in) {
          uint8_t* dst = sKV + st * kStage + (keys ? 0 : C::NSUB) * kSub + lane * rows * 128;
          const int y = x & ((1 << shift) - 1);     // its first row within the page
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s)
            tma_load_4d(dst + s * kSub, map, &bars->full[st], 64 * s, y, sg.head, p);
        }
      }
      ++nu;
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      bool ok = true;
      int n = 0, nu = 0;
      if (warp == 1) {
        constexpr uint32_t idS = idesc_bf16(128, kN, false, false);
        while (ok && walk.next(sg)) {
          ok = mbar_wait(&bars->q_full[nu & 1], (nu >> 1) & 1, abort_flag, a.err, a.wait_ns);
          for (int k0 = sg.k0; ok && k0 < sg.k1; k0 += kKeys, ++n) {
            const int st = n % kStages;
            ok = mbar_wait(&bars->full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dK = sw128_desc(smem_u32(sKV + st * kStage), 16, 1024);
            const uint64_t dQ = sw128_desc(smem_u32(sQ + (nu & 1) * kQBytes), 16, 1024);
#pragma unroll
            for (int g = 0; g < C::NSUB; ++g) {
              uint64_t da[4], db[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                da[k] = dK + static_cast<uint64_t>((g * kSub + k * 32) >> 4);
                db[k] = dQ + static_cast<uint64_t>((g * (kN * 128) + k * 32) >> 4);
              }
              mma_ss_x4(tb + st * kN, da, db, idS, g > 0 ? 1u : 0u);
            }
            mma_commit(&bars->s_full[st]);
            if (k0 + kKeys >= sg.k1) mma_commit(&bars->q_empty[nu & 1]);
          }
          ++nu;
        }
      } else {
        constexpr uint32_t idO = idesc_bf16(128, kN, true, false);
        while (ok && walk.next(sg)) {
          for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
            const int st = n % kStages;
            ok = mbar_wait(&bars->p_full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            // A = V^T, M = 128: the second group of 64 rows is the next 64 columns of V (d =
            // 128) or, with no offset, the same ones again (d = 64: those rows are never read).
            const uint64_t dV = sw128_desc(smem_u32(sKV + st * kStage + C::NSUB * kSub),
                                           D == 128 ? kSub : 0, 1024);
            const uint64_t dP = sw128_desc(smem_u32(sP + st * kPBytes), 16, 1024);
            const uint32_t tO = tb + kO + ((nu & 1) * 2 + (n & 1)) * kN;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint64_t da[4], db[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                da[k] = dV + static_cast<uint64_t>((2048 * (4 * g + k)) >> 4);
                db[k] = dP + static_cast<uint64_t>((g * (kN * 128) + k * 32) >> 4);
              }
              // a group's first tile of the segment is one of its first two
              mma_ss_x4(tO, da, db, idO, (k0 - sg.k0 > kKeys || g > 0) ? 1u : 0u);
            }
            mma_commit(&bars->empty[st]);
            if (k0 + kKeys >= sg.k1) mma_commit(&bars->o_full[nu & 1]);
          }
          ++nu;
        }
      }
      // Every MMA issued by either thread has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, a.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax (thread = key row)
    // Group grp has the tiles whose number n (over all segments) is grp mod 2.
    const int w4 = warp & 3, grp = (warp - 4) >> 2;
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
      bool first = true;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        if ((n & 1) != grp) continue;
        const int st = n % kStages;
        // The stage has landed (its MMAs wait for it too); the wait orders the row mask.
        ok = mbar_wait_warp(&bars->full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        const bool vis = k0 + r < sg.k1 && ((bars->seen[st] >> (r >> 4)) & 1u);
        ok = mbar_wait_warp(&bars->s_full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[16];
        tmem_ld16_wait(lane_base + st * kN, sv);
        float x[GP];
#pragma unroll
        for (int h = 0; h < GP; ++h) x[h] = vis ? __uint_as_float(sv[h]) * a.c : -INFINITY;
        // The group's maximum per head: warp maxima through shared memory and an mbarrier.
        const int turn = (n >> 1) & 1;
        float* rm = red_m + (grp * 2 + turn) * 4 * kN;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float v = warp_max(x[h]);
          if (lane == 0) rm[w4 * kN + h] = v;
        }
        mbar_arrive(&bars->xmax[grp]);
        ok = mbar_wait_warp(&bars->xmax[grp], turn, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        float alpha[GP];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float mt = fmaxf(fmaxf(rm[h], rm[kN + h]), fmaxf(rm[2 * kN + h], rm[3 * kN + h]));
          const float mn = mt > m_run[h] + kRescaleThreshold ? mt : m_run[h];
          const bool ch = mn != m_run[h];
          alpha[h] = ch ? ex2(m_run[h] - mn) : 1.f;   // m_run = -inf gives 0
          grow |= ch;
          m_run[h] = mn;
          x[h] -= mn == -INFINITY ? 0.f : mn;
        }
        uint8_t* pt = sP + st * kPBytes;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float p = ex2(x[h]);   // x = -inf gives 0
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
        // Rescale the group's O^T (lane = d) when a maximum moved after its first tile; the
        // product of its previous tile must have completed.
        if (grow && !first) {
          ok = mbar_wait_warp(&bars->empty[(n - 2) % kStages], ((n - 2) / kStages) & 1, abort_flag,
                              a.err, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          uint32_t ov[16];
          const uint32_t oaddr = lane_base + kO + ((nu & 1) * 2 + grp) * kN;
          tmem_ld16_wait(oaddr, ov);
#pragma unroll
          for (int h = 0; h < GP; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * alpha[h]);
          tmem_st16(oaddr, ov);
          tmem_wait_st();
        }
        first = false;
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_full[st]);
      }
      if (!ok) break;
      // ---- the segment's statistics; then the groups in turn write its result
      float* rl = red_l + (nu & 1) * 2 * 4 * kN;
      float* sm = seg_m + (nu & 1) * 2 * 4 * kN;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        float v = l_run[h];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) rl[(grp * 4 + w4) * kN + h] = v;
        if (r == 0) sm[grp * 4 * kN + h] = m_run[h];
      }
      mbar_arrive(&bars->xsum[nu & 1]);
      if ((nu & 1) == grp) {
        ok = mbar_wait_warp(&bars->xsum[nu & 1], (nu >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        ok = mbar_wait_warp(&bars->o_full[nu & 1], (nu >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t o0[16], o1[16];
        tmem_ld16_wait(lane_base + kO + (nu & 1) * 2 * kN, o0);
        tmem_ld16_wait(lane_base + kO + ((nu & 1) * 2 + 1) * kN, o1);
        tc_fence_before();
        const int slot = sched::slot(sg.pair_start, start.first, blockIdx.x);
        float* out = a.part + static_cast<size_t>(slot) * G * kPStride;
        const size_t head0 = static_cast<size_t>(sg.b) * a.Hq + sg.head * G;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          if (h >= G) break;
          float l[2], w[2];
          const float m0 = sm[h], m1 = sm[4 * kN + h], M = fmaxf(m0, m1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* li = rl + i * 4 * kN + h;
            l[i] = li[0] + li[kN] + li[2 * kN] + li[3 * kN];
            w[i] = ex2((i ? m1 : m0) - (M == -INFINITY ? 0.f : M));   // -inf gives 0
          }
          const float lt = l[0] * w[0] + l[1] * w[1];
          // A group without a tile has left its O^T as it was.
          const float oh = (w[0] > 0.f ? __uint_as_float(o0[h]) * w[0] : 0.f) +
                           (w[1] > 0.f ? __uint_as_float(o1[h]) * w[1] : 0.f);
          if (sg.whole) {
            if (r < D) a.o[(head0 + h) * D + r] = __float2bfloat16_rn(lt == 0.f ? 0.f : oh / lt);
            if (r == 0) a.lse[head0 + h] = lt == 0.f ? -INFINITY : (M + __log2f(lt)) * kLn2;
          } else {
            if (r < D) out[h * kPStride + r] = oh;
            if (r == 0) {
              out[h * kPStride + D] = M;
              out[h * kPStride + D + 1] = lt;
            }
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
    tmem_dealloc(tb, 256);
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
