// What the decode kernels over a paged cache have in common: a CTA that walks segments of (sequence,
// key/value head) pairs, tile by tile, keys as the rows of the tensor cores' products.  Its
// mathematics and its layout are described where it is launched from (fa_decode_paged.cu).
//
// Walk yields the CTA's segments in order (every role has a copy): next(Segment&) -> bool.  A
// segment's keys are tokens [k0, k1) of the sequence, k0 a multiple of a box's rows; one that is
// `whole` is all that its rows attend to and becomes their output, the others leave partial results
// (unnormalised o, maximum, sum) in place `slot`.
#pragma once

#include <cuda.h>
#include <math.h>

#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace decode {

using namespace ptx;

struct Segment : sched::Segment {
  int slot;                // place of its partial result
};

constexpr int kKeys = 128;                    // keys per tile
// Most keys of a TMA box, so of what a sequence's last box loads in vain (pages of 256, sequences of up
// to 2000 tokens: 51.1 us; boxes of 128 keys 53.1, of 64 52.0).
constexpr int kBox = 32;
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

// A CTA's shared memory, from a 1024-byte boundary on.
template <int D>
struct Smem {
  uint8_t *sKV, *sQ, *sP;              // [STAGES][K subtiles, V subtiles], [2][QBYTES], [STAGES][kPBytes]
  // A group's exchange of maxima: [2 groups][2][4 warps][16 heads]; a segment's statistics:
  // [2 segments][2 groups][4 warps: sums][16 heads], then the same of maxima (one row used).
  float *red_m, *red_l, *seg_m;
  Bars* bars;
  __device__ __forceinline__ explicit Smem(uint8_t* base) {
    using C = TC<D>;
    sKV = base;
    sQ = sKV + C::STAGES * C::STAGE;
    sP = sQ + 2 * C::QBYTES;
    red_m = reinterpret_cast<float*>(sP + C::STAGES * kPBytes);
    red_l = red_m + 2 * 2 * 4 * kN;
    seg_m = red_l + 2 * 2 * 4 * kN;
    bars = reinterpret_cast<Bars*>(seg_m + 2 * 2 * 4 * kN);
  }
};

// By one thread, before the block's barrier.
template <int D>
__device__ __forceinline__ void init_bars(Bars* bars) {
  for (int s = 0; s < TC<D>::STAGES; ++s) {
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

// Columns of tensor memory from tb on.
constexpr int kDecodeColumns = 256;

// The roles of the CTA's warps.  GP: query heads per key/value head rounded up to a power of two.
template <int D, int GP, class Walk>
__device__ __forceinline__ void segments(const CUtensorMap& mk, const CUtensorMap& mv,
                                         const CUtensorMap& mq, const PagedArgs& a,
                                         const Smem<D>& sh, uint32_t tb, Walk walk) {
  using C = TC<D>;
  constexpr int kStages = C::STAGES, kStage = C::STAGE, kQBytes = C::QBYTES;
  constexpr int kPStride = C::PSTRIDE;
  uint8_t *sKV = sh.sKV, *sQ = sh.sQ, *sP = sh.sP;
  float *red_m = sh.red_m, *red_l = sh.red_l, *seg_m = sh.seg_m;
  Bars* bars = sh.bars;
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  Segment sg;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    // Warp 0 has the queries and the keys, warp 2 the values: one warp issues a box in some 70
    // cycles, and small pages make many.  Lane i < boxes takes the i-th box of every tile.
    const bool keys = warp == 0;
    const CUtensorMap* map = keys ? &mk : &mv;
    const int shift = a.page_shift;
    const int rows = min(kBox, 1 << shift);         // rows of a box
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
          // every lane from another 16 bytes on: all at the same would be the same banks (sequences of
          // up to 256 tokens, B = 256: 63 us, so 50)
          uint8_t* vt = sKV + st * kStage + C::NSUB * kSub + r * 128;
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<uint4*>(vt + s * kSub + ((ch + lane) & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
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
        float* out = a.part + static_cast<size_t>(sg.slot) * G * kPStride;
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
}

}  // namespace decode
}  // namespace fa
