// Absorbed latent decode over a paged latent cache: one new query token per sequence, up to
// 128 heads that all read the sequence's one latent row a token.
//
// More than 16 heads; fa_latent_decode_few.cu has the others.
//
// Mathematics.  A cached row is (c, r), c the latent vector (512) that stands for keys and
// values of every head and r the rotated key part (64) the heads share.  With the key
// up-projection absorbed into the query, s_hj = scale q_h . (c_j, r_j) over 576 columns and
// o_h = softmax(s_h) c over the first 512; the value up-projection is left to the caller.
// One pass with a running maximum and sum per head (log2 domain); parts join as in
// fa_decode_paged.cu.  Everything but the operands of the two products is fp32; P is rounded
// once to bf16 as the operand of P V.
//
// What bounds it: a token costs 1152 bytes and 2176 H operations, so H = 128 asks for 242
// operations a byte, near the card's 295: HBM and the tensor cores are both close, and few
// heads leave HBM alone.  All heads of a sequence are the M = 128 rows of one tile (rows past H
// compute what is never read), so a cached row is read once for all of them.
//
// Tensor memory sets the layout: O for 128 heads x 512 columns would fill all of it.  Two CTAs
// share a worker's keys, each forms the scores of all 576 columns and keeps O for its own half
// of the 512: 1.53 times the operations, but no exchange between the two.  512 columns then hold
// O (256), one score tile of 128 keys (128, P overwrites S as bf16) and the own half's 256
// columns of Q (128, the A operand of 16 of the 36 score steps); the other 320 columns of Q stay
// in shared memory (80 KB).  A score tile of 128 keys and not two of 64: an MMA takes the pipe
// and its issuer 70 to 130 cycles here whether N is 64 or 128 (traced: 3950 cycles of scores a
// 64-key tile), so half as many of them beat the overlap that two tiles would give.
//
// A tile of 128 keys is 144 KB, all that is left of shared memory.  Only the own half (64 KB)
// has to stay until P V; the other 80 KB are refilled as soon as their score MMAs have run, behind
// the rest of the tile's work, so the next tile's are there when its scores begin, and the own
// half, fetched behind P V (from L2: the other CTA has had it), when they get to it.  One barrier
// for the 80 KB: a wait and a commit between four MMAs cost as much as the four.
//   warp 0     producer: Q, then the tiles page by page;  warp 1  MMA issuer (one thread);
//   warp 2     tensor memory;                             warps 4-11 softmax, a row in 4 threads.
// Measured: 32 sequences of 4096 to 8192 tokens, 128 heads: 78 us for 35 us of bytes (L2 serves the
// other CTA of the pair).  A tile takes 5k cycles, of which the pipe runs 3.4k: the rest's scores
// 1445, the own half's 950, the softmax 1070 between them and P V; joining the parts adds 8 us.
// Work is shared out as fa_paged_sched.cuh says, over pairs of CTAs.  Every wait is bounded; on
// expiry the CTA records FA_ERR_TIMEOUT and leaves.
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <math.h>

#include "fa_internal.cuh"
#include "fa_latent_decode.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;
using sched::Segment;

constexpr int kRank = FA_LATENT_RANK, kRow = FA_LATENT_RANK + FA_LATENT_ROPE;
constexpr int kHeads = 128;                   // rows of a tile
constexpr int kKeys = 128;                    // keys per tile
constexpr int kSub = kKeys * 128;             // [128 keys][64 columns], 16 KB
constexpr int kHalf = kRank / 2;              // columns of O per CTA
constexpr int kOwnSubs = kHalf / 64;          // subtiles of the own half
constexpr int kOwn = kOwnSubs * kSub;
constexpr int kRestSubs = kRow / 64 - kOwnSubs;   // the other half's, then the rotated part's
constexpr int kQSub = kHeads * 128;           // [128 heads][64 columns], 16 KB
constexpr int kThreads = 384;
constexpr uint32_t kTS = kHalf, kTQ = kHalf + kKeys;       // columns of S and of Q's own half
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units; exact, see fa_fwd_sm103.cu

struct Bars {
  uint64_t own_full;
  uint64_t own_empty;   // P V of a tile has completed
  uint64_t rest_full;
  uint64_t rest_empty;  // the rest's score products of a tile have completed
  uint64_t q_full;      // Q's columns of the rest have landed in shared memory
  uint64_t q_own;       // Q's own half is in tensor memory
  uint64_t q_empty;     // every score product of the segment has completed
  uint64_t s_full;
  uint64_t p_full[2];   // of each half of the tile's keys
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t seen[2];  // bit i: rows 16 i ... 16 i + 15 of the tile are in the pool
  int abort;
  int never;  // stays 0: the drain wait must not be cut short by an abort
};

constexpr int kSmem = 1024 + kRestSubs * kQSub + kOwn + kRestSubs * kSub +
                      static_cast<int>(sizeof(Bars));
static_assert(kSmem <= 226 * 1024, "shared memory");

template <int LINES>
__device__ __forceinline__ void prefetch_l2(const __nv_bfloat16* p) {   // LINES lines of 128 bytes
#pragma unroll
  for (int i = 0; i < LINES; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 64 * i));
}

__global__ void __launch_bounds__(kThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mq,
                     LatentArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                        // [kRestSubs][128 heads][64]
  uint8_t* sOwn = sQ + kRestSubs * kQSub;    // [kOwnSubs][128 keys][64]
  uint8_t* sRest = sOwn + kOwn;             // [kRestSubs][128 keys][64]
  Bars* bars = reinterpret_cast<Bars*>(sRest + kRestSubs * kSub);
  __shared__ sched::Start start;
  __shared__ long long scan[kThreads / 32 + 1];
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x & 1, worker = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const int cap = a.max_pages << a.page_shift;
  // First column of the i-th subtile of the rest: the other half's, then the rotated part's.
  auto rest_col = [&](int i) { return i < kOwnSubs ? (1 - half) * kHalf + 64 * i : kRank; };

  if (tid == 0) {
    mbar_init(&bars->own_full, 1);
    mbar_init(&bars->own_empty, 1);
    mbar_init(&bars->rest_full, 1);
    mbar_init(&bars->rest_empty, 1);
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_own, 256);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->p_full[0], 256);
    mbar_init(&bars->p_full[1], 256);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->never = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mc);
    tma_prefetch_desc(&mq);
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  sched::find_start<kKeys, kThreads>(&start, scan, a.cache_len, a.B, 1, cap, worker, workers,
                                        blockIdx.x == 0 ? a.prefix : nullptr);
  const uint32_t tb = bars->tmem_base;
  sched::Walk<kKeys> walk(start, a.cache_len, 1, cap);
  Segment sg;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const int shift = a.page_shift;
    const int rows = min(kKeys, 1 << shift);        // rows of a box
    const int boxes = kKeys / rows;
    const uint32_t bits = (1u << (rows / 16)) - 1u; // of a box in the tile's row mask
    bool ok = true;
    int n = 0, nu = 0;                              // tiles, segments so far
    while (ok && walk.next(sg)) {
      if (nu > 0) {
        ok = mbar_wait_warp(&bars->q_empty, (nu - 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, kRestSubs * kQSub);
        for (int s = 0; s < kRestSubs; ++s)
          tma_load_3d(sQ + s * kQSub, &mq, &bars->q_full, rest_col(s), sg.b * a.H, 0);
      }
      const int32_t* row = a.table + sg.b * a.table_stride;
      for (int k0 = sg.k0; ok && k0 < sg.k1; k0 += kKeys, ++n) {
        const int x = k0 + lane * rows;             // first token of box `lane`
        int p = -1;
        if (lane < boxes && x < sg.len) p = row[x >> shift];
        const bool in = p >= 0 && p < a.num_pages;
        const uint32_t pages = __ballot_sync(0xffffffffu, in);
        const uint32_t bytes = static_cast<uint32_t>(__popc(pages)) * rows * 128;  // a subtile's
        const int in_page = (1 << shift) - 1;
        if (lane == 0) {
          uint32_t seen = 0;
          for (int i = 0; i < boxes; ++i)
            if (pages >> i & 1u) seen |= bits << (i * (rows / 16));
          bars->seen[n & 1] = seen;                 // released with own_full below
        }
        ok = mbar_wait_warp(&bars->rest_empty, (n & 1) ^ 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars->rest_full, kRestSubs * bytes);
        __syncwarp();
        if (in) {
#pragma unroll
          for (int i = 0; i < kRestSubs; ++i)
            tma_load_4d(sRest + i * kSub + lane * rows * 128, &mc, &bars->rest_full, rest_col(i),
                        x & in_page, 0, p);
        }
        ok = mbar_wait_warp(&bars->own_empty, (n & 1) ^ 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars->own_full, kOwnSubs * bytes);
        __syncwarp();
        // Box lane / 4, subtile lane % 4 of the own half.
        const int box = lane >> 2, s = lane & 3;
        const int pb = __shfl_sync(0xffffffffu, p, box);
        if (box < boxes && (pages >> box & 1u))
          tma_load_4d(sOwn + s * kSub + box * rows * 128, &mc, &bars->own_full,
                      half * kHalf + 64 * s, (k0 + box * rows) & in_page, 0, pb);
      }
      ++nu;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, kKeys, false, false);
      constexpr uint32_t idO = idesc_bf16(128, kHalf, false, true);
      const uint64_t dQ = sw128_desc(smem_u32(sQ), 16, 1024);
      const uint64_t dRest = sw128_desc(smem_u32(sRest), 16, 1024);
      const uint64_t dOwn = sw128_desc(smem_u32(sOwn), 16, 1024);     // own half, K-major
      const uint64_t dV = sw128_desc(smem_u32(sOwn), kSub, 1024);     // the same, along the keys
      const uint32_t tS = tb + kTS;
      bool ok = true;
      int n = 0, nu = 0;
      while (ok && walk.next(sg)) {
        ok = mbar_wait(&bars->q_full, nu & 1, abort_flag, a.err, a.wait_ns) &&
             mbar_wait(&bars->q_own, nu & 1, abort_flag, a.err, a.wait_ns);
        for (int k0 = sg.k0; ok && k0 < sg.k1; k0 += kKeys, ++n) {
          ok = mbar_wait(&bars->rest_full, n & 1, abort_flag, a.err, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kRestSubs; ++i) {
            uint64_t da[4], db[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              da[k] = dQ + static_cast<uint64_t>((i * kQSub + k * 32) >> 4);
              db[k] = dRest + static_cast<uint64_t>((i * kSub + k * 32) >> 4);
            }
            mma_ss_x4(tS, da, db, idS, i > 0 ? 1u : 0u);
          }
          mma_commit(&bars->rest_empty);
          ok = mbar_wait(&bars->own_full, n & 1, abort_flag, a.err, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kOwnSubs; ++g) {
            uint32_t ta[4];
            uint64_t db[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ta[k] = tb + kTQ + 8 * (4 * g + k);
              db[k] = dOwn + static_cast<uint64_t>((g * kSub + k * 32) >> 4);
            }
            mma_ts_x4(tS, ta, db, idS, 1u);
          }
          mma_commit(&bars->s_full);
          if (k0 + kKeys >= sg.k1) mma_commit(&bars->q_empty);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            ok = ok && mbar_wait(&bars->p_full[g], n & 1, abort_flag, a.err, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            uint32_t ta[4];
            uint64_t db[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ta[k] = tS + 8 * (4 * g + k);
              db[k] = dV + static_cast<uint64_t>((2048 * (4 * g + k)) >> 4);
            }
            mma_ts_x4(tb, ta, db, idO, (k0 > sg.k0 || g > 0) ? 1u : 0u);
          }
          if (!ok) break;
          mma_commit(&bars->own_empty);
        }
        ++nu;
      }
      // Every MMA issued has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, a.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    // Warp 4 + q + 4h owns heads 32q + 16h + [0, 16) through the 16-lane shapes: thread t holds
    // heads A = 32q + 16h + t/4 and B = A + 8, keys 8c + 2(t%4) + {0, 1} for c = 0..15.
    const int q4 = warp & 3, hh = (warp - 4) >> 2, t4 = lane & 3;
    const int rA = 32 * q4 + 16 * hh + (lane >> 2), rB = rA + 8;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * q4 + 16 * hh) << 16);
    const uint64_t c2 = f2_pack(a.c, a.c);
    // The own half of the segment's queries into tensor memory: this warp's 16 rows, four threads
    // to 32 bytes of a row (a row per thread touches four times the lines a load: 83 us for 79 us
    // at 32 x 128 heads).  The score products of the segment before have completed: this warp has
    // read the last of them.
    auto write_q = [&](const Segment& s) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q) +
                            (static_cast<size_t>(s.b) * a.H * kRow + half * kHalf) / 2 + 2 * t4;
      uint32_t w[64];
#pragma unroll
      for (int cc = 0; cc < 16; ++cc) {
        uint2 x = make_uint2(0u, 0u), y = x;
        if (rA < a.H) x = *reinterpret_cast<const uint2*>(src + rA * (kRow / 2) + 8 * cc);
        if (rB < a.H) y = *reinterpret_cast<const uint2*>(src + rB * (kRow / 2) + 8 * cc);
        w[4 * cc] = x.x;
        w[4 * cc + 1] = x.y;
        w[4 * cc + 2] = y.x;
        w[4 * cc + 3] = y.y;
      }
      tmem_st_16x256b_x16(lane_base + kTQ, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->q_own);
    };
    bool ok = true;
    int n = 0;
    bool have = walk.next(sg);
    if (have) write_q(sg);
    while (ok && have) {
      Segment nx;
      const bool more = walk.next(nx);
      if (more && 32 * q4 + lane < a.H)   // the next segment's queries into L2 meanwhile
        prefetch_l2<5>(a.q + (static_cast<size_t>(nx.b) * a.H + 32 * q4 + lane) * kRow + 256 * hh);
      float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        // The own half has landed (its MMAs wait for it too); the wait orders the row mask.
        ok = mbar_wait_warp(&bars->own_full, n & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        const uint32_t seen = bars->seen[n & 1];
        const int valid = sg.k1 - k0;
        ok = mbar_wait_warp(&bars->s_full, n & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[64];
        tmem_ld_16x256b_x16_wait(lane_base + kTS, v);
        float sv[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) sv[i] = __uint_as_float(v[i]);
        if (valid < kKeys || seen != 0xffu) {
#pragma unroll
          for (int cc = 0; cc < 16; ++cc) {
            const int key = 8 * cc + 2 * t4;
            const bool page = (seen >> (cc >> 1)) & 1u;
            if (!page || key >= valid) sv[4 * cc] = sv[4 * cc + 2] = -INFINITY;
            if (!page || key + 1 >= valid) sv[4 * cc + 1] = sv[4 * cc + 3] = -INFINITY;
          }
          // Hidden rows: zero the values this CTA multiplies, so that 0 x (anything) stays 0.
          const int row = (tid - 128) & 127, s0 = (tid - 128) >> 7;
          if (row >= valid || !((seen >> (row >> 4)) & 1u)) {
            uint8_t* vt = sOwn + s0 * 2 * kSub + row * 128;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(vt + s * kSub + ch * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        float ma0 = fmaxf(sv[0], sv[1]), ma1 = fmaxf(sv[4], sv[5]);
        float mb0 = fmaxf(sv[2], sv[3]), mb1 = fmaxf(sv[6], sv[7]);
#pragma unroll
        for (int cc = 2; cc < 16; cc += 2) {
          ma0 = fmax3(ma0, sv[4 * cc], sv[4 * cc + 1]);
          mb0 = fmax3(mb0, sv[4 * cc + 2], sv[4 * cc + 3]);
          ma1 = fmax3(ma1, sv[4 * cc + 4], sv[4 * cc + 5]);
          mb1 = fmax3(mb1, sv[4 * cc + 6], sv[4 * cc + 7]);
        }
        float tA = fmaxf(ma0, ma1) * a.c, tB = fmaxf(mb0, mb1) * a.c;
        // As in fa_latent_fwd.cu: rows' maxima only where one passes the running reference.
        float alphaA = 1.f, alphaB = 1.f;
        const bool grew = __any_sync(0xffffffffu, tA > mA + kRescaleThreshold ||
                                                      tB > mB + kRescaleThreshold);
        if (grew) {
          tA = fmaxf(tA, __shfl_xor_sync(0xffffffffu, tA, 1));
          tB = fmaxf(tB, __shfl_xor_sync(0xffffffffu, tB, 1));
          tA = fmaxf(tA, __shfl_xor_sync(0xffffffffu, tA, 2));
          tB = fmaxf(tB, __shfl_xor_sync(0xffffffffu, tB, 2));
          if (tA > mA + kRescaleThreshold) {
            alphaA = ex2(mA - tA);   // m = -inf gives 0
            mA = tA;
          }
          if (tB > mB + kRescaleThreshold) {
            alphaB = ex2(mB - tB);
            mB = tB;
          }
        }
        const float useA = mA == -INFINITY ? 0.f : mA, useB = mB == -INFINITY ? 0.f : mB;
        const uint64_t negA = f2_pack(-useA, -useA), negB = f2_pack(-useB, -useB);
        // Rescale the running O when a maximum moved after the first tile: its products were
        // issued before these scores, so they have completed.
        if (k0 > sg.k0 && grew) {
#pragma unroll 1
          for (int i = 0; i < kHalf / 64; ++i) {
            uint32_t o[32];
            tmem_ld_16x256b_x8_wait(lane_base + 64 * i, o);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint(__uint_as_float(o[k]) * ((k & 2) ? alphaB : alphaA));
            tmem_st_16x256b_x8(lane_base + 64 * i, o);
          }
        }
        // P over the first 64 columns of S in this warp's 16 lanes, which no other warp reads; the
        // product starts on each half of the keys as it comes.
        uint64_t accA = f2_pack(0.f, 0.f), accB = accA;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* x = sv + 4 * (8 * g + i);
            const float2 xa = f2_unpack(ffma2(f2_pack(x[0], x[1]), c2, negA));
            const float2 xb = f2_unpack(ffma2(f2_pack(x[2], x[3]), c2, negB));
            const float pa0 = ex2(xa.x), pa1 = ex2(xa.y);
            const float pb0 = ex2(xb.x), pb1 = ex2(xb.y);
            accA = fadd2(accA, f2_pack(pa0, pa1));
            accB = fadd2(accB, f2_pack(pb0, pb1));
            pk[2 * i] = pack_bf16x2(pa0, pa1);
            pk[2 * i + 1] = pack_bf16x2(pb0, pb1);
          }
          tmem_st_16x128b_x8(lane_base + kTS + 32 * g, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[g]);
        }
        const float2 sa = f2_unpack(accA), sb = f2_unpack(accB);
        lA = lA * alphaA + (sa.x + sa.y);
        lB = lB * alphaB + (sb.x + sb.y);
      }
      if (!ok) break;
      // The next segment's queries first: the issuer's next scores wait for them.
      have = more;
      if (have) write_q(nx);
      ok = mbar_wait_warp(&bars->own_empty, (n - 1) & 1, abort_flag, a.err, a.wait_ns);
      if (!ok) break;
      tc_fence_after();
      lA += __shfl_xor_sync(0xffffffffu, lA, 1);
      lB += __shfl_xor_sync(0xffffffffu, lB, 1);
      lA += __shfl_xor_sync(0xffffffffu, lA, 2);
      lB += __shfl_xor_sync(0xffffffffu, lB, 2);
      const float invA = lA == 0.f ? 0.f : 1.f / lA;        // a NaN sum stays one
      const float invB = lB == 0.f ? 0.f : 1.f / lB;
      const size_t head0 = static_cast<size_t>(sg.b) * a.H;
      const int slot = sched::slot(sg.pair_start, start.first, worker);
      const size_t prow0 = static_cast<size_t>(slot) * a.H;
#pragma unroll 1
      for (int i = 0; i < kHalf / 64; ++i) {
        uint32_t ov[32];
        __syncwarp();
        tmem_ld_16x256b_x8_wait(lane_base + 64 * i, ov);
        const int col = half * kHalf + 64 * i + 2 * t4;
#pragma unroll
        for (int ab = 0; ab < 2; ++ab) {
          const int r = ab ? rB : rA;
          const float inv = ab ? invB : invA;
          if (r >= a.H) continue;
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {
            const float x0 = __uint_as_float(ov[4 * cc + 2 * ab]);
            const float x1 = __uint_as_float(ov[4 * cc + 2 * ab + 1]);
            if (sg.whole)
              *reinterpret_cast<uint32_t*>(a.o + (head0 + r) * kRank + col + 8 * cc) =
                  pack_bf16x2(x0 * inv, x1 * inv);
            else
              *reinterpret_cast<float2*>(a.part + (prow0 + r) * kRank + col + 8 * cc) =
                  make_float2(x0, x1);
          }
        }
      }
      tc_fence_before();
      if (t4 == 0) {
#pragma unroll
        for (int ab = 0; ab < 2; ++ab) {
          const int r = ab ? rB : rA;
          const float m = ab ? mB : mA, l = ab ? lB : lA;
          if (r >= a.H) continue;
          if (!sg.whole)
            a.stat[(static_cast<size_t>(slot) * 2 + half) * a.H + r] = make_float2(m, l);
          else if (half == 0)
            a.lse[head0 + r] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
        }
      }
      sg = nx;
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
    tmem_dealloc(tb, 512);
  }
}

// Joins the parts of a sequence that more than one worker had; o = 0, lse = -inf for an empty
// sequence.  A warp adds a quarter of the columns (four a lane) of HEADS heads.  Each half of the
// columns has statistics of its own (its CTAs add the score products in another order), which
// every warp reads for itself, a part in a lane: no barrier.  What it costs is a chain of loads
// (prefix, statistics, rows), so the rows of the first parts are asked for with the statistics.
//   GROUPS = 1  block = the four quarters of HEADS heads of a sequence;
//   GROUPS > 1  block = one quarter of one head, each warp with its share of the parts.
template <int GROUPS, int HEADS>
__global__ void __launch_bounds__(GROUPS == 1 ? 128 : 32 * GROUPS)
latent_combine_kernel(LatentArgs a, int workers) {
  static_assert(GROUPS == 1 || HEADS == 1, "a block's share");
  constexpr int kAhead = GROUPS == 1 ? 4 : 8;
  __shared__ float4 rows[GROUPS][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = GROUPS == 1 ? 0 : warp, quarter = GROUPS == 1 ? warp : blockIdx.x & 3;
  const int hc = quarter >> 1, col = 32 * quarter + lane;   // columns 4 col ... of half hc
  const int per = (a.H + HEADS - 1) / HEADS, unit = GROUPS == 1 ? blockIdx.x : blockIdx.x >> 2;
  const int b = unit / per, h0 = unit % per * HEADS, heads = min(HEADS, a.H - h0);
  const size_t head0 = static_cast<size_t>(b) * a.H + h0;
  const long long p0 = a.prefix[b], p1 = a.prefix[b + 1], total = a.prefix[a.B];
  if (p0 == p1) {
    for (int k = 0; k < heads; ++k) {
      if (g == 0)
        reinterpret_cast<uint2*>(a.o + (head0 + k) * kRank)[col] = make_uint2(0u, 0u);
      if (g == 0 && col == 0) a.lse[head0 + k] = -INFINITY;
    }
    return;
  }
  workers = sched::active(total, workers);
  const int w0 = sched::owner(p0, total, workers);
  const int parts = sched::owner(p1 - 1, total, workers) - w0 + 1;
  if (parts == 1) return;   // finished by its CTAs
  // Only the first part can sit in the second of its worker's slots.
  const int slot0 = sched::slot(p0, sched::range_start(total, w0, workers), w0);
  auto slot = [&](int i) { return i == 0 ? slot0 : 2 * (w0 + i); };
  auto row = [&](int i, int k) {
    return reinterpret_cast<const float4*>(a.part + (static_cast<size_t>(slot(i)) * a.H + h0 + k) *
                                                        kRank)[col];
  };
  auto stat = [&](int i, int k) {
    return i < parts ? a.stat[(static_cast<size_t>(slot(i)) * 2 + hc) * a.H + h0 + k]
                     : make_float2(-INFINITY, 0.f);
  };
  const int i0 = parts * g / GROUPS, i1 = parts * (g + 1) / GROUPS;
  float4 first[HEADS][kAhead];
  float2 own[HEADS];
#pragma unroll
  for (int k = 0; k < HEADS; ++k) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      first[k][i] = k < heads && i0 + i < i1 ? row(i0 + i, k) : make_float4(0.f, 0.f, 0.f, 0.f);
    own[k] = k < heads ? stat(lane, k) : make_float2(-INFINITY, 0.f);
  }
#pragma unroll
  for (int k = 0; k < HEADS; ++k) {
    if (k >= heads) break;
    float M = own[k].x;
    for (int i = 32; i < parts; i += 32) M = fmaxf(M, stat(i + lane, k).x);
    M = warp_max(M);
    if (M == -INFINITY) M = 0.f;
    float l = own[k].y * ex2(own[k].x - M);   // a part without a visible key (-inf) weighs 0
    for (int i = 32; i < parts; i += 32) {
      const float2 s = stat(i + lane, k);
      l += s.y * ex2(s.x - M);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& v) {
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    };
    for (int c = i0; c < i1; c += 32) {   // the weights of 32 parts, one in a lane
      const float w = ex2(stat(c + lane, k).x - M);
      const int n = min(32, i1 - c);
      int i = 0;
      if (c == i0) {
#pragma unroll
        for (; i < kAhead; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
          if (i < n) add(wi, first[k][i]);
        }
      }
#pragma unroll 4
      for (; i < n; ++i) add(__shfl_sync(0xffffffffu, w, i), row(c + i, k));
    }
    if constexpr (GROUPS > 1) {
      rows[g][lane] = acc;
      __syncthreads();
      if (g > 0) return;
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) add(1.f, rows[i][lane]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;   // a NaN sum stays one
    reinterpret_cast<uint2*>(a.o + (head0 + k) * kRank)[col] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (col == 0) a.lse[head0 + k] = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
  }
}

// Up to 16 heads leave the tensor cores idle here (M = 128) and fit one tile of the warp-level MMA:
// 57 us in fa_latent_decode_few.cu, 69 us here at 16 heads (32 sequences of 4096 to 8192); 17 heads
// would take two such tiles, whose registers there are not.
bool few_heads(int H) { return H <= kFewHeads; }

// Workers, and with it two parts' room each: pairs of CTAs, or CTAs.
int max_workers(int H) { return few_heads(H) ? sm_count() : sm_count() / 2; }

size_t part_bytes(int H) {
  return 2 * static_cast<size_t>(max_workers(H)) * H * kRank * sizeof(float);
}
size_t stat_bytes(int H) {
  return round_up(2 * static_cast<size_t>(max_workers(H)) * 2 * H * sizeof(float2), 256);
}

}  // namespace

size_t latent_decode_bytes(int B, int H) {
  return part_bytes(H) + stat_bytes(H) + (static_cast<size_t>(B) + 1) * sizeof(long long);
}

cudaError_t launch_latent_decode(const void* q, const void* cache, long long page_stride,
                                 const int32_t* table, long long table_stride, int max_pages,
                                 int page_shift, int num_pages, const int32_t* cache_len, void* o,
                                 float* lse, int B, int H, float scale, void* workspace, int* err,
                                 unsigned long long wait_ns, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  LatentArgs a{static_cast<const __nv_bfloat16*>(q), table, table_stride, max_pages, page_shift,
               num_pages, cache_len, B, H, scale * kLog2e, static_cast<__nv_bfloat16*>(o), lse,
               reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + part_bytes(H)),
               reinterpret_cast<long long*>(ws + part_bytes(H) + stat_bytes(H)), err, wait_ns};
  // No more workers than there can be tiles.
  const int keys = few_heads(H) ? kFewKeys : kKeys;
  const long long most = static_cast<long long>(B) *
                         (((static_cast<long long>(max_pages) << page_shift) + keys - 1) / keys);
  const int workers = static_cast<int>(std::min<long long>(most, max_workers(H)));
  CUtensorMap mc, mq;
  const int page = 1 << page_shift;
  if (!make_page_map(&mc, cache, num_pages, 1, page, kRow, page_stride, page < keys ? page : keys))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (few_heads(H)) {
    e = launch_latent_decode_few(mc, a, workers, s);
  } else {
    if (!make_head_map_rows(&mq, q, 1, B * H, kRow, kHeads)) return cudaErrorInvalidValue;
    static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
      e = cudaFuncSetAttribute(latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) attr_set[dev].store(true);
    }
    e = launch_dependent(latent_decode_kernel, dim3(2 * workers), dim3(kThreads), kSmem, s, mc, mq,
                         a);
  }
  if (e != cudaSuccess) return e;
  // Warps to a row by the parts of an average sequence: every block costs a chain of loads, so more
  // of them only pay where a warp's own sum would be longer (1 x 16 heads, 152 parts: 16, 8, 4 warps
  // 18.9, 21.6, 24.4 us; 1 x 128, 76 parts: 26.4, 23.0, 24.2; 2 x 128, 38 parts: 8, 4 warps 24.6,
  // 22.2; 4 x 128, 19 parts: 4, 1 warps 30.3, 33.5; 8 x 128, 9 parts, many rows: 41, 37.5).
  const unsigned rows = static_cast<unsigned>(B) * H;
  const int parts = workers / B;
  auto combine = [&](auto kernel, unsigned blocks, unsigned threads) {
    return launch_dependent(kernel, dim3(blocks), dim3(threads), 0, s, a, workers);
  };
  if (parts >= 128) return combine(latent_combine_kernel<16, 1>, 4 * rows, 512);
  if (parts >= 64) return combine(latent_combine_kernel<8, 1>, 4 * rows, 256);
  if (parts >= 8 && rows <= 512) return combine(latent_combine_kernel<4, 1>, 4 * rows, 128);
  return combine(latent_combine_kernel<1, 2>, static_cast<unsigned>(B) * ((H + 1) / 2), 128);
}

}  // namespace fa
