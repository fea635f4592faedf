// Absorbed latent decode over a paged latent cache: one new query token per sequence, up to
// 128 heads that all read the sequence's one latent row a token.
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
// heads leave HBM alone.  All heads of a sequence are therefore the M = 128 rows of one tile
// (rows past H compute what is never read), so a cached row is read once for all of them.
//
// Tensor memory sets the layout: O for 128 heads x 512 columns would fill all of it.  Two CTAs
// share a worker's keys, each forms the scores of all 576 columns and keeps O for one half of
// the 512: 1.53 times the operations, but no exchange between the two.  512 columns then hold
// O (256), two score tiles of 64 keys (128, P overwrites S as bf16) and the last 256 columns
// of Q (128, the A operand of 16 of the 36 score steps); the first 320 columns of Q stay in
// shared memory (80 KB) beside two stages of [64 keys][576] (144 KB).
//   warp 0     producer: Q, then K tiles page by page;   warp 1  MMA issuer (one thread);
//   warp 2     tensor memory;                            warps 4-7 softmax, thread = head.
// Scores of tile n + 1 are issued before O += P V of tile n.  Work is shared out as
// fa_paged_sched.cuh says, over pairs of CTAs.  Every wait is bounded; on expiry the CTA
// records FA_ERR_TIMEOUT and leaves.
#include <atomic>

#include <cuda.h>
#include <math.h>

#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;
using sched::Segment;

constexpr int kRank = FA_LATENT_RANK, kRow = FA_LATENT_RANK + FA_LATENT_ROPE;
constexpr int kHeads = 128;                   // rows of a tile
constexpr int kKeys = 64;                     // keys per tile
constexpr int kGranule = 128;                 // keys of the smallest share of the work
constexpr int kStages = 2;
constexpr int kSubs = kRow / 64;              // 64-column subtiles of a row
constexpr int kKSub = kKeys * 128;            // [64 keys][64 columns], 8 KB
constexpr int kStage = kSubs * kKSub;
constexpr int kQSubs = 5;                     // subtiles of Q in shared memory
constexpr int kQSub = kHeads * 128;           // [128 heads][64 columns], 16 KB
constexpr int kHalf = kRank / 2;              // columns of O per CTA
constexpr int kThreads = 256;
constexpr uint32_t kTS = kHalf, kTQ = kHalf + 2 * kKeys;   // columns of S and of Q's rest
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units; exact, see fa_fwd_sm103.cu

struct Bars {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t q_full;      // Q's first columns have landed in shared memory
  uint64_t q_rest;      // Q's last columns are in tensor memory
  uint64_t q_empty;     // every score product of the segment has completed
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t pv_done[2];
  uint64_t o_full;
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t seen[kStages];  // bit i: rows 16 i ... 16 i + 15 of the stage are in the pool
  int abort;
  int never;  // stays 0: the drain wait must not be cut short by an abort
};

constexpr int kSmem = 1024 + kQSubs * kQSub + kStages * kStage + static_cast<int>(sizeof(Bars));
static_assert(kSmem <= 226 * 1024, "shared memory");

struct LatentArgs {
  const __nv_bfloat16* q;  // [B, H, 576]
  const int32_t* table;
  long long table_stride;
  int max_pages, page_shift, num_pages;
  const int32_t* cache_len;
  int B, H;
  float c;                 // scale log2 e
  __nv_bfloat16* o;        // [B, H, 512]
  float* lse;
  float* part;             // [2 workers][2 halves][H][256]
  float2* stat;            // [2 workers][2 halves][H]: maximum, sum
  long long* prefix;       // [B + 1] granules before each sequence
  int* err;
  unsigned long long wait_ns;
};

__global__ void __launch_bounds__(kThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mq,
                     LatentArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                        // [kQSubs][128 heads][64]
  uint8_t* sK = sQ + kQSubs * kQSub;         // [kStages][kSubs][64 keys][64]
  Bars* bars = reinterpret_cast<Bars*>(sK + kStages * kStage);
  __shared__ sched::Start start;
  __shared__ long long scan[kThreads / 32 + 1];
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x & 1, worker = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const int cap = a.max_pages << a.page_shift;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_rest, 128);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 128);
      mbar_init(&bars->pv_done[i], 1);
    }
    mbar_init(&bars->o_full, 1);
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
  sched::find_start<kGranule, kThreads>(&start, scan, a.cache_len, a.B, 1, cap, worker, workers,
                                        blockIdx.x == 0 ? a.prefix : nullptr);
  const uint32_t tb = bars->tmem_base;
  sched::Walk<kGranule> walk(start, a.cache_len, 1, cap);
  Segment sg;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const int shift = a.page_shift;
    const int rows = min(kKeys, 1 << shift);        // rows of a box
    const int boxes = kKeys / rows;
    const uint32_t bits = (1u << (rows / 16)) - 1u; // of a box in the stage's row mask
    bool ok = true;
    int n = 0, nu = 0;
    while (ok && walk.next(sg)) {
      if (nu > 0) {
        ok = mbar_wait_warp(&bars->q_empty, (nu - 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, kQSubs * kQSub);
        for (int s = 0; s < kQSubs; ++s)
          tma_load_3d(sQ + s * kQSub, &mq, &bars->q_full, 64 * s, sg.b * a.H, 0);
      }
      const int32_t* row = a.table + sg.b * a.table_stride;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        const int st = n % kStages;
        const int x = k0 + lane * rows;             // first token of box `lane`
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
                                static_cast<uint32_t>(__popc(pages)) * rows * kRow * 2);
        }
        __syncwarp();
        // Box i / kSubs, subtile i % kSubs, spread over the lanes.
        for (int i0 = 0; i0 < boxes * kSubs; i0 += 32) {
          const int i = i0 + lane, box = i / kSubs, s = i - box * kSubs;
          const int pb = __shfl_sync(0xffffffffu, p, box & 31);
          if (i < boxes * kSubs && (pages >> box & 1u))
            tma_load_4d(sK + st * kStage + s * kKSub + box * rows * 128, &mc, &bars->full[st],
                        64 * s, (k0 + box * rows) & ((1 << shift) - 1), 0, pb);
        }
      }
      ++nu;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, kKeys, false, false);
      constexpr uint32_t idO = idesc_bf16(128, kHalf, false, true);
      bool ok = true;
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
      const uint64_t dQ = sw128_desc(smem_u32(sQ), 16, 1024);
      auto issue_s = [&](const Cur& c, int m) -> bool {
        const int st = m % kStages;
        if (c.t == 0) {
          if (!mbar_wait(&bars->q_full, c.nu & 1, abort_flag, a.err, a.wait_ns)) return false;
          if (!mbar_wait(&bars->q_rest, c.nu & 1, abort_flag, a.err, a.wait_ns)) return false;
        }
        if (!mbar_wait(&bars->full[st], (m / kStages) & 1, abort_flag, a.err, a.wait_ns))
          return false;
        tc_fence_after();
        const uint64_t dK = sw128_desc(smem_u32(sK + st * kStage), 16, 1024);
        const uint32_t tS = tb + kTS + (m & 1) * kKeys;
#pragma unroll
        for (int g = 0; g < kSubs; ++g) {
          uint64_t db[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) db[k] = dK + static_cast<uint64_t>((g * kKSub + k * 32) >> 4);
          if (g < kQSubs) {
            uint64_t da[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              da[k] = dQ + static_cast<uint64_t>((g * kQSub + k * 32) >> 4);
            mma_ss_x4(tS, da, db, idS, g > 0 ? 1u : 0u);
          } else {
            uint32_t ta[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ta[k] = tb + kTQ + 8 * (4 * (g - kQSubs) + k);
            mma_ts_x4(tS, ta, db, idS, 1u);
          }
        }
        mma_commit(&bars->s_full[m & 1]);
        if (c.t == c.nt - 1) mma_commit(&bars->q_empty);
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
        // V: this CTA's four subtiles of the same tile, read along the keys.
        const uint64_t dV = sw128_desc(smem_u32(sK + st * kStage + half * 4 * kKSub), kKSub, 1024);
        uint32_t ta[4];
        uint64_t db[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ta[k] = tb + kTS + (n & 1) * kKeys + 8 * k;
          db[k] = dV + static_cast<uint64_t>((2048 * k) >> 4);
        }
        mma_ts_x4(tb, ta, db, idO, cur.t > 0 ? 1u : 0u);
        mma_commit(&bars->pv_done[n & 1]);
        mma_commit(&bars->empty[st]);
        if (cur.t == cur.nt - 1) mma_commit(&bars->o_full);
        cur = nxt;
        have = have_next;
        ++n;
      }
      // Every MMA issued has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, a.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax (thread = head)
    const int w4 = warp & 3;
    const int r = 32 * w4 + lane;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * w4) << 16);
    // The last 256 columns of the segment's queries into tensor memory.  The score products of
    // the segment before have completed: this warp has read the last of them.
    auto write_q = [&](const Segment& s) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(s.b) * a.H + (r < a.H ? r : 0)) * kRow + kQSubs * 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 x = r < a.H ? src[8 * i + k] : make_uint4(0u, 0u, 0u, 0u);
          w[4 * k] = x.x;
          w[4 * k + 1] = x.y;
          w[4 * k + 2] = x.z;
          w[4 * k + 3] = x.w;
        }
        tmem_st32(lane_base + kTQ + 32 * i, w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->q_rest);
    };
    bool ok = true;
    int n = 0, nu = 0;
    bool have = walk.next(sg);
    if (have) write_q(sg);
    while (ok && have) {
      float m_run = -INFINITY, l_run = 0.f;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        const int st = n % kStages;
        // The stage has landed (its MMAs wait for it too); the wait orders the row mask.
        ok = mbar_wait_warp(&bars->full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        const uint32_t seen = bars->seen[st];
        const int valid = sg.k1 - k0;
        ok = mbar_wait_warp(&bars->s_full[n & 1], (n >> 1) & 1, abort_flag, a.err, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = lane_base + kTS + (n & 1) * kKeys;
        uint32_t sv[64];
        tmem_ld64_wait(tS, tS + 32, sv);
        float x[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = __uint_as_float(sv[i]);
        if (valid < kKeys || seen != 0xfu) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= valid || !((seen >> (i >> 4)) & 1u)) x[i] = -INFINITY;
          // Hidden rows: zero the values this CTA multiplies, so that 0 x (anything) stays 0.
          const int row = r & 63;
          if (row >= valid || !((seen >> (row >> 4)) & 1u)) {
            uint8_t* vt = sK + st * kStage + (half * 4 + (r >> 6) * 2) * kKSub + row * 128;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(vt + s * kKSub + ch * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmax3(mx[j], x[i + 2 * j], x[i + 2 * j + 1]);
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
        const float mn = mt > m_run + kRescaleThreshold ? mt : m_run;
        const bool ch = mn != m_run;
        const float alpha = ch ? ex2(m_run - mn) : 1.f;   // m_run = -inf gives 0
        m_run = mn;
        const float muse = mn == -INFINITY ? 0.f : mn;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = ex2(fmaf(x[2 * i], a.c, -muse));
          const float p1 = ex2(fmaf(x[2 * i + 1], a.c, -muse));
          sum[i & 3] += p0 + p1;
          pk[i] = pack_bf16x2(p0, p1);
        }
        tmem_st32(tS, pk);
        l_run = l_run * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        // Rescale the running O when a maximum moved after the first tile; the product of the
        // previous tile must have completed.
        if (k0 > sg.k0 && __any_sync(0xffffffffu, ch)) {
          ok = mbar_wait_warp(&bars->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.err,
                              a.wait_ns);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < kHalf / 32; ++i) {
            uint32_t ov[32];
            tmem_ld32_wait(lane_base + 32 * i, ov);
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
            tmem_st32(lane_base + 32 * i, ov);
          }
        }
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_full[n & 1]);
      }
      if (!ok) break;
      // The next segment's queries first: the issuer's next scores wait for them.
      Segment nx;
      have = walk.next(nx);
      if (have) write_q(nx);
      ok = mbar_wait_warp(&bars->o_full, nu & 1, abort_flag, a.err, a.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const int slot = 2 * sched::slot(sg.pair_start, start.first, worker) + half;
      const size_t head = static_cast<size_t>(sg.b) * a.H + r;
      const size_t prow = static_cast<size_t>(slot) * a.H + r;
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;   // a NaN sum stays one
#pragma unroll 1
      for (int i = 0; i < kHalf / 32; ++i) {
        uint32_t ov[32];
        __syncwarp();
        tmem_ld32_wait(lane_base + 32 * i, ov);
        if (r < a.H) {
          if (sg.whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + head * kRank + half * kHalf + 32 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack_bf16x2(__uint_as_float(ov[8 * k + 2 * j]) * inv,
                                   __uint_as_float(ov[8 * k + 2 * j + 1]) * inv);
              dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(a.part + prow * kHalf + 32 * i);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
      if (r < a.H) {
        if (!sg.whole)
          a.stat[prow] = make_float2(m_run, l_run);
        else if (half == 0)
          a.lse[head] = l_run == 0.f ? -INFINITY : (m_run + __log2f(l_run)) * kLn2;
      }
      sg = nx;
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
    tmem_dealloc(tb, 512);
  }
}

// One block per (b, h), four columns a thread: joins the parts of a sequence that more than
// one worker had; o = 0, lse = -inf for an empty sequence.
__global__ void __launch_bounds__(128) latent_combine_kernel(LatentArgs a, int workers) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int col = 4 * threadIdx.x, half = col / kHalf;
  const long long p0 = a.prefix[b], p1 = a.prefix[b + 1], total = a.prefix[a.B];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  if (p1 > p0) {
    workers = sched::active(total, workers);
    const int w0 = sched::owner(p0, total, workers), w1 = sched::owner(p1 - 1, total, workers);
    if (w0 == w1) return;   // finished by its CTAs
    auto row = [&](int w) {
      const int slot = 2 * sched::slot(p0, sched::range_start(total, w, workers), w) + half;
      return static_cast<size_t>(slot) * a.H + h;
    };
    for (int w = w0; w <= w1; ++w) M = fmaxf(M, a.stat[row(w)].x);
    if (M == -INFINITY) M = 0.f;
    for (int w = w0; w <= w1; ++w) {
      const size_t i = row(w);
      const float2 s = a.stat[i];
      const float wt = ex2(s.x - M);   // a part without a visible key (-inf) weighs 0
      const float4 v = *reinterpret_cast<const float4*>(a.part + i * kHalf + (col & (kHalf - 1)));
      l += s.y * wt;
      acc.x = fmaf(wt, v.x, acc.x);
      acc.y = fmaf(wt, v.y, acc.y);
      acc.z = fmaf(wt, v.z, acc.z);
      acc.w = fmaf(wt, v.w, acc.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;   // a NaN sum stays one
  const size_t head = blockIdx.x;
  *reinterpret_cast<uint2*>(a.o + head * kRank + col) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (threadIdx.x == 0) a.lse[head] = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
}

int latent_workers() { return sm_count() / 2; }

size_t part_bytes(int H) { return static_cast<size_t>(2 * latent_workers()) * H * kRank * 4; }
size_t stat_bytes(int H) {
  return round_up(static_cast<size_t>(2 * latent_workers()) * 2 * H * sizeof(float2), 256);
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
  CUtensorMap mc, mq;
  const int page = 1 << page_shift;
  if (!make_page_map(&mc, cache, num_pages, 1, page, kRow, page_stride,
                     page < kKeys ? page : kKeys) ||
      !make_head_map_rows(&mq, q, 1, B * H, kRow, kHeads))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  // No more workers than there can be granules.
  const long long most = static_cast<long long>(B) *
                         (((static_cast<long long>(max_pages) << page_shift) + kGranule - 1) / kGranule);
  const int workers = most < latent_workers() ? static_cast<int>(most) : latent_workers();
  cudaError_t e = launch_dependent(latent_decode_kernel, dim3(2 * workers), dim3(kThreads), kSmem,
                                   s, mc, mq, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(latent_combine_kernel, dim3(static_cast<unsigned>(B) * H), dim3(128), 0,
                          s, a, workers);
}

}  // namespace fa
