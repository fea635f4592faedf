// Expanded latent attention, backward, on sm_103a tensor cores (tcgen05 + TMA), bf16 in, fp32
// accumulation.  The formulas stand in fa_latent_simt.cu.
//
// Two kinds of CTAs of one template, without atomics (the result does not depend on scheduling):
//   dK, dV  a CTA owns 128 keys of a head (k, v stay in shared memory) and streams the blocks of
//           128 query rows that may see them:
//             S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q;
//   dQ      a CTA owns 128 query rows (q, dO stay) and streams key blocks of 128:
//             S = Q K^T, dP = dO V^T, dQ += dS K.
// Seven products instead of five (S and dP are formed twice: 1152 columns of MMA a pair against
// 832), because dK (192) + dV (128) + dQ (192) and two score tiles do not fit tensor memory's 512
// columns, and dQ needs no fp32 sums through global memory this way.
//
// What bounds it: the issue and the pipe.  An MMA costs 65 to 90 cycles whether N is 64 or 128, so
// the blocks are 128 wide although tensor memory then holds one score tile at a time: 4.3k (dK, dV)
// + 2.7k (dQ) cycles a 128 x 128 block traced, against 6.4k + 5.2k with 64-wide blocks, two in
// flight.  dK, dV: 2.9k of MMAs and the chain S^T, softmax, dP^T, softmax, dK between them.
//   dK, dV  columns: dV 128, dK 192, one region of 128 for S^T, then dP^T (once the softmax warps
//           have S^T in registers), then dS^T in place; 64 for P^T.
//   dQ      columns: dQ 192, S 128, dP 128 (dS in place), the owned dO 64 as an A operand:
//           S(n + 1) starts as soon as the softmax warps have read S(n).
// Of shared memory the owned rows hold 80 KB (dQ: 48, which makes room for a third stage of X);
// the streamed side X (q or k, 192 columns: scores early, gradient product late) has two or three
// stages of 48 KB and Y (dO or v, 128) one of 32.  Both lie as [128 rows][64 columns] subtiles
// that the score products read K-major and the gradient products MN-major.
//   warp 0 producer; warps 1, 3 MMA issuers; warp 2 tensor memory and (dK, dV) the block's lse and
//   D; warps 4-11 softmax, two threads a row, 64 columns each.
// Every wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and exits.
#include <atomic>

#include <cuda.h>
#include <math.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kRows = 128;              // rows a CTA owns, rows of a streamed block
constexpr int kXSubs = (FA_LATENT_NOPE + FA_LATENT_ROPE) / 64, kYSubs = FA_LATENT_V / 64;
constexpr int kQK = FA_LATENT_NOPE + FA_LATENT_ROPE, kV = FA_LATENT_V;
constexpr int kSub = kRows * 128;       // [128 rows][64] subtile, 16 KB
constexpr int kX = kXSubs * kSub, kY = kYSubs * kSub;
constexpr int kMaxXStages = 3;
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f;

struct Bars {
  uint64_t fixed_full;
  uint64_t x_full[kMaxXStages];
  uint64_t x_empty[kMaxXStages];  // the block's last product has completed
  uint64_t y_full;
  uint64_t y_empty;
  uint64_t s_full;
  uint64_t s_read;             // the softmax warps have the scores in registers
  uint64_t dp_full;
  uint64_t p_half;             // of each 64 columns the first 32
  uint64_t p_ready;
  uint64_t ds_half;            // of each 64 columns the first 32
  uint64_t ds_ready;
  uint64_t ds_taken;           // the product with dS's first term has completed
  uint64_t do_ready;           // dQ: the owned dO is in tensor memory
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int never;  // stays 0: waits that must not be cut short by an abort
};

struct Stats {                          // of a streamed query block (dK, dV)
  float lse2[kRows];                    // lse log2 e; +inf for rows that see no key or none are
  float D[kRows];
};

template <bool DQ>
struct Lay {
  static constexpr int XS = DQ ? 3 : 2;                 // stages of X
  static constexpr int FIXED = DQ ? kX : kX + kY;       // owned rows in shared memory
  static constexpr int SMEM = 1024 + FIXED + XS * kX + kY +
                              (DQ ? 0 : XS * static_cast<int>(sizeof(Stats))) +
                              static_cast<int>(sizeof(Bars));
  static_assert(XS <= kMaxXStages && SMEM <= 227 * 1024, "shared memory");
};

struct BwdArgs {
  const __nv_bfloat16* dO;
  const float* lse;
  const float* D;
  __nv_bfloat16* dq;       // dQ kernel
  __nv_bfloat16* dkn;      // dK, dV kernel
  float* dkr;              // [B, H, N, 64], one head's share
  __nv_bfloat16* dv;
};

// lse as the exponent's offset: a row that saw no key (lse = -inf) gets P = 0 everywhere.
__device__ __forceinline__ float exponent_of(float lse) {
  return lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// DQ = false: X = q, Y = dO streamed, k and v owned.  DQ = true: k, v streamed, q and dO owned.
// `cta`: its number among those of its kind.
template <bool DQ>
__device__ __forceinline__ void bwd_cta(const CUtensorMap& mq, const CUtensorMap& mkn,
                                        const CUtensorMap& mkr, const CUtensorMap& mv,
                                        const CUtensorMap& mdo, const BwdArgs& a,
                                        const LatentProblem& p, int cta) {
  constexpr uint32_t kAccX = DQ ? 0 : kV;            // columns of dQ or dK (dV sits before dK)
  constexpr uint32_t kS = kAccX + kQK;               // the scores
  constexpr uint32_t kDP = DQ ? kS + 128 : kS;       // dP
  constexpr uint32_t kDS = kDP;                      // dS as bf16 in place, ...
  constexpr uint32_t kDSHalf = 64;                   // ... each 64 columns' pairs at their start
  constexpr uint32_t kP = kS + 128;                  // dK, dV: P^T as bf16
  constexpr uint32_t kDO = kDP + 128;                // dQ: the owned dO
  constexpr int kXStages = Lay<DQ>::XS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sF = base;                                // owned rows: X subtiles (dK, dV: then Y)
  uint8_t* sX = sF + Lay<DQ>::FIXED;                 // [kXStages]
  uint8_t* sY = sX + kXStages * kX;
  Stats* stats = reinterpret_cast<Stats*>(sY + kY);
  Bars* bars = reinterpret_cast<Bars*>(stats + (DQ ? 0 : kXStages));
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Work: groups of heads whose streamed rows (640 N bytes a head) fit 64 MiB of L2; in each
  // group the tiles with the most blocks first (causal: early keys, late queries), the group's
  // heads fastest.
  const int tiles = (p.N + kRows - 1) / kRows, bhs = p.B * p.H;
  int bh, row0;
  {
    const int G = static_cast<int>(max(1ll, min(static_cast<long long>(bhs),
                                                (64ll << 20) / (640ll * p.N))));
    const int g = cta / (G * tiles), r = cta - g * G * tiles;
    const int Gg = min(G, bhs - g * G);
    bh = g * G + r % Gg;
    row0 = (DQ ? tiles - 1 - r / Gg : r / Gg) * kRows;
  }
  const int seq = bh / p.H;

  if (tid == 0) {
    mbar_init(&bars->fixed_full, 1);
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&bars->x_full[s], DQ ? 1 : 33);
      mbar_init(&bars->x_empty[s], 1);
    }
    mbar_init(&bars->y_full, 1);
    mbar_init(&bars->y_empty, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_read, 256);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_half, 256);
    mbar_init(&bars->p_ready, 256);
    mbar_init(&bars->ds_half, 256);
    mbar_init(&bars->ds_ready, 256);
    mbar_init(&bars->ds_taken, 1);
    mbar_init(&bars->do_ready, 256);
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->drain, DQ ? 2 : 1);
    bars->abort = 0;
    bars->never = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = bars->tmem_base;
  griddep_wait();
  griddep_launch_dependents();
  int L = p.N;
  if (p.kv_len) {
    L = p.kv_len[seq];
    L = L < 0 ? 0 : (L > p.N ? p.N : L);
  }
  // The streamed rows [begin, end) in blocks of 128.
  const int begin = !DQ && p.causal ? row0 : 0;
  const int end = DQ ? (p.causal ? min(L, row0 + kRows) : L) : (row0 < L ? p.N : begin);
  const int blocks = end > begin ? (end - begin + kRows - 1) / kRows : 0;
  // One rounding of dS leaves dq 0.0024 of its norm off at any length, where the result's own leaves
  // 0.0017.  But the fewer keys a query sees, the fewer roundings its row of dq holds and the farther
  // off a single row can be: 0.0045 of it over 2 keys, 0.0035 over 300 (the result's rounding alone:
  // 0.0021; the largest of 2400 rows, D taken as given).  An accuracy choice for such rows: queries
  // that see at most 128 keys, whose row of dS is one block, have it in the products as two bf16
  // terms, the second in the first's place when its product is done: the same instructions once
  // more, since further MMAs in the issuers' loops slow every block (side by side, 6% and more).
  // `fine`: the CTA's first blocks that hold such queries.  A training step of 16 heads x 8192,
  // causal, takes 1137 us with it and 1113 without, 4 x 64 heads x 100 61.5 and 57.3, 2 x 8 x 1000
  // 56.4 both; 4 x 8 x 1000 with 2 visible keys each 62 and 55.
  const int fine = DQ ? (end <= kRows ? blocks : 0)
                      : row0 > 0 ? 0 : L <= kRows ? blocks : p.causal ? 1 : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && blocks > 0) {
      const auto load_x = [&](uint8_t* dst, uint64_t* bar, int row, bool keys) {
        if (keys) {
          tma_load_3d(dst, &mkn, bar, 0, row, bh);
          tma_load_3d(dst + kSub, &mkn, bar, 64, row, bh);
          tma_load_3d(dst + 2 * kSub, &mkr, bar, 0, row, seq);
        } else {
          for (int s = 0; s < kXSubs; ++s) tma_load_3d(dst + s * kSub, &mq, bar, 64 * s, row, bh);
        }
      };
      const auto load_y = [&](uint8_t* dst, uint64_t* bar, int row, bool keys) {
        for (int s = 0; s < kYSubs; ++s)
          tma_load_3d(dst + s * kSub, keys ? &mv : &mdo, bar, 64 * s, row, bh);
      };
      mbar_arrive_expect_tx(&bars->fixed_full, Lay<DQ>::FIXED);
      load_x(sF, &bars->fixed_full, row0, !DQ);
      if (!DQ) load_y(sF + kX, &bars->fixed_full, row0, true);
      for (int n = 0; n < blocks; ++n) {
        const int st = n % kXStages, row = begin + n * kRows;
        if (!mbar_wait(&bars->x_empty[st], ((n / kXStages) & 1) ^ 1, abort_flag, p.err, p.wait_ns))
          break;
        mbar_arrive_expect_tx(&bars->x_full[st], kX);
        load_x(sX + st * kX, &bars->x_full[st], row, DQ);
        if (!mbar_wait(&bars->y_empty, (n & 1) ^ 1, abort_flag, p.err, p.wait_ns)) break;
        mbar_arrive_expect_tx(&bars->y_full, kY);
        load_y(sY, &bars->y_full, row, DQ);
      }
    }
  } else if (warp == 1 || (DQ && warp == 3)) {
    // ------------------------------------------------------------ MMA issuers
    // dK, dV: one thread, since S^T follows dK in the region dS^T leaves.  dQ: one for the scores,
    // which wait for their keys, and one for dQ and then dP in the region dS leaves.
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(kRows, kRows, false, false);
      constexpr uint32_t idX = idesc_bf16(kRows, kQK, false, true);
      constexpr uint32_t idV = idesc_bf16(kRows, kV, false, true);
      // Descriptors by their low words (the start address); the high words hold the strides, alike
      // for K-major and for MN-major operands.
      auto low = [](const uint8_t* p, uint32_t lbo) {
        return static_cast<uint32_t>(sw128_desc(smem_u32(p), lbo, 1024));
      };
      const uint32_t hi = static_cast<uint32_t>(sw128_desc(0, 16, 1024) >> 32);
      const uint32_t dF = low(sF, 16), dXk = low(sX, 16), dYk = low(sY, 16);   // K-major
      const uint32_t dXm = low(sX, kSub), dYm = low(sY, kSub);                 // MN-major
      // Score product over `subs` subtiles from descriptors a0 and b0 on.
      auto scores = [&](uint32_t d, uint32_t a0, uint32_t b0, int subs) {
#pragma unroll
        for (int g = 0; g < subs; ++g) {
          uint32_t da[4], db[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            da[k] = a0 + ((g * kSub + k * 32) >> 4);
            db[k] = b0 + ((g * kSub + k * 32) >> 4);
          }
          mma_ss_x4_lo(d, da, hi, db, hi, idS, g > 0 ? 1u : 0u);
        }
      };
      // Half of a gradient product: A from the bf16 pairs at `t` (64 rows of the block each `half`
      // columns), of each 64 rows the first or the last 32, B the stage's subtiles along the rows.
      auto halves = [&](uint32_t d, uint32_t t, uint32_t half, uint32_t b0, uint32_t id, int q,
                        bool acc) {
        uint32_t ta[4], db[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ta[k] = t + (k >> 1) * half + 8 * (2 * q + (k & 1));
          db[k] = b0 + ((2048 * (4 * (k >> 1) + 2 * q + (k & 1))) >> 4);
        }
        mma_ts_x4_lo(d, ta, db, hi, id, acc ? 1u : 0u);
      };
      auto start_s = [&](int n) -> bool {
        const int st = n % kXStages;
        if (!mbar_wait(&bars->x_full[st], (n / kXStages) & 1, abort_flag, p.err, p.wait_ns))
          return false;
        tc_fence_after();
        scores(tb + kS, dF, dXk + ((st * kX) >> 4), kXSubs);
        mma_commit(&bars->s_full);
        return true;
      };
      auto start_dp = [&](int n) -> bool {
        if (!mbar_wait(&bars->y_full, n & 1, abort_flag, p.err, p.wait_ns)) return false;
        tc_fence_after();
        if (DQ) {   // A = dO from tensor memory
#pragma unroll
          for (int g = 0; g < kYSubs; ++g) {
            uint32_t ta[4], db[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ta[k] = tb + kDO + 8 * (4 * g + k);
              db[k] = dYk + ((g * kSub + k * 32) >> 4);
            }
            mma_ts_x4_lo(tb + kDP, ta, db, hi, idS, g > 0 ? 1u : 0u);
          }
        } else {
          scores(tb + kDP, dF + (kX >> 4), dYk, kYSubs);
        }
        mma_commit(&bars->dp_full);
        if (DQ) mma_commit(&bars->y_empty);
        return true;
      };
      auto wait = [&](uint64_t* bar, int n) -> bool {
        if (!mbar_wait(bar, n & 1, abort_flag, p.err, p.wait_ns)) return false;
        tc_fence_after();
        return true;
      };
      // dQ += dS K, dK += dS^T Q, in one term or (the first `fine` blocks) in two; begun on the first
      // half of dS while the softmax warps form the second, as dV += P^T dO is (16 heads x 8192: 1199
      // -> 1169 us, 2 x 8 x 1000: 62.5 -> 63.5).
      int nd = 0;
      auto dS_product = [&](int st, int n) -> bool {
        bool more = n < fine;
#pragma unroll 1
        for (bool acc = n > 0;; acc = true) {
          const uint32_t b0 = dXm + ((st * kX) >> 4);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (!wait(q ? &bars->ds_ready : &bars->ds_half, nd)) return false;
            halves(tb + kAccX, tb + kDS, kDSHalf, b0, idX, q, acc || q > 0);
          }
          ++nd;
          if (!more) return true;
          more = false;
          mma_commit(&bars->ds_taken);
        }
      };
      bool ok = blocks > 0;
      if (DQ && warp == 3) {
        ok = ok && mbar_wait(&bars->do_ready, 0, abort_flag, p.err, p.wait_ns) && start_dp(0);
        for (int n = 0; ok && n < blocks; ++n) {
          const int st = n % kXStages;
          ok = mbar_wait(&bars->x_full[st], (n / kXStages) & 1, abort_flag, p.err, p.wait_ns) &&
               dS_product(st, n);
          if (!ok) break;
          mma_commit(&bars->x_empty[st]);
          if (n + 1 < blocks) ok = start_dp(n + 1);   // over dS, behind the product that reads it
        }
      } else if (DQ) {
        ok = ok && mbar_wait(&bars->fixed_full, 0, abort_flag, p.err, p.wait_ns);
        for (int n = 0; ok && n < blocks; ++n) {
          if (n > 0) ok = wait(&bars->s_read, n - 1);
          ok = ok && start_s(n);
        }
      } else {
        ok = ok && mbar_wait(&bars->fixed_full, 0, abort_flag, p.err, p.wait_ns) && start_s(0);
        for (int n = 0; ok && n < blocks; ++n) {
          const int st = n % kXStages;
          ok = wait(&bars->s_read, n) && start_dp(n);
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            ok = ok && wait(q ? &bars->p_ready : &bars->p_half, n);
            if (!ok) break;
            halves(tb, tb + kP, 32, dYm, idV, q, n > 0 || q > 0);
          }
          if (!ok) break;
          mma_commit(&bars->y_empty);
          ok = dS_product(st, n);
          if (!ok) break;
          mma_commit(&bars->x_empty[st]);
          if (n + 1 < blocks) ok = start_s(n + 1);
        }
      }
      if (ok && warp == (DQ ? 3 : 1)) mma_commit(&bars->acc_full);
      // Every MMA issued by either thread has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, p.wait_ns);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ lse and D of the query block
    if (!DQ) {
      const size_t rows = static_cast<size_t>(bh) * p.N;
      bool ok = true;
      for (int n = 0; ok && n < blocks; ++n) {
        const int st = n % kXStages;
        float l2[4], Dr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = begin + n * kRows + 32 * i + lane;
          l2[i] = row < p.N ? exponent_of(a.lse[rows + row]) : INFINITY;
          Dr[i] = row < p.N ? a.D[rows + row] : 0.f;
        }
        ok = mbar_wait_warp(&bars->x_empty[st], ((n / kXStages) & 1) ^ 1, abort_flag, p.err,
                            p.wait_ns);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          stats[st].lse2[32 * i + lane] = l2[i];
          stats[st].D[32 * i + lane] = Dr[i];
        }
        mbar_arrive(&bars->x_full[st]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    // Thread = row r of the owned side, columns 64 half ... + 63 of the streamed block.
    const int w4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * w4 + lane, row = row0 + r;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * w4) << 16);
    const float c = p.scale * kLog2e;
    float row_l2 = INFINITY, row_D = 0.f;
    if (DQ && row < p.N) {
      row_l2 = exponent_of(a.lse[static_cast<size_t>(bh) * p.N + row]);
      row_D = a.D[static_cast<size_t>(bh) * p.N + row];
    }
    if (DQ && blocks > 0) {
      // The owned dO as the A operand of dP: 16 rows a warp, four threads to 32 bytes of a row.
      const int rA = row0 + 32 * w4 + 16 * half + (lane >> 2), rB = rA + 8;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.dO) +
                            static_cast<size_t>(bh) * p.N * (kV / 2) + 2 * (lane & 3);
      uint32_t w[32];
#pragma unroll
      for (int cc = 0; cc < 8; ++cc) {
        uint2 x = make_uint2(0u, 0u), y = x;
        if (rA < p.N)
          x = *reinterpret_cast<const uint2*>(src + static_cast<size_t>(rA) * (kV / 2) + 8 * cc);
        if (rB < p.N)
          y = *reinterpret_cast<const uint2*>(src + static_cast<size_t>(rB) * (kV / 2) + 8 * cc);
        w[4 * cc] = x.x;
        w[4 * cc + 1] = x.y;
        w[4 * cc + 2] = y.x;
        w[4 * cc + 3] = y.y;
      }
      tmem_st_16x256b_x8(lane_base + (static_cast<uint32_t>(16 * half) << 16) + kDO, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->do_ready);
    }
    bool ok = true;
    for (int n = 0; ok && n < blocks; ++n) {
      const int st = n % kXStages;
      const int col0 = begin + n * kRows + 64 * half;   // this thread's first streamed row
      const bool tail = DQ && begin + (n + 1) * kRows > L;
      if (!DQ || tail) {
        // The stage has landed (its MMAs wait for it too); the wait orders the statistics.
        ok = mbar_wait_warp(&bars->x_full[st], (n / kXStages) & 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
      }
      ok = mbar_wait_warp(&bars->s_full, n & 1, abort_flag, p.err, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[64];
      tmem_ld64_wait(lane_base + kS + 64 * half, lane_base + kS + 64 * half + 32, sv);
      tc_fence_before();
      mbar_arrive(&bars->s_read);
      // Visible: key < L, and key <= query where causal.
      int lo = 0, hi = 64;                        // visible columns of this thread's 64
      if (DQ) {
        hi = min(hi, L - col0);
        if (p.causal) hi = min(hi, row - col0 + 1);
      } else {
        if (row >= L) hi = 0;
        if (p.causal) lo = max(lo, row - col0);
      }
      const bool edge = lo > 0 || hi < 64;
      float P[64];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 32 * q; i < 32 * q + 32; i += 4) {
          float4 l2 = make_float4(row_l2, row_l2, row_l2, row_l2);
          if (!DQ) l2 = *reinterpret_cast<const float4*>(&stats[st].lse2[64 * half + i]);
          P[i] = ex2(fmaf(__uint_as_float(sv[i]), c, -l2.x));
          P[i + 1] = ex2(fmaf(__uint_as_float(sv[i + 1]), c, -l2.y));
          P[i + 2] = ex2(fmaf(__uint_as_float(sv[i + 2]), c, -l2.z));
          P[i + 3] = ex2(fmaf(__uint_as_float(sv[i + 3]), c, -l2.w));
        }
        if (edge) {
#pragma unroll
          for (int i = 32 * q; i < 32 * q + 32; ++i)
            if (i < lo || i >= hi) P[i] = 0.f;
        }
        if (!DQ) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(P[32 * q + 2 * i], P[32 * q + 2 * i + 1]);
          tmem_st16(lane_base + kP + 32 * half + 16 * q, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(q ? &bars->p_ready : &bars->p_half);
        }
      }
      ok = mbar_wait_warp(&bars->dp_full, n & 1, abort_flag, p.err, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      if (tail) {
        // Keys past the length: zero their rows before dS K reads them, so that 0 x (anything)
        // stays 0 (the scores of this block have been formed).
        const int key = (tid - 128) >> 1;
        if (begin + n * kRows + key >= L) {
          uint8_t* kr = sX + st * kX + key * 128 + 64 * (tid & 1);
#pragma unroll
          for (int s = 0; s < kXSubs; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(kr + s * kSub)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t dv[32], pk[16];
        tmem_ld32_wait(lane_base + kDP + 64 * half + 32 * q, dv);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 D = make_float4(row_D, row_D, row_D, row_D);
          if (!DQ) D = *reinterpret_cast<const float4*>(&stats[st].D[64 * half + 32 * q + i]);
          P[32 * q + i] *= __uint_as_float(dv[i]) - D.x;
          P[32 * q + i + 1] *= __uint_as_float(dv[i + 1]) - D.y;
          P[32 * q + i + 2] *= __uint_as_float(dv[i + 2]) - D.z;
          P[32 * q + i + 3] *= __uint_as_float(dv[i + 3]) - D.w;
        }
        if (edge) {   // a hidden key's v may hold anything
#pragma unroll
          for (int i = 32 * q; i < 32 * q + 32; ++i)
            if (i < lo || i >= hi) P[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[i] = pack_bf16x2(P[32 * q + 2 * i], P[32 * q + 2 * i + 1]);
        // In place: columns of this thread's own that it has read.
        tmem_st16(lane_base + kDS + kDSHalf * half + 16 * q, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(q ? &bars->ds_ready : &bars->ds_half);
      }
      if (n < fine) {   // what the rounding left
        ok = mbar_wait_warp(&bars->ds_taken, n & 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = P[32 * q + 2 * i], y = P[32 * q + 2 * i + 1];
            pk[i] = pack_bf16x2(x - __bfloat162float(__float2bfloat16_rn(x)),
                                y - __bfloat162float(__float2bfloat16_rn(y)));
          }
          tmem_st16(lane_base + kDS + kDSHalf * half + 16 * q, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(q ? &bars->ds_ready : &bars->ds_half);
        }
      }
    }
    // ------------------------------------------------------------ epilogue
    if (ok && blocks > 0) {
      ok = mbar_wait_warp(&bars->acc_full, 0, abort_flag, p.err, p.wait_ns);
      tc_fence_after();
    }
    // Rows A and B of the tile, 16 a warp: the four threads of a row exchange their column pairs so
    // that each stores 16 bytes, 64 in a row (a row per thread touches four times the lines: 4 x 64
    // heads x 100 66 -> 61 us, 16 x 8192 1159 -> 1147).
    const int t4 = lane & 3, rA = row0 + 32 * w4 + 16 * half + (lane >> 2), rB = rA + 8;
    const uint32_t quarter = lane_base + (static_cast<uint32_t>(16 * half) << 16);
    if (ok) {
#pragma unroll 1
      for (int i = 0; i < (DQ ? 3 : 5); ++i) {   // 64 columns: three of dQ or dK, then two of dV
        uint32_t v[32];
        __syncwarp();
        if (blocks > 0) tmem_ld_16x256b_x8_wait(quarter + (i < 3 ? kAccX + 64 * i : 64 * (i - 3)), v);
#pragma unroll
        for (int ab = 0; ab < 2; ++ab) {
          const int r = ab ? rB : rA;
          const bool live = blocks > 0 && (DQ || r < L), in = r < p.N;
          const size_t at = static_cast<size_t>(bh) * p.N + r;
          const float mul = i < 3 ? p.scale : 1.f;
          float f[16];
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {
            f[2 * cc] = live ? __uint_as_float(v[4 * cc + 2 * ab]) * mul : 0.f;
            f[2 * cc + 1] = live ? __uint_as_float(v[4 * cc + 2 * ab + 1]) * mul : 0.f;
          }
          if (!DQ && i == 2) {   // the head's share of dk_rope
            float* dst = a.dkr + at * FA_LATENT_ROPE + 2 * t4;
#pragma unroll
            for (int cc = 0; cc < 8; ++cc)
              if (in) *reinterpret_cast<float2*>(dst + 8 * cc) = make_float2(f[2 * cc], f[2 * cc + 1]);
          } else {
            __nv_bfloat16* out = DQ ? a.dq + at * kQK + 64 * i
                                    : i < 3 ? a.dkn + at * FA_LATENT_NOPE + 64 * i
                                            : a.dv + at * kV + 64 * (i - 3);
#pragma unroll
            for (int c4 = 0; c4 < 2; ++c4) {
              const float* g = f + 8 * c4;
              const uint4 x = quad_transpose(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                                             pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]), t4);
              if (in) *reinterpret_cast<uint4*>(out + 32 * c4 + 8 * t4) = x;
            }
          }
        }
      }
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

// Both kinds in one grid, dK, dV first (their CTAs take longer): neither needs the other, and the
// second fills the SMs that the first leaves idle at its end (short sequences: from the start).
__global__ void __launch_bounds__(kThreads, 1)
latent_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkn,
                  const __grid_constant__ CUtensorMap mkr, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mdo, BwdArgs a, LatentProblem p) {
  const int half = gridDim.x / 2, cta = blockIdx.x;
  if (cta < half)
    bwd_cta<false>(mq, mkn, mkr, mv, mdo, a, p, cta);
  else
    bwd_cta<true>(mq, mkn, mkr, mv, mdo, a, p, cta - half);
}

constexpr int kSmem = Lay<false>::SMEM > Lay<true>::SMEM ? Lay<false>::SMEM : Lay<true>::SMEM;

}  // namespace

cudaError_t launch_latent_bwd_sm103(const LatentProblem& p, const void* q, const void* kn,
                                    const void* kr, const void* v, const float* lse,
                                    const void* dO, const float* Dsum, void* dq, void* dkn,
                                    float* dkr_part, void* dv, cudaStream_t s) {
  BwdArgs a{static_cast<const __nv_bfloat16*>(dO), lse, Dsum, static_cast<__nv_bfloat16*>(dq),
            static_cast<__nv_bfloat16*>(dkn), dkr_part, static_cast<__nv_bfloat16*>(dv)};
  CUtensorMap mq, mkn, mkr, mv, mdo;
  const int BH = p.B * p.H;
  if (!make_head_map(&mq, q, BH, p.N, kQK) || !make_head_map(&mkn, kn, BH, p.N, FA_LATENT_NOPE) ||
      !make_head_map(&mkr, kr, p.B, p.N, FA_LATENT_ROPE) ||
      !make_head_map(&mv, v, BH, p.N, kV) || !make_head_map(&mdo, dO, BH, p.N, kV))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(latent_bwd_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  const long long tiles = (p.N + kRows - 1) / kRows;
  return launch_dependent(latent_bwd_kernel, dim3(static_cast<unsigned>(2 * BH * tiles)),
                          dim3(kThreads), kSmem, s, mq, mkn, mkr, mv, mdo, a, p);
}

}  // namespace fa
