// Expanded latent attention, backward, on sm_103a tensor cores (tcgen05 + TMA), bf16 in, fp32
// accumulation.  The formulas stand in fa_latent_simt.cu.
//
// Two kernels of one template, without atomics (the result does not depend on scheduling):
//   dK, dV  a CTA owns 128 keys of a head (k, v stay in shared memory) and streams the query
//           blocks of 64 rows that may see them:
//             S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q;
//   dQ      a CTA owns 128 query rows (q, dO stay) and streams key blocks of 64:
//             S = Q K^T, dP = dO V^T, dQ += dS K.
// Seven products instead of five (S and dP are formed twice: 1152 columns of MMA a pair against
// 832), because dK (192) + dV (128) + dQ (192) and two score tiles do not fit tensor memory's 512
// columns, and dQ needs no fp32 sums through global memory this way.
//
// What bounds it: the score products, whose N = 64 makes shared memory feed 6 KB an MMA of 32
// cycles' work (48 cycles at 128 B a cycle), about 1600 + 1344 cycles a 128 x 64 block.
//
// Both score operands of the streamed side come from one stage: X (192 columns: q or k) and Y
// (128: dO or v) lie as [64 rows][64 columns] subtiles that the score products read K-major and
// the gradient products MN-major.  Tensor memory: the accumulators, then regions of 64 columns
// for S and dP, whose rows P and dS overwrite as bf16 (the A operand of the gradient products).
// dK, dV has three regions: S(n) sits in region 2n mod 3 and dP(n) in 2n + 1 mod 3, so S(n + 1)
// starts while block n is in the softmax and dP(n + 1) takes the region that P(n) leaves after
// its product.  dQ has four.
//   warp 0 producer; warp 1 MMA issuer; warp 2 tensor memory and (dK, dV) the block's lse and
//   D; warps 4-11 softmax, two threads a row, 32 columns each.
// Every wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and exits.
#include <atomic>

#include <cuda.h>
#include <math.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kRows = 128;              // rows a CTA owns
constexpr int kCols = 64;               // rows of a streamed block
constexpr int kXSubs = (FA_LATENT_NOPE + FA_LATENT_ROPE) / 64, kYSubs = FA_LATENT_V / 64;
constexpr int kQK = FA_LATENT_NOPE + FA_LATENT_ROPE, kV = FA_LATENT_V;
constexpr int kFSub = kRows * 128;      // [128 rows][64] subtile of the owned side, 16 KB
constexpr int kSSub = kCols * 128;      // [64 rows][64] subtile of the streamed side, 8 KB
constexpr int kFixed = (kXSubs + kYSubs) * kFSub;
constexpr int kStage = (kXSubs + kYSubs) * kSSub;
constexpr int kStages = 3;
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f;

struct Bars {
  uint64_t fixed_full;
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t s_full[2];
  uint64_t dp_full[2];
  uint64_t p_ready[2];
  uint64_t ds_ready[2];
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int never;  // stays 0: waits that must not be cut short by an abort
};

struct Stats {                          // of a streamed query block (dK, dV)
  float lse2[kCols];                    // lse log2 e; +inf for rows that see no key or none are
  float D[kCols];
};

constexpr int kSmem = 1024 + kFixed + kStages * kStage +
                      kStages * static_cast<int>(sizeof(Stats)) + static_cast<int>(sizeof(Bars));
static_assert(kSmem <= 227 * 1024, "shared memory");

struct BwdArgs {
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
// Maps: boxes of 128 rows on the owned side, of 64 on the streamed side.
template <bool DQ>
__global__ void __launch_bounds__(kThreads, 1)
latent_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkn,
                  const __grid_constant__ CUtensorMap mkr, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mdo, BwdArgs a, LatentProblem p) {
  constexpr uint32_t kAccX = DQ ? 0 : kV;            // columns of dQ or dK (dV sits before dK)
  constexpr uint32_t kRegions = kAccX + kQK;         // first column of the S and dP regions
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sF = base;                                // owned rows: X subtiles, Y subtiles
  uint8_t* sS = sF + kFixed;                         // [kStages] X subtiles, Y subtiles
  Stats* stats = reinterpret_cast<Stats*>(sS + kStages * kStage);
  Bars* bars = reinterpret_cast<Bars*>(stats + kStages);
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
    const int x = blockIdx.x, g = x / (G * tiles), r = x - g * G * tiles;
    const int Gg = min(G, bhs - g * G);
    bh = g * G + r % Gg;
    row0 = (DQ ? tiles - 1 - r / Gg : r / Gg) * kRows;
  }
  const int seq = bh / p.H;

  if (tid == 0) {
    mbar_init(&bars->fixed_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], DQ ? 1 : 33);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->dp_full[i], 1);
      mbar_init(&bars->p_ready[i], 256);
      mbar_init(&bars->ds_ready[i], 256);
    }
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->drain, 1);
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
  // The streamed rows [begin, end) in blocks of 64.
  const int begin = !DQ && p.causal ? row0 : 0;
  const int end = DQ ? (p.causal ? min(L, row0 + kRows) : L) : (row0 < L ? p.N : begin);
  const int blocks = end > begin ? (end - begin + kCols - 1) / kCols : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && blocks > 0) {
      const auto load = [&](uint8_t* dst, int sub, uint64_t* bar, int row, bool keys) {
        if (keys) {
          tma_load_3d(dst, &mkn, bar, 0, row, bh);
          tma_load_3d(dst + sub, &mkn, bar, 64, row, bh);
          tma_load_3d(dst + 2 * sub, &mkr, bar, 0, row, seq);
          tma_load_3d(dst + 3 * sub, &mv, bar, 0, row, bh);
          tma_load_3d(dst + 4 * sub, &mv, bar, 64, row, bh);
        } else {
          tma_load_3d(dst, &mq, bar, 0, row, bh);
          tma_load_3d(dst + sub, &mq, bar, 64, row, bh);
          tma_load_3d(dst + 2 * sub, &mq, bar, 128, row, bh);
          tma_load_3d(dst + 3 * sub, &mdo, bar, 0, row, bh);
          tma_load_3d(dst + 4 * sub, &mdo, bar, 64, row, bh);
        }
      };
      mbar_arrive_expect_tx(&bars->fixed_full, kFixed);
      load(sF, kFSub, &bars->fixed_full, row0, !DQ);
      for (int n = 0; n < blocks; ++n) {
        const int st = n % kStages;
        if (!mbar_wait(&bars->empty[st], ((n / kStages) & 1) ^ 1, abort_flag, p.err, p.wait_ns))
          break;
        mbar_arrive_expect_tx(&bars->full[st], kStage);
        load(sS + st * kStage, kSSub, &bars->full[st], begin + n * kCols, DQ);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(kRows, kCols, false, false);
      constexpr uint32_t idX = idesc_bf16(kRows, kQK, false, true);
      constexpr uint32_t idV = idesc_bf16(kRows, kV, false, true);
      const uint64_t dF = sw128_desc(smem_u32(sF), 16, 1024);
      const uint64_t dSk = sw128_desc(smem_u32(sS), 16, 1024);     // streamed, K-major
      const uint64_t dSm = sw128_desc(smem_u32(sS), kSSub, 1024);  // streamed, MN-major
      auto s_col = [&](int n) { return tb + kRegions + 64 * (DQ ? (n & 1) : (2 * n) % 3); };
      auto dp_col = [&](int n) { return tb + kRegions + 64 * (DQ ? 2 + (n & 1) : (2 * n + 1) % 3); };
      // Score product over subtiles [s0, s1) of both sides.
      auto scores = [&](uint32_t d, int st, int s0, int s1) {
#pragma unroll
        for (int g = s0; g < s1; ++g) {
          uint64_t da[4], db[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            da[k] = dF + static_cast<uint64_t>((g * kFSub + k * 32) >> 4);
            db[k] = dSk + static_cast<uint64_t>((st * kStage + g * kSSub + k * 32) >> 4);
          }
          mma_ss_x4(d, da, db, idS, g > s0 ? 1u : 0u);
        }
      };
      // Gradient product: A from the bf16 pairs in region `t` (32 rows of the block in its
      // columns 0-15, 32 in 32-47), B the stage's subtiles from `sub` on, along the rows.
      auto grads = [&](uint32_t d, uint32_t t, int st, int sub, uint32_t id, bool acc) {
        uint32_t ta[4];
        uint64_t db[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ta[k] = t + 32 * (k >> 1) + 8 * (k & 1);
          db[k] = dSm + static_cast<uint64_t>((st * kStage + sub * kSSub + 2048 * k) >> 4);
        }
        mma_ts_x4(d, ta, db, id, acc ? 1u : 0u);
      };
      auto start_s = [&](int n) -> bool {
        const int st = n % kStages;
        if (!mbar_wait(&bars->full[st], (n / kStages) & 1, abort_flag, p.err, p.wait_ns))
          return false;
        tc_fence_after();
        scores(s_col(n), st, 0, kXSubs);
        mma_commit(&bars->s_full[n & 1]);
        return true;
      };
      auto start_dp = [&](int n) {
        scores(dp_col(n), n % kStages, kXSubs, kXSubs + kYSubs);
        mma_commit(&bars->dp_full[n & 1]);
      };
      bool ok = blocks > 0;
      if (ok) ok = mbar_wait(&bars->fixed_full, 0, abort_flag, p.err, p.wait_ns);
      if (ok) ok = start_s(0);
      if (ok) start_dp(0);
      for (int n = 0; ok && n < blocks; ++n) {
        const int st = n % kStages;
        if (n + 1 < blocks) {
          ok = start_s(n + 1);
          if (!ok) break;
          if (DQ) start_dp(n + 1);
        }
        if (!DQ) {
          ok = mbar_wait(&bars->p_ready[n & 1], (n >> 1) & 1, abort_flag, p.err, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          grads(tb, s_col(n), st, kXSubs, idV, n > 0);
          if (n + 1 < blocks) start_dp(n + 1);
        }
        ok = mbar_wait(&bars->ds_ready[n & 1], (n >> 1) & 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        grads(tb + kAccX, dp_col(n), st, 0, idX, n > 0);
        mma_commit(&bars->empty[st]);
      }
      if (ok) mma_commit(&bars->acc_full);
      // Every MMA issued has completed before tensor memory is released.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, p.wait_ns);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ lse and D of the query block
    if (!DQ) {
      const size_t rows = static_cast<size_t>(bh) * p.N;
      bool ok = true;
      for (int n = 0; ok && n < blocks; ++n) {
        const int st = n % kStages;
        float l2[2], Dr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = begin + n * kCols + 32 * i + lane;
          l2[i] = row < p.N ? exponent_of(a.lse[rows + row]) : INFINITY;
          Dr[i] = row < p.N ? a.D[rows + row] : 0.f;
        }
        ok = mbar_wait_warp(&bars->empty[st], ((n / kStages) & 1) ^ 1, abort_flag, p.err,
                            p.wait_ns);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          stats[st].lse2[32 * i + lane] = l2[i];
          stats[st].D[32 * i + lane] = Dr[i];
        }
        mbar_arrive(&bars->full[st]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    // Thread = row r of the owned side, columns 32 half ... + 31 of the streamed block.
    const int w4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * w4 + lane, row = row0 + r;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * w4) << 16);
    const float c = p.scale * kLog2e;
    float row_l2 = INFINITY, row_D = 0.f;
    if (DQ && row < p.N) {
      row_l2 = exponent_of(a.lse[static_cast<size_t>(bh) * p.N + row]);
      row_D = a.D[static_cast<size_t>(bh) * p.N + row];
    }
    bool ok = true;
    for (int n = 0; ok && n < blocks; ++n) {
      const int st = n % kStages;
      const int col0 = begin + n * kCols + 32 * half;   // this thread's first streamed row
      if (!DQ || begin + (n + 1) * kCols > L) {
        // The stage has landed (its MMAs wait for it too); the wait orders the statistics.
        ok = mbar_wait_warp(&bars->full[st], (n / kStages) & 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
      }
      ok = mbar_wait_warp(&bars->s_full[n & 1], (n >> 1) & 1, abort_flag, p.err, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tS = lane_base + kRegions + 64 * (DQ ? (n & 1) : (2 * n) % 3) + 32 * half;
      const uint32_t tD =
          lane_base + kRegions + 64 * (DQ ? 2 + (n & 1) : (2 * n + 1) % 3) + 32 * half;
      uint32_t sv[32];
      tmem_ld32_wait(tS, sv);
      float P[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float l2 = DQ ? row_l2 : stats[st].lse2[32 * half + i];
        P[i] = ex2(fmaf(__uint_as_float(sv[i]), c, -l2));
      }
      // Visible: key < L, and key <= query where causal.
      int lo = 0, hi = 32;                        // visible columns of this thread's 32
      if (DQ) {
        hi = min(hi, L - col0);
        if (p.causal) hi = min(hi, row - col0 + 1);
      } else {
        if (row >= L) hi = 0;
        if (p.causal) lo = max(lo, row - col0);
      }
      const bool edge = lo > 0 || hi < 32;
      if (edge) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < lo || i >= hi) P[i] = 0.f;
      }
      uint32_t pk[16];
      if (!DQ) {
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(P[2 * i], P[2 * i + 1]);
        tmem_st16(tS, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_ready[n & 1]);
      }
      ok = mbar_wait_warp(&bars->dp_full[n & 1], (n >> 1) & 1, abort_flag, p.err, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32_wait(tD, sv);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float D = DQ ? row_D : stats[st].D[32 * half + i];
        P[i] *= __uint_as_float(sv[i]) - D;
      }
      if (edge) {   // a hidden key's v may hold anything
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < lo || i >= hi) P[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(P[2 * i], P[2 * i + 1]);
      tmem_st16(tD, pk);
      if (DQ && begin + (n + 1) * kCols > L) {
        // Keys past the length: zero their rows before dS K reads them, so that 0 x (anything)
        // stays 0 (the scores of this block have been formed).
        const int t = tid - 128, key = t >> 2;
        if (begin + n * kCols + key >= L && (t & 3) < kXSubs) {
          uint4* kr = reinterpret_cast<uint4*>(sS + st * kStage + (t & 3) * kSSub + key * 128);
#pragma unroll
          for (int i = 0; i < 8; ++i) kr[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->ds_ready[n & 1]);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && blocks > 0) {
      ok = mbar_wait_warp(&bars->acc_full, 0, abort_flag, p.err, p.wait_ns);
      tc_fence_after();
    }
    const bool live = blocks > 0 && (DQ || row < L);
    const size_t at = static_cast<size_t>(bh) * p.N + row;
    if (ok) {
#pragma unroll 1
      for (int i = 0; i < (DQ ? 3 : 5); ++i) {
        // Chunks of 32 columns: three of dQ or dK (96 half ... ), then two of dV (64 half ...).
        const int col = i < 3 ? 96 * half + 32 * i : 64 * half + 32 * (i - 3);
        uint32_t v[32];
        __syncwarp();
        if (blocks > 0) tmem_ld32_wait(lane_base + (i < 3 ? kAccX : 0) + col, v);
        float f[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
          f[k] = live ? __uint_as_float(v[k]) * (i < 3 ? p.scale : 1.f) : 0.f;
        if (row >= p.N) {
          // a row of the tile past the sequence
        } else if (!DQ && i < 3 && col >= FA_LATENT_NOPE) {
          float4* dst = reinterpret_cast<float4*>(a.dkr + at * FA_LATENT_ROPE + col - FA_LATENT_NOPE);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
        } else {
          __nv_bfloat16* out = DQ ? a.dq + at * kQK : i < 3 ? a.dkn + at * FA_LATENT_NOPE
                                                            : a.dv + at * kV;
          uint4* dst = reinterpret_cast<uint4*>(out + col);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack_bf16x2(f[8 * k], f[8 * k + 1]),
                                pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                                pack_bf16x2(f[8 * k + 4], f[8 * k + 5]),
                                pack_bf16x2(f[8 * k + 6], f[8 * k + 7]));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (bars->abort && tid == 0) {
    // Let any bulk copy still in flight land before the CTA's shared memory is released.
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

template <bool DQ>
cudaError_t launch_one(const LatentProblem& p, const void* q, const void* kn, const void* kr,
                       const void* v, const void* dO, const BwdArgs& a, cudaStream_t s) {
  CUtensorMap mq, mkn, mkr, mv, mdo;
  const int BH = p.B * p.H, q_rows = DQ ? kRows : kCols, k_rows = DQ ? kCols : kRows;
  if (!make_head_map_rows(&mq, q, BH, p.N, kQK, q_rows) ||
      !make_head_map_rows(&mkn, kn, BH, p.N, FA_LATENT_NOPE, k_rows) ||
      !make_head_map_rows(&mkr, kr, p.B, p.N, FA_LATENT_ROPE, k_rows) ||
      !make_head_map_rows(&mv, v, BH, p.N, kV, k_rows) ||
      !make_head_map_rows(&mdo, dO, BH, p.N, kV, q_rows))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(latent_bwd_kernel<DQ>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  const long long tiles = (p.N + kRows - 1) / kRows;
  return launch_dependent(latent_bwd_kernel<DQ>, dim3(static_cast<unsigned>(BH * tiles)),
                          dim3(kThreads), kSmem, s, mq, mkn, mkr, mv, mdo, a, p);
}

}  // namespace

cudaError_t launch_latent_bwd_sm103(const LatentProblem& p, const void* q, const void* kn,
                                    const void* kr, const void* v, const float* lse,
                                    const void* dO, const float* Dsum, void* dq, void* dkn,
                                    float* dkr_part, void* dv, cudaStream_t s) {
  BwdArgs a{lse, Dsum, static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dkn), dkr_part,
            static_cast<__nv_bfloat16*>(dv)};
  cudaError_t e = launch_one<false>(p, q, kn, kr, v, dO, a, s);
  if (e != cudaSuccess) return e;
  return launch_one<true>(p, q, kn, kr, v, dO, a, s);
}

}  // namespace fa
