// Expanded latent attention, forward, on sm_103a tensor cores (tcgen05 + TMA), bf16 in, fp32
// accumulation.
//
// Mathematics.  Head h's key is (k_nope_h, k_rope): 128 columns of its own and 64 that all heads
// of the sequence share; queries have 192 columns, values 128.  O = softmax(scale q k^T) v with
// the running maximum and sum of fa_fwd_sm103.cu (log2 domain, O unnormalised until the end and
// rescaled only past a 2^8 growth of the maximum).  The shared part is never copied per head: a
// key tile is two subtiles of the head's own tensor and one of the shared one.
//
// What bounds it: 640 operations a (query, key) pair against 640 bytes a key, read once for 256
// queries, so the tensor cores, and beside them the softmax.  As in fa_fwd_sm103.cu a CTA owns two tiles
// of 128 query rows, one MMA-issuing thread each, and all eight softmax warps take the tiles in
// turn: 540 us for 16 heads x 8192 without a mask (1.27 PFLOP/s), 4.1k cycles a pair of tiles
// and block of which 2.8k are MMAs.  Softmax warps of a tile's own measured slower, both four (a
// row per thread, 678 us) and eight (scores read twice, 627 us), and a P V product in two halves of
// the keys, the first while the second half of P is formed, gains nothing (566 us).
// A CTA takes further units of the grid with cluster launch control, for a unit's own cost (Q's and
// the first K's way from HBM, the first scores, O's way out) is that of two blocks: the roles walk
// the units on their own, so the next unit's loads and scores run while the softmax warps finish
// this one (causal, 4 x 16 heads x 2000: 90 -> 82 us, 16 x 8192: 268 -> 264; a grid that fits the SMs
// pays 0.2).  O goes out from the registers, as Q's buffers are by then the next unit's.
// Of the 227 KB of shared memory Q's two tiles hold 96, two K stages 96 and one V stage 32:
// V(j + 1) is fetched behind P V(j), while the scores of block j + 1 and their
// softmax run.  Tensor memory: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512).
// Every mbarrier wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and exits.
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <math.h>

#include "fa_fwd_units.cuh"
#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;
using namespace units;

constexpr int kSub = 128 * 128;         // bytes of a [128 rows][64 bf16] 128B-swizzled subtile
constexpr int kQKSubs = (FA_LATENT_NOPE + FA_LATENT_ROPE) / 64, kVSubs = FA_LATENT_V / 64;
constexpr int kQTile = kQKSubs * kSub, kVTile = kVSubs * kSub;
constexpr int kKStages = 2;
constexpr int kSmem = 1024 + (2 + kKStages) * kQTile + kVTile + 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kThreads = 384;
constexpr int kAsk = 2;             // key blocks before its end at which a unit asks for the next
constexpr int kRoles = 1 + 2 + 8;   // producer, issuers, softmax warps
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Bars {
  uint64_t q_full;
  uint64_t q_empty;     // every score product of the unit has completed
  uint64_t k_full[kKStages];
  uint64_t k_empty[kKStages];
  uint64_t v_full;
  uint64_t v_empty;
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_done[2];
  uint64_t next_full[2];   // the answer to a request for a further unit is there
  uint64_t next_empty[2];  // every role has read it
  uint64_t drain;
  alignas(16) uint4 next[2];
  uint32_t tmem_base;
  int abort;
  int never;  // stays 0: waits that must not be cut short by an abort
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__global__ void __launch_bounds__(kThreads, 1)
latent_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkn,
                  const __grid_constant__ CUtensorMap mkr, const __grid_constant__ CUtensorMap mv,
                  __nv_bfloat16* __restrict__ o, float* __restrict__ o_acc,
                  float* __restrict__ lse, LatentProblem p, int G) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                           // [2][kQTile]
  uint8_t* sK = sQ + 2 * kQTile;                // [kKStages][kQTile]
  uint8_t* sV = sK + kKStages * kQTile;         // [kVTile]
  Bars* bars = reinterpret_cast<Bars*>(sV + kVTile);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Work unit of a block index: groups of G heads; in each group heavy (late, causal) query blocks
  // first, the group's heads fastest.
  auto place = [&](int b) {
    const int nqb = (p.N + 2 * kBlk - 1) / (2 * kBlk), bhs = p.B * p.H;
    const int g = b / (G * nqb), r = b - g * G * nqb;
    const int Gg = min(G, bhs - g * G);
    Unit u;
    u.bh = g * G + r % Gg;
    u.q0 = (nqb - 1 - r / Gg) * 2 * kBlk;
    u.nb = (p.N + kBlk - 1) / kBlk;
    u.L = p.N;
    return u;
  };
  const Unit first_unit = place(blockIdx.x);
  auto unit = [&](int i, int b) {   // the i-th of this CTA
    Unit u = first_unit;
    if (i > 0) u = place(b);
    if (p.kv_len) u.L = max(0, min(p.kv_len[u.bh / p.H], p.N));
    return u;
  };

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 2);
    }
    mbar_init(&bars->v_full, 1);
    mbar_init(&bars->v_empty, 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 2 * kBlk);
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->next_full[t], 1);
      mbar_init(&bars->next_empty[t], kRoles);
    }
    mbar_init(&bars->drain, 2);
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
  // The unit after the i-th, or -1; one thread of each role.
  auto next_unit = [&](int i) -> int {
    if (!mbar_wait(&bars->next_full[i & 1], (i >> 1) & 1, abort_flag, p.err, p.wait_ns)) return -1;
    const int b = next_block_answer(&bars->next[i & 1]);
    fence_proxy_async_smem();   // read before it is written again
    mbar_arrive(&bars->next_empty[i & 1]);
    return b;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mkn);
      tma_prefetch_desc(&mkr);
      tma_prefetch_desc(&mv);
      bool ok = true;
      int n = 0, nu = 0;   // key blocks, units with any
      for (int i = 0, blk = blockIdx.x; ok && blk >= 0; ++i) {
        const Unit u = unit(i, blk);
        const int jend = key_blocks(p, u), seq = u.bh / p.H;
        // The next unit is asked for two blocks before this one's end: early enough for the answer,
        // and late enough that no block waits here while another CTA runs dry.
        auto request = [&]() -> bool {
          if (!mbar_wait(&bars->next_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, p.err,
                         p.wait_ns))
            return false;
          mbar_arrive_expect_tx(&bars->next_full[i & 1], sizeof(uint4));
          next_block_request(&bars->next[i & 1], &bars->next_full[i & 1]);
          return true;
        };
        const int j_ask = max(jend - kAsk, 0);
        if (jend == 0) ok = request();
        bool q_asked = false;
        for (int j = next_any(p, u, -1, jend); ok && j >= 0; j = next_any(p, u, j, jend), ++n) {
          const int st = n % kKStages;
          ok = mbar_wait(&bars->k_empty[st], ((n / kKStages) & 1) ^ 1, abort_flag, p.err,
                         p.wait_ns);
          if (!ok) break;
          if (j == j_ask && !request()) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->k_full[st], kQTile);
          uint8_t* dk = sK + st * kQTile;
          tma_load_3d(dk, &mkn, &bars->k_full[st], 0, j * kBlk, u.bh);
          tma_load_3d(dk + kSub, &mkn, &bars->k_full[st], 64, j * kBlk, u.bh);
          tma_load_3d(dk + 2 * kSub, &mkr, &bars->k_full[st], 0, j * kBlk, seq);
          if (!q_asked) {
            q_asked = true;
            ok = mbar_wait(&bars->q_empty, (nu & 1) ^ 1, abort_flag, p.err, p.wait_ns);
            if (!ok) break;
            ++nu;
            mbar_arrive_expect_tx(&bars->q_full, 2 * kQTile);
            for (int t = 0; t < 2; ++t)
              for (int s = 0; s < kQKSubs; ++s)
                tma_load_3d(sQ + t * kQTile + s * kSub, &mq, &bars->q_full, 64 * s,
                            u.q0 + t * kBlk, u.bh);
          }
          ok = mbar_wait(&bars->v_empty, (n & 1) ^ 1, abort_flag, p.err, p.wait_ns);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars->v_full, kVTile);
          for (int s = 0; s < kVSubs; ++s)
            tma_load_3d(sV + s * kSub, &mv, &bars->v_full, 64 * s, j * kBlk, u.bh);
        }
        if (ok) blk = next_unit(i);
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers
    // One thread per query tile: each walks every key block, and per block issues
    // O_t += P_t V_j after its softmax handshake, then S_t = Q_t K_{j+1}^T.
    if (lane == 0) {
      const int t = warp == 1 ? 0 : 1;
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = idesc_bf16(128, FA_LATENT_V, false, true);
      const uint64_t dQ = sw128_desc(smem_u32(sQ + t * kQTile), 16, 1024);  // K-major Q_t
      const uint64_t dK = sw128_desc(smem_u32(sK), 16, 1024);               // K-major K stages
      const uint64_t dV = sw128_desc(smem_u32(sV), kSub, 1024);             // MN-major V
      // Descriptors differ in their low words only (the start address).
      const uint32_t loQ = static_cast<uint32_t>(dQ), loK = static_cast<uint32_t>(dK);
      const uint32_t loV = static_cast<uint32_t>(dV);
      const uint32_t hiK = static_cast<uint32_t>(dK >> 32), hiV = static_cast<uint32_t>(dV >> 32);
      const uint32_t tS = tb + t * 128, tO = tb + 256 + t * 128;
      int nk = 0, nv = 0, nu = 0, np = 0;   // K and V blocks, units with any, P V products
      bool ok = true;
      for (int i = 0, blk = blockIdx.x; ok && blk >= 0; ++i) {
        const Unit u = unit(i, blk);
        const int jend = key_blocks(p, u);
        int last = -1;
        for (int j = jend - 1; j >= 0 && last < 0; --j)
          if (need(p, u, t, j)) last = j;
        // The scores of key block j, if this tile needs them; releases the stage, and Q behind
        // the unit's last block.
        auto take_k = [&](int j, bool end) -> bool {
          const int st = nk % kKStages;
          if (!mbar_wait(&bars->k_full[st], (nk / kKStages) & 1, abort_flag, p.err, p.wait_ns))
            return false;
          ++nk;
          tc_fence_after();
          if (need(p, u, t, j)) {
            const uint32_t loKs = loK + ((st * kQTile) >> 4);
#pragma unroll
            for (int g = 0; g < kQKSubs; ++g) {
              uint32_t da[4], db[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t off = (g * kSub + k * 32) >> 4;
                da[k] = loQ + off;
                db[k] = loKs + off;
              }
              mma_ss_x4_lo(tS, da, hiK, db, hiK, idS, g > 0 ? 1u : 0u);
            }
            mma_commit(&bars->s_full[t]);
          }
          mma_commit(&bars->k_empty[st]);
          if (end) mma_commit(&bars->q_empty);
          return true;
        };
        int j = next_any(p, u, -1, jend);
        int jn = j >= 0 ? next_any(p, u, j, jend) : -1;
        if (j >= 0) {
          ok = mbar_wait(&bars->q_full, nu & 1, abort_flag, p.err, p.wait_ns);
          if (!ok) break;
          ++nu;
          tc_fence_after();
          ok = take_k(j, jn < 0);
        }
        bool first = true;   // P V of the unit's first block overwrites O
        while (ok && j >= 0) {
          ok = mbar_wait(&bars->v_full, nv & 1, abort_flag, p.err, p.wait_ns);
          if (!ok) break;
          ++nv;
          tc_fence_after();
          if (need(p, u, t, j)) {
            ok = mbar_wait(&bars->p_full[t], np & 1, abort_flag, p.err, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t ta[4], db[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ta[k] = tS + 8 * (4 * g + k);
                db[k] = loV + ((2048 * (4 * g + k)) >> 4);
              }
              mma_ts_x4_lo(tO, ta, db, hiV, idO, (!first || g > 0) ? 1u : 0u);
            }
            first = false;
            ++np;
            if (j == last) mma_commit(&bars->o_done[t]);
          }
          mma_commit(&bars->v_empty);
          j = jn;
          if (j >= 0) {
            jn = next_any(p, u, j, jend);
            ok = take_k(j, jn < 0);
          }
        }
        if (ok) blk = next_unit(i);
      }
      // Drain: every MMA issued by either thread has completed before tensor memory is
      // released (the barrier counts one arrival per issuer).
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, p.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    // Warp 4 + q + 4h owns rows 32q + 16h + [0, 16) of both tiles through the 16-lane shapes:
    // thread t holds rows A = 32q + 16h + t/4 and B = A + 8, keys 8c + 2(t%4) + {0, 1}.
    const int q4 = warp & 3, h = (warp - 4) >> 2, t4 = lane & 3;
    const int rA = 32 * q4 + 16 * h + (lane >> 2), rB = rA + 8;   // rows within a tile
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * q4 + 16 * h) << 16);
    const float c = p.scale * kLog2e;
    const uint64_t c2 = f2_pack(c, c);
    bool ok = true;
    int n_s[2] = {0, 0}, n_o[2] = {0, 0}, n_v = 0;   // score tiles, outputs, key blocks so far
    for (int i = 0, blk = blockIdx.x; ok && blk >= 0; ++i) {
      const Unit u = unit(i, blk);
      const int jend = key_blocks(p, u);
      float m_run[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};  // [tile][A/B]
      float l_part[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      bool any[2] = {false, false};
      for (int j = 0; j < jend && ok; ++j, ++n_v) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || !need(p, u, t, j)) continue;
          ok = mbar_wait_warp(&bars->s_full[t], n_s[t] & 1, abort_flag, p.err, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          uint32_t v[64];
          tmem_ld_16x256b_x16_wait(lane_base + t * 128, v);
          float sv[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) sv[i] = __uint_as_float(v[i]);
          const int k0 = j * kBlk;
          const int row0 = u.q0 + t * kBlk;
          const bool edge = (p.causal && k0 + kBlk - 1 > row0) || (k0 + kBlk > u.L);
          if (edge) {
            const int lim_len = u.L - 1 - k0;
            const int limA = min(p.causal ? row0 + rA - k0 : kBlk - 1, lim_len);
            const int limB = min(p.causal ? row0 + rB - k0 : kBlk - 1, lim_len);
#pragma unroll
            for (int cc = 0; cc < 16; ++cc) {
              const int key = 8 * cc + 2 * t4;
              if (key > limA) sv[4 * cc] = -INFINITY;
              if (key + 1 > limA) sv[4 * cc + 1] = -INFINITY;
              if (key > limB) sv[4 * cc + 2] = -INFINITY;
              if (key + 1 > limB) sv[4 * cc + 3] = -INFINITY;
            }
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
          float mA = fmaxf(ma0, ma1) * c, mB = fmaxf(mb0, mb1) * c;
          // The rows' maxima are only formed where a thread's own part of one passes the running
          // reference by 2^8, in the first block and rarely after it.
          const float oldA = m_run[t][0], oldB = m_run[t][1];
          float newA = oldA, newB = oldB, alphaA = 1.f, alphaB = 1.f;
          const bool grew = __any_sync(0xffffffffu, mA > oldA + kRescaleThreshold ||
                                                        mB > oldB + kRescaleThreshold);
          if (grew) {
            mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 1));
            mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 1));
            mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 2));
            mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 2));
            if (mA > oldA + kRescaleThreshold) {
              newA = mA;
              alphaA = ex2(oldA - newA);   // old = -inf gives 0
            }
            if (mB > oldB + kRescaleThreshold) {
              newB = mB;
              alphaB = ex2(oldB - newB);
            }
          }
          const float useA = newA == -INFINITY ? 0.f : newA;
          const float useB = newB == -INFINITY ? 0.f : newB;
          const uint64_t nA = f2_pack(-useA, -useA), nB = f2_pack(-useB, -useB);
          uint64_t accA = f2_pack(0.f, 0.f), accB = accA;
          uint32_t pk[32];
#pragma unroll
          for (int cc = 0; cc < 16; ++cc) {
            const float2 xa = f2_unpack(ffma2(f2_pack(sv[4 * cc], sv[4 * cc + 1]), c2, nA));
            const float2 xb = f2_unpack(ffma2(f2_pack(sv[4 * cc + 2], sv[4 * cc + 3]), c2, nB));
            const float pa0 = ex2(xa.x), pa1 = ex2(xa.y);
            const float pb0 = ex2(xb.x), pb1 = ex2(xb.y);
            accA = fadd2(accA, f2_pack(pa0, pa1));
            accB = fadd2(accB, f2_pack(pb0, pb1));
            pk[2 * cc] = pack_bf16x2(pa0, pa1);
            pk[2 * cc + 1] = pack_bf16x2(pb0, pb1);
          }
          // P (bf16 pairs) overwrites the first 64 columns of this tile's S region in this
          // warp's 16 lanes, which no other warp reads; the load above has completed.
          tmem_st_16x128b_x16(lane_base + t * 128, pk);
          const float2 sa = f2_unpack(accA), sb = f2_unpack(accB);
          l_part[t][0] = l_part[t][0] * alphaA + (sa.x + sa.y);
          l_part[t][1] = l_part[t][1] * alphaB + (sb.x + sb.y);
          m_run[t][0] = newA;
          m_run[t][1] = newB;
          // Rescale the running O (the P V products issued before the S just read are done).
          if (any[t] && grew) {
#pragma unroll
            for (int half = 0; half < kVSubs; ++half) {
              uint32_t o[32];
              const uint32_t oaddr = lane_base + 256 + t * 128 + 64 * half;
              tmem_ld_16x256b_x8_wait(oaddr, o);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * ((i & 2) ? alphaB : alphaA));
              tmem_st_16x256b_x8(oaddr, o);
            }
          }
          if (k0 + kBlk > u.L) {
            // Keys past the length: zero their V rows before the product reads them, so that
            // 0 x (anything) stays 0.
            ok = mbar_wait_warp(&bars->v_full, n_v & 1, abort_flag, p.err, p.wait_ns);
            if (!ok) break;
            const int row = (tid - 128) >> 1;
            if (k0 + row >= u.L) {
              uint4* vr = reinterpret_cast<uint4*>(sV + (tid & 1) * kSub + row * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[t]);
          ++n_s[t];
          any[t] = true;
        }
      }
      // ------------------------------------------------------------ epilogue
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && any[t]) {
          ok = mbar_wait_warp(&bars->o_done[t], n_o[t] & 1, abort_flag, p.err, p.wait_ns);
          tc_fence_after();
          ++n_o[t];
        }
        if (!ok) break;
        float lA = l_part[t][0], lB = l_part[t][1];
        lA += __shfl_xor_sync(0xffffffffu, lA, 1);
        lB += __shfl_xor_sync(0xffffffffu, lB, 1);
        lA += __shfl_xor_sync(0xffffffffu, lA, 2);
        lB += __shfl_xor_sync(0xffffffffu, lB, 2);
        const float invA = lA == 0.f ? 0.f : 1.f / lA, invB = lB == 0.f ? 0.f : 1.f / lB;
        const int rowA = u.q0 + t * kBlk + rA, rowB = rowA + 8;
        // O / l as bf16.  The four threads of a row exchange their column pairs so that each
        // stores 16 bytes, 64 in a row; the fp32 O, where asked for, goes out as it lies.
#pragma unroll
        for (int half = 0; half < kVSubs; ++half) {
          uint32_t ov[32];
          if (any[t]) {
            tmem_ld_16x256b_x8_wait(lane_base + 256 + t * 128 + 64 * half, ov);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = 0u;
          }
#pragma unroll
          for (int ab = 0; ab < 2; ++ab) {
            const int row = ab ? rowB : rowA;
            const float inv = ab ? invB : invA;
            const size_t at = (static_cast<size_t>(u.bh) * p.N + row) * FA_LATENT_V + 64 * half;
            uint32_t w[8];
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
              const float x0 = __uint_as_float(ov[4 * cc + 2 * ab]) * inv;
              const float x1 = __uint_as_float(ov[4 * cc + 2 * ab + 1]) * inv;
              w[cc] = pack_bf16x2(x0, x1);
              if (o_acc && row < p.N)
                *reinterpret_cast<float2*>(o_acc + at + 8 * cc + 2 * t4) = make_float2(x0, x1);
            }
#pragma unroll
            for (int c4 = 0; c4 < 2; ++c4) {
              const uint4 x = quad_transpose(w[4 * c4], w[4 * c4 + 1], w[4 * c4 + 2],
                                             w[4 * c4 + 3], t4);
              if (row < p.N) *reinterpret_cast<uint4*>(o + at + 32 * c4 + 8 * t4) = x;
            }
          }
        }
        if (t4 == 0) {
          float* lrow = lse + static_cast<size_t>(u.bh) * p.N;
          if (rowA < p.N)
            lrow[rowA] = lA == 0.f ? -INFINITY : (m_run[t][0] + __log2f(lA)) * kLn2;
          if (rowB < p.N)
            lrow[rowB] = lB == 0.f ? -INFINITY : (m_run[t][1] + __log2f(lB)) * kLn2;
        }
      }
      if (ok) {
        tc_fence_before();   // O has been read: the next unit's first P V comes behind p_full
        int nb = 0;
        if (lane == 0) nb = next_unit(i);
        blk = __shfl_sync(0xffffffffu, nb, 0);
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

}  // namespace

cudaError_t launch_latent_fwd_sm103(const LatentProblem& p, const void* q, const void* kn,
                                    const void* kr, const void* v, void* o, float* o_acc,
                                    float* lse, cudaStream_t s) {
  CUtensorMap mq, mkn, mkr, mv;
  const int BH = p.B * p.H;
  if (!make_head_map(&mq, q, BH, p.N, FA_LATENT_NOPE + FA_LATENT_ROPE) ||
      !make_head_map(&mkn, kn, BH, p.N, FA_LATENT_NOPE) ||
      !make_head_map(&mkr, kr, p.B, p.N, FA_LATENT_ROPE) ||
      !make_head_map(&mv, v, BH, p.N, FA_LATENT_V))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(latent_fwd_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  const long long nqb = (p.N + 255) / 256;
  // Equal groups of heads whose K and V (640 N bytes a head) fit 96 MiB of L2 (all heads at once: 4%
  // slower at 200 MB; 64 MiB, more groups: 3% at 82 MB, as a group that starts late ends late).
  const int most = static_cast<int>(
      std::max(1ll, std::min<long long>(BH, (96ll << 20) / (640ll * p.N))));
  const int groups = (BH + most - 1) / most, G = (BH + groups - 1) / groups;
  return launch_dependent(latent_fwd_kernel, dim3(static_cast<unsigned>(BH * nqb)),
                          dim3(kThreads), kSmem, s, mq, mkn, mkr, mv, static_cast<__nv_bfloat16*>(o),
                          o_acc, lse, p, G);
}

}  // namespace fa
