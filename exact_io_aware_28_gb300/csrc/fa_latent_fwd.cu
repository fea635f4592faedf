// Expanded latent attention, forward, on sm_103a tensor cores (tcgen05 + TMA), bf16 in, fp32
// accumulation.
//
// Mathematics.  Head h's key is (k_nope_h, k_rope): 128 columns of its own and 64 that all heads
// of the sequence share; queries have 192 columns, values 128.  O = softmax(scale q k^T) v with
// the running maximum and sum of fa_fwd_sm103.cu (log2 domain, O unnormalised until the end and
// rescaled only past a 2^8 growth of the maximum).  The shared part is never copied per head: a
// key tile is two subtiles of the head's own tensor and one of the shared one.
//
// What bounds it: 640 operations a (query, key) pair against 832 bytes a key and 128 queries,
// so the tensor cores, and beside them the softmax.  As in fa_fwd_sm103.cu a CTA owns two tiles
// of 128 query rows, one MMA-issuing thread each, and all eight softmax warps take the tiles in
// turn: 545 us for 16 heads x 8192 without a mask (1.26 PFLOP/s), 4.2k cycles a pair of tiles
// and block of which 2.8k are MMAs.  Softmax warps of a tile's own measured slower, both four (a
// row per thread, 678 us) and eight (scores read twice, 627 us).
// Of the 227 KB of shared memory Q's two tiles hold 96, two K stages 96 and one V stage 32:
// V(j + 1) is fetched behind P V(j), while the scores of block j + 1 and their
// softmax run.  Tensor memory: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512).
// Every mbarrier wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and exits.
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
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages];
  uint64_t k_empty[kKStages];
  uint64_t v_full;
  uint64_t v_empty;
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_done[2];
  uint64_t o_staged[2];  // a tile of O is in shared memory, ready for the TMA store
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int never;  // stays 0: waits that must not be cut short by an abort
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__global__ void __launch_bounds__(kThreads, 1)
latent_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkn,
                  const __grid_constant__ CUtensorMap mkr, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mo, float* __restrict__ o_acc,
                  float* __restrict__ lse, LatentProblem p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                           // [2][kQTile]
  uint8_t* sK = sQ + 2 * kQTile;                // [kKStages][kQTile]
  uint8_t* sV = sK + kKStages * kQTile;         // [kVTile]
  Bars* bars = reinterpret_cast<Bars*>(sV + kVTile);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Work unit: groups of heads whose K and V (640 N bytes a head) fit 64 MiB of L2; in each
  // group heavy (late, causal) query blocks first, the group's heads fastest.
  const int nqb = (p.N + 2 * kBlk - 1) / (2 * kBlk);
  const int bhs = p.B * p.H;
  Unit u;
  {
    const long long per_head = 640ll * p.N;
    const int G = static_cast<int>(max(1ll, min(static_cast<long long>(bhs),
                                                (64ll << 20) / per_head)));
    const int b = blockIdx.x, g = b / (G * nqb), r = b - g * G * nqb;
    const int Gg = min(G, bhs - g * G);
    u.bh = g * G + r % Gg;
    u.q0 = (nqb - 1 - r / Gg) * 2 * kBlk;
  }
  u.nb = (p.N + kBlk - 1) / kBlk;
  const int seq = u.bh / p.H;

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
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
      mbar_init(&bars->o_staged[t], 2 * kBlk);
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
  {
    int L = p.N;
    if (p.kv_len) {
      L = p.kv_len[seq];
      L = L < 0 ? 0 : (L > p.N ? p.N : L);
    }
    u.L = L;
  }
  const int jend = key_blocks(p, u);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mkn);
      tma_prefetch_desc(&mkr);
      tma_prefetch_desc(&mv);
      mbar_arrive_expect_tx(&bars->q_full, 2 * kQTile);
      for (int t = 0; t < 2; ++t)
        for (int s = 0; s < kQKSubs; ++s)
          tma_load_3d(sQ + t * kQTile + s * kSub, &mq, &bars->q_full, 64 * s, u.q0 + t * kBlk,
                      u.bh);
      bool ok = true;
      int n = 0;
      for (int j = next_any(p, u, -1, jend); ok && j >= 0; j = next_any(p, u, j, jend), ++n) {
        const int st = n % kKStages;
        ok = mbar_wait(&bars->k_empty[st], ((n / kKStages) & 1) ^ 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars->k_full[st], kQTile);
        uint8_t* dk = sK + st * kQTile;
        tma_load_3d(dk, &mkn, &bars->k_full[st], 0, j * kBlk, u.bh);
        tma_load_3d(dk + kSub, &mkn, &bars->k_full[st], 64, j * kBlk, u.bh);
        tma_load_3d(dk + 2 * kSub, &mkr, &bars->k_full[st], 0, j * kBlk, seq);
        ok = mbar_wait(&bars->v_empty, (n & 1) ^ 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars->v_full, kVTile);
        for (int s = 0; s < kVSubs; ++s)
          tma_load_3d(sV + s * kSub, &mv, &bars->v_full, 64 * s, j * kBlk, u.bh);
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
      int last = -1;
      for (int j = jend - 1; j >= 0 && last < 0; --j)
        if (need(p, u, t, j)) last = j;
      int nk = 0, nv = 0, npv = 0;   // K and V blocks taken, P V products issued
      bool ok = mbar_wait(&bars->q_full, 0, abort_flag, p.err, p.wait_ns);
      tc_fence_after();
      // The scores of the next key block, if this tile needs them; releases the stage.
      auto take_k = [&](int j) -> bool {
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
        return true;
      };
      int j = next_any(p, u, -1, jend);
      if (ok && j >= 0) ok = take_k(j);
      while (ok && j >= 0) {
        const int jn = next_any(p, u, j, jend);
        ok = mbar_wait(&bars->v_full, nv & 1, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
        ++nv;
        tc_fence_after();
        if (need(p, u, t, j)) {
          ok = mbar_wait(&bars->p_full[t], npv & 1, abort_flag, p.err, p.wait_ns);
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
            mma_ts_x4_lo(tO, ta, db, hiV, idO, (npv > 0 || g > 0) ? 1u : 0u);
          }
          ++npv;
          if (j == last) mma_commit(&bars->o_done[t]);
        }
        mma_commit(&bars->v_empty);
        if (jn >= 0) ok = take_k(jn);
        j = jn;
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
    float m_run[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};  // [tile][A/B]
    float l_part[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    int n_t[2] = {0, 0};
    bool ok = true;
    for (int j = 0; j < jend && ok; ++j) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || !need(p, u, t, j)) continue;
        ok = mbar_wait_warp(&bars->s_full[t], n_t[t] & 1, abort_flag, p.err, p.wait_ns);
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
        float mA = fmaxf(ma0, ma1), mB = fmaxf(mb0, mb1);
        mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 1));
        mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 1));
        mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 2));
        mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 2));
        mA *= c;
        mB *= c;
        const float oldA = m_run[t][0], oldB = m_run[t][1];
        const float newA = mA > oldA + kRescaleThreshold ? mA : oldA;
        const float newB = mB > oldB + kRescaleThreshold ? mB : oldB;
        const bool chA = newA != oldA, chB = newB != oldB;
        const float alphaA = chA ? ex2(oldA - newA) : 1.f;  // old = -inf gives 0
        const float alphaB = chB ? ex2(oldB - newB) : 1.f;
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
        if (n_t[t] > 0 && __any_sync(0xffffffffu, chA || chB)) {
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
          // 0 x (anything) stays 0.  Block j is the (j + 1)-th fill of the V stage.
          ok = mbar_wait_warp(&bars->v_full, j & 1, abort_flag, p.err, p.wait_ns);
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
        ++n_t[t];
      }
    }
    // ------------------------------------------------------------ epilogue
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (ok && n_t[t] > 0) {
        ok = mbar_wait_warp(&bars->o_done[t], 0, abort_flag, p.err, p.wait_ns);
        tc_fence_after();
      }
      if (!ok) break;
      if (n_t[t] == 0) {
        // No product has read Q's tile, so nothing says that its load has landed; O goes over it.
        ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.err, p.wait_ns);
        if (!ok) break;
      }
      float lA = l_part[t][0], lB = l_part[t][1];
      lA += __shfl_xor_sync(0xffffffffu, lA, 1);
      lB += __shfl_xor_sync(0xffffffffu, lB, 1);
      lA += __shfl_xor_sync(0xffffffffu, lA, 2);
      lB += __shfl_xor_sync(0xffffffffu, lB, 2);
      const float invA = lA == 0.f ? 0.f : 1.f / lA, invB = lB == 0.f ? 0.f : 1.f / lB;
      const int rowA = u.q0 + t * kBlk + rA, rowB = rowA + 8;
      // O / l as bf16 into this tile's Q buffer (every S MMA that read it has completed), in the
      // 128-byte-swizzled layout of the TMA box; one thread then stores the tile (rows past N
      // are clipped).  The fp32 O, where asked for, goes out from the registers.
      uint8_t* stage = sQ + t * kQTile;
#pragma unroll
      for (int half = 0; half < kVSubs; ++half) {
        uint32_t ov[32];
        if (n_t[t] > 0) {
          tmem_ld_16x256b_x8_wait(lane_base + 256 + t * 128 + 64 * half, ov);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = 0u;
        }
        uint8_t* sub = stage + half * kSub;
        float* accA = o_acc ? o_acc + (static_cast<size_t>(u.bh) * p.N + rowA) * FA_LATENT_V +
                                  64 * half + 2 * t4
                            : nullptr;
        float* accB = o_acc ? accA + 8 * FA_LATENT_V : nullptr;
#pragma unroll
        for (int cc = 0; cc < 8; ++cc) {
          const uint32_t byte = static_cast<uint32_t>(4 * t4);   // column 8cc + 2t4, bf16
          const float a0 = __uint_as_float(ov[4 * cc]) * invA;
          const float a1 = __uint_as_float(ov[4 * cc + 1]) * invA;
          const float b0 = __uint_as_float(ov[4 * cc + 2]) * invB;
          const float b1 = __uint_as_float(ov[4 * cc + 3]) * invB;
          *reinterpret_cast<uint32_t*>(sub + rA * 128 + ((cc ^ (rA & 7)) << 4) + byte) =
              pack_bf16x2(a0, a1);
          *reinterpret_cast<uint32_t*>(sub + rB * 128 + ((cc ^ (rB & 7)) << 4) + byte) =
              pack_bf16x2(b0, b1);
          if (o_acc) {
            if (rowA < p.N) *reinterpret_cast<float2*>(accA + 8 * cc) = make_float2(a0, a1);
            if (rowB < p.N) *reinterpret_cast<float2*>(accB + 8 * cc) = make_float2(b0, b1);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->o_staged[t]);
      if (warp == 4 && lane == 0 && u.q0 + t * kBlk < p.N) {
        if (mbar_wait(&bars->o_staged[t], 0, abort_flag, p.err, p.wait_ns)) {
#pragma unroll
          for (int half = 0; half < kVSubs; ++half)
            tma_store_3d(&mo, stage + half * kSub, 64 * half, u.q0 + t * kBlk, u.bh);
          bulk_commit_group();
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
  }

  if (warp == 4 && lane == 0) bulk_wait_group_all();
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
  CUtensorMap mq, mkn, mkr, mv, mo;
  const int BH = p.B * p.H;
  if (!make_head_map(&mq, q, BH, p.N, FA_LATENT_NOPE + FA_LATENT_ROPE) ||
      !make_head_map(&mkn, kn, BH, p.N, FA_LATENT_NOPE) ||
      !make_head_map(&mkr, kr, p.B, p.N, FA_LATENT_ROPE) ||
      !make_head_map(&mv, v, BH, p.N, FA_LATENT_V) || !make_head_map(&mo, o, BH, p.N, FA_LATENT_V))
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
  return launch_dependent(latent_fwd_kernel, dim3(static_cast<unsigned>(BH * nqb)),
                          dim3(kThreads), kSmem, s, mq, mkn, mkr, mv, mo, o_acc, lse, p);
}

}  // namespace fa
