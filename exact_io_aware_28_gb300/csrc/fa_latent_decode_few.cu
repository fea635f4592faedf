// Absorbed latent decode over a paged latent cache for at most 16 heads (a shard of the heads);
// the mathematics stands in fa_latent_decode.cu.
//
// What bounds it: HBM.  16 heads ask for 30 operations a byte, a tenth of what the tensor cores
// could do, but a tcgen05 MMA takes the pipe 47 cycles however few its columns are, and 68 of them
// a 128-key tile with the hand-overs between them measured twice the time of the bytes.  Sixteen
// rows are one tile of the warp-level MMA (m16n8k16), whose operands and results stay in the
// warps' registers: no hand-over but two block barriers a tile.
//   tile    64 keys x 576 columns (72 KB), three stages;
//   scores  warp w of 8 has keys 8 w ... 8 w + 7 and all 576 columns, q in registers (144);
//   softmax a warp's maxima through shared memory, P as bf16 [16][64] in shared memory;
//   P V     warp w has columns 64 w ... 64 w + 63 of the output (32 registers) and all keys.
// The rows of a thread's scores and of its outputs are the same two heads, so maxima, sums and
// the rescaling (only past a 2^8 growth) need no exchange of their own.  There is no loading
// warp, since a ninth warp would halve the registers: behind the first barrier of tile n every
// warp is done with tile n - 1, and each warp asks for one subtile of tile n + 2 in its stage (all
// nine by one warp took 1.4k cycles, which the others waited out at the second barrier), the page
// numbers looked up a tile ago.
// All 255 registers are taken, and 72 bytes of a thread's values spill.
// Measured: 32 sequences of 4096 to 8192 tokens, 16 heads: 58 us for 34 us of bytes (3.9 TB/s), the
// join in it; 2 sequences of 901 tokens 11.4 us.
// Work is shared out as fa_paged_sched.cuh says.  Waits are bounded: after an expiry the block
// runs on without waiting, in step with its barriers, and records FA_ERR_TIMEOUT.
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
constexpr int kSubs = kRow / 64;              // 64-column subtiles of a row
constexpr int kSub = kFewKeys * 128;          // [64 keys][64 columns], 128-byte swizzled
constexpr int kStage = kSubs * kSub;
constexpr int kStages = 3;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPStride = 2 * kFewKeys + 16;   // bytes of a row of P: 16 past a multiple of 128
constexpr int kQPart = 3 * 64;                // columns of q that pass through shared memory at once
constexpr int kQStride = 2 * kQPart + 16;     // bytes of a row of them: 16 past a multiple of 128
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units; exact, see fa_fwd_sm103.cu
static_assert(kRank == 64 * kWarps && kFewKeys == 8 * kWarps, "a warp's share");

struct Shared {
  uint64_t full[kStages];
  uint32_t seen[kStages];     // bit i: rows 16 i ... 16 i + 15 of the stage are in the pool
  int abort;
  sched::Start start;
  long long scan[kThreads / 32 + 1];
  float wmax[2][kWarps][kFewHeads];
  float wsum[kWarps][kFewHeads];
  alignas(16) uint8_t pq[kFewHeads * kQStride];   // P; between segments a third of q
};

constexpr int kSmem = 1024 + kStages * kStage + static_cast<int>(sizeof(Shared));
static_assert(kSmem <= 227 * 1024 && kPStride <= kQStride, "shared memory");

__global__ void __launch_bounds__(kThreads, 1)
latent_decode_few_kernel(const __grid_constant__ CUtensorMap mc, LatentArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sC = base;                                  // [kStages][kSubs][64 keys][64]
  Shared* sh = reinterpret_cast<Shared*>(sC + kStages * kStage);
  volatile int* abort_flag = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.max_pages << a.page_shift;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sh->full[s], 1);
    sh->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mc);
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  sched::find_start<kFewKeys, kThreads>(&sh->start, sh->scan, a.cache_len, a.B, 1, cap, blockIdx.x,
                                        gridDim.x, blockIdx.x == 0 ? a.prefix : nullptr);
  // ------------------------------------------------------------ loading
  // The next tile to ask for: segment ls, keys from lk on; lp is the page of the lane's box.
  const int shift = a.page_shift;
  const int rows = min(kFewKeys, 1 << shift);       // rows of a box
  const int boxes = kFewKeys / rows;
  sched::Walk<kFewKeys> ahead(sh->start, a.cache_len, 1, cap);
  Segment ls;
  int lk = 0, lp = -1, ln = 0;
  bool left = ahead.next(ls);
  auto look_up = [&]() {
    const int x = lk + lane * rows;                 // first token of box `lane`
    lp = -1;
    if (lane < boxes && x < ls.len) {
      const int p = a.table[ls.b * a.table_stride + (x >> shift)];
      lp = p >= 0 && p < a.num_pages ? p : -1;
    }
  };
  if (left) {
    lk = ls.k0;
    look_up();
  }
  // What the tile's stage expects: warp 0, before a barrier that the copies come behind.
  auto expect = [&]() {
    if (warp != 0 || !left || *abort_flag) return;
    const uint32_t pages = __ballot_sync(0xffffffffu, lp >= 0);
    if (lane == 0) {
      const uint32_t bits = (1u << (rows / 16)) - 1u;
      uint32_t seen = 0;
      for (int i = 0; i < boxes; ++i)
        if (pages >> i & 1u) seen |= bits << (i * (rows / 16));
      sh->seen[ln % kStages] = seen;
      mbar_arrive_expect_tx(&sh->full[ln % kStages],
                            static_cast<uint32_t>(__popc(pages)) * rows * kRow * 2);
    }
  };
  auto ask = [&]() {
    if (!left || *abort_flag) return;
    if (lp >= 0) {
      const int st = ln % kStages, y = (lk + lane * rows) & ((1 << shift) - 1);
      for (int s = warp; s < kSubs; s += kWarps)
        tma_load_4d(sC + st * kStage + s * kSub + lane * rows * 128, &mc, &sh->full[st], 64 * s, y,
                    0, lp);
    }
    ++ln;
    lk += kFewKeys;
    if (lk >= ls.k1) {
      left = ahead.next(ls);
      lk = ls.k0;
    }
    if (left) look_up();
  };
  for (int i = 0; i < kStages - 1; ++i) {
    expect();
    __syncthreads();
    ask();
  }

  // ------------------------------------------------------------ products and softmax
  sched::Walk<kFewKeys> walk(sh->start, a.cache_len, 1, cap);
  Segment sg;
  {
    // A thread's heads are hA = lane / 4 and hB = hA + 8; its keys of a score tile are
    // 8 warp + 2 (lane % 4) + {0, 1}, its columns of an output tile 2 (lane % 4) + {0, 1}.
    const int t4 = lane & 3, hA = lane >> 2, hB = hA + 8;
    const int key = 8 * warp + 2 * t4;
    // Addresses of the thread's rows for ldmatrix: of the warp's keys for the scores (matrix
    // lane / 8 is the 16-byte piece), of P, and of the keys for P V (transposed).
    const uint32_t uC = smem_u32(sC), uP = smem_u32(sh->pq);
    const int srow = 8 * warp + (lane & 7), spiece = lane >> 3;
    const uint32_t uPl = uP + ((lane & 7) + ((lane >> 3) & 1) * 8) * kPStride + (lane >> 4) * 16;
    const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vpiece = lane >> 4;
    bool ok = true;
    int n = 0;
    while (walk.next(sg)) {
      // q as A operands of the 36 steps of 16 columns; heads past H are zero.  The rows come in
      // one piece of coalesced loads, then a third at a time through shared memory (fragments
      // straight from global memory took 4.6 us a segment: 144 scattered loads a thread).
      uint32_t qa[kRow / 16][4];
      {
        constexpr int kPieces = kFewHeads * kRow / 8, kPer = (kPieces + kThreads - 1) / kThreads;
        constexpr int kPartPieces = kQPart / 8;
        const uint4* src = reinterpret_cast<const uint4*>(a.q) +
                           static_cast<size_t>(sg.b) * a.H * (kRow / 8);
        uint4 raw[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = tid + i * kThreads;
          raw[i] = e < a.H * (kRow / 8) ? src[e] : make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t uQl = smem_u32(sh->pq) +
                             ((lane & 7) + ((lane >> 3) & 1) * 8) * kQStride + (lane >> 4) * 16;
#pragma unroll
        for (int part = 0; part < kRow / kQPart; ++part) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int e = tid + i * kThreads, h = e / (kRow / 8);
            const int c = e - h * (kRow / 8) - part * kPartPieces;
            if (e < kPieces && c >= 0 && c < kPartPieces)
              *reinterpret_cast<uint4*>(sh->pq + h * kQStride + 16 * c) = raw[i];
          }
          __syncthreads();
#pragma unroll
          for (int k = 0; k < kQPart / 16; ++k) ldmatrix_x4(qa[part * (kQPart / 16) + k], uQl + 32 * k);
        }
      }
      float acc[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kFewKeys, ++n) {
        const int st = n % kStages;
        if (ok)
          ok = mbar_wait_warp(&sh->full[st], (n / kStages) & 1, abort_flag, a.err, a.wait_ns);
        const uint32_t seen = sh->seen[st];
        const int valid = sg.k1 - k0;
        // ---- scores of the warp's 8 keys, in four chains
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
        const uint32_t rowC = uC + st * kStage + srow * 128;
#pragma unroll
        for (int j = 0; j < kRow / 32; ++j) {      // 32 columns: four pieces of a subtile
          uint32_t b[4];
          ldmatrix_x4(b, rowC + (j >> 1) * kSub + (((4 * (j & 1) + spiece) ^ (srow & 7)) << 4));
          mma_16816(sc[2 * (j & 1)], qa[2 * j], b[0], b[1]);
          mma_16816(sc[2 * (j & 1) + 1], qa[2 * j + 1], b[2], b[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[0][j] = ((sc[0][j] + sc[1][j]) + (sc[2][j] + sc[3][j])) * a.c;
        const bool page = (seen >> (warp >> 1)) & 1u;
        const bool v0 = page && key < valid, v1 = page && key + 1 < valid;
        float x[4];
        x[0] = v0 ? sc[0][0] : -INFINITY;
        x[1] = v1 ? sc[0][1] : -INFINITY;
        x[2] = v0 ? sc[0][2] : -INFINITY;
        x[3] = v1 ? sc[0][3] : -INFINITY;
        float tA = fmaxf(x[0], x[1]), tB = fmaxf(x[2], x[3]);
        tA = fmaxf(tA, __shfl_xor_sync(0xffffffffu, tA, 1));
        tB = fmaxf(tB, __shfl_xor_sync(0xffffffffu, tB, 1));
        tA = fmaxf(tA, __shfl_xor_sync(0xffffffffu, tA, 2));
        tB = fmaxf(tB, __shfl_xor_sync(0xffffffffu, tB, 2));
        float (&wm)[kWarps][kFewHeads] = sh->wmax[n & 1];
        if (t4 == 0) {
          wm[warp][hA] = tA;
          wm[warp][hB] = tB;
        }
        if (valid < kFewKeys || seen != 0xfu) {
          // Hidden rows: zero their values, so that 0 x (anything) stays 0.
          const int r = tid >> 2;
          if (r >= valid || !((seen >> (r >> 4)) & 1u)) {
            uint8_t* vt = sC + st * kStage + r * 128 + (tid & 3) * 2 * kSub;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint4*>(vt + (i >> 3) * kSub + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();              // before the stage's next fill
          }
        }
        expect();
        __syncthreads();
        ask();                                     // over tile n - 1
        tA = wm[0][hA];
        tB = wm[0][hB];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          tA = fmaxf(tA, wm[w][hA]);
          tB = fmaxf(tB, wm[w][hB]);
        }
        const float nA = tA > mA + kRescaleThreshold ? tA : mA;
        const float nB = tB > mB + kRescaleThreshold ? tB : mB;
        const bool ch = nA != mA || nB != mB;
        const float alphaA = nA != mA ? ex2(mA - nA) : 1.f;   // m = -inf gives 0
        const float alphaB = nB != mB ? ex2(mB - nB) : 1.f;
        mA = nA;
        mB = nB;
        const float useA = nA == -INFINITY ? 0.f : nA, useB = nB == -INFINITY ? 0.f : nB;
        const float p0 = ex2(x[0] - useA), p1 = ex2(x[1] - useA);
        const float p2 = ex2(x[2] - useB), p3 = ex2(x[3] - useB);
        lA = fmaf(lA, alphaA, p0 + p1);
        lB = fmaf(lB, alphaB, p2 + p3);
        *reinterpret_cast<uint32_t*>(sh->pq + hA * kPStride + 2 * key) = pack_bf16x2(p0, p1);
        *reinterpret_cast<uint32_t*>(sh->pq + hB * kPStride + 2 * key) = pack_bf16x2(p2, p3);
        if (ch) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[i][0] *= alphaA;
            acc[i][1] *= alphaA;
            acc[i][2] *= alphaB;
            acc[i][3] *= alphaB;
          }
        }
        __syncthreads();
        // ---- P V: 16 keys a step, the warp's 64 columns
        const uint32_t tileV = uC + st * kStage + warp * kSub;
#pragma unroll
        for (int k = 0; k < kFewKeys / 16; ++k) {
          uint32_t pa[4];
          ldmatrix_x4(pa, uPl + 32 * k);
          const int r = 16 * k + vrow;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b[4];
            ldmatrix_x4_trans(b, tileV + r * 128 + (((2 * i + vpiece) ^ (r & 7)) << 4));
            mma_16816(acc[2 * i], pa, b[0], b[1]);
            mma_16816(acc[2 * i + 1], pa, b[2], b[3]);
          }
        }
      }
      // ---- the segment's result
      lA += __shfl_xor_sync(0xffffffffu, lA, 1);
      lB += __shfl_xor_sync(0xffffffffu, lB, 1);
      lA += __shfl_xor_sync(0xffffffffu, lA, 2);
      lB += __shfl_xor_sync(0xffffffffu, lB, 2);
      if (t4 == 0) {
        sh->wsum[warp][hA] = lA;
        sh->wsum[warp][hB] = lB;
      }
      __syncthreads();
      lA = lB = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lA += sh->wsum[w][hA];
        lB += sh->wsum[w][hB];
      }
      const int slot = sched::slot(sg.pair_start, sh->start.first, blockIdx.x);
      const size_t head0 = static_cast<size_t>(sg.b) * a.H;
      const size_t prow0 = static_cast<size_t>(slot) * a.H;
#pragma unroll
      for (int ab = 0; ab < 2; ++ab) {
        const int h = ab ? hB : hA;
        if (h >= a.H) continue;
        const float l = ab ? lB : lA, m = ab ? mB : mA;
        const float inv = l == 0.f ? 0.f : 1.f / l;           // a NaN sum stays one
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int col = 64 * warp + 8 * i + 2 * t4;
          const float o0 = acc[i][2 * ab], o1 = acc[i][2 * ab + 1];
          if (sg.whole)
            *reinterpret_cast<uint32_t*>(a.o + (head0 + h) * kRank + col) =
                pack_bf16x2(o0 * inv, o1 * inv);
          else
            *reinterpret_cast<float2*>(a.part + (prow0 + h) * kRank + col) = make_float2(o0, o1);
        }
        if (warp == 0 && t4 == 0) {
          if (sg.whole) {
            a.lse[head0 + h] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
          } else {
            // The same statistics serve both halves of the columns.
            a.stat[static_cast<size_t>(slot) * 2 * a.H + h] = make_float2(m, l);
            a.stat[(static_cast<size_t>(slot) * 2 + 1) * a.H + h] = make_float2(m, l);
          }
        }
      }
      // The sums are rewritten only behind the next segment's first barrier.
    }
  }

  __syncthreads();
  if (sh->abort && tid == 0) {
    // Let any copy still in flight land before the CTA's shared memory is released.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncthreads();
}

}  // namespace

cudaError_t launch_latent_decode_few(const CUtensorMap& mc, const LatentArgs& a, int workers,
                                     cudaStream_t s) {
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(latent_decode_few_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  return launch_dependent(latent_decode_few_kernel, dim3(workers), dim3(kThreads), kSmem, s, mc, a);
}

}  // namespace fa
