// Expanded latent attention on the CUDA cores (fp32 arithmetic), and the two row kernels of
// its backward that both paths use.
//
// Mathematics.  Head h has the key k_j = (k_nope_hj, k_rope_j) of 128 + 64 columns, the last 64
// shared by all heads, and values of 128 columns.  With s_ij = scale q_i . k_j, P = softmax(s):
//   O = P V,  D_i = dO_i . O_i,  dS_ij = P_ij (dO_i . v_j - D_i),  dV_j = sum_i P_ij dO_i,
//   dQ_i = scale sum_j dS_ij k_j,  dK_nope_j = scale sum_i dS_ij q_i[0:128],
//   dK_rope_j = scale sum_h sum_i dS_hij q_hi[128:192].
// D is formed from the fp32 O that the forward leaves: a row's dS sums P (dP - D) over all its
// keys, so a D that is off by O's rounding to bf16 moves dQ and dK by as much as the rounding of
// dS itself (1.5 to 2 times a single rounding in causal rows, against 1.43 with fp32 O).
// The heads' shares of dK_rope go to the workspace in fp32 and are added in order of the heads,
// so the result does not depend on scheduling.
//
// This path serves fp32 tensors and runs at the rate of the FMA pipes, if shared memory lets it:
// a dot product per thread reads as many words as it does multiply-adds (549 us for a training
// step of 2 x 3 heads x 333 rows).  So both products of a tile are register tiles: a CTA of
// 16 x 16 threads owns 16 RT rows and streams 64 rows at a time; a thread forms RT x 4 scores
// from four columns of a row per 16-byte load, and RT x 4 of every 64 columns of the result from
// P or dS in shared memory (140 us).  Scores are in the log2 domain.
#include <math.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNope = FA_LATENT_NOPE, kRope = FA_LATENT_ROPE, kQK = kNope + kRope;
constexpr int kV = FA_LATENT_V;
constexpr int kCols = 64;      // rows of the streamed side per tile
constexpr int kThreads = 256;  // 16 x 16
constexpr int kDotRows = 32;   // rows of a block of latent_rowdot_kernel
// Row strides in shared memory: 16 bytes past a multiple of 128, so that eight rows' pieces of
// 16 bytes lie in different banks.
constexpr int kSX = kQK + 4, kSY = kV + 4, kSP = kCols + 4;

__device__ __forceinline__ int key_limit(const LatentProblem& p, int b) {
  if (!p.kv_len) return p.N;
  const int L = p.kv_len[b];
  return L < 0 ? 0 : (L > p.N ? p.N : L);
}

// Sum and maximum over the 16 threads that share a row.
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// `count` rows of `src` from row r0 on (W columns each) into `dst`; rows from `limit` on are 0.
template <int W, int STRIDE>
__device__ __forceinline__ void load_rows(float* dst, const float* src, int r0, int limit,
                                          int count) {
  for (int e = threadIdx.x; e < count * (W / 4); e += kThreads) {
    const int i = e / (W / 4), c = e % (W / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + i < limit) x = reinterpret_cast<const float4*>(src + static_cast<size_t>(r0 + i) * W)[c];
    *reinterpret_cast<float4*>(dst + i * STRIDE + 4 * c) = x;
  }
}

// The rows (k_nope, k_rope) of a head's keys.
__device__ __forceinline__ void load_keys(float* dst, const float* kn, const float* kr, int r0,
                                          int limit, int count) {
  load_rows<kNope, kSX>(dst, kn, r0, limit, count);
  load_rows<kRope, kSX>(dst + kNope, kr, r0, limit, count);
}

// acc[i][j] = own row (RT ty + i) . streamed row (tx + 16 j) over W columns.
template <int RT, int W, int STRIDE>
__device__ __forceinline__ void dots(float (&acc)[RT][4], const float* own, const float* str) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int k = 0; k < W; k += 4) {
    float4 a[RT], b[4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
      a[i] = *reinterpret_cast<const float4*>(own + (RT * ty + i) * STRIDE + k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b[j] = *reinterpret_cast<const float4*>(str + (tx + 16 * j) * STRIDE + k);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y,
                    fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
  }
}

// acc[i][4 g + c] += sum over the tile's rows j of w[RT ty + i][j] x[j][64 g + 4 tx + c].
template <int RT, int G, int STRIDE>
__device__ __forceinline__ void mix(float (&acc)[RT][4 * G], const float* w, const float* x) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int j = 0; j < kCols; j += 4) {
    float a[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float4 x4 = *reinterpret_cast<const float4*>(w + (RT * ty + i) * kSP + j);
      a[i][0] = x4.x;
      a[i][1] = x4.y;
      a[i][2] = x4.z;
      a[i][3] = x4.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float4 b = *reinterpret_cast<const float4*>(x + (j + jj) * STRIDE + 64 * g + 4 * tx);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          acc[i][4 * g] = fmaf(a[i][jj], b.x, acc[i][4 * g]);
          acc[i][4 * g + 1] = fmaf(a[i][jj], b.y, acc[i][4 * g + 1]);
          acc[i][4 * g + 2] = fmaf(a[i][jj], b.z, acc[i][4 * g + 2]);
          acc[i][4 * g + 3] = fmaf(a[i][jj], b.w, acc[i][4 * g + 3]);
        }
      }
  }
}

template <int RT>
constexpr int fwd_smem() {
  return (16 * RT * (kSX + kSP) + kCols * (kSX + kSY)) * static_cast<int>(sizeof(float));
}
template <int RT>
constexpr int bwd_smem() {
  return (16 * RT * (kSX + kSY + 2 * kSP) + kCols * (kSX + kSY + 2)) *
         static_cast<int>(sizeof(float));
}
static_assert(bwd_smem<4>() <= 227 * 1024, "shared memory");

template <int RT>
__global__ void __launch_bounds__(kThreads)
latent_fwd_simt_kernel(const float* __restrict__ q, const float* __restrict__ kn,
                       const float* __restrict__ kr, const float* __restrict__ v, float* o,
                       float* o_acc, float* __restrict__ lse, LatentProblem p) {
  constexpr int R = 16 * RT;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);   // [R][kSX]
  float* ps = qs + R * kSX;                      // [R][kSP]
  float* ks = ps + R * kSP;                      // [64][kSX]
  float* vs = ks + kCols * kSX;                  // [64][kSY]
  const int N = p.N, bh = blockIdx.y, b = bh / p.H;
  const size_t head = static_cast<size_t>(bh) * N, seq = static_cast<size_t>(b) * N;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int row0 = (gridDim.x - 1 - blockIdx.x) * R;       // the longest (causal) rows first
  const float c = p.scale * kLog2e;
  load_rows<kQK, kSX>(qs, q + head * kQK, row0, N, R);
  float acc[RT][8], m[RT], l[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  int kend = key_limit(p, b);
  if (p.causal) kend = min(kend, row0 + R);
  for (int k0 = 0; k0 < kend; k0 += kCols) {
    __syncthreads();
    load_keys(ks, kn + head * kNope, kr + seq * kRope, k0, kend, kCols);
    load_rows<kV, kSY>(vs, v + head * kV, k0, kend, kCols);
    __syncthreads();
    float s[RT][4];
    dots<RT, kQK, kSX>(s, qs, ks);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = row0 + RT * ty + i;
      const int lim = p.causal ? min(kend, row + 1) : kend;
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = k0 + tx + 16 * j < lim ? s[i][j] * c : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
      mt = fmaxf(m[i], row_max(mt));
      const float use = mt == -INFINITY ? 0.f : mt;
      const float alpha = exp2f(m[i] - use);      // m = -inf gives 0
      m[i] = mt;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pj = exp2f(s[i][j] - use);
        sum += pj;
        ps[(RT * ty + i) * kSP + tx + 16 * j] = pj;
      }
      l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] *= alpha;
    }
    __syncthreads();
    mix<RT, 2, kSY>(acc, ps, vs);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = row0 + RT * ty + i;
    const float lt = row_sum(l[i]);
    const float inv = lt == 0.f ? 0.f : 1.f / lt;   // a NaN sum stays one
    if (row >= N) continue;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float4 x = make_float4(acc[i][4 * g] * inv, acc[i][4 * g + 1] * inv,
                                   acc[i][4 * g + 2] * inv, acc[i][4 * g + 3] * inv);
      const size_t at = (head + row) * kV + 64 * g + 4 * tx;
      *reinterpret_cast<float4*>(o + at) = x;
      if (o_acc) *reinterpret_cast<float4*>(o_acc + at) = x;
    }
    if (tx == 0) lse[head + row] = lt == 0.f ? -INFINITY : (m[i] + log2f(lt)) * kLn2;
  }
}

// DQ = false: the CTA owns keys and streams queries (dK, dV); DQ = true: the other way (dQ).
template <bool DQ, int RT>
__device__ __forceinline__ void bwd_tile(const float* __restrict__ q, const float* __restrict__ kn,
                                         const float* __restrict__ kr, const float* __restrict__ v,
                                         const float* __restrict__ lse,
                                         const float* __restrict__ dO,
                                         const float* __restrict__ Dsum, float* __restrict__ dq,
                                         float* __restrict__ dkn, float* __restrict__ dkr_part,
                                         float* __restrict__ dv, const LatentProblem& p) {
  constexpr int R = 16 * RT;
  extern __shared__ float4 smem4[];
  float* ox = reinterpret_cast<float*>(smem4);   // owned: q or k, [R][kSX]
  float* oy = ox + R * kSX;                      // owned: dO or v, [R][kSY]
  float* ps = oy + R * kSY;                      // [R][kSP], P (dK, dV)
  float* ds = ps + R * kSP;                      // [R][kSP], dS
  float* sx = ds + R * kSP;                      // streamed: k or q, [64][kSX]
  float* sy = sx + kCols * kSX;                  // streamed: v or dO, [64][kSY]
  float* sl = sy + kCols * kSY;                  // streamed rows' lse and D (dK, dV)
  float* sd = sl + kCols;
  const int N = p.N, bh = blockIdx.y, b = bh / p.H;
  const size_t head = static_cast<size_t>(bh) * N, seq = static_cast<size_t>(b) * N;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // The tiles with the most work first (causal: early keys, late queries).
  const int row0 = (DQ ? gridDim.x - 1 - blockIdx.x : blockIdx.x) * R;
  const int L = key_limit(p, b);
  const float c = p.scale * kLog2e;
  float ax[RT][12], ay[RT][8];                   // dQ or dK; dV
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int j = 0; j < 12; ++j) ax[i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ay[i][j] = 0.f;
  }
  float own_lse[RT], own_D[RT];
  if constexpr (DQ) {
    load_rows<kQK, kSX>(ox, q + head * kQK, row0, N, R);
    load_rows<kV, kSY>(oy, dO + head * kV, row0, N, R);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = row0 + RT * ty + i;
      own_lse[i] = row < N ? lse[head + row] : -INFINITY;
      own_D[i] = row < N ? Dsum[head + row] : 0.f;
    }
  } else {
    load_keys(ox, kn + head * kNope, kr + seq * kRope, row0, L, R);
    load_rows<kV, kSY>(oy, v + head * kV, row0, L, R);
  }
  int begin = 0, end = DQ ? L : (row0 < L ? N : 0);
  if (p.causal && DQ) end = min(end, row0 + R);
  if (p.causal && !DQ) begin = row0 / kCols * kCols;
  for (int c0 = begin; c0 < end; c0 += kCols) {
    __syncthreads();
    if constexpr (DQ) {
      load_keys(sx, kn + head * kNope, kr + seq * kRope, c0, end, kCols);
      load_rows<kV, kSY>(sy, v + head * kV, c0, end, kCols);
    } else {
      load_rows<kQK, kSX>(sx, q + head * kQK, c0, end, kCols);
      load_rows<kV, kSY>(sy, dO + head * kV, c0, end, kCols);
      if (threadIdx.x < kCols) {
        const int row = c0 + threadIdx.x;
        sl[threadIdx.x] = row < N ? lse[head + row] : -INFINITY;
        sd[threadIdx.x] = row < N ? Dsum[head + row] : 0.f;
      }
    }
    __syncthreads();
    float s[RT][4], dp[RT][4];
    dots<RT, kQK, kSX>(s, ox, sx);
    dots<RT, kV, kSY>(dp, oy, sy);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int own = row0 + RT * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = c0 + tx + 16 * j;
        const int key = DQ ? col : own, row = DQ ? own : col;
        const float rl = DQ ? own_lse[i] : sl[tx + 16 * j];   // -inf: no key seen, or no such row
        const float rd = DQ ? own_D[i] : sd[tx + 16 * j];
        const bool seen = key < L && !(p.causal && key > row) && rl != -INFINITY;
        const float pij = seen ? exp2f(fmaf(-kLog2e, rl, s[i][j] * c)) : 0.f;
        if (!DQ) ps[(RT * ty + i) * kSP + tx + 16 * j] = pij;
        ds[(RT * ty + i) * kSP + tx + 16 * j] = seen ? pij * (dp[i][j] - rd) : 0.f;
      }
    }
    __syncthreads();
    mix<RT, 3, kSX>(ax, ds, sx);
    if constexpr (!DQ) mix<RT, 2, kSY>(ay, ps, sy);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int own = row0 + RT * ty + i;
    if (own >= N) continue;
    const size_t at = head + own;
#pragma unroll
    for (int g = 0; g < 3; ++g) {
      const float4 x = make_float4(ax[i][4 * g] * p.scale, ax[i][4 * g + 1] * p.scale,
                                   ax[i][4 * g + 2] * p.scale, ax[i][4 * g + 3] * p.scale);
      float* dst = DQ ? dq + at * kQK + 64 * g
                      : g < 2 ? dkn + at * kNope + 64 * g : dkr_part + at * kRope;
      *reinterpret_cast<float4*>(dst + 4 * tx) = x;
    }
    if constexpr (!DQ) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
        *reinterpret_cast<float4*>(dv + at * kV + 64 * g + 4 * tx) =
            make_float4(ay[i][4 * g], ay[i][4 * g + 1], ay[i][4 * g + 2], ay[i][4 * g + 3]);
    }
  }
}

// Both in one grid (z): neither needs the other, and short sequences do not fill the card twice.
template <int RT>
__global__ void __launch_bounds__(kThreads)
latent_bwd_simt_kernel(const float* __restrict__ q, const float* __restrict__ kn,
                       const float* __restrict__ kr, const float* __restrict__ v,
                       const float* __restrict__ lse, const float* __restrict__ dO,
                       const float* __restrict__ Dsum, float* __restrict__ dq,
                       float* __restrict__ dkn, float* __restrict__ dkr_part,
                       float* __restrict__ dv, LatentProblem p) {
  if (blockIdx.z == 0)
    bwd_tile<false, RT>(q, kn, kr, v, lse, dO, Dsum, dq, dkn, dkr_part, dv, p);
  else
    bwd_tile<true, RT>(q, kn, kr, v, lse, dO, Dsum, dq, dkn, dkr_part, dv, p);
}

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
}

// Eight values from 16-byte loads.
__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = load4(p), b = load4(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(float (&x)[8], const __nv_bfloat16* p) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}

// D_i = dO_i . O_i: sixteen threads a row with eight columns each, two rows a thread whose loads are
// all under way at once.  HBM-bound; with fewer rows, one round of loads (2 x 8 heads x 1000: a warp
// per row, row after row, took the step 8 us longer; four rows a thread 1 us).
template <typename T>
__global__ void __launch_bounds__(256)
latent_rowdot_kernel(const float* __restrict__ o_acc, const T* __restrict__ dO,
                     float* __restrict__ Dsum, long long rows) {
  constexpr int kEach = kDotRows / 16;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int col = 8 * (threadIdx.x & 15);
  const long long step = static_cast<long long>(gridDim.x) * kDotRows;
  for (long long r0 = static_cast<long long>(blockIdx.x) * kDotRows; r0 < rows; r0 += step) {
    float a[kEach][8], b[kEach][8];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const long long row = r0 + 16 * j + (threadIdx.x >> 4);
      if (row < rows) {
        load8(a[j], o_acc + row * kV + col);
        load8(b[j], dO + row * kV + col);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[j][i] = b[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(a[j][i], b[j][i], s);
      s = row_sum(s);
      const long long row = r0 + 16 * j + (threadIdx.x >> 4);
      if (col == 0 && row < rows) Dsum[row] = s;
    }
  }
}

// dK_rope = the heads' shares added in order: four columns a thread.  HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256)
latent_rope_sum_kernel(const float* __restrict__ part, T* __restrict__ dkr, int H, long long NR,
                       long long total) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long step = static_cast<long long>(gridDim.x) * 256;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += step) {
    const long long b = 4 * i / NR, at = 4 * i - b * NR;   // NR = N * 64 values a sequence
    const float* src = part + b * H * NR + at;
    float4 s = load4(src);
    for (int h = 1; h < H; ++h) {
      const float4 x = load4(src + h * NR);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    store4(dkr + b * NR + at, s);
  }
}

}  // namespace

namespace {

// Rows per thread: four (64-row CTAs) where that still gives every SM two CTAs, else two.
bool wide_rows(const LatentProblem& p) {
  return static_cast<long long>(p.B) * p.H * ((p.N + 63) / 64) >= 2ll * sm_count();
}

template <typename... KArgs, typename... Args>
cudaError_t launch_tiles(void (*kernel)(KArgs...), int smem, int rows, int passes,
                         const LatentProblem& p, cudaStream_t s, Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.N + rows - 1) / rows, p.B * p.H, passes);
  kernel<<<grid, kThreads, smem, s>>>(args..., p);
  return cudaGetLastError();
}

template <int RT>
cudaError_t fwd_rows(const LatentProblem& p, const float* q, const float* kn, const float* kr,
                     const float* v, float* o, float* o_acc, float* lse, cudaStream_t s) {
  return launch_tiles(latent_fwd_simt_kernel<RT>, fwd_smem<RT>(), 16 * RT, 1, p, s, q, kn, kr, v,
                      o, o_acc, lse);
}

template <int RT>
cudaError_t bwd_rows(const LatentProblem& p, const float* q, const float* kn, const float* kr,
                     const float* v, const float* lse, const float* dO, const float* Dsum,
                     float* dq, float* dkn, float* dkr_part, float* dv, cudaStream_t s) {
  return launch_tiles(latent_bwd_simt_kernel<RT>, bwd_smem<RT>(), 16 * RT, 2, p, s, q, kn, kr, v,
                      lse, dO, Dsum, dq, dkn, dkr_part, dv);
}

}  // namespace

cudaError_t launch_latent_fwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, void* o, float* o_acc,
                                   float* lse, cudaStream_t s) {
  const float *qf = static_cast<const float*>(q), *knf = static_cast<const float*>(kn);
  const float *krf = static_cast<const float*>(kr), *vf = static_cast<const float*>(v);
  float* of = static_cast<float*>(o);
  return wide_rows(p) ? fwd_rows<4>(p, qf, knf, krf, vf, of, o_acc, lse, s)
                      : fwd_rows<2>(p, qf, knf, krf, vf, of, o_acc, lse, s);
}

cudaError_t launch_latent_bwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, const float* lse,
                                   const void* dO, const float* Dsum, void* dq, void* dkn,
                                   float* dkr_part, void* dv, cudaStream_t s) {
  const float *qf = static_cast<const float*>(q), *knf = static_cast<const float*>(kn);
  const float *krf = static_cast<const float*>(kr), *vf = static_cast<const float*>(v);
  const float* dof = static_cast<const float*>(dO);
  float *dqf = static_cast<float*>(dq), *dknf = static_cast<float*>(dkn);
  float* dvf = static_cast<float*>(dv);
  return wide_rows(p)
             ? bwd_rows<4>(p, qf, knf, krf, vf, lse, dof, Dsum, dqf, dknf, dkr_part, dvf, s)
             : bwd_rows<2>(p, qf, knf, krf, vf, lse, dof, Dsum, dqf, dknf, dkr_part, dvf, s);
}

cudaError_t launch_latent_rowdot(const LatentProblem& p, fa_dtype dt, const float* o_acc,
                                 const void* dO, float* Dsum, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.N;
  long long blocks = (rows + kDotRows - 1) / kDotRows;
  if (blocks > 8ll * sm_count()) blocks = 8ll * sm_count();
  const dim3 grid(static_cast<unsigned>(blocks));
  return dt == FA_FP32
             ? launch_dependent(latent_rowdot_kernel<float>, grid, dim3(256), 0, s, o_acc,
                                static_cast<const float*>(dO), Dsum, rows)
             : launch_dependent(latent_rowdot_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, o_acc,
                                static_cast<const __nv_bfloat16*>(dO), Dsum, rows);
}

cudaError_t launch_latent_rope_sum(const LatentProblem& p, fa_dtype dt, const float* part,
                                   void* dkr, cudaStream_t s) {
  const long long NR = static_cast<long long>(p.N) * kRope, total = p.B * NR / 4;
  long long blocks = (total + 255) / 256;
  if (blocks > 8ll * sm_count()) blocks = 8ll * sm_count();
  const dim3 grid(static_cast<unsigned>(blocks));
  return dt == FA_FP32
             ? launch_dependent(latent_rope_sum_kernel<float>, grid, dim3(256), 0, s, part,
                                static_cast<float*>(dkr), p.H, NR, total)
             : launch_dependent(latent_rope_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, part,
                                static_cast<__nv_bfloat16*>(dkr), p.H, NR, total);
}

}  // namespace fa
