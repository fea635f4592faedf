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
// This path serves fp32 tensors.  Four threads per row, each owning every fourth column; a CTA
// owns 64 rows and walks the other operand in tiles of 32 rows in shared memory.  Scores are in
// the log2 domain (scale log2 e folded into the row held in registers).
#include <math.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNope = FA_LATENT_NOPE, kRope = FA_LATENT_ROPE, kQK = kNope + kRope;
constexpr int kV = FA_LATENT_V;
constexpr int kTPR = 4;        // threads per row
constexpr int kRows = 64;      // rows owned by one CTA
constexpr int kTile = 32;      // rows of the other operand staged per shared-memory tile
constexpr int kThreads = kRows * kTPR;
constexpr int kNQ = kQK / kTPR, kNV = kV / kTPR;   // columns per thread

__device__ __forceinline__ int key_limit(const LatentProblem& p, int b) {
  if (!p.kv_len) return p.N;
  const int L = p.kv_len[b];
  return L < 0 ? 0 : (L > p.N ? p.N : L);
}

__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x;
}

// Column c of key j's row of head bh.
__device__ __forceinline__ float key_at(const LatentProblem& p, const float* kn, const float* kr,
                                        int bh, int b, int j, int c) {
  return c < kNope ? kn[(static_cast<size_t>(bh) * p.N + j) * kNope + c]
                   : kr[(static_cast<size_t>(b) * p.N + j) * kRope + c - kNope];
}

__global__ void __launch_bounds__(kThreads)
latent_fwd_simt_kernel(const float* __restrict__ q, const float* __restrict__ kn,
                       const float* __restrict__ kr, const float* __restrict__ v,
                       float* __restrict__ o, float* __restrict__ o_acc, float* __restrict__ lse,
                       LatentProblem p) {
  __shared__ float ks[kTile][kQK];
  __shared__ float vs[kTile][kV];
  const int N = p.N, bh = blockIdx.y, b = bh / p.H;
  const size_t rows0 = static_cast<size_t>(bh) * N;
  const int tid = threadIdx.x, part = tid % kTPR;
  const int row0 = blockIdx.x * kRows, row = row0 + tid / kTPR;
  const bool valid_row = row < N;
  const float c = p.scale * kLog2e;
  float qr[kNQ], acc[kNV];
#pragma unroll
  for (int t = 0; t < kNQ; ++t)
    qr[t] = valid_row ? q[(rows0 + row) * kQK + part + kTPR * t] * c : 0.f;
#pragma unroll
  for (int t = 0; t < kNV; ++t) acc[t] = 0.f;
  float m = -INFINITY, l = 0.f;
  int kend = key_limit(p, b);
  if (p.causal) kend = min(kend, min(N, row0 + kRows));
  for (int k0 = 0; k0 < kend; k0 += kTile) {
    const int jmax = min(kTile, kend - k0);
    __syncthreads();
    for (int e = tid; e < jmax * kQK; e += kThreads)
      ks[e / kQK][e % kQK] = key_at(p, kn, kr, bh, b, k0 + e / kQK, e % kQK);
    for (int e = tid; e < jmax * kV; e += kThreads)
      vs[e / kV][e % kV] = v[(rows0 + k0 + e / kV) * kV + e % kV];
    __syncthreads();
    for (int j = 0; j < jmax; ++j) {
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < kNQ; ++t) s = fmaf(qr[t], ks[j][part + kTPR * t], s);
      s = group_sum(s);
      if (!valid_row || (p.causal && k0 + j > row)) continue;
      if (s > m) {
        const float alpha = exp2f(m - s);
        l *= alpha;
#pragma unroll
        for (int t = 0; t < kNV; ++t) acc[t] *= alpha;
        m = s;
      }
      const float pj = exp2f(s - m);
      l += pj;
#pragma unroll
      for (int t = 0; t < kNV; ++t) acc[t] = fmaf(pj, vs[j][part + kTPR * t], acc[t]);
    }
  }
  if (valid_row) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int t = 0; t < kNV; ++t) {
      const size_t at = (rows0 + row) * kV + part + kTPR * t;
      o[at] = acc[t] * inv;
      if (o_acc) o_acc[at] = acc[t] * inv;
    }
    if (part == 0) lse[rows0 + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// Key-outer: one CTA owns 64 keys of one head and walks every query row that may see them.
__global__ void __launch_bounds__(kThreads)
latent_dkdv_simt_kernel(const float* __restrict__ q, const float* __restrict__ kn,
                        const float* __restrict__ kr, const float* __restrict__ v,
                        const float* __restrict__ lse, const float* __restrict__ dO,
                        const float* __restrict__ Dsum, float* __restrict__ dkn,
                        float* __restrict__ dkr_part, float* __restrict__ dv, LatentProblem p) {
  __shared__ float qs[kTile][kQK];
  __shared__ float dos[kTile][kV];
  __shared__ float lses[kTile], Ds[kTile];
  const int N = p.N, bh = blockIdx.y, b = bh / p.H;
  const size_t rows0 = static_cast<size_t>(bh) * N;
  const int tid = threadIdx.x, part = tid % kTPR;
  const int key0 = blockIdx.x * kRows, key = key0 + tid / kTPR;
  const int L = key_limit(p, b);
  const bool live_key = key < L;
  const float c = p.scale * kLog2e;
  float kreg[kNQ], vr[kNV], dka[kNQ], dva[kNV];
#pragma unroll
  for (int t = 0; t < kNQ; ++t) {
    kreg[t] = live_key ? key_at(p, kn, kr, bh, b, key, part + kTPR * t) * c : 0.f;
    dka[t] = 0.f;
  }
#pragma unroll
  for (int t = 0; t < kNV; ++t) {
    vr[t] = live_key ? v[(rows0 + key) * kV + part + kTPR * t] : 0.f;
    dva[t] = 0.f;
  }
  if (key0 < L) {
    for (int i0 = p.causal ? key0 : 0; i0 < N; i0 += kTile) {
      const int imax = min(kTile, N - i0);
      __syncthreads();
      for (int e = tid; e < imax * kQK; e += kThreads)
        qs[e / kQK][e % kQK] = q[(rows0 + i0) * kQK + e];
      for (int e = tid; e < imax * kV; e += kThreads)
        dos[e / kV][e % kV] = dO[(rows0 + i0) * kV + e];
      if (tid < imax) {
        lses[tid] = lse[rows0 + i0 + tid];
        Ds[tid] = Dsum[rows0 + i0 + tid];
      }
      __syncthreads();
      for (int ii = 0; ii < imax; ++ii) {
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int t = 0; t < kNQ; ++t) s = fmaf(kreg[t], qs[ii][part + kTPR * t], s);
#pragma unroll
        for (int t = 0; t < kNV; ++t) dp = fmaf(vr[t], dos[ii][part + kTPR * t], dp);
        s = group_sum(s);
        dp = group_sum(dp);
        if (!live_key || (p.causal && key > i0 + ii)) continue;
        const float pij = exp2f(fmaf(-kLog2e, lses[ii], s));
        const float ds = pij * (dp - Ds[ii]);
#pragma unroll
        for (int t = 0; t < kNV; ++t) dva[t] = fmaf(pij, dos[ii][part + kTPR * t], dva[t]);
#pragma unroll
        for (int t = 0; t < kNQ; ++t) dka[t] = fmaf(ds, qs[ii][part + kTPR * t], dka[t]);
      }
    }
  }
  if (key < N) {
#pragma unroll
    for (int t = 0; t < kNV; ++t) dv[(rows0 + key) * kV + part + kTPR * t] = dva[t];
#pragma unroll
    for (int t = 0; t < kNQ; ++t) {
      const int cc = part + kTPR * t;
      if (cc < kNope) dkn[(rows0 + key) * kNope + cc] = dka[t] * p.scale;
      else dkr_part[(rows0 + key) * kRope + cc - kNope] = dka[t] * p.scale;
    }
  }
}

// Query-outer: one CTA owns 64 query rows and walks every key they may see.
__global__ void __launch_bounds__(kThreads)
latent_dq_simt_kernel(const float* __restrict__ q, const float* __restrict__ kn,
                      const float* __restrict__ kr, const float* __restrict__ v,
                      const float* __restrict__ lse, const float* __restrict__ dO,
                      const float* __restrict__ Dsum, float* __restrict__ dq, LatentProblem p) {
  __shared__ float ks[kTile][kQK];
  __shared__ float vs[kTile][kV];
  const int N = p.N, bh = blockIdx.y, b = bh / p.H;
  const size_t rows0 = static_cast<size_t>(bh) * N;
  const int tid = threadIdx.x, part = tid % kTPR;
  const int row0 = blockIdx.x * kRows, row = row0 + tid / kTPR;
  const bool valid_row = row < N;
  const float c = p.scale * kLog2e;
  float qr[kNQ], dor[kNV], acc[kNQ];
#pragma unroll
  for (int t = 0; t < kNQ; ++t) {
    qr[t] = valid_row ? q[(rows0 + row) * kQK + part + kTPR * t] * c : 0.f;
    acc[t] = 0.f;
  }
#pragma unroll
  for (int t = 0; t < kNV; ++t)
    dor[t] = valid_row ? dO[(rows0 + row) * kV + part + kTPR * t] : 0.f;
  const float row_lse = valid_row ? lse[rows0 + row] : -INFINITY;
  const float Di = valid_row ? Dsum[rows0 + row] : 0.f;
  int kend = key_limit(p, b);
  if (p.causal) kend = min(kend, min(N, row0 + kRows));
  for (int k0 = 0; k0 < kend; k0 += kTile) {
    const int jmax = min(kTile, kend - k0);
    __syncthreads();
    for (int e = tid; e < jmax * kQK; e += kThreads)
      ks[e / kQK][e % kQK] = key_at(p, kn, kr, bh, b, k0 + e / kQK, e % kQK);
    for (int e = tid; e < jmax * kV; e += kThreads)
      vs[e / kV][e % kV] = v[(rows0 + k0 + e / kV) * kV + e % kV];
    __syncthreads();
    for (int j = 0; j < jmax; ++j) {
      float s = 0.f, dp = 0.f;
#pragma unroll
      for (int t = 0; t < kNQ; ++t) s = fmaf(qr[t], ks[j][part + kTPR * t], s);
#pragma unroll
      for (int t = 0; t < kNV; ++t) dp = fmaf(dor[t], vs[j][part + kTPR * t], dp);
      s = group_sum(s);
      dp = group_sum(dp);
      if (!valid_row || (p.causal && k0 + j > row)) continue;
      const float ds = exp2f(fmaf(-kLog2e, row_lse, s)) * (dp - Di);
#pragma unroll
      for (int t = 0; t < kNQ; ++t) acc[t] = fmaf(ds, ks[j][part + kTPR * t], acc[t]);
    }
  }
  if (valid_row) {
#pragma unroll
    for (int t = 0; t < kNQ; ++t)
      dq[(rows0 + row) * kQK + part + kTPR * t] = acc[t] * p.scale;
  }
}

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 raw = *reinterpret_cast<const uint2*>(p);
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
}

// D_i = dO_i . O_i: a warp per row, four columns a lane.  HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256)
latent_rowdot_kernel(const float* __restrict__ o_acc, const T* __restrict__ dO,
                     float* __restrict__ Dsum, long long rows) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  for (long long row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < rows; row += step) {
    const float4 x = load4(o_acc + row * kV + 4 * lane), g = load4(dO + row * kV + 4 * lane);
    float s = fmaf(x.x, g.x, fmaf(x.y, g.y, fmaf(x.z, g.z, x.w * g.w)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) Dsum[row] = s;
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

cudaError_t launch_latent_fwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, void* o, float* o_acc,
                                   float* lse, cudaStream_t s) {
  const dim3 grid((p.N + kRows - 1) / kRows, p.B * p.H);
  latent_fwd_simt_kernel<<<grid, kThreads, 0, s>>>(
      static_cast<const float*>(q), static_cast<const float*>(kn), static_cast<const float*>(kr),
      static_cast<const float*>(v), static_cast<float*>(o), o_acc, lse, p);
  return cudaGetLastError();
}

cudaError_t launch_latent_bwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, const float* lse,
                                   const void* dO, const float* Dsum, void* dq, void* dkn,
                                   float* dkr_part, void* dv, cudaStream_t s) {
  const dim3 grid((p.N + kRows - 1) / kRows, p.B * p.H);
  const float *qf = static_cast<const float*>(q), *knf = static_cast<const float*>(kn);
  const float *krf = static_cast<const float*>(kr), *vf = static_cast<const float*>(v);
  const float* dof = static_cast<const float*>(dO);
  latent_dkdv_simt_kernel<<<grid, kThreads, 0, s>>>(qf, knf, krf, vf, lse, dof, Dsum,
                                                    static_cast<float*>(dkn), dkr_part,
                                                    static_cast<float*>(dv), p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  latent_dq_simt_kernel<<<grid, kThreads, 0, s>>>(qf, knf, krf, vf, lse, dof, Dsum,
                                                  static_cast<float*>(dq), p);
  return cudaGetLastError();
}

cudaError_t launch_latent_rowdot(const LatentProblem& p, fa_dtype dt, const float* o_acc,
                                 const void* dO, float* Dsum, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.N;
  long long blocks = (rows + 7) / 8;
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
