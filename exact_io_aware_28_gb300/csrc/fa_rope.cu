// Rotary positions: pairs of channels turned by an angle that grows with the token's position on
// one of several axes (one for text; time, height and width for images and video), on tensors of
// any strides, forwards and backwards, and fused with the write of new rows into a paged cache.
//
// Mathematics.  Pair i of a row at positions n_0, n_1, ... turns by the angle n_a w_i, a = axis[i]:
//   y_1 = x_1 cos - x_2 sin,   y_2 = x_2 cos + x_1 sin,
// and the gradient is the turn back, by minus the angle.  Frequencies come as turns a position in
// units of 2^-64 turn: the product with a position, modulo 2^64, is the angle modulo a full turn,
// without error however far the position is, so that no range reduction is left; the upper 32 bits,
// rounded to fp32 (2^-25 of half a turn), are what sine and cosine are taken of.  Values are turned
// in fp32 and rounded once.
//
// What bounds it: every value is read and written once, so HBM does: 32 + 32 heads x 16384 x 128 in bf16
// and their gradients (1.07 GB) 170 us, 6.3 TB/s, 0.93 of a plain copy's rate; 16384 new rows of 48
// heads (0.4 GB) 64 us, 6.3 TB/s; 64 of them 2.8 us.  A thread has eight pairs of a
// token (two 16-byte pieces of bf16) and goes over a share of the heads with the same sines and
// cosines, four heads' loads at a time; the channels that are not turned go to further threads.
//
// All launch as dependent kernels (they wait for the previous kernel in the stream before touching
// global memory).
#include <math.h>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kPairs = 8;          // pairs a thread turns
constexpr int kUnroll = 4;         // heads in flight

struct Angles {
  const int32_t* pos;
  long long axis_stride, batch_stride;   // of pos, elements
  int axes;
  const unsigned long long* turns;
  const int32_t* axis;
  int inverse;
};

// Cosines and sines of pairs p0 ... p0 + 7 of a token.
__device__ __forceinline__ void angles(const Angles& g, long long token, int p0, float (&c)[kPairs],
                                       float (&s)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int a = min(max(g.axis[p0 + i], 0), g.axes - 1);
    const long long n = g.pos[a * g.axis_stride + token];
    const unsigned long long t = g.turns[p0 + i] * static_cast<unsigned long long>(n);
    const int half = static_cast<int>(t >> 32);       // half turns, in 2^-31
    sincospif(static_cast<float>(half) * 0x1p-31f, &s[i], &c[i]);
    if (g.inverse) s[i] = -s[i];
  }
}

template <typename T>
struct Eight;    // eight neighbouring channels

template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = v;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    v = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                   ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
  }
};

template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Sixteen channels turned: u the first piece, v the second.  INTER: the pieces are neighbours and a
// pair is two neighbouring channels; else u has the pairs' first channels and v their second ones.
template <bool INTER, typename T>
__device__ __forceinline__ void turn(Eight<T>& u, Eight<T>& v, const float (&c)[kPairs],
                                     const float (&s)[kPairs]) {
  float a[8], b[8], p[8], q[8];
  u.get(a);
  v.get(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (INTER) {
      float* x = i < 4 ? &a[2 * i] : &b[2 * (i - 4)];
      float* y = i < 4 ? &p[2 * i] : &q[2 * (i - 4)];
      y[0] = x[0] * c[i] - x[1] * s[i];
      y[1] = x[1] * c[i] + x[0] * s[i];
    } else {
      p[i] = a[i] * c[i] - b[i] * s[i];
      q[i] = b[i] * c[i] + a[i] * s[i];
    }
  }
  u.set(p);
  v.set(q);
}

struct RopeArgs {
  const void* x;
  void* y;
  long long xb, xh, xn, yb, yh, yn;    // strides of batch, head and token, elements
  Angles g;
  int H, N, pairs, tail;               // tail: pieces of eight channels copied as they are
  int heads;                           // heads a thread
};

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int chunks = a.pairs / kPairs, per = chunks + a.tail;
  const long long item = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x;
  const long long n = item / per;
  const int c = static_cast<int>(item - n * per);
  if (n >= a.N) return;
  const int b = blockIdx.z, h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  const T* x = static_cast<const T*>(a.x) + b * a.xb + n * a.xn;
  T* y = static_cast<T*>(a.y) + b * a.yb + n * a.yn;
  if (c >= chunks) {
    const int at = 2 * a.pairs + 8 * (c - chunks);
    for (int h = h0; h < h1; ++h) {
      Eight<T> u;
      u.load(x + h * a.xh + at);
      u.store(y + h * a.yh + at);
    }
    return;
  }
  const int at = INTER ? 16 * c : 8 * c, to = INTER ? at + 8 : at + a.pairs;
  float cs[kPairs], sn[kPairs];
  angles(a.g, b * a.g.batch_stride + n, kPairs * c, cs, sn);
  for (int h = h0; h < h1; h += kUnroll) {
    Eight<T> u[kUnroll], v[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (h + j < h1) {
        u[j].load(x + (h + j) * a.xh + at);
        v[j].load(x + (h + j) * a.xh + to);
      }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (h + j < h1) {
        turn<INTER>(u[j], v[j], cs, sn);
        u[j].store(y + (h + j) * a.yh + at);
        v[j].store(y + (h + j) * a.yh + to);
      }
  }
}

// Rows of new tokens: Hq of queries, turned into q_out; Hkv of keys, turned into the cache; Hkv of
// values, copied into the cache.
struct RopeAppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;    // between tokens, elements
  __nv_bfloat16* q_out;
  long long qo_stride;
  __nv_bfloat16 *k_cache, *v_cache;
  long long page_stride;
  const int32_t* slots;
  Angles g;
  int T, Hq, Hkv, d, pairs, tail, shift, num_slots;
  int heads;                                 // rows a thread
};

template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeAppendArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int chunks = a.pairs / kPairs, per = chunks + a.tail;
  const int item = blockIdx.x * kRopeThreads + threadIdx.x;
  const int t = item / per, c = item - t * per;
  if (t >= a.T) return;
  const bool copy = c >= chunks;             // channels behind the turned ones: one piece
  const int at = copy ? 2 * a.pairs + 8 * (c - chunks) : INTER ? 16 * c : 8 * c;
  const int to = copy ? at : INTER ? at + 8 : at + a.pairs;
  const int h0 = blockIdx.y * a.heads, h1 = min(a.Hq + 2 * a.Hkv, h0 + a.heads);
  const int slot = a.slots[t];
  const bool kept = slot >= 0 && slot < a.num_slots;
  const long long row =
      kept ? (slot >> a.shift) * a.page_stride + (slot & ((1 << a.shift) - 1)) * a.d : 0;
  const long long head = static_cast<long long>(a.d) << a.shift;
  float cs[kPairs], sn[kPairs];
  if (!copy && h0 < a.Hq + a.Hkv) angles(a.g, t, kPairs * c, cs, sn);
  using E = Eight<__nv_bfloat16>;
  for (int h = h0; h < h1; h += kUnroll) {
    E u[kUnroll], v[kUnroll];
    __nv_bfloat16* dst[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int r = h + j, g = r - a.Hq;
      dst[j] = nullptr;
      if (r >= h1) continue;
      const __nv_bfloat16* src;
      if (g < 0) {
        src = a.q + t * a.q_stride + static_cast<long long>(r) * a.d;
        dst[j] = a.q_out + t * a.qo_stride + static_cast<long long>(r) * a.d;
      } else if (g < a.Hkv) {
        src = a.k + t * a.k_stride + static_cast<long long>(g) * a.d;
        if (kept) dst[j] = a.k_cache + row + g * head;
      } else {
        src = a.v + t * a.v_stride + static_cast<long long>(g - a.Hkv) * a.d;
        if (kept) dst[j] = a.v_cache + row + (g - a.Hkv) * head;
      }
      if (dst[j]) {
        u[j].load(src + at);
        if (!copy) v[j].load(src + to);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (!dst[j]) continue;
      if (!copy && h + j < a.Hq + a.Hkv) turn<INTER>(u[j], v[j], cs, sn);
      u[j].store(dst[j] + at);
      if (!copy) v[j].store(dst[j] + to);
    }
  }
}

// Heads a thread: as many as leave the grid 32 blocks an SM, so that few tokens are spread over the
// heads and many share their sines and cosines; from the heads in flight on a multiple of them.
// (Blocks of 256, 8 an SM, never fewer than 4 heads: 176 for 170 us for 2 x 32 heads x 16384 and back,
// 67.4 for 64.1 for 16384 rows into the cache, 3.6 for 2.8 for 64, 13.5 for 8.8 for four calls of 2 x
// 3 heads x 333 in fp32; 8 heads in flight 200.)
int heads_each(long long blocks, int heads) {
  long long split = blocks > 0 ? 32ll * sm_count() / blocks : 1;
  if (split < 1) split = 1;
  if (split > heads) split = heads;
  const int each = static_cast<int>((heads + split - 1) / split);
  return each > kUnroll ? (each + kUnroll - 1) / kUnroll * kUnroll : each;
}

}  // namespace

cudaError_t launch_rope(const void* x, void* y, const long long (&xs)[3], const long long (&ys)[3],
                        const int32_t* pos, long long pos_axis, long long pos_batch, int axes,
                        const long long* turns, const int32_t* axis, int B, int H, int N, int d,
                        int rot, int interleaved, int inverse, fa_dtype dt, cudaStream_t s) {
  RopeArgs a{x, y, xs[0], xs[1], xs[2], ys[0], ys[1], ys[2],
             {pos, pos_axis, pos_batch, axes,
              reinterpret_cast<const unsigned long long*>(turns), axis, inverse},
             H, N, rot / 2, x == y ? 0 : (d - rot) / 8, 0};
  const long long items = static_cast<long long>(N) * (a.pairs / kPairs + a.tail);
  const long long blocks = (items + kRopeThreads - 1) / kRopeThreads;
  a.heads = heads_each(blocks * B, H);
  const dim3 grid(static_cast<unsigned>(blocks), (H + a.heads - 1) / a.heads, B);
  if (dt == FA_BF16)
    return interleaved ? launch_dependent(rope_kernel<__nv_bfloat16, true>, grid,
                                          dim3(kRopeThreads), 0, s, a)
                       : launch_dependent(rope_kernel<__nv_bfloat16, false>, grid,
                                          dim3(kRopeThreads), 0, s, a);
  return interleaved
             ? launch_dependent(rope_kernel<float, true>, grid, dim3(kRopeThreads), 0, s, a)
             : launch_dependent(rope_kernel<float, false>, grid, dim3(kRopeThreads), 0, s, a);
}

cudaError_t launch_rope_append(const void* q, const void* k, const void* v, long long q_stride,
                               long long k_stride, long long v_stride, void* q_out,
                               long long qo_stride, void* k_cache, void* v_cache,
                               long long page_stride, const int32_t* slots, const int32_t* pos,
                               long long pos_axis, int axes, const long long* turns,
                               const int32_t* axis, int T, int Hq, int Hkv, int num_pages,
                               int page_shift, int d, int rot, int interleaved, cudaStream_t s) {
  using bf = __nv_bfloat16;
  RopeAppendArgs a{static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v),
                   q_stride, k_stride, v_stride, static_cast<bf*>(q_out), qo_stride,
                   static_cast<bf*>(k_cache), static_cast<bf*>(v_cache), page_stride, slots,
                   {pos, pos_axis, 0, axes, reinterpret_cast<const unsigned long long*>(turns),
                    axis, 0},
                   T, Hq, Hkv, d, rot / 2, (d - rot) / 8, page_shift, num_pages << page_shift, 0};
  const long long items = static_cast<long long>(T) * (a.pairs / kPairs + a.tail);
  const long long blocks = (items + kRopeThreads - 1) / kRopeThreads;
  const int rows = Hq + 2 * Hkv;
  a.heads = heads_each(blocks, rows);
  const dim3 grid(static_cast<unsigned>(blocks), (rows + a.heads - 1) / a.heads);
  return interleaved
             ? launch_dependent(rope_append_kernel<true>, grid, dim3(kRopeThreads), 0, s, a)
             : launch_dependent(rope_append_kernel<false>, grid, dim3(kRopeThreads), 0, s, a);
}

}  // namespace fa
