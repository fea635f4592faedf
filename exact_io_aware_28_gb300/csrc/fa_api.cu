// C-ABI boundary of libfa_gb300.so: argument validation, workspace carving and kernel
// dispatch.  Every entry point validates on the host before launching anything; no entry
// point allocates device memory or synchronises the stream (fa_device_error excepted).
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>

#include "fa_internal.cuh"

namespace fa {

namespace {
constexpr int kMaxDevices = 64;
// Per-device caches.  Host threads may fill them concurrently: each slot is atomic and a
// race only stores the same value twice.
std::atomic<int> g_sm_count[kMaxDevices];    // 0 = not yet queried
std::atomic<int*> g_err_ptr[kMaxDevices];    // device address of the error word
}  // namespace

// Device error word: a kernel whose bounded wait runs out stores FA_ERR_TIMEOUT here.
static __device__ int g_device_error;

int sm_count() {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return 148;
  int n = g_sm_count[dev].load();
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    g_sm_count[dev].store(n);
  }
  return n;
}

int* error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  int* cached = g_err_ptr[dev].load();
  if (!cached) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_device_error) != cudaSuccess || !ptr) return nullptr;
    cached = static_cast<int*>(ptr);
    g_err_ptr[dev].store(cached);
  }
  return cached;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

fa_status check_shape(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((long long)B * H > 65535) return FA_ERR_UNSUPPORTED;
  if (N > (1 << 24)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

unsigned long long wait_limit_ns() {
  // Initialised once (a function-local static is thread-safe).
  static const unsigned long long ns = [] {
    unsigned long long v = 2000ull;
    if (const char* s = getenv("FA_WAIT_LIMIT_MS")) {
      const long long ms = atoll(s);
      if (ms > 0 && ms < 600000) v = static_cast<unsigned long long>(ms);
    }
    return v * 1000000ull;
  }();
  return ns;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_decode_workspace_bytes(int B, int Hq, int Hkv, int Lmax, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lmax < 1 || Hq % Hkv != 0) return 0;
  if (d != 64 && d != 128) return 0;
  const size_t splits = static_cast<size_t>(decode_splits(B, Hkv, Lmax, d));
  return static_cast<size_t>(B) * Hq * splits * (d + 4) * sizeof(float);
}

fa_status fa_decode(const void* q, const void* k, const void* v, void* o, float* lse,
                    int B, int Hq, int Hkv, int Lmax, int d, const int32_t* cache_len,
                    float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lmax < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > 65535 || Lmax > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace))
    return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cache_len) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_decode_workspace_bytes(B, Hq, Hkv, Lmax, d)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  const int splits = decode_splits(B, Hkv, Lmax, d);
  cudaError_t e = launch_decode(q, k, v, o, lse, B, Hq, Hkv, Lmax, d, cache_len, scale,
                                static_cast<float*>(workspace), splits, err, wait_limit_ns(),
                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG: invalid argument";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: shape not supported";
    case FA_ERR_CUDA: return "FA_ERR_CUDA: CUDA runtime error";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a bounded device wait ran out";
  }
  return "FA_ERR_UNKNOWN";
}

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d) {
  if (check_shape(B, H, N, d) != FA_OK) return 0;
  const size_t rows = (size_t)B * H * N;
  return round_up(rows * sizeof(float), 256) + rows * (size_t)d * sizeof(float);
}

}  // extern "C"

namespace fa {
namespace {

// Dropout arguments as the kernels take them; threshold 0 is no dropout.
void set_dropout(Problem* p, int threshold, uint64_t seed, uint32_t offset) {
  p->drop_threshold = threshold;
  p->drop_seed_lo = static_cast<uint32_t>(seed);
  p->drop_seed_hi = static_cast<uint32_t>(seed >> 32);
  p->drop_offset = offset;
  p->drop_scale = 256.f / static_cast<float>(256 - threshold);
}

fa_status fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse,
                   int B, int H, int N, int d, int causal,
                   const uint8_t* blockmask, const int32_t* kv_len,
                   float scale, fa_dtype dtype, void* stream,
                   int drop_threshold, uint64_t seed, uint32_t offset) {
  fa_status st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(kv_len) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  Problem p{B, H, N, d, causal ? 1 : 0, blockmask, kv_len, scale, err, wait_limit_ns()};
  set_dropout(&p, drop_threshold, seed, offset);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == FA_BF16 ? launch_fwd_sm103(p, q, k, v, o, lse, s)
                                   : launch_fwd_simt(p, dtype, q, k, v, o, lse, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int H, int N, int d, int causal,
                 const uint8_t* blockmask, const int32_t* kv_len,
                 float scale, fa_dtype dtype, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, N, d, causal, blockmask, kv_len, scale, dtype, stream,
                  0, 0, 0);
}

fa_status fa_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse,
                         int B, int H, int N, int d, int causal,
                         const uint8_t* blockmask, const int32_t* kv_len,
                         float scale, fa_dtype dtype, int drop_threshold,
                         unsigned long long seed, unsigned int offset, void* stream) {
  if (drop_threshold < 0 || drop_threshold > 255) return FA_ERR_INVALID_ARG;
  return fwd_impl(q, k, v, o, lse, B, H, N, d, causal, blockmask, kv_len, scale, dtype, stream,
                  drop_threshold, seed, offset);
}

namespace {

struct Workspace {
  float* Dsum;
  float* dq_acc;
};

Workspace carve(void* workspace, int B, int H, int N) {
  const size_t rows = (size_t)B * H * N;
  Workspace w;
  w.Dsum = static_cast<float*>(workspace);
  w.dq_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      fa::round_up(rows * sizeof(float), 256));
  return w;
}

fa_status check_common(int B, int H, int N, int d, fa_dtype dtype, void* workspace,
                       size_t workspace_bytes) {
  fa_status st = fa::check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_bwd_workspace_bytes(B, H, N, d)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

bool bad_ptr(const void* p) { return !p || !fa::aligned16(p); }

fa_status check_masks_scale(const int32_t* kv_len, const float* lse, float scale) {
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(kv_len) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status to_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace

fa_status fa_bwd_preprocess(const void* o, const void* dO, int B, int H, int N, int d,
                            fa_dtype dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  fa_status st = check_common(B, H, N, d, dtype, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  if (bad_ptr(o) || bad_ptr(dO)) return FA_ERR_INVALID_ARG;
  Problem p{B, H, N, d, 0, nullptr, nullptr, 1.f, nullptr, 0};
  Workspace w = carve(workspace, B, H, N);
  return to_status(launch_bwd_preprocess(p, dtype, o, dO, w.Dsum,
                                         dtype == FA_BF16 ? w.dq_acc : nullptr,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

fa_status bwd_main_impl(const void* q, const void* k, const void* v, const float* lse,
                        const void* dO, void* dq, void* dk, void* dv,
                        int B, int H, int N, int d, int causal,
                        const uint8_t* blockmask, const int32_t* kv_len,
                        float scale, fa_dtype dtype,
                        void* workspace, size_t workspace_bytes, void* stream,
                        int drop_threshold, uint64_t seed, uint32_t offset) {
  fa_status st = check_common(B, H, N, d, dtype, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k) || bad_ptr(v) || bad_ptr(dO) || bad_ptr(dk) || bad_ptr(dv))
    return FA_ERR_INVALID_ARG;
  if (dtype == FA_FP32 && bad_ptr(dq)) return FA_ERR_INVALID_ARG;
  st = check_masks_scale(kv_len, lse, scale);
  if (st != FA_OK) return st;
  int* err = fa::error_word();
  if (!err) return FA_ERR_CUDA;
  Problem p{B, H, N, d, causal ? 1 : 0, blockmask, kv_len, scale, err, wait_limit_ns()};
  fa::set_dropout(&p, drop_threshold, seed, offset);
  Workspace w = carve(workspace, B, H, N);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FA_BF16)
    return to_status(launch_bwd_sm103(p, q, k, v, lse, dO, w.Dsum, w.dq_acc, dk, dv, s));
  return to_status(launch_bwd_simt(p, dtype, q, k, v, lse, dO, w.Dsum, dq, dk, dv, s));
}

fa_status bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv,
                   int B, int H, int N, int d, int causal,
                   const uint8_t* blockmask, const int32_t* kv_len,
                   float scale, fa_dtype dtype,
                   void* workspace, size_t workspace_bytes, void* stream,
                   int drop_threshold, uint64_t seed, uint32_t offset) {
  fa_status st = check_common(B, H, N, d, dtype, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k) || bad_ptr(v) || bad_ptr(o) || bad_ptr(dO) || bad_ptr(dq) ||
      bad_ptr(dk) || bad_ptr(dv))
    return FA_ERR_INVALID_ARG;
  st = check_masks_scale(kv_len, lse, scale);
  if (st != FA_OK) return st;
  st = fa_bwd_preprocess(o, dO, B, H, N, d, dtype, workspace, workspace_bytes, stream);
  if (st != FA_OK) return st;
  st = bwd_main_impl(q, k, v, lse, dO, dq, dk, dv, B, H, N, d, causal, blockmask, kv_len, scale,
                     dtype, workspace, workspace_bytes, stream, drop_threshold, seed, offset);
  if (st != FA_OK) return st;
  return fa_bwd_dq_convert(dq, B, H, N, d, scale, dtype, workspace, workspace_bytes, stream);
}

}  // namespace

namespace {

// A call's memory: where some CTAs read what others write, no output shares memory with an input
// or with another output.
struct Span {
  uintptr_t begin, end;
  Span(const void* p, long long bytes)
      : begin(reinterpret_cast<uintptr_t>(p)),
        end(p ? reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(bytes) : 0) {}
  bool meets(const Span& o) const { return begin < o.end && o.begin < end; }
};
template <size_t I, size_t O>
bool apart(const Span (&ins)[I], const Span (&outs)[O]) {
  for (size_t j = 0; j < O; ++j) {
    for (const Span& in : ins)
      if (outs[j].meets(in)) return false;
    for (size_t i = 0; i < j; ++i)
      if (outs[j].meets(outs[i])) return false;
  }
  return true;
}
// Bytes of a bf16 pool.
long long pool_bytes(int num_pages, long long page_stride, long long page_elems) {
  return 2 * ((num_pages - 1) * page_stride + page_elems);
}

}  // namespace

extern "C" {

fa_status fa_bwd_main(const void* q, const void* k, const void* v, const float* lse,
                      const void* dO, void* dq, void* dk, void* dv,
                      int B, int H, int N, int d, int causal,
                      const uint8_t* blockmask, const int32_t* kv_len,
                      float scale, fa_dtype dtype,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_main_impl(q, k, v, lse, dO, dq, dk, dv, B, H, N, d, causal, blockmask, kv_len,
                       scale, dtype, workspace, workspace_bytes, stream, 0, 0, 0);
}

fa_status fa_bwd_main_dropout(const void* q, const void* k, const void* v, const float* lse,
                              const void* dO, void* dq, void* dk, void* dv,
                              int B, int H, int N, int d, int causal,
                              const uint8_t* blockmask, const int32_t* kv_len,
                              float scale, fa_dtype dtype, int drop_threshold,
                              unsigned long long seed, unsigned int offset,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (drop_threshold < 0 || drop_threshold > 255) return FA_ERR_INVALID_ARG;
  return bwd_main_impl(q, k, v, lse, dO, dq, dk, dv, B, H, N, d, causal, blockmask, kv_len,
                       scale, dtype, workspace, workspace_bytes, stream, drop_threshold, seed,
                       offset);
}

fa_status fa_bwd_dq_convert(void* dq, int B, int H, int N, int d, float scale, fa_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_common(B, H, N, d, dtype, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  if (bad_ptr(dq)) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (dtype == FA_FP32) return FA_OK;
  Problem p{B, H, N, d, 0, nullptr, nullptr, scale, nullptr, 0};
  Workspace w = carve(workspace, B, H, N);
  return to_status(launch_dq_convert(p, w.dq_acc, dq, static_cast<cudaStream_t>(stream)));
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dO, void* dq, void* dk, void* dv,
                 int B, int H, int N, int d, int causal,
                 const uint8_t* blockmask, const int32_t* kv_len,
                 float scale, fa_dtype dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, causal, blockmask, kv_len, scale,
                  dtype, workspace, workspace_bytes, stream, 0, 0, 0);
}

fa_status fa_bwd_dropout(const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dO, void* dq, void* dk, void* dv,
                         int B, int H, int N, int d, int causal,
                         const uint8_t* blockmask, const int32_t* kv_len,
                         float scale, fa_dtype dtype, int drop_threshold,
                         unsigned long long seed, unsigned int offset,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (drop_threshold < 0 || drop_threshold > 255) return FA_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, causal, blockmask, kv_len, scale,
                  dtype, workspace, workspace_bytes, stream, drop_threshold, seed, offset);
}

fa_status fa_dropout_random_bytes(void* out, int BH, int n_q, int n_k, unsigned long long seed,
                                  unsigned int offset, void* stream) {
  if (!out || BH < 1 || n_q < 1 || n_k < 1 || BH > 65535) return FA_ERR_INVALID_ARG;
  if ((long long)n_q * n_k > (1ll << 31)) return FA_ERR_UNSUPPORTED;
  Problem p{1, BH, n_q, 64, 0, nullptr, nullptr, 1.f, nullptr, 0};
  set_dropout(&p, 0, seed, offset);
  return to_status(launch_dropout_bytes(p, static_cast<uint8_t*>(out), BH, n_q, n_k,
                                        static_cast<cudaStream_t>(stream)));
}

size_t fa_fp8_vt_bytes(int B, int H, int N, int d) {
  if (check_shape(B, H, N, d) != FA_OK || d != 128) return 0;
  return static_cast<size_t>(B) * H * d * round_up(static_cast<size_t>(N), 128);
}

namespace {

fa_status check_fp8(int B, int H, int N, int d) {
  fa_status st = fa::check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  return d == 128 ? FA_OK : FA_ERR_UNSUPPORTED;
}

bool bad_scale(const float* s) { return !s || (reinterpret_cast<uintptr_t>(s) & 3u) != 0; }

}  // namespace

fa_status fa_fp8_quantize_qk(const void* x, void* x8, float* scale, int B, int H, int N, int d,
                             void* stream) {
  fa_status st = check_fp8(B, H, N, d);
  if (st != FA_OK) return st;
  if (bad_ptr(x) || bad_ptr(x8) || bad_scale(scale)) return FA_ERR_INVALID_ARG;
  return to_status(launch_fp8_quantize_rows(x, x8, scale, B * H, N,
                                            static_cast<cudaStream_t>(stream)));
}

fa_status fa_fp8_quantize_v(const void* v, void* vt8, float* scale, int B, int H, int N, int d,
                            void* stream) {
  fa_status st = check_fp8(B, H, N, d);
  if (st != FA_OK) return st;
  if (bad_ptr(v) || bad_ptr(vt8) || bad_scale(scale)) return FA_ERR_INVALID_ARG;
  return to_status(launch_fp8_quantize_v(v, vt8, scale, B * H, N,
                                         static_cast<cudaStream_t>(stream)));
}

fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, const float* q_scale,
                     const float* k_scale, const float* v_scale, void* o, float* lse,
                     int B, int H, int N, int d, int causal, const uint8_t* blockmask,
                     const int32_t* kv_len, float scale, void* stream) {
  fa_status st = check_fp8(B, H, N, d);
  if (st != FA_OK) return st;
  if (bad_ptr(q8) || bad_ptr(k8) || bad_ptr(vt8) || bad_ptr(o)) return FA_ERR_INVALID_ARG;
  if (bad_scale(q_scale) || bad_scale(k_scale) || bad_scale(v_scale)) return FA_ERR_INVALID_ARG;
  st = check_masks_scale(kv_len, lse, scale);
  if (st != FA_OK) return st;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  Problem p{B, H, N, d, causal ? 1 : 0, blockmask, kv_len, scale, err, wait_limit_ns()};
  return to_status(launch_fwd_fp8(p, q8, k8, vt8, q_scale, k_scale, v_scale, o, lse,
                                  static_cast<cudaStream_t>(stream)));
}

namespace {

bool bad4(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// log2 of a supported page size, or -1.
int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// The pool: its sizes, and pages at least `page_elems` elements apart.
fa_status check_pool(int num_pages, int page_size, long long page_stride, long long page_elems) {
  if (num_pages < 1) return FA_ERR_INVALID_ARG;
  if (page_shift(page_size) < 0) return FA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page_size >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (page_stride < page_elems || page_stride % 8 != 0) return FA_ERR_INVALID_ARG;
  if (page_stride > (1ll << 38)) return FA_ERR_UNSUPPORTED;   // the tensor map's limit
  return FA_OK;
}

fa_status check_table(const int32_t* table, long long table_stride, int max_pages, int page_size) {
  if (bad4(table) || max_pages < 1 || table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if ((long long)max_pages * page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Two pools of pages of E elements, S apart, have no element in common: pages i and j lie
// delta + (j - i) S apart, and the two distances nearest to 0 are delta mod S and that less S.
bool pools_apart(const void* a, const void* b, long long S, long long E, int num_pages) {
  S *= 2, E *= 2;   // bytes
  const long long delta = static_cast<long long>(reinterpret_cast<intptr_t>(b) -
                                                 reinterpret_cast<intptr_t>(a));
  const long long r = ((delta % S) + S) % S, i = (delta - r) / S;
  return !(r < E && i > -num_pages && i < num_pages) &&
         !(S - r < E && i + 1 > -num_pages && i + 1 < num_pages);
}

bool bad_row_stride(long long stride, long long row) { return stride < row || stride % 8 != 0; }

constexpr int kLatentQK = FA_LATENT_NOPE + FA_LATENT_ROPE;

bool bad_softmax_scale(float scale) { return !(isfinite(scale) && scale > 0.f); }

}  // namespace

fa_status fa_paged_tables(const int32_t* cache_len, const int32_t* new_len,
                          const int32_t* free_pages, int n_free, int32_t* block_table,
                          long long table_stride, int max_pages, int32_t* total_len,
                          int32_t* token_start, int32_t* slots, int n_slots,
                          int32_t* pages_taken, int B, int page_size, int num_pages,
                          void* stream) {
  if (B < 1 || n_free < 0 || n_slots < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(num_pages, page_size, 8, 8);
  if (st == FA_OK) st = check_table(block_table, table_stride, max_pages, page_size);
  if (st != FA_OK) return st;
  if (B > 8192 || n_slots > (1 << 30) || (long long)B * max_pages * page_size >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  if (bad4(cache_len) || bad4(new_len) || bad4(total_len) || bad4(token_start) ||
      bad4(pages_taken))
    return FA_ERR_INVALID_ARG;
  if ((n_free > 0 && bad4(free_pages)) || (n_slots > 0 && bad4(slots))) return FA_ERR_INVALID_ARG;
  const Span ins[] = {{cache_len, 4ll * B}, {new_len, 4ll * B}, {free_pages, 4ll * n_free}};
  const Span outs[] = {{total_len, 4ll * B}, {token_start, 4 * (B + 1ll)}, {slots, 4ll * n_slots},
                       {pages_taken, 4}, {block_table, 4 * ((B - 1) * table_stride + max_pages)}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_tables(cache_len, new_len, free_pages, n_free, block_table,
                                       table_stride, max_pages, total_len, token_start, slots,
                                       n_slots, pages_taken, B, page_shift(page_size), num_pages,
                                       static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_append(const void* k, const void* v, long long k_stride, long long v_stride,
                          void* k_cache, void* v_cache, long long page_stride,
                          const int32_t* slots, int T, int num_pages, int Hkv, int page_size,
                          int d, void* stream) {
  if (T < 0 || Hkv < 1) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  fa_status st = check_pool(num_pages, page_size, page_stride, (long long)Hkv * page_size * d);
  if (st != FA_OK) return st;
  if (T == 0) return FA_OK;
  if (bad_ptr(k) || bad_ptr(v) || bad_ptr(k_cache) || bad_ptr(v_cache) || bad4(slots))
    return FA_ERR_INVALID_ARG;
  if (bad_row_stride(k_stride, (long long)Hkv * d) || bad_row_stride(v_stride, (long long)Hkv * d))
    return FA_ERR_INVALID_ARG;
  const bool same = k == v && k_stride == v_stride && k_cache == v_cache;   // the same bytes twice
  if (!same && !pools_apart(k_cache, v_cache, page_stride, (long long)Hkv * page_size * d, num_pages))
    return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_append(k, v, k_stride, v_stride, k_cache, v_cache, page_stride,
                                       slots, T, num_pages, Hkv, page_shift(page_size), d,
                                       static_cast<cudaStream_t>(stream)));
}

fa_status fa_latent_append(const void* c, const void* k_rope, long long c_stride,
                           long long rope_stride, void* cache, long long page_stride,
                           const int32_t* slots, int T, int num_pages, int page_size,
                           void* stream) {
  if (T < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(num_pages, page_size, page_stride,
                            (long long)page_size * (FA_LATENT_RANK + FA_LATENT_ROPE));
  if (st != FA_OK) return st;
  if (T == 0) return FA_OK;
  if (bad_ptr(c) || bad_ptr(k_rope) || bad_ptr(cache) || bad4(slots)) return FA_ERR_INVALID_ARG;
  if (bad_row_stride(c_stride, FA_LATENT_RANK) || bad_row_stride(rope_stride, FA_LATENT_ROPE))
    return FA_ERR_INVALID_ARG;
  return to_status(launch_latent_append(c, k_rope, c_stride, rope_stride, cache, page_stride,
                                        slots, T, num_pages, page_shift(page_size),
                                        static_cast<cudaStream_t>(stream)));
}

namespace {

fa_status check_decode_paged(int B, int Hq, int Hkv, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq / Hkv > 16) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > 65535) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status check_latent_decode(int B, int H) {
  if (B < 1 || H < 1) return FA_ERR_INVALID_ARG;
  return H <= 128 && B <= 65535 ? FA_OK : FA_ERR_UNSUPPORTED;
}

}  // namespace

size_t fa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (check_decode_paged(B, Hq, Hkv, d) != FA_OK) return 0;
  return decode_paged_part_bytes(Hq / Hkv, d) + (static_cast<size_t>(B) + 1) * sizeof(long long);
}

fa_status fa_decode_paged(const void* q, const void* k, const void* v, long long page_stride,
                          const int32_t* block_table, long long table_stride, int max_pages,
                          const int32_t* cache_len, void* o, float* lse, int B, int Hq, int Hkv,
                          int num_pages, int page_size, int d, float scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
  fa_status st = check_decode_paged(B, Hq, Hkv, d);
  if (st == FA_OK)
    st = check_pool(num_pages, page_size, page_stride, (long long)Hkv * page_size * d);
  if (st == FA_OK) st = check_table(block_table, table_stride, max_pages, page_size);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k) || bad_ptr(v) || bad_ptr(o) || bad_ptr(workspace) || bad4(lse) ||
      bad4(cache_len) || bad_softmax_scale(scale))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_decode_paged_workspace_bytes(B, Hq, Hkv, d);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  const long long rows = (long long)B * Hq;
  const long long pool = pool_bytes(num_pages, page_stride, (long long)Hkv * page_size * d);
  const Span ins[] = {{q, rows * d * 2}, {k, pool}, {v, pool}, {cache_len, 4ll * B},
                      {block_table, 4 * ((B - 1) * table_stride + max_pages)}};
  const Span outs[] = {{o, rows * d * 2}, {lse, rows * 4}, {workspace, (long long)need}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  return to_status(launch_decode_paged(q, k, v, page_stride, block_table, table_stride, max_pages,
                                       page_shift(page_size), num_pages, cache_len, o, lse, B, Hq,
                                       Hkv, d, scale, workspace, err, wait_limit_ns(),
                                       static_cast<cudaStream_t>(stream)));
}

namespace {

bool bad8(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 7u) != 0; }

// Rotary positions' plan: axes, turns of the rot / 2 pairs and the axis of each.
fa_status check_rope(const int32_t* pos, int axes, const int64_t* turns, const int32_t* axis, int d,
                     int rot) {
  if (d < 16 || d % 8 != 0 || d > 1024 || rot < 16 || rot % 16 != 0 || rot > d)
    return FA_ERR_UNSUPPORTED;
  if (axes < 1 || bad4(pos) || bad8(turns) || bad4(axis)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// A [B, H, N, d] tensor by its strides (elements): bytes from its first to its last element.
struct Strided {
  long long n[3], st[3];
  int d, esz;
  Strided(int B, int H, int N, int d_, long long sb, long long sh, long long sn, int esz_)
      : n{B, H, N}, st{sb, sh, sn}, d(d_), esz(esz_) {}
  bool fits() const {              // pieces of 16 bytes
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (st[i] < 0 || st[i] * esz % 16 != 0 || st[i] > (1ll << 40))) return false;
    return true;
  }
  long long bytes() const {
    long long e = d;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * st[i];
    return e * esz;
  }
  // Every element has a place of its own: each stride passes all that the smaller ones reach.
  bool distinct() const {
    bool used[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
    long long reach = d;
    for (int k = 0; k < 3; ++k) {
      int least = -1;
      for (int i = 0; i < 3; ++i)
        if (!used[i] && (least < 0 || st[i] < st[least])) least = i;
      if (least < 0) break;
      if (st[least] < reach) return false;
      reach += (n[least] - 1) * st[least];
      used[least] = true;
    }
    return true;
  }
  bool same(const Strided& o) const {
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && st[i] != o.st[i]) return false;
    return true;
  }
};

// T rows of ea elements at a, sa apart, and of eb at b, sb apart (bf16), have no element in common.
// Rows of one buffer (equal strides) may lie between one another.
bool rows_apart(const void* a, long long sa, long long ea, const void* b, long long sb, long long eb,
                int T) {
  const Span x(a, 2 * ((T - 1) * sa + ea)), y(b, 2 * ((T - 1) * sb + eb));
  if (!x.meets(y)) return true;
  if (sa != sb || T == 1) return false;
  const long long S = 2 * sa;
  const long long r = ((static_cast<long long>(y.begin - x.begin) % S) + S) % S;
  return r >= 2 * ea && S - r >= 2 * eb;
}

}  // namespace

fa_status fa_rope(const void* x, void* y, long long x_batch, long long x_head, long long x_token,
                  long long y_batch, long long y_head, long long y_token, const int32_t* pos,
                  long long pos_axis, long long pos_batch, int axes, const int64_t* turns,
                  const int32_t* axis, int B, int H, int N, int d, int rot, int interleaved,
                  int inverse, fa_dtype dtype, void* stream) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  fa_status st = check_rope(pos, axes, turns, axis, d, rot);
  if (st != FA_OK) return st;
  if (B > 65535 || H > 65535 || N > (1 << 30)) return FA_ERR_UNSUPPORTED;
  const int esz = dtype == FA_BF16 ? 2 : 4;
  const Strided xs(B, H, N, d, x_batch, x_head, x_token, esz);
  const Strided ys(B, H, N, d, y_batch, y_head, y_token, esz);
  if (bad_ptr(x) || bad_ptr(y) || !xs.fits() || !ys.fits() || !ys.distinct())
    return FA_ERR_INVALID_ARG;
  if ((axes > 1 && pos_axis < 0) || (B > 1 && pos_batch < 0)) return FA_ERR_INVALID_ARG;
  const long long places = (axes - 1) * pos_axis + (B - 1) * pos_batch + N;
  const bool in_place = x == y && xs.same(ys);
  const Span ins[] = {{in_place ? nullptr : x, xs.bytes()}, {pos, 4 * places}, {turns, 4ll * rot},
                      {axis, 2ll * rot}};
  const Span outs[] = {{y, ys.bytes()}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  return to_status(launch_rope(x, y, {x_batch, x_head, x_token}, {y_batch, y_head, y_token}, pos,
                               pos_axis, pos_batch, axes, reinterpret_cast<const long long*>(turns),
                               axis, B, H, N, d, rot, interleaved ? 1 : 0, inverse ? 1 : 0, dtype,
                               static_cast<cudaStream_t>(stream)));
}

fa_status fa_rope_append(const void* q, const void* k, const void* v, long long q_stride,
                         long long k_stride, long long v_stride, void* q_out, long long qo_stride,
                         void* k_cache, void* v_cache, long long page_stride, const int32_t* slots,
                         const int32_t* pos, long long pos_axis, int axes, const int64_t* turns,
                         const int32_t* axis, int T, int Hq, int Hkv, int num_pages, int page_size,
                         int d, int rot, int interleaved, void* stream) {
  if (T < 0 || Hq < 1 || Hkv < 1) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq > 65535 || Hkv > 65535 || T > (1 << 26)) return FA_ERR_UNSUPPORTED;
  const long long page = (long long)Hkv * page_size * d;
  fa_status st = check_pool(num_pages, page_size, page_stride, page);
  if (st != FA_OK) return st;
  if (T == 0) return FA_OK;
  st = check_rope(pos, axes, turns, axis, d, rot);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k) || bad_ptr(v) || bad_ptr(q_out) || bad_ptr(k_cache) ||
      bad_ptr(v_cache) || bad4(slots) || (axes > 1 && pos_axis < 0))
    return FA_ERR_INVALID_ARG;
  const long long qe = (long long)Hq * d, ke = (long long)Hkv * d;
  if (bad_row_stride(q_stride, qe) || bad_row_stride(qo_stride, qe) ||
      bad_row_stride(k_stride, ke) || bad_row_stride(v_stride, ke))
    return FA_ERR_INVALID_ARG;
  const bool in_place = q == q_out && (T == 1 || q_stride == qo_stride);
  if ((!in_place && !rows_apart(q_out, qo_stride, qe, q, q_stride, qe, T)) ||
      !rows_apart(q_out, qo_stride, qe, k, k_stride, ke, T) ||
      !rows_apart(q_out, qo_stride, qe, v, v_stride, ke, T) ||
      !pools_apart(k_cache, v_cache, page_stride, page, num_pages))
    return FA_ERR_INVALID_ARG;
  const Span small[] = {{slots, 4ll * T}, {pos, 4 * ((axes - 1) * pos_axis + T)}, {turns, 4ll * rot},
                        {axis, 2ll * rot}};
  const Span rows[] = {{q, 2 * ((T - 1) * q_stride + qe)}, {k, 2 * ((T - 1) * k_stride + ke)},
                       {v, 2 * ((T - 1) * v_stride + ke)}};
  const long long pool = pool_bytes(num_pages, page_stride, page);
  const Span out(q_out, 2 * ((T - 1) * qo_stride + qe)), kc(k_cache, pool), vc(v_cache, pool);
  if (kc.meets(out) || vc.meets(out)) return FA_ERR_INVALID_ARG;
  for (const Span& s : small)
    if (s.meets(out) || s.meets(kc) || s.meets(vc)) return FA_ERR_INVALID_ARG;
  for (const Span& s : rows)
    if (s.meets(kc) || s.meets(vc)) return FA_ERR_INVALID_ARG;
  return to_status(launch_rope_append(q, k, v, q_stride, k_stride, v_stride, q_out, qo_stride,
                                      k_cache, v_cache, page_stride, slots, pos, pos_axis, axes,
                                      reinterpret_cast<const long long*>(turns), axis, T, Hq, Hkv,
                                      num_pages, page_shift(page_size), d, rot, interleaved ? 1 : 0,
                                      static_cast<cudaStream_t>(stream)));
}

namespace {

// What the operators on a cache's tables have in common.
fa_status check_pages(const int32_t* cache_len, const int32_t* table, long long table_stride,
                      int max_pages, int B, int page_size, int num_pages) {
  if (B < 1) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(num_pages, page_size, 8, 8);
  if (st == FA_OK) st = check_table(table, table_stride, max_pages, page_size);
  if (st != FA_OK) return st;
  if (B > 8192 || (long long)B * max_pages * page_size >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return bad4(cache_len) ? FA_ERR_INVALID_ARG : FA_OK;
}

}  // namespace

fa_status fa_paged_fork(int32_t* cache_len, int32_t* block_table, long long table_stride,
                        int max_pages, const int32_t* free_pages, int n_free, const int32_t* src,
                        const int32_t* dst, int n, int32_t* copy_src, int32_t* copy_dst,
                        int32_t* copy_rows, int32_t* pages_taken, int B, int page_size,
                        int num_pages, void* stream) {
  if (n < 0 || n_free < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pages(cache_len, block_table, table_stride, max_pages, B, page_size,
                             num_pages);
  if (st != FA_OK) return st;
  if (n > 8192) return FA_ERR_UNSUPPORTED;
  if (bad4(pages_taken) || (n_free > 0 && bad4(free_pages))) return FA_ERR_INVALID_ARG;
  if (n > 0 && (bad4(src) || bad4(dst) || bad4(copy_src) || bad4(copy_dst) || bad4(copy_rows)))
    return FA_ERR_INVALID_ARG;
  const Span ins[] = {{n ? src : nullptr, 4ll * n}, {n ? dst : nullptr, 4ll * n},
                      {n_free ? free_pages : nullptr, 4ll * n_free}};
  const Span outs[] = {{cache_len, 4ll * B}, {block_table, 4 * ((B - 1) * table_stride + max_pages)},
                       {n ? copy_src : nullptr, 4ll * n}, {n ? copy_dst : nullptr, 4ll * n},
                       {n ? copy_rows : nullptr, 4ll * n}, {pages_taken, 4}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_fork(cache_len, block_table, table_stride, max_pages, free_pages,
                                     n_free, src, dst, n, copy_src, copy_dst, copy_rows,
                                     pages_taken, B, page_shift(page_size), num_pages,
                                     static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_free(int32_t* cache_len, int32_t* block_table, long long table_stride,
                        int max_pages, const int32_t* rows, int n, int32_t* refs,
                        int32_t* free_pages, int32_t* n_free, int B, int page_size, int num_pages,
                        void* stream) {
  if (n < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pages(cache_len, block_table, table_stride, max_pages, B, page_size,
                             num_pages);
  if (st != FA_OK) return st;
  if ((n > 0 && bad4(rows)) || bad4(refs) || bad4(free_pages) || bad4(n_free))
    return FA_ERR_INVALID_ARG;
  const Span ins[] = {{n ? rows : nullptr, 4ll * n}};
  const Span outs[] = {{cache_len, 4ll * B}, {block_table, 4 * ((B - 1) * table_stride + max_pages)},
                       {refs, 4ll * num_pages}, {free_pages, 4ll * num_pages}, {n_free, 4}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_free(cache_len, block_table, table_stride, max_pages, rows, n, refs,
                                     free_pages, n_free, B, page_shift(page_size), num_pages,
                                     static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_compact(const int32_t* cache_len, int32_t* block_table, long long table_stride,
                           int max_pages, int32_t* moved, int32_t* copy_src, int32_t* copy_dst,
                           int n_copies, int32_t* n_used, int B, int page_size, int num_pages,
                           void* stream) {
  fa_status st = check_pages(cache_len, block_table, table_stride, max_pages, B, page_size,
                             num_pages);
  if (st != FA_OK) return st;
  if (n_copies < num_pages / 2 || bad4(moved) || bad4(n_used)) return FA_ERR_INVALID_ARG;
  if (n_copies > 0 && (bad4(copy_src) || bad4(copy_dst))) return FA_ERR_INVALID_ARG;
  const Span ins[] = {{cache_len, 4ll * B}};
  const Span outs[] = {{block_table, 4 * ((B - 1) * table_stride + max_pages)},
                       {moved, 4ll * num_pages}, {n_copies ? copy_src : nullptr, 4ll * n_copies},
                       {n_copies ? copy_dst : nullptr, 4ll * n_copies}, {n_used, 4}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_compact(cache_len, block_table, table_stride, max_pages, moved,
                                        copy_src, copy_dst, n_copies, n_used, B,
                                        page_shift(page_size), num_pages,
                                        static_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_copy(void* k_cache, void* v_cache, long long page_stride,
                        const int32_t* copy_src, const int32_t* copy_dst, const int32_t* copy_rows,
                        int n, int num_pages, int Hkv, int page_size, int d, void* stream) {
  if (n < 0 || Hkv < 1) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128 && d != FA_LATENT_RANK + FA_LATENT_ROPE) || Hkv > 65535)
    return FA_ERR_UNSUPPORTED;
  const long long page = (long long)Hkv * page_size * d;
  fa_status st = check_pool(num_pages, page_size, page_stride, page);
  if (st != FA_OK) return st;
  if (page / 8 >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (n == 0) return FA_OK;
  if (bad_ptr(k_cache) || !aligned16(v_cache) || bad4(copy_src) || bad4(copy_dst) ||
      (copy_rows && bad4(copy_rows)))
    return FA_ERR_INVALID_ARG;
  if (v_cache && !pools_apart(k_cache, v_cache, page_stride, page, num_pages))
    return FA_ERR_INVALID_ARG;
  const long long pool = pool_bytes(num_pages, page_stride, page);
  const Span ins[] = {{copy_src, 4ll * n}, {copy_dst, 4ll * n}, {copy_rows, 4ll * n}};
  for (const Span& s : ins)
    if (s.meets(Span(k_cache, pool)) || s.meets(Span(v_cache, pool))) return FA_ERR_INVALID_ARG;
  return to_status(launch_paged_copy(k_cache, v_cache, page_stride, copy_src, copy_dst, copy_rows,
                                     n, num_pages, Hkv, page_shift(page_size), d,
                                     static_cast<cudaStream_t>(stream)));
}

size_t fa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int d) {
  return check_decode_paged(B, Hq, Hkv, d) == FA_OK ? decode_shared_bytes(B, Hq, Hkv, d) : 0;
}

fa_status fa_decode_shared(const void* q, const void* k, const void* v, long long page_stride,
                           const int32_t* block_table, long long table_stride, int max_pages,
                           const int32_t* cache_len, const int32_t* group_start,
                           const int32_t* shared_len, int groups, void* o, float* lse, int B,
                           int Hq, int Hkv, int num_pages, int page_size, int d, float scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_decode_paged(B, Hq, Hkv, d);
  if (st == FA_OK)
    st = check_pool(num_pages, page_size, page_stride, (long long)Hkv * page_size * d);
  if (st == FA_OK) st = check_table(block_table, table_stride, max_pages, page_size);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k) || bad_ptr(v) || bad_ptr(o) || bad_ptr(workspace) || bad4(lse) ||
      bad4(cache_len) || bad4(group_start) || bad4(shared_len) || groups < 1 || groups > B ||
      bad_softmax_scale(scale))
    return FA_ERR_INVALID_ARG;
  // tiles of 128 tokens are counted in 32 bits
  if ((long long)B * Hkv * (((long long)max_pages * page_size + 127) / 128) >= (1ll << 29))
    return FA_ERR_UNSUPPORTED;
  const size_t need = fa_decode_shared_workspace_bytes(B, Hq, Hkv, d);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  const long long rows = (long long)B * Hq;
  const long long pool = pool_bytes(num_pages, page_stride, (long long)Hkv * page_size * d);
  const Span ins[] = {{q, rows * d * 2}, {k, pool}, {v, pool}, {cache_len, 4ll * B},
                      {block_table, 4 * ((B - 1) * table_stride + max_pages)},
                      {group_start, 4 * (groups + 1ll)}, {shared_len, 4ll * groups}};
  const Span outs[] = {{o, rows * d * 2}, {lse, rows * 4}, {workspace, (long long)need}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  return to_status(launch_decode_shared(q, k, v, page_stride, block_table, table_stride, max_pages,
                                        page_shift(page_size), num_pages, cache_len, group_start,
                                        shared_len, groups, o, lse, B, Hq, Hkv, d, scale, workspace,
                                        err, wait_limit_ns(), static_cast<cudaStream_t>(stream)));
}

size_t fa_latent_decode_workspace_bytes(int B, int H) {
  return check_latent_decode(B, H) == FA_OK ? latent_decode_bytes(B, H) : 0;
}

fa_status fa_latent_decode(const void* q, const void* cache, long long page_stride,
                           const int32_t* block_table, long long table_stride, int max_pages,
                           const int32_t* cache_len, void* o, float* lse, int B, int H,
                           int num_pages, int page_size, float scale, void* workspace,
                           size_t workspace_bytes, void* stream) {
  fa_status st = check_latent_decode(B, H);
  if (st == FA_OK)
    st = check_pool(num_pages, page_size, page_stride,
                    (long long)page_size * (FA_LATENT_RANK + FA_LATENT_ROPE));
  if (st == FA_OK) st = check_table(block_table, table_stride, max_pages, page_size);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(cache) || bad_ptr(o) || bad_ptr(workspace) || bad4(lse) ||
      bad4(cache_len) || bad_softmax_scale(scale))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_latent_decode_workspace_bytes(B, H);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  constexpr int kRow = FA_LATENT_RANK + FA_LATENT_ROPE;
  const long long rows = (long long)B * H;
  const Span ins[] = {{q, rows * kRow * 2}, {cache_len, 4ll * B},
                      {cache, pool_bytes(num_pages, page_stride, (long long)page_size * kRow)},
                      {block_table, 4 * ((B - 1) * table_stride + max_pages)}};
  const Span outs[] = {{o, rows * FA_LATENT_RANK * 2}, {lse, rows * 4},
                       {workspace, (long long)need}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  return to_status(launch_latent_decode(q, cache, page_stride, block_table, table_stride,
                                        max_pages, page_shift(page_size), num_pages, cache_len, o,
                                        lse, B, H, scale, workspace, err, wait_limit_ns(),
                                        static_cast<cudaStream_t>(stream)));
}

fa_status fa_latent_fwd(const void* q, const void* k_nope, const void* k_rope, const void* v,
                        void* o, float* o_acc, float* lse, int B, int H, int N, int causal,
                        const int32_t* kv_len, float scale, fa_dtype dtype, void* stream) {
  fa_status st = fa::check_shape(B, H, N, FA_LATENT_V);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k_nope) || bad_ptr(k_rope) || bad_ptr(v) || bad_ptr(o) ||
      !aligned16(o_acc))
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  st = check_masks_scale(kv_len, lse, scale);
  if (st != FA_OK) return st;
  const long long rows = (long long)B * H * N, esz = dtype == FA_BF16 ? 2 : 4;
  const bool same = o_acc == o && dtype == FA_FP32;   // allowed: the same values
  const Span ins[] = {{q, rows * kLatentQK * esz}, {k_nope, rows * FA_LATENT_NOPE * esz},
                      {k_rope, (long long)B * N * FA_LATENT_ROPE * esz}, {v, rows * FA_LATENT_V * esz},
                      {kv_len, 4ll * B}};
  const Span outs[] = {{o, rows * FA_LATENT_V * esz}, {same ? nullptr : o_acc, rows * FA_LATENT_V * 4},
                       {lse, rows * 4}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  LatentProblem p{B, H, N, FA_LATENT_V, causal ? 1 : 0, nullptr, kv_len, scale, err,
                  wait_limit_ns()};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return to_status(dtype == FA_BF16
                       ? launch_latent_fwd_sm103(p, q, k_nope, k_rope, v, o, o_acc, lse, s)
                       : launch_latent_fwd_simt(p, q, k_nope, k_rope, v, o, o_acc, lse, s));
}

size_t fa_latent_bwd_workspace_bytes(int B, int H, int N) {
  if (check_shape(B, H, N, FA_LATENT_V) != FA_OK) return 0;
  const size_t rows = (size_t)B * H * N;
  return round_up(rows * sizeof(float), 256) + rows * FA_LATENT_ROPE * sizeof(float);
}

fa_status fa_latent_bwd(const void* q, const void* k_nope, const void* k_rope, const void* v,
                        const float* o_acc, const float* lse, const void* dO, void* dq,
                        void* dk_nope, void* dk_rope, void* dv, int B, int H, int N, int causal,
                        const int32_t* kv_len, float scale, fa_dtype dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  fa_status st = fa::check_shape(B, H, N, FA_LATENT_V);
  if (st != FA_OK) return st;
  if (bad_ptr(q) || bad_ptr(k_nope) || bad_ptr(k_rope) || bad_ptr(v) || bad_ptr(o_acc) ||
      bad_ptr(dO) || bad_ptr(dq) || bad_ptr(dk_nope) || bad_ptr(dk_rope) || bad_ptr(dv))
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  st = check_masks_scale(kv_len, lse, scale);
  if (st != FA_OK) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < fa_latent_bwd_workspace_bytes(B, H, N))
    return FA_ERR_INVALID_ARG;
  const long long rows = (long long)B * H * N, esz = dtype == FA_BF16 ? 2 : 4;
  const long long rope = (long long)B * N * FA_LATENT_ROPE * esz;
  const Span ins[] = {{q, rows * kLatentQK * esz}, {k_nope, rows * FA_LATENT_NOPE * esz},
                      {k_rope, rope}, {v, rows * FA_LATENT_V * esz}, {o_acc, rows * FA_LATENT_V * 4},
                      {lse, rows * 4}, {dO, rows * FA_LATENT_V * esz}, {kv_len, 4ll * B}};
  const Span outs[] = {{dq, rows * kLatentQK * esz}, {dk_nope, rows * FA_LATENT_NOPE * esz},
                       {dk_rope, rope}, {dv, rows * FA_LATENT_V * esz},
                       {workspace, (long long)fa_latent_bwd_workspace_bytes(B, H, N)}};
  if (!apart(ins, outs)) return FA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  LatentProblem p{B, H, N, FA_LATENT_V, causal ? 1 : 0, nullptr, kv_len, scale, err,
                  wait_limit_ns()};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* Dsum = static_cast<float*>(workspace);
  float* dkr_part = reinterpret_cast<float*>(
      static_cast<char*>(workspace) + round_up((size_t)B * H * N * sizeof(float), 256));
  cudaError_t e = launch_latent_rowdot(p, dtype, o_acc, dO, Dsum, s);
  if (e == cudaSuccess)
    e = dtype == FA_BF16 ? launch_latent_bwd_sm103(p, q, k_nope, k_rope, v, lse, dO, Dsum, dq,
                                                   dk_nope, dkr_part, dv, s)
                         : launch_latent_bwd_simt(p, q, k_nope, k_rope, v, lse, dO, Dsum, dq,
                                                  dk_nope, dkr_part, dv, s);
  if (e == cudaSuccess) e = launch_latent_rope_sum(p, dtype, dkr_part, dk_rope, s);
  return to_status(e);
}

fa_status fa_device_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  int* err = error_word();
  if (!err) return FA_ERR_CUDA;
  int host = 0;
  if (cudaMemcpy(&host, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return FA_ERR_CUDA;
  return host == 0 ? FA_OK : static_cast<fa_status>(host);
}

}  // extern "C"
