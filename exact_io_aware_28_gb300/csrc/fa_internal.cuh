// Internal declarations shared by the translation units of libfa_gb300.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <utility>

#include "fa.h"

namespace fa {

constexpr int kMaskBlock = FA_MASK_BLOCK;

// Problem description handed from the C-ABI layer to the launchers.  Pointers are
// device pointers; element pointers are typed by the launcher.
struct Problem {
  int B, H, N, d;
  int causal;
  const uint8_t* blockmask;  // [nb, nb] or nullptr
  const int32_t* kv_len;     // [B] or nullptr
  float scale;
  int* err;                  // device error word
  unsigned long long wait_ns;  // bound of every mbarrier wait in the tensor-core kernels
  // Dropout on the probabilities (threshold 0: none): element (bh, i, j) is dropped when its
  // generator byte is below drop_threshold, kept ones are scaled by drop_scale.
  int drop_threshold = 0;
  uint32_t drop_seed_lo = 0, drop_seed_hi = 0, drop_offset = 0;
  float drop_scale = 1.f;    // 256 / (256 - drop_threshold)
};

// Bound of device-side waits: FA_WAIT_LIMIT_MS from the environment (read once), else 2 s.
unsigned long long wait_limit_ns();

// Device error codes written into the error word (match fa_status).
constexpr int kErrTimeout = FA_ERR_TIMEOUT;

// Launch of a kernel of the training step (forward, preprocess, backward main, dQ convert)
// with programmatic stream serialization: it may be scheduled while the previous kernel in
// the stream drains, runs its set-up (barriers, tensor memory, descriptor prefetch), and waits
// in griddep_wait before it touches global memory.  Every such kernel calls griddep_wait in
// every CTA before it can exit, so completion stays ordered along the stream.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Launchers.  Each returns cudaSuccess or the launch error.
cudaError_t launch_fwd_simt(const Problem& p, fa_dtype dt, const void* q, const void* k,
                            const void* v, void* o, float* lse, cudaStream_t s);
cudaError_t launch_bwd_simt(const Problem& p, fa_dtype dt, const void* q, const void* k,
                            const void* v, const float* lse, const void* dO, const float* D,
                            void* dq, void* dk, void* dv, cudaStream_t s);
cudaError_t launch_bwd_preprocess(const Problem& p, fa_dtype dt, const void* o, const void* dO,
                                  float* D, float* dq_acc, cudaStream_t s);
cudaError_t launch_dq_convert(const Problem& p, const float* dq_acc, void* dq, cudaStream_t s);
cudaError_t launch_fwd_sm103(const Problem& p, const void* q, const void* k, const void* v,
                             void* o, float* lse, cudaStream_t s);
cudaError_t launch_bwd_sm103(const Problem& p, const void* q, const void* k, const void* v,
                             const float* lse, const void* dO, const float* D, float* dq_acc,
                             void* dk, void* dv, cudaStream_t s);

// Generator bytes of dropout for [BH, n_q, n_k] elements (fa_dropout.cu).
cudaError_t launch_dropout_bytes(const Problem& p, uint8_t* out, int BH, int n_q, int n_k,
                                 cudaStream_t s);

// Tensor map of a [B*H, N, d] bf16 tensor (d innermost) with 64 x 128 boxes and 128-byte
// swizzle; rows beyond N read as zero.  Returns false if the driver rejects it.
bool make_head_map(CUtensorMap* map, const void* ptr, int BH, int N, int d);
// The same view with 64-column boxes of `box_rows` rows (1..256).
bool make_head_map_rows(CUtensorMap* map, const void* ptr, int BH, int N, int d, int box_rows);

// Tensor map of a [BH, rows, inner] byte tensor (inner contiguous, a multiple of 16) with
// 128 x 128 boxes and 128-byte swizzle; bytes outside the tensor read as zero.
bool make_u8_map(CUtensorMap* map, const void* ptr, int BH, int rows, int inner);

// FP8 (e4m3) path, d = 128 (fa_fp8.cu): encoders and the forward.
cudaError_t launch_fp8_quantize_rows(const void* x, void* x8, float* scale, int BH, int N,
                                     cudaStream_t s);
cudaError_t launch_fp8_quantize_v(const void* v, void* vt8, float* scale, int BH, int N,
                                  cudaStream_t s);
cudaError_t launch_fwd_fp8(const Problem& p, const void* q8, const void* k8, const void* vt8,
                           const float* q_scale, const float* k_scale, const float* v_scale,
                           void* o, float* lse, cudaStream_t s);

// Decode over a key/value cache (split kernel + combine kernel); see fa_decode.cu.
cudaError_t launch_decode(const void* q, const void* k, const void* v, void* o, float* lse,
                          int B, int Hq, int Hkv, int Lmax, int d, const int32_t* cache_len,
                          float scale, float* partials, int splits, int* err,
                          unsigned long long wait_ns, cudaStream_t s);
// Number of key splits per (sequence, key/value head) the decode uses on this device.
int decode_splits(int B, int Hkv, int Lmax, int d);
// The tensor-core split kernel (fa_decode_tc.cu, d = 64 or 128) and its number of splits.
int decode_tc_splits(int B, int Hkv, int Lmax);
cudaError_t launch_decode_tc(const void* q, const void* k, const void* v, int B, int Hq,
                             int Hkv, int Lmax, int d, const int32_t* cache_len, float scale,
                             float* part, int splits, int* err, unsigned long long wait_ns,
                             cudaStream_t s);

// Sequence sharding (fa_shard.cu): merge of partial (O, lse) results, fp32 gradient sums.
cudaError_t launch_merge(const void* o_parts, const float* lse_parts, int S, void* o, float* lse,
                         long long rows, int d, fa_dtype dt, cudaStream_t s);
cudaError_t launch_accumulate(float* acc, const void* x, long long n, fa_dtype dt,
                              cudaStream_t s);
cudaError_t launch_finish(void* out, const float* acc, long long n, fa_dtype dt, cudaStream_t s);

// Paged cache (fa_paged.cu): block tables and slot maps, rows into their slots.  page_shift is
// log2 of the page size; strides count elements.
cudaError_t launch_paged_tables(const int32_t* cache_len, const int32_t* new_len,
                                const int32_t* free_pages, int n_free, int32_t* table,
                                long long table_stride, int max_pages, int32_t* total_len,
                                int32_t* token_start, int32_t* slots, int n_slots,
                                int32_t* pages_taken, int B, int page_shift, int num_pages,
                                cudaStream_t s);
cudaError_t launch_paged_append(const void* k, const void* v, long long k_stride,
                                long long v_stride, void* k_cache, void* v_cache,
                                long long page_stride, const int32_t* slots, int T, int num_pages,
                                int Hkv, int page_shift, int d, cudaStream_t s);
cudaError_t launch_latent_append(const void* c, const void* k_rope, long long c_stride,
                                 long long rope_stride, void* cache, long long page_stride,
                                 const int32_t* slots, int T, int num_pages, int page_shift,
                                 cudaStream_t s);

// Decode over a paged cache (fa_decode_paged.cu) and absorbed latent decode
// (fa_latent_decode.cu); the workspace holds partial results, then the sequences' tile sums.
size_t decode_paged_part_bytes(int G, int d);
cudaError_t launch_decode_paged(const void* q, const void* k, const void* v,
                                long long page_stride, const int32_t* table,
                                long long table_stride, int max_pages, int page_shift,
                                int num_pages, const int32_t* cache_len, void* o, float* lse,
                                int B, int Hq, int Hkv, int d, float scale, void* workspace,
                                int* err, unsigned long long wait_ns, cudaStream_t s);
size_t latent_decode_bytes(int B, int H);
cudaError_t launch_latent_decode(const void* q, const void* cache, long long page_stride,
                                 const int32_t* table, long long table_stride, int max_pages,
                                 int page_shift, int num_pages, const int32_t* cache_len, void* o,
                                 float* lse, int B, int H, float scale, void* workspace, int* err,
                                 unsigned long long wait_ns, cudaStream_t s);

// Decode for groups of sequences with a prefix in common (fa_decode_shared.cu).
size_t decode_shared_bytes(int B, int Hq, int Hkv, int d);
cudaError_t launch_decode_shared(const void* q, const void* k, const void* v,
                                 long long page_stride, const int32_t* table,
                                 long long table_stride, int max_pages, int page_shift,
                                 int num_pages, const int32_t* cache_len, const int32_t* start,
                                 const int32_t* shared_len, int groups, void* o, float* lse, int B,
                                 int Hq, int Hkv, int d, float scale, void* workspace, int* err,
                                 unsigned long long wait_ns, cudaStream_t s);
// Tensor map of decode queries [B, heads, group, d] with boxes of `seqs` sequences of one head.
bool make_query_map(CUtensorMap* map, const void* ptr, int B, int heads, int group, int d,
                    int seqs);

// Rotary positions (fa_rope.cu); strides of batch, head and token in elements.
cudaError_t launch_rope(const void* x, void* y, const long long (&xs)[3], const long long (&ys)[3],
                        const int32_t* pos, long long pos_axis, long long pos_batch, int axes,
                        const long long* turns, const int32_t* axis, int B, int H, int N, int d,
                        int rot, int interleaved, int inverse, fa_dtype dt, cudaStream_t s);
cudaError_t launch_rope_append(const void* q, const void* k, const void* v, long long q_stride,
                               long long k_stride, long long v_stride, void* q_out,
                               long long qo_stride, void* k_cache, void* v_cache,
                               long long page_stride, const int32_t* slots, const int32_t* pos,
                               long long pos_axis, int axes, const long long* turns,
                               const int32_t* axis, int T, int Hq, int Hkv, int num_pages,
                               int page_shift, int d, int rot, int interleaved, cudaStream_t s);

// The pages of a paged cache (fa_pages.cu).
cudaError_t launch_paged_fork(int32_t* cache_len, int32_t* table, long long table_stride,
                              int max_pages, const int32_t* free_pages, int n_free,
                              const int32_t* src, const int32_t* dst, int n, int32_t* copy_src,
                              int32_t* copy_dst, int32_t* copy_rows, int32_t* pages_taken, int B,
                              int page_shift, int num_pages, cudaStream_t s);
cudaError_t launch_paged_free(int32_t* cache_len, int32_t* table, long long table_stride,
                              int max_pages, const int32_t* rows, int n, int32_t* refs,
                              int32_t* free_pages, int32_t* n_free, int B, int page_shift,
                              int num_pages, cudaStream_t s);
cudaError_t launch_paged_compact(const int32_t* cache_len, int32_t* table, long long table_stride,
                                 int max_pages, int32_t* moved, int32_t* copy_src,
                                 int32_t* copy_dst, int n_copies, int32_t* n_used, int B,
                                 int page_shift, int num_pages, cudaStream_t s);
cudaError_t launch_paged_copy(void* k_cache, void* v_cache, long long page_stride,
                              const int32_t* src, const int32_t* dst, const int32_t* rows, int n,
                              int num_pages, int heads, int page_shift, int d, cudaStream_t s);

// Expanded latent attention: fp32 tensors on the CUDA cores (fa_latent_simt.cu), bf16 on the
// tensor cores (fa_latent_fwd.cu, fa_latent_bwd.cu).  Problem::d and the block mask are unused.
using LatentProblem = Problem;
cudaError_t launch_latent_fwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, void* o, float* o_acc,
                                   float* lse, cudaStream_t s);
cudaError_t launch_latent_fwd_sm103(const LatentProblem& p, const void* q, const void* kn,
                                    const void* kr, const void* v, void* o, float* o_acc,
                                    float* lse, cudaStream_t s);
cudaError_t launch_latent_rowdot(const LatentProblem& p, fa_dtype dt, const float* o_acc,
                                 const void* dO, float* Dsum, cudaStream_t s);
cudaError_t launch_latent_bwd_simt(const LatentProblem& p, const void* q, const void* kn,
                                   const void* kr, const void* v, const float* lse,
                                   const void* dO, const float* Dsum, void* dq, void* dkn,
                                   float* dkr_part, void* dv, cudaStream_t s);
cudaError_t launch_latent_bwd_sm103(const LatentProblem& p, const void* q, const void* kn,
                                    const void* kr, const void* v, const float* lse,
                                    const void* dO, const float* Dsum, void* dq, void* dkn,
                                    float* dkr_part, void* dv, cudaStream_t s);
cudaError_t launch_latent_rope_sum(const LatentProblem& p, fa_dtype dt, const float* part,
                                   void* dkr, cudaStream_t s);

// Tensor map of a pool of pages [P, heads, page, d] bf16 with 64 x box_rows boxes.
bool make_page_map(CUtensorMap* map, const void* ptr, int P, int heads, int page, int d,
                   long long page_stride, int box_rows);

// x rounded up to a multiple of a.
size_t round_up(size_t x, size_t a);

// Tensor map of a [B*H, N, d] fp32 accumulator with 32 x 32 boxes (128-byte swizzle), for bulk
// reduce-add; rows beyond N are outside the map.
bool make_acc_map(CUtensorMap* map, const void* ptr, int BH, int N, int d);

// Device address of the library's error word on the current device (nullptr on failure).
int* error_word();

// Number of SMs of the current device (cached per device).
int sm_count();

}  // namespace fa
