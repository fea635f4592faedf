// What the kernels of the absorbed latent decode share.
#pragma once

#include <cuda.h>

#include "fa_internal.cuh"

namespace fa {

struct LatentArgs {
  const __nv_bfloat16* q;  // [B, H, 576]
  const int32_t* table;
  long long table_stride;
  int max_pages, page_shift, num_pages;
  const int32_t* cache_len;
  int B, H;
  float c;                 // scale log2 e
  __nv_bfloat16* o;        // [B, H, 512]
  float* lse;
  float* part;             // [2 workers][H][512]
  float2* stat;            // [2 workers][2 halves of the columns][H]: maximum, sum
  long long* prefix;       // [B + 1] tiles before each sequence
  int* err;
  unsigned long long wait_ns;
};

constexpr int kFewHeads = 16;   // most heads of launch_latent_decode_few
constexpr int kFewKeys = 64;    // keys of its tile, and of the boxes of its map of the cache

// At most 16 heads (fa_latent_decode_few.cu); `workers` CTAs, partial results and prefix as for
// the combine kernel of fa_latent_decode.cu.
cudaError_t launch_latent_decode_few(const CUtensorMap& mc, const LatentArgs& a, int workers,
                                     cudaStream_t s);

}  // namespace fa
