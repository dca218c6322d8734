// kv_append.h -- parameters and launcher of the rotated append to bf16 and per-token
// E4M3 caches (kv_append.cu).  Not part of the public ABI.
#pragma once

#include "internal.h"

namespace gqa {

struct KvAppendParams {
  // token (b, i) of [B, T]: rows of H_q * d (q) and H_kv * d (k, v) elements, token
  // b * T + i at q_stride or kv_stride elements times that
  const __nv_bfloat16 *q, *k, *v;  // q may be null
  long long q_stride, kv_stride;
  const float* freqs;        // [rot / 2] radians per position
  int rot, interleaved;      // rot == 0: nothing is turned
  const int32_t* n_new;      // [B] or null: every one T
  const int32_t* seq_lens;   // [B] lengths after the call
  const int32_t* positions;  // [B, T] or null: the token's place in its sequence
  const int32_t* block_table;
  int B, T, S_max, H_q, H_kv, d;
  int max_blocks, page_size, num_pages;
  void *k_cache, *v_cache;   // bf16, or E4M3 codes if k_scale is set
  float *k_scale, *v_scale;  // one per cache row
  __nv_bfloat16* q_out;      // [B, T, H_q, d]
  unsigned* err;
};

cudaError_t launch_kv_append_rot(const KvAppendParams& p, int sms, cudaStream_t stream);

}  // namespace gqa
