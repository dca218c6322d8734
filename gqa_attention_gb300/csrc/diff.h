// diff.h -- parameter blocks, launchers and the epilogue of differential attention
// (decode_diff.cu, prefill.cu).  Not part of the public ABI.
#pragma once

#include "internal.h"

namespace gqa {

// What follows the two maps of a head: O = O_1 - lam O_2, and if norm_eps >= 0
// O / sqrt(mean(O^2) + norm_eps) * norm_weight, times out_scale.
struct DiffParams {
  const float* lam;                // lam[b * lam_b + t * lam_t + h * lam_h]
  long long lam_b, lam_t, lam_h;   // strides in elements, 0 for a value that is shared
  const float* norm_weight;        // [d], or null (ones)
  float norm_eps;                  // negative: no norm
  float out_scale;
  int split_keys;  // the maps are the halves of a query and a key row, not two query heads
};

// Decode: H_q and G of `dec` count maps (two per head), out is [B, T_q, H_q / 2, d],
// lse and the workspace have a row per map; q is [B, T_q, H_q, d], or
// [B, T_q, H_q / 2, d] with split keys.
struct DecodeDiffParams {
  DecodeParams dec;
  DiffParams diff;
  // > 0: the batch is cut by its lengths into at most as many pieces, at most n_split of a
  // sequence, and grid x is the piece; 0: split x of sequence z has dec.chunk keys.
  int pieces;
};

// The merge of a head's partials, two maps of n_part parts each, and the epilogue.
struct DiffMergeParams {
  DiffParams diff;
  const float2* ws_ml;  // [B * T * H_maps][n_part] (m, l)
  const float* ws_O;    // [B * T * H_maps][n_part][d]
  float m_log2;         // m times this is in base-2 units
  int B, T, H_maps, d, n_part;
  __nv_bfloat16* out;   // [B, T, H_maps / 2, d]
  float* lse;           // element (b, t, map) at b * lse_b + t * lse_t + map * lse_m
  long long lse_b, lse_t, lse_m;
  unsigned* err;
};

struct PrefillDiffParams {
  PrefillParams pre;  // H_q and G count maps, as above
  DiffParams diff;
};

cudaError_t launch_decode_diff(const DecodeDiffParams& p, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, cudaStream_t stream);
// `general`: lengths, a window or parts (else plain causal prefill).  With parts the kernel
// leaves the maps' partials; launch_diff_merge finishes.
cudaError_t launch_prefill_diff(const PrefillDiffParams& p, bool general, const CUtensorMap& tm_q,
                                const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                                cudaStream_t stream);
// d = 128, up to 128 rows of maps per KV head in one tensor-core tile (decode_tc.cu), 128-key
// boxes and chunks.  tm_q: q as [B * T_q][2 H][d], box {64, G, T_q}; with split keys as
// [B * T_q][H][2][64], box {64, 2, G / 2, T_q}.
cudaError_t launch_decode_diff_tc(const DecodeDiffParams& p, const CUtensorMap& tm_q,
                                  const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                  cudaStream_t stream);
cudaError_t launch_diff_merge(const DiffMergeParams& p, cudaStream_t stream);

}  // namespace gqa
