// api.cu -- the C ABI of libgqa_attn.so (declared in include/gqa_attn.h):
// argument checks, TMA tensor-map encoding, the per-device error word and the
// kernel launches.  Nothing here computes attention.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "diff.h"
#include "gqa_attn.h"
#include "internal.h"
#include "kv_append.h"

namespace {

// One error word per device (a module global is instantiated per context).
__device__ unsigned g_error_word;

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
unsigned* g_err_ptr[kMaxDevices] = {};
int g_num_sms[kMaxDevices] = {};
std::atomic<uint64_t> g_wait_ns{2000000000ull};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

gqa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA; }

// Device pointer of the error word of the current device (looked up once).
gqa_status error_word(unsigned** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GQA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return GQA_ERR_CUDA;
    g_err_ptr[dev] = static_cast<unsigned*>(p);
  }
  *out = g_err_ptr[dev];
  return GQA_OK;
}

int num_sms_current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_num_sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
      n = 148;
    g_num_sms[dev] = n;
  }
  return g_num_sms[dev];
}

gqa_status get_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !f)
      return GQA_ERR_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  *fn = g_encode;
  return GQA_OK;
}

// A tensor map of `rank` dims (innermost first); strides in bytes for dims 1.. .
gqa_status encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swz);

gqa_status encode_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                       const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swz) {
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, strides, box, swz);
}

gqa_status encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swz) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  gqa_status st = get_encoder(&enc);
  if (st != GQA_OK) return st;
  cuuint64_t gdim[5], gstr[4];
  cuuint32_t bdim[5], estr[5];
  for (int i = 0; i < rank; ++i) {
    gdim[i] = dims[i];
    bdim[i] = box[i];
    estr[i] = 1;
    if (i + 1 < rank) gstr[i] = strides[i];
  }
  CUresult r = enc(map, type, rank, const_cast<void*>(base), gdim,
                   gstr, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GQA_OK : GQA_ERR_INVALID_ARG;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

// Query rows (T_q x G) a multi-token decode folds per KV head: four row groups
// of 16, each its own CTA; with d = 128, up to 128 rows in one tensor-core
// tile (used above 16 rows).
constexpr int kMaxMultiRows = 64;
constexpr int kMaxMultiRowsTc = 128;
// Splits of a sequence in differential decode, at most.
constexpr int kMaxDiffSplits = 65535;
// Token rows of a cache, at most, where a last tile may reach past them in 32 bits.
constexpr long long kMaxCacheRows = 0x7fff0000LL;
bool multi_uses_tc(int T_q, int G, int d) { return d == 128 && T_q * G > 16; }

}  // namespace

extern "C" {

const char* gqa_status_str(int status) {
  switch (status) {
    case GQA_OK: return "GQA_OK";
    case GQA_ERR_INVALID_ARG: return "GQA_ERR_INVALID_ARG";
    case GQA_ERR_UNSUPPORTED: return "GQA_ERR_UNSUPPORTED";
    case GQA_ERR_CUDA: return "GQA_ERR_CUDA";
    case GQA_ERR_TIMEOUT: return "GQA_ERR_TIMEOUT";
    default: return "GQA_ERR_UNKNOWN";
  }
}

int gqa_version(void) { return 100; }

int gqa_attn_decode_split_chunk(int S_max, int n_split) {
  if (S_max < 1 || n_split < 1) return 0;
  const long long per = ((long long)S_max + n_split - 1) / n_split;
  const long long t = gqa::kDecodeTile;
  return (int)((per + t - 1) / t * t);
}

size_t gqa_attn_decode_workspace_bytes(int B, int H_q, int d, int n_split) {
  if (B < 1 || H_q < 1 || d < 1 || n_split <= 1) return 0;
  return gqa::decode_ws_O_offset(B, H_q, n_split) + (size_t)B * H_q * n_split * d * sizeof(float);
}

int gqa_attn_decode_default_splits(int B, int H_kv, int S_max, int device) {
  if (B < 1 || H_kv < 1 || S_max < 1) return 1;
  int sms = 0;
  if (device < 0) {
    sms = num_sms_current_device();
  } else if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
             sms < 1) {
    cudaGetLastError();  // (a device that cannot be queried leaves no sticky error)
    return 1;
  }
  // Up to 1024 tokens one CTA streams the whole sequence: the combine launch
  // then costs more than the split saves (measured: d = 32, 1024 tokens, 6.1 us
  // unsplit against 9.0 us with 8 splits + combine; d = 128 about equal).
  if (S_max <= 1024) return 1;
  // About one CTA per SM (measured best for a single long sequence), with
  // splits of at least 128 tokens and at most 8192 tokens (ragged batches then
  // have enough CTAs to balance).
  const long long groups = (long long)B * H_kv;
  long long n = (sms + groups - 1) / groups;
  const long long most = (S_max + 127) / 128;
  const long long fill = (S_max + 8191) / 8192;
  if (n > most) n = most;
  if (n < fill) n = fill;
  if (n < 1) n = 1;
  if (n > 65535) n = 65535;
  return (int)n;
}

}  // extern "C"

namespace {

// Checks the decode arguments shared by the contiguous and the paged cache,
// encodes the K/V tensor maps (cache viewed as [rows][H_kv][d], boxes of
// box_rows token rows of one head, at most 64 elements / 128 bytes wide,
// swizzled for ldmatrix) and fills the kernel parameters.
gqa_status prepare_decode(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* seq_lens, int B, int S_max, long long rows, int box_rows,
                          int H_q, int H_kv, int d, float scale, int n_split, void* workspace,
                          void* out, float* lse, CUtensorMap* tm_k, CUtensorMap* tm_v,
                          gqa::DecodeParams* p, bool needs_workspace = true) {
  if (!q || !k_cache || !v_cache || !seq_lens || !out || !lse) return GQA_ERR_INVALID_ARG;
  if (B < 1 || S_max < 1 || H_q < 1 || H_kv < 1 || n_split < 1) return GQA_ERR_INVALID_ARG;
  if (B > 65535 || H_kv > 65535 || H_q % H_kv != 0) return GQA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return GQA_ERR_INVALID_ARG;
  if (rows > 0x7fffffffLL || n_split > 0x7fffffff) return GQA_ERR_INVALID_ARG;
  if (!head_dim_ok(d) || H_q / H_kv > 16) return GQA_ERR_UNSUPPORTED;
  if (needs_workspace && n_split > 1 && !workspace) return GQA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(seq_lens, 4) || (workspace && !aligned(workspace, 256)))
    return GQA_ERR_INVALID_ARG;

  unsigned* err = nullptr;
  gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;

  const int box_d = d >= 64 ? 64 : d;
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)H_kv, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)H_kv * d * 2};
  const uint32_t box[3] = {(uint32_t)box_d, 1u, (uint32_t)box_rows};
  const CUtensorMapSwizzle swz = box_d == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if ((st = encode_bf16(tm_k, k_cache, 3, dims, strides, box, swz)) != GQA_OK) return st;
  if ((st = encode_bf16(tm_v, v_cache, 3, dims, strides, box, swz)) != GQA_OK) return st;

  *p = gqa::DecodeParams{};
  p->q = static_cast<const __nv_bfloat16*>(q);
  p->seq_lens = seq_lens;
  p->T_q = 1;
  p->n_rg = 1;
  p->B = B;
  p->S_max = S_max;
  p->H_q = H_q;
  p->H_kv = H_kv;
  p->G = H_q / H_kv;
  p->d = d;
  p->n_split = n_split;
  p->chunk = gqa_attn_decode_split_chunk(S_max, n_split);
  p->scale_log2 = scale * 1.4426950408889634f;
  p->ws_ml = static_cast<float2*>(workspace);
  p->ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                 gqa::decode_ws_O_offset(B, H_q, n_split))
                      : nullptr;
  p->out = static_cast<__nv_bfloat16*>(out);
  p->lse = lse;
  p->err = err;
  p->wait_ns = g_wait_ns.load();
  return GQA_OK;
}

}  // namespace

extern "C" {

gqa_status gqa_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* seq_lens, int B, int S_max, int H_q, int H_kv, int d,
                           float scale, int n_split, void* workspace, void* out, float* lse,
                           gqa_stream_t stream) {
  CUtensorMap tm_k, tm_v;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_cache, v_cache, seq_lens, B, S_max, (long long)B * S_max,
                                 gqa::kDecodeTile, H_q, H_kv, d, scale, n_split, workspace, out,
                                 lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  return cuda_status(gqa::launch_decode_split(p, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gqa_attn_decode_counter_bytes(int B, int H_kv) {
  if (B < 1 || H_kv < 1) return 0;
  return (size_t)B * H_kv * 2 * sizeof(int32_t);
}

gqa_status gqa_attn_decode_balanced(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* seq_lens, int B, int S_max, int H_q, int H_kv,
                                    int d, float scale, int n_split, void* workspace,
                                    int32_t* counters, void* out, float* lse,
                                    gqa_stream_t stream) {
  if (n_split > 1 && (!counters || !aligned(counters, 4))) return GQA_ERR_INVALID_ARG;
  CUtensorMap tm_k, tm_v;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_cache, v_cache, seq_lens, B, S_max, (long long)B * S_max,
                                 gqa::kDecodeTile, H_q, H_kv, d, scale, n_split, workspace, out,
                                 lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  if (n_split > 1) p.tile_ctr = counters;
  return cuda_status(gqa::launch_decode_split(p, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
}

int gqa_attn_decode_multi_default_splits(int B, int T_q, int H_q, int H_kv, int S_max, int d) {
  if (B < 1 || T_q < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0) return 1;
  const int n = gqa_attn_decode_default_splits(B, H_kv, S_max, -1);
  const long long groups = (T_q * (long long)(H_q / H_kv) + 15) / 16;
  if (groups <= 1) return n;
  // The tensor-core kernel: one CTA per SM, K/V read once per split.
  if (multi_uses_tc(T_q, H_q / H_kv, d)) return n;
  // Several row groups: keep every CTA of a split resident at once (two per
  // SM), so the groups' reads of the same K/V tiles meet in L2 (measured for
  // Llama3-70B at 32K: 19 / 12 / 9 splits best for 2 / 3 / 4 groups).
  const long long fit = 2LL * num_sms_current_device() / ((long long)B * H_kv * groups);
  return (int)std::max(1LL, std::min((long long)n, fit));
}

gqa_status gqa_attn_decode_multi(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* seq_lens, int B, int T_q, int S_max, int H_q,
                                 int H_kv, int d, float scale, int n_split, void* workspace,
                                 void* out, float* lse, gqa_stream_t stream) {
  if (T_q < 1 || T_q > 64 || T_q > S_max) return GQA_ERR_INVALID_ARG;
  if (H_kv < 1 || H_q % H_kv != 0) return GQA_ERR_INVALID_ARG;
  const bool tc = multi_uses_tc(T_q, H_q / H_kv, d);
  if (T_q * (H_q / H_kv) > (tc ? kMaxMultiRowsTc : kMaxMultiRows)) return GQA_ERR_UNSUPPORTED;
  if ((long long)B * T_q > 65535) return GQA_ERR_INVALID_ARG;
  CUtensorMap tm_k, tm_v;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_cache, v_cache, seq_lens, B, S_max, (long long)B * S_max,
                                 tc ? 128 : gqa::kDecodeTile, H_q, H_kv, d, scale, n_split,
                                 workspace, out, lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  if (tc) {
    // All T_q * G rows of a KV head in one tile: Q as [B * T_q][H_q][d], one
    // box of G heads x T_q queries per d half; 128-key splits.
    CUtensorMap tm_q;
    const uint64_t qdims[3] = {(uint64_t)d, (uint64_t)H_q, (uint64_t)B * T_q};
    const uint64_t qstrides[2] = {(uint64_t)d * 2, (uint64_t)H_q * d * 2};
    const uint32_t qbox[3] = {64u, (uint32_t)(H_q / H_kv), (uint32_t)T_q};
    if ((st = encode_bf16(&tm_q, q, 3, qdims, qstrides, qbox, CU_TENSOR_MAP_SWIZZLE_128B)) !=
        GQA_OK)
      return st;
    p.T_q = T_q;
    p.n_rg = 1;
    const long long per = ((long long)S_max + n_split - 1) / n_split;
    p.chunk = (int)((per + 127) / 128 * 128);
    p.ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                  gqa::decode_ws_O_offset(B * T_q, H_q, n_split))
                       : nullptr;
    return cuda_status(
        gqa::launch_decode_tc(p, tm_q, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
  }
  p.T_q = T_q;
  p.n_rg = (T_q * p.G + 15) / 16;
  if ((long long)n_split * p.n_rg > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
  // the partials are laid out for B * T_q rows of H_q heads
  p.ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                gqa::decode_ws_O_offset(B * T_q, H_q, n_split))
                     : nullptr;
  return cuda_status(gqa::launch_decode_split(p, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
}

int gqa_attn_decode_fused_splits(int B, int H_q, int H_kv, int d) {
  if (B < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0 || !head_dim_ok(d) || H_q / H_kv > 16)
    return 0;
  // The largest cluster (16, else 8) whose CTAs can be resident together,
  // probed once per device and head shape class.
  static int cache[64][3][2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int di = d == 32 ? 0 : d == 64 ? 1 : 2, gi = H_q / H_kv > 8 ? 1 : 0;
  if (dev >= 0 && dev < 64 && cache[dev][di][gi] != 0) return cache[dev][di][gi] > 0 ? cache[dev][di][gi] : 0;
  int found = -1;
  for (int c : {16, 8}) {
    gqa::DecodeParams p{};
    p.B = 1;
    p.H_kv = 1;
    p.G = H_q / H_kv;
    p.d = d;
    p.n_split = c;
    CUtensorMap dummy{};
    if (gqa::launch_decode_fused(p, dummy, dummy, true, nullptr) == cudaSuccess) {
      found = c;
      break;
    }
    cudaGetLastError();  // clear a failed probe
  }
  if (dev >= 0 && dev < 64) cache[dev][di][gi] = found;
  return found > 0 ? found : 0;
}

gqa_status gqa_attn_decode_fused(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* seq_lens, int B, int S_max, int H_q, int H_kv,
                                 int d, float scale, void* out, float* lse, gqa_stream_t stream) {
  if (B < 1 || H_q < 1 || H_kv < 1) return GQA_ERR_INVALID_ARG;
  if (H_q % H_kv != 0) return GQA_ERR_INVALID_ARG;
  const int c = gqa_attn_decode_fused_splits(B, H_q, H_kv, d);
  if (c == 0) return GQA_ERR_UNSUPPORTED;
  CUtensorMap tm_k, tm_v;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_cache, v_cache, seq_lens, B, S_max, (long long)B * S_max,
                                 gqa::kDecodeTile, H_q, H_kv, d, scale, c, nullptr, out, lse,
                                 &tm_k, &tm_v, &p, /*needs_workspace=*/false);
  if (st != GQA_OK) return st;
  return cuda_status(
      gqa::launch_decode_fused(p, tm_k, tm_v, false, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status gqa_attn_decode_paged_multi(const void* q, const void* k_pool, const void* v_pool,
                                       const int32_t* block_table, const int32_t* seq_lens, int B,
                                       int T_q, int num_pages, int page_size, int max_blocks,
                                       int H_q, int H_kv, int d, float scale, int n_split,
                                       void* workspace, void* out, float* lse,
                                       gqa_stream_t stream) {
  if (T_q < 1 || T_q > 64) return GQA_ERR_INVALID_ARG;
  if (H_kv < 1 || H_q % H_kv != 0) return GQA_ERR_INVALID_ARG;
  const bool tc = multi_uses_tc(T_q, H_q / H_kv, d);
  if (T_q * (H_q / H_kv) > (tc ? kMaxMultiRowsTc : kMaxMultiRows)) return GQA_ERR_UNSUPPORTED;
  if ((long long)B * T_q > 65535) return GQA_ERR_INVALID_ARG;
  if (!block_table || !aligned(block_table, 4)) return GQA_ERR_INVALID_ARG;
  if (num_pages < 1 || max_blocks < 1 || page_size < 1) return GQA_ERR_INVALID_ARG;
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return GQA_ERR_UNSUPPORTED;
  const long long S_max = (long long)max_blocks * page_size;
  const long long rows = (long long)num_pages * page_size;
  if (S_max > 0x7fffffffLL || rows > 0x7ffffffeLL) return GQA_ERR_INVALID_ARG;
  if (tc) {
    // All T_q * G rows of a KV head in one tensor-core tile; each 128-key tile
    // arrives as boxes of min(page_size, 128) rows, one page each.
    CUtensorMap tm_k, tm_v, tm_q;
    gqa::DecodeParams p;
    gqa_status st = prepare_decode(q, k_pool, v_pool, seq_lens, B, (int)S_max, rows,
                                   page_size < 128 ? page_size : 128, H_q, H_kv, d, scale,
                                   n_split, workspace, out, lse, &tm_k, &tm_v, &p);
    if (st != GQA_OK) return st;
    const uint64_t qdims[3] = {(uint64_t)d, (uint64_t)H_q, (uint64_t)B * T_q};
    const uint64_t qstrides[2] = {(uint64_t)d * 2, (uint64_t)H_q * d * 2};
    const uint32_t qbox[3] = {64u, (uint32_t)(H_q / H_kv), (uint32_t)T_q};
    if ((st = encode_bf16(&tm_q, q, 3, qdims, qstrides, qbox, CU_TENSOR_MAP_SWIZZLE_128B)) !=
        GQA_OK)
      return st;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.T_q = T_q;
    p.n_rg = 1;
    const long long per = (S_max + n_split - 1) / n_split;
    p.chunk = (int)((per + 127) / 128 * 128);
    p.ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                  gqa::decode_ws_O_offset(B * T_q, H_q, n_split))
                       : nullptr;
    return cuda_status(
        gqa::launch_decode_tc(p, tm_q, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
  }
  if (n_split >= 1) {
    const int chunk = gqa_attn_decode_split_chunk((int)S_max, n_split);
    if (chunk / page_size + 2 > gqa::kMaxPagesPerCta) return GQA_ERR_UNSUPPORTED;
  }
  CUtensorMap tm_k, tm_v;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_pool, v_pool, seq_lens, B, (int)S_max, rows,
                                 page_size < gqa::kDecodeTile ? page_size : gqa::kDecodeTile, H_q,
                                 H_kv, d, scale, n_split, workspace, out, lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.T_q = T_q;
  p.n_rg = (T_q * p.G + 15) / 16;
  p.ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                gqa::decode_ws_O_offset(B * T_q, H_q, n_split))
                     : nullptr;
  return cuda_status(gqa::launch_decode_paged(p, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status gqa_attn_decode_paged(const void* q, const void* k_pool, const void* v_pool,
                                 const int32_t* block_table, const int32_t* seq_lens, int B,
                                 int num_pages, int page_size, int max_blocks, int H_q, int H_kv,
                                 int d, float scale, int n_split, void* workspace, void* out,
                                 float* lse, gqa_stream_t stream) {
  return gqa_attn_decode_paged_multi(q, k_pool, v_pool, block_table, seq_lens, B, 1, num_pages,
                                     page_size, max_blocks, H_q, H_kv, d, scale, n_split,
                                     workspace, out, lse, stream);
}

}  // extern "C"

namespace {

// The arguments of differential attention beside those of the two maps.
gqa_status diff_params(const float* lam, int64_t lam_b, int64_t lam_t, int64_t lam_h, int H,
                       int H_kv, int split_keys, const float* norm_weight, float norm_eps,
                       float out_scale, gqa::DiffParams* p) {
  if (!lam || !aligned(lam, 4) || lam_b < 0 || lam_t < 0 || lam_h < 0) return GQA_ERR_INVALID_ARG;
  if (H < 1 || H > 32767 || H_kv < 1 || H % H_kv != 0) return GQA_ERR_INVALID_ARG;
  if (split_keys != 0 && split_keys != 1) return GQA_ERR_INVALID_ARG;
  if (!std::isfinite(norm_eps) || !std::isfinite(out_scale)) return GQA_ERR_INVALID_ARG;
  if (norm_weight && (norm_eps < 0.f || !aligned(norm_weight, 4))) return GQA_ERR_INVALID_ARG;
  *p = gqa::DiffParams{lam, lam_b, lam_t, lam_h, norm_weight, norm_eps, out_scale, split_keys};
  return GQA_OK;
}

// The shape of a paged cache: S_max and the pools' token rows.
gqa_status paged_shape(const int32_t* block_table, int num_pages, int page_size, int max_blocks,
                       int* S_max, long long* rows) {
  if (!block_table || !aligned(block_table, 4)) return GQA_ERR_INVALID_ARG;
  if (num_pages < 1 || max_blocks < 1 || page_size < 1) return GQA_ERR_INVALID_ARG;
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return GQA_ERR_UNSUPPORTED;
  const long long s = (long long)max_blocks * page_size;
  *rows = (long long)num_pages * page_size;
  if (s > kMaxCacheRows) return GQA_ERR_INVALID_ARG;
  *S_max = (int)s;
  return GQA_OK;
}

int length_pieces(int B, long long groups, int rows, int S_max);

// Pieces for every KV head that a batch of differential decode on mma.sync is cut into by its
// lengths, or 0: even splits.  One piece for each CTA that the GPU holds (two to an SM, one
// of more than 16 rows).  Where a piece has 32 tiles of 64 keys (8 sequences of 1K to 64K, 8 KV
// heads of 128: 174 us, 238 in 8 even splits, 177 in 12), or, of more than 16 rows, 4 (8 x
// 20K, 3 heads of 64, 30 rows: all equally long 38.7 us, even 48.8; 3K to 20K 28.8 and
// 28.0); with less the cut takes what it saves (4 x 8K, 4 heads of 128: 14.6 and 12.9).
// Fewer than four pieces a sequence fill the GPU badly (24 x 20K, 5 heads of 32: 102 and 69).
int diff_pieces(int B, int H_kv, int rows, int S_max) {
  const long long groups = (long long)H_kv * (rows <= 16 ? 1 : (rows + 31) / 32);
  const long long slots = (rows <= 16 ? 2LL : 1LL) * num_sms_current_device();
  const long long pieces = slots / groups, tiles = ((long long)S_max + 63) / 64;
  const long long least = rows <= 16 ? 32 : 4;
  return B > 1 && B <= 96 && pieces >= 4LL * B && tiles * B * groups >= least * slots ? (int)pieces : 0;
}

gqa_status run_decode_diff(const void* q, const void* k, const void* v, const int32_t* block_table,
                           const int32_t* seq_lens, const gqa::DiffParams& diff, int B, int T_q,
                           int S_max, long long rows, int num_pages, int page_size, int max_blocks,
                           int H, int H_kv, int d, float scale, int n_split, void* workspace,
                           void* out, float* lse, gqa_stream_t stream) {
  // (rows and tokens stay below 2^31 with the last tile's overhang)
  if (rows < 1 || rows > kMaxCacheRows || S_max < 1 || S_max > kMaxCacheRows)
    return GQA_ERR_INVALID_ARG;
  if (T_q < 1 || T_q > 64 || T_q > S_max || n_split > kMaxDiffSplits)
    return GQA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !aligned(lse, 8)) return GQA_ERR_INVALID_ARG;
  if (head_dim_ok(d) && T_q * (2 * H / H_kv) > kMaxMultiRows) return GQA_ERR_UNSUPPORTED;
  // More than 16 rows of d = 128: one tensor-core tile of 128 keys.
  const bool tc = multi_uses_tc(T_q, 2 * H / H_kv, d);
  const int tile = tc ? 128 : gqa::kDecodeTile;
  CUtensorMap tm_k, tm_v;
  gqa::DecodeDiffParams p{};
  gqa_status st = prepare_decode(q, k, v, seq_lens, B, S_max, rows,
                                 block_table && page_size < tile ? page_size : tile, 2 * H, H_kv, d,
                                 scale, n_split, workspace, out, lse, &tm_k, &tm_v, &p.dec);
  if (st != GQA_OK) return st;
  p.diff = diff;
  p.dec.T_q = T_q;
  p.dec.block_table = block_table;
  p.dec.max_blocks = max_blocks;
  p.dec.page_size = page_size;
  p.dec.num_pages = num_pages;
  // the partials are laid out for B * T_q rows of 2 H maps
  if ((long long)B * T_q > 0x7fffffffLL / (2 * H)) return GQA_ERR_INVALID_ARG;
  p.dec.ws_O = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                    gqa::decode_ws_O_offset(B * T_q, 2 * H, n_split))
                         : nullptr;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tc) {
    const uint64_t G = 2 * H / H_kv, BT = (uint64_t)B * T_q;
    CUtensorMap tm_q;
    if (diff.split_keys) {
      const uint64_t dims[4] = {64, 2, (uint64_t)H, BT}, strides[3] = {128, 256, (uint64_t)H * 256};
      const uint32_t box[4] = {64u, 2u, (uint32_t)G / 2, (uint32_t)T_q};
      st = encode_bf16(&tm_q, q, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
      const uint64_t dims[3] = {128, 2 * (uint64_t)H, BT}, strides[2] = {256, 2 * (uint64_t)H * 256};
      const uint32_t box[3] = {64u, (uint32_t)G, (uint32_t)T_q};
      st = encode_bf16(&tm_q, q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (st != GQA_OK) return st;
    const long long per = ((long long)S_max + n_split - 1) / n_split;
    p.dec.n_rg = 1;
    p.dec.chunk = (int)((per + 127) / 128 * 128);
    p.pieces = n_split == 1 ? 0 : length_pieces(B, H_kv, T_q * (int)G, S_max);
    if ((long long)n_split * p.dec.chunk > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
    st = cuda_status(gqa::launch_decode_diff_tc(p, tm_q, tm_k, tm_v, s));
  } else {
    if ((long long)n_split * p.dec.chunk > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
    p.pieces = n_split == 1 ? 0 : diff_pieces(B, H_kv, T_q * (2 * H / H_kv), S_max);
    st = cuda_status(gqa::launch_decode_diff(p, tm_k, tm_v, s));
  }
  if (st != GQA_OK || n_split == 1) return st;
  gqa::DiffMergeParams m{};
  m.diff = diff;
  m.ws_ml = p.dec.ws_ml;
  m.ws_O = p.dec.ws_O;
  m.m_log2 = 1.4426950408889634f;
  m.B = B;
  m.T = T_q;
  m.H_maps = 2 * H;
  m.d = d;
  m.n_part = n_split;
  m.out = p.dec.out;
  m.lse = lse;
  m.lse_b = (long long)T_q * 2 * H;
  m.lse_t = 2 * H;
  m.lse_m = 1;
  m.err = p.dec.err;
  return cuda_status(gqa::launch_diff_merge(m, s));
}

// Checks what the appends share and launches; the cache's shape is in `p` already.
gqa_status run_kv_append_rot(gqa::KvAppendParams* p, long long rows, const void* q,
                             const void* k_new, const void* v_new, int64_t q_stride,
                             int64_t kv_stride, const float* freqs, int rot, int interleaved,
                             const int32_t* n_new, const int32_t* positions,
                             const int32_t* seq_lens, int B, int T, int H_q, int H_kv, int d,
                             void* k_cache, void* v_cache, void* q_out, gqa_stream_t stream) {
  if (!k_new || !v_new || !seq_lens || !k_cache || !v_cache) return GQA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return GQA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || H_kv < 1 || H_kv > 65535 || (q && (H_q < 1 || H_q > 65535)))
    return GQA_ERR_INVALID_ARG;
  if (d != 16 && !head_dim_ok(d)) return GQA_ERR_UNSUPPORTED;
  if (rows < 1 || rows > kMaxCacheRows || (long long)B * T > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || (rot > 0 && (!freqs || !aligned(freqs, 4)))) return GQA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return GQA_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return GQA_ERR_INVALID_ARG;
  if (kv_stride < (int64_t)H_kv * d || kv_stride % 8 != 0) return GQA_ERR_INVALID_ARG;
  if (q && (q_stride < (int64_t)H_q * d || q_stride % 8 != 0)) return GQA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(seq_lens, 4) ||
      !aligned(n_new, 4) || !aligned(positions, 4) || !aligned(p->k_scale, 4) ||
      !aligned(p->v_scale, 4))
    return GQA_ERR_INVALID_ARG;
  unsigned* err = nullptr;
  const gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;
  p->q = static_cast<const __nv_bfloat16*>(q);
  p->k = static_cast<const __nv_bfloat16*>(k_new);
  p->v = static_cast<const __nv_bfloat16*>(v_new);
  p->q_stride = q_stride;
  p->kv_stride = kv_stride;
  p->freqs = freqs;
  p->rot = rot;
  p->interleaved = interleaved;
  p->n_new = n_new;
  p->seq_lens = seq_lens;
  p->positions = positions;
  p->B = B;
  p->T = T;
  p->H_q = q ? H_q : 0;
  p->H_kv = H_kv;
  p->d = d;
  p->k_cache = k_cache;
  p->v_cache = v_cache;
  p->q_out = static_cast<__nv_bfloat16*>(q_out);
  p->err = err;
  return cuda_status(gqa::launch_kv_append_rot(*p, num_sms_current_device(),
                                               reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

gqa_status gqa_kv_append(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                         int64_t kv_stride, const float* freqs, int rot, int interleaved,
                         const int32_t* n_new, const int32_t* positions, const int32_t* seq_lens,
                         int B, int T, int S_max, int H_q, int H_kv, int d, void* k_cache,
                         void* v_cache, void* q_out, gqa_stream_t stream) {
  gqa::KvAppendParams p{};
  p.S_max = S_max;
  return run_kv_append_rot(&p, S_max < 1 ? 0 : (long long)B * S_max, q, k_new, v_new, q_stride,
                           kv_stride, freqs, rot, interleaved, n_new, positions, seq_lens, B, T,
                           H_q, H_kv, d, k_cache, v_cache, q_out, stream);
}

gqa_status gqa_kv_append_paged(const void* q, const void* k_new, const void* v_new,
                               int64_t q_stride, int64_t kv_stride, const float* freqs, int rot,
                               int interleaved, const int32_t* n_new, const int32_t* positions,
                               const int32_t* block_table, const int32_t* seq_lens, int B, int T,
                               int num_pages, int page_size, int max_blocks, int H_q, int H_kv,
                               int d, void* k_pool, void* v_pool, void* q_out,
                               gqa_stream_t stream) {
  gqa::KvAppendParams p{};
  long long rows = 0;
  const gqa_status st = paged_shape(block_table, num_pages, page_size, max_blocks, &p.S_max, &rows);
  if (st != GQA_OK) return st;
  p.block_table = block_table;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_blocks = max_blocks;
  return run_kv_append_rot(&p, rows, q, k_new, v_new, q_stride, kv_stride, freqs, rot, interleaved,
                           n_new, positions, seq_lens, B, T, H_q, H_kv, d, k_pool, v_pool, q_out,
                           stream);
}

gqa_status gqa_kv_append_fp8(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                             int64_t kv_stride, const float* freqs, int rot, int interleaved,
                             const int32_t* n_new, const int32_t* positions,
                             const int32_t* seq_lens, int B, int T, int S_max, int H_q, int H_kv,
                             int d, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                             void* q_out, gqa_stream_t stream) {
  if (!k_scale || !v_scale) return GQA_ERR_INVALID_ARG;
  gqa::KvAppendParams p{};
  p.S_max = S_max;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  return run_kv_append_rot(&p, S_max < 1 ? 0 : (long long)B * S_max, q, k_new, v_new, q_stride,
                           kv_stride, freqs, rot, interleaved, n_new, positions, seq_lens, B, T,
                           H_q, H_kv, d, k_cache, v_cache, q_out, stream);
}

gqa_status gqa_kv_append_paged_fp8(const void* q, const void* k_new, const void* v_new,
                                   int64_t q_stride, int64_t kv_stride, const float* freqs,
                                   int rot, int interleaved, const int32_t* n_new,
                                   const int32_t* positions, const int32_t* block_table,
                                   const int32_t* seq_lens, int B, int T, int num_pages,
                                   int page_size, int max_blocks, int H_q, int H_kv, int d,
                                   void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                                   void* q_out, gqa_stream_t stream) {
  if (!k_scale || !v_scale) return GQA_ERR_INVALID_ARG;
  gqa::KvAppendParams p{};
  long long rows = 0;
  const gqa_status st = paged_shape(block_table, num_pages, page_size, max_blocks, &p.S_max, &rows);
  if (st != GQA_OK) return st;
  p.block_table = block_table;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_blocks = max_blocks;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  return run_kv_append_rot(&p, rows, q, k_new, v_new, q_stride, kv_stride, freqs, rot, interleaved,
                           n_new, positions, seq_lens, B, T, H_q, H_kv, d, k_pool, v_pool, q_out,
                           stream);
}

int gqa_attn_decode_diff_default_splits(int B, int T_q, int H, int H_kv, int S_max, int d) {
  if (B < 1 || T_q < 1 || H < 1 || H_kv < 1 || H % H_kv != 0) return 1;
  const int rows = (int)std::min<long long>((long long)T_q * (2LL * H / H_kv), 1 << 20);
  if (multi_uses_tc(T_q, (int)std::min(2LL * H / H_kv, 1LL << 20), d)) {
    // Cut by the lengths: room for twice as many pieces of a sequence as they have on average.
    const int pieces = length_pieces(B, H_kv, rows, S_max);
    if (pieces > 0) return 2 * ((pieces + B - 1) / B);
    // One CTA on an SM: no more than fill them once (4 sequences of 8K, 8 KV heads, 32 rows:
    // 45 us in five splits, 26 in four), from 16 on a multiple of eight (32 rows, 8 KV heads,
    // in 16 splits / 19: 8K tokens 10.9 / 11.8 us, 32K 23.7 / 24.1), and of four tiles or more
    // no more than one for each (64 rows, 900 tokens in 8 / 4: 9.0 / 10.0; 200 in 2 / 1: 9.5 / 8.8).
    const long long sms = num_sms_current_device();
    long long fill = sms / ((long long)B * H_kv);
    if (fill >= 16) fill -= fill % 8;
    const long long tiles = ((long long)S_max + 127) / 128;
    long long n = std::min(fill, tiles < 4 ? (tiles + 1) / 2 : tiles);
    // Several sequences that are not cut, there being too many: splits of up to 8192 tokens, but
    // no more than eight CTAs to an SM, or one CTA walks through the longest sequence after
    // the others are done (32 rows, 8 KV heads, in one split / so: 10 sequences of 1K to 64K 595
    // / 222 us, 16 592 / 390, 24 649 / 527; 10 of 1K to 16K 152 / 81, 16 152 / 94; 20 of 1K to 32K, 4
    // heads, 299 / 140).  It costs equally long ones that fill one wave (10 of 16K 153 / 167, 16
    // 155 / 171; 24, more than a wave, 325 / 259), and short ones behind a wide table, whose
    // splits are empty (0.5K to 1K of 64K: 10 sequences 15.5 / 22.7, 24 29.7 / 36.5).
    if (B > 1)
      n = std::max(n, std::min(((long long)S_max + 8191) / 8192, 8 * sms / ((long long)B * H_kv)));
    return (int)std::max(1LL, n);
  }
  // Up to 1024 tokens one launch, which is a cluster of CTAs where the grid leaves room, and up
  // to 2048 if it leaves room for eight CTAs (8 KV heads of 128, 2K tokens: 6.6 us, 5.6 in 16
  // splits, but a second launch takes the host 2.5 us).  More than 32 rows are no clusters:
  // up to 384 (900 tokens, 8 heads of 64, 64 rows: 12.0 us, 6.6 in eight splits).
  const long long sms = num_sms_current_device();
  const long long groups =
      std::min((long long)B * H_kv, 1LL << 40) * (rows <= 16 ? 1 : (rows + 31) / 32);
  const int pieces = diff_pieces(B, H_kv, rows, S_max);
  if (pieces > 0 && S_max > 1024) return 2 * ((pieces + B - 1) / B);
  if (S_max <= (rows > 32 ? 384 : 1024) || (S_max <= 2048 && rows <= 32 && groups * 8 <= sms))
    return 1;
  // One sequence: a CTA to an SM, or somewhat fewer, a multiple of eight (8 KV heads of 128 in 16
  // splits / 19: 4K tokens 6.2 us / 6.8, 8K 8.3 / 9.4, 32K 22.5-23.1 / 23.1-23.4; 4 of 64 in
  // 32 / 38: 4K 4.3 / 5.4, 32K 9.4 / 10.3, 64K 16.0 / 15.9).  Small heads do not fill HBM with
  // a CTA to an SM: two, unless that takes more than 32 splits, which the merge folds in two
  // rounds (8 heads in 16 / 32: of 64, 8K 6.6 / 5.9, 64K 28.9 / 22.2; of 32, 64K 24.1 /
  // 16.9).  Several: two (one and a half of more than 16 rows of 64, which have an
  // SM to themselves; three of up to 16 of d = 32), since sequences are seldom equally long
  // and two fill it better: 2 x 4K-30K tokens, 8 KV heads of 128, 35 us in 9 splits, 28 in 18
  // (all of 30K 39 and 39); 8 x 8K, 4 of 64, 21.7 in four, 13.9 in eight; 32 x 0.5K-2.5K, 5 of
  // 32, 14.4 in one, 12.5 in two; 26 x 5K-9K, one of 32, 42 rows, 28.6 in two, 19.2 in five.
  // (Short ones, up to 1024 tokens of more than 32 rows: a CTA to an SM.)  Splits of 128 to
  // 8192 tokens, or as many as the call takes.
  long long n = sms / groups;
  if (B > 1 && S_max > 1024)
    n = (rows > 16 ? (d == 32 ? 4 : 3) : d == 32 && S_max >= 1536 ? 6 : 4) * sms / (2 * groups);
  else if (B == 1 && rows <= 16 && d < 128)
    n = std::max(n, std::min(32LL, 2 * sms / groups));
  if (B == 1 && n >= 16) n -= n % 8;
  n = std::min(n, ((long long)S_max + 127) / 128);
  n = std::max({1LL, n, ((long long)S_max + 8191) / 8192});
  return (int)std::min<long long>(n, kMaxDiffSplits);
}

gqa_status gqa_attn_decode_diff(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* seq_lens, const float* lam, int64_t lam_stride_b,
                                int64_t lam_stride_t, int64_t lam_stride_h, int B, int T_q,
                                int S_max, int H, int H_kv, int d, int split_keys, float scale,
                                const float* norm_weight, float norm_eps, float out_scale,
                                int n_split, void* workspace, void* out, float* lse,
                                gqa_stream_t stream) {
  gqa::DiffParams diff;
  const gqa_status st = diff_params(lam, lam_stride_b, lam_stride_t, lam_stride_h, H, H_kv,
                                    split_keys, norm_weight, norm_eps, out_scale, &diff);
  if (st != GQA_OK) return st;
  return run_decode_diff(q, k_cache, v_cache, nullptr, seq_lens, diff, B, T_q, S_max,
                         (long long)B * S_max, 0, 0, 0, H, H_kv, d, scale, n_split, workspace, out,
                         lse, stream);
}

gqa_status gqa_attn_decode_paged_diff(const void* q, const void* k_pool, const void* v_pool,
                                      const int32_t* block_table, const int32_t* seq_lens,
                                      const float* lam, int64_t lam_stride_b, int64_t lam_stride_t,
                                      int64_t lam_stride_h, int B, int T_q, int num_pages,
                                      int page_size, int max_blocks, int H, int H_kv, int d,
                                      int split_keys, float scale, const float* norm_weight,
                                      float norm_eps, float out_scale, int n_split,
                                      void* workspace, void* out, float* lse,
                                      gqa_stream_t stream) {
  gqa::DiffParams diff;
  gqa_status st = diff_params(lam, lam_stride_b, lam_stride_t, lam_stride_h, H, H_kv, split_keys,
                              norm_weight, norm_eps, out_scale, &diff);
  if (st != GQA_OK) return st;
  int S_max = 0;
  long long rows = 0;
  st = paged_shape(block_table, num_pages, page_size, max_blocks, &S_max, &rows);
  if (st != GQA_OK) return st;
  return run_decode_diff(q, k_pool, v_pool, block_table, seq_lens, diff, B, T_q, S_max, rows,
                         num_pages, page_size, max_blocks, H, H_kv, d, scale, n_split, workspace,
                         out, lse, stream);
}

}  // extern "C"

namespace {

// E4M3 cache maps: codes viewed as [rows][H_kv][d] bytes (boxes of box_rows rows
// of one head, swizzled over d bytes) and the per-token scales as [outer][inner] fp32.
gqa_status prepare_fp8_maps(const void* k8, const void* v8, const float* k_scale,
                            const float* v_scale, long long rows, int box_rows, int H_kv, int d,
                            int sc_inner, int sc_outer, CUtensorMap* tm_k, CUtensorMap* tm_v,
                            CUtensorMap* tm_ks, CUtensorMap* tm_vs) {
  if (!k8 || !v8 || !k_scale || !v_scale) return GQA_ERR_INVALID_ARG;
  if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return GQA_ERR_INVALID_ARG;
  if ((sc_inner * 4) % 16 != 0) return GQA_ERR_UNSUPPORTED;
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)H_kv, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)d, (uint64_t)H_kv * d};
  const uint32_t box[3] = {(uint32_t)d, 1u, (uint32_t)box_rows};
  // rows of d bytes, swizzled over all of them (the kernel reads 4-byte pieces
  // of eight different rows per instruction without bank conflicts)
  const CUtensorMapSwizzle swz = d == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                 : d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_32B;
  gqa_status st;
  if ((st = encode_map(tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, k8, 3, dims, strides, box, swz)) !=
      GQA_OK)
    return st;
  if ((st = encode_map(tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, v8, 3, dims, strides, box, swz)) !=
      GQA_OK)
    return st;
  const uint64_t sdims[2] = {(uint64_t)sc_inner, (uint64_t)sc_outer};
  const uint64_t sstr[1] = {(uint64_t)sc_inner * 4};
  const uint32_t sbox[2] = {(uint32_t)box_rows, 1u};
  if ((st = encode_map(tm_ks, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, k_scale, 2, sdims, sstr, sbox,
                       CU_TENSOR_MAP_SWIZZLE_NONE)) != GQA_OK)
    return st;
  return encode_map(tm_vs, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, v_scale, 2, sdims, sstr, sbox,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

extern "C" {

gqa_status gqa_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale,
                               const int32_t* seq_lens, int B, int S_max, int H_q, int H_kv,
                               int d, float scale, int n_split, void* workspace, void* out,
                               float* lse, gqa_stream_t stream) {
  CUtensorMap tm_k, tm_v, tm_ks, tm_vs;
  gqa::DecodeParams p;
  // the bf16 maps encoded here are replaced below; this runs the shared checks
  gqa_status st = prepare_decode(q, k_cache, v_cache, seq_lens, B, S_max, (long long)B * S_max,
                                 gqa::kDecodeTile, H_q, H_kv, d, scale, n_split, workspace, out,
                                 lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  if ((st = prepare_fp8_maps(k_cache, v_cache, k_scale, v_scale, (long long)B * S_max,
                             gqa::kDecodeTile, H_kv, d, S_max, B, &tm_k, &tm_v, &tm_ks,
                             &tm_vs)) != GQA_OK)
    return st;
  return cuda_status(
      gqa::launch_decode_fp8(p, tm_k, tm_v, tm_ks, tm_vs, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status gqa_attn_decode_paged_fp8(const void* q, const void* k_pool, const void* v_pool,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* block_table, const int32_t* seq_lens, int B,
                                     int num_pages, int page_size, int max_blocks, int H_q,
                                     int H_kv, int d, float scale, int n_split, void* workspace,
                                     void* out, float* lse, gqa_stream_t stream) {
  if (!block_table || !aligned(block_table, 4)) return GQA_ERR_INVALID_ARG;
  if (num_pages < 1 || max_blocks < 1 || page_size < 1) return GQA_ERR_INVALID_ARG;
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return GQA_ERR_UNSUPPORTED;
  const long long S_max = (long long)max_blocks * page_size;
  const long long rows = (long long)num_pages * page_size;
  if (S_max > 0x7fffffffLL || rows > 0x7ffffffeLL) return GQA_ERR_INVALID_ARG;
  if (n_split >= 1) {
    const int chunk = gqa_attn_decode_split_chunk((int)S_max, n_split);
    if (chunk / page_size + 2 > gqa::kMaxPagesPerCta) return GQA_ERR_UNSUPPORTED;
  }
  const int h = page_size < gqa::kDecodeTile ? page_size : gqa::kDecodeTile;
  CUtensorMap tm_k, tm_v, tm_ks, tm_vs;
  gqa::DecodeParams p;
  gqa_status st = prepare_decode(q, k_pool, v_pool, seq_lens, B, (int)S_max, rows, h, H_q, H_kv,
                                 d, scale, n_split, workspace, out, lse, &tm_k, &tm_v, &p);
  if (st != GQA_OK) return st;
  if ((st = prepare_fp8_maps(k_pool, v_pool, k_scale, v_scale, rows, h, H_kv, d, page_size,
                             num_pages, &tm_k, &tm_v, &tm_ks, &tm_vs)) != GQA_OK)
    return st;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  return cuda_status(
      gqa::launch_decode_fp8(p, tm_k, tm_v, tm_ks, tm_vs, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Token rows of a block-scaled cache: row and key indices, also those that a kernel
// works out up to 2^15 keys past the end before it compares them, stay within 32 bits.
constexpr long long kMaxBlockRows = 0x7fff0000LL;

// The layout of a block-scaled E4M3 cache: checks what the calls on it share and
// fills the units of the parameter block (a unit is a sequence of a contiguous
// cache, block_table null, or a page of a pool).
gqa_status kv_block_layout(const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* block_table,
                           const int32_t* seq_lens, int B, int S_max, bool paged, int num_pages,
                           int page_size, int max_blocks, int H_kv, int d, int block,
                           gqa::KvBlockParams* p) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !seq_lens) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || H_kv < 1 || H_kv > 32767) return GQA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(seq_lens, 4))
    return GQA_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return GQA_ERR_UNSUPPORTED;
  if (block != 16 && block != 32 && block != 64 && block != 128) return GQA_ERR_UNSUPPORTED;
  *p = gqa::KvBlockParams{};
  if (paged) {
    if (!block_table || !aligned(block_table, 4)) return GQA_ERR_INVALID_ARG;
    if (num_pages < 1 || max_blocks < 1 || page_size < 1) return GQA_ERR_INVALID_ARG;
    if (page_size < 16 || (page_size & (page_size - 1)) != 0) return GQA_ERR_UNSUPPORTED;
    if (block > page_size) return GQA_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > kMaxBlockRows ||
        (long long)num_pages * page_size > kMaxBlockRows)
      return GQA_ERR_INVALID_ARG;
    S_max = max_blocks * page_size;
    p->units = num_pages;
    p->per = page_size;
    p->block_table = block_table;
    p->max_blocks = max_blocks;
    p->page_size = page_size;
    p->num_pages = num_pages;
  } else {
    if (S_max < 1 || (long long)B * S_max > kMaxBlockRows) return GQA_ERR_INVALID_ARG;
    p->units = B;
    p->per = S_max;
  }
  p->per_blk = p->per / block + (p->per % block != 0);
  while ((1 << p->block_log2) < block) ++p->block_log2;
  while (paged && (1 << p->page_log2) < page_size) ++p->page_log2;
  p->B = B;
  p->S_max = S_max;
  p->H_kv = H_kv;
  p->d = d;
  p->block = block;
  p->seq_lens = seq_lens;
  p->k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  p->v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  p->k_scale = const_cast<float*>(k_scale);
  p->v_scale = const_cast<float*>(v_scale);
  return GQA_OK;
}

gqa_status run_kv_append(gqa::KvBlockParams* p, const void* k_new, const void* v_new,
                         long long new_stride, const int32_t* n_new, int T, gqa_stream_t stream) {
  if (!k_new || !v_new || T < 1) return GQA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || (n_new && !aligned(n_new, 4)))
    return GQA_ERR_INVALID_ARG;
  if (new_stride < (long long)p->H_kv * p->d || new_stride % 8 != 0) return GQA_ERR_INVALID_ARG;
  p->k_new = static_cast<const __nv_bfloat16*>(k_new);
  p->v_new = static_cast<const __nv_bfloat16*>(v_new);
  p->new_stride = new_stride;
  p->n_new = n_new;
  p->T = T;
  const gqa_status st = error_word(&p->err);
  if (st != GQA_OK) return st;
  return cuda_status(gqa::launch_kv_append(*p, reinterpret_cast<cudaStream_t>(stream)));
}

gqa_status run_kv_read(gqa::KvBlockParams* p, int start, int S_out, void* k_out, void* v_out,
                       gqa_stream_t stream) {
  if (!k_out || !v_out || start < 0 || S_out < 1) return GQA_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return GQA_ERR_INVALID_ARG;
  if ((long long)start + S_out > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
  p->start = start;
  p->S_out = S_out;
  p->k_out = static_cast<__nv_bfloat16*>(k_out);
  p->v_out = static_cast<__nv_bfloat16*>(v_out);
  const gqa_status st = error_word(&p->err);
  if (st != GQA_OK) return st;
  return cuda_status(gqa::launch_kv_read(*p, reinterpret_cast<cudaStream_t>(stream)));
}

// Pieces of a batch that the kernel cuts by its lengths, for each of `groups` groups of heads
// that a CTA takes, with `rows` query rows together; 0: splits are even ones of S_max.  For
// more than 16 rows, which are bound by the softmax, so that an SM without work is lost
// (fewer are bound by HBM, and ragged batches within 10% either way), where that leaves at
// least two pieces a sequence and pieces of 16 tiles on average.  64 rows, 8 sequences, 8 KV
// heads: 100 to 10K tokens 64.7 us in even splits, 47.9 cut by the lengths; 100 to 33K 165
// and 112; all of 10K 65.8 and 69.1, since the cut takes time before the first load.  32
// rows: 37.6 and 28.6, all of 10K 39.0 and 42.2; 32 rows of four packed heads of d = 32 (32
// sequences of 100 to 19K) 50.5 and 46.5, all of 16K 62.6 and 56.9.  One sequence, and few
// pieces each (64 rows, 16 sequences: 104 and 104 us, all of 10K 104 and 120), are split
// evenly.
int length_pieces(int B, long long groups, int rows, int S_max) {
  const long long sms = num_sms_current_device(), pieces = sms / groups;
  const long long tiles = ((long long)S_max + 127) / 128;
  return rows > 16 && B > 1 && B <= 96 && pieces >= 2LL * B && tiles * B * groups >= 16 * sms ? (int)pieces : 0;
}

gqa_status run_decode_fp8_block(const gqa::KvBlockParams& c, const void* q, int T_q, int H_q,
                                float scale, int n_split, void* workspace, void* out, float* lse,
                                gqa_stream_t stream) {
  if (!q || !out || !lse || H_q < 1 || n_split < 1) return GQA_ERR_INVALID_ARG;
  if (H_q % c.H_kv != 0 || H_q > 65535) return GQA_ERR_INVALID_ARG;
  if (T_q < 1 || T_q > 64 || T_q > c.S_max) return GQA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return GQA_ERR_INVALID_ARG;
  if ((long long)c.B * T_q > 65535) return GQA_ERR_INVALID_ARG;
  const int G = H_q / c.H_kv;
  if (G > 16 || T_q * G > kMaxMultiRows) return GQA_ERR_UNSUPPORTED;
  if (n_split > 1 && !workspace) return GQA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      (workspace && !aligned(workspace, 256)))
    return GQA_ERR_INVALID_ARG;
  // Codes as [rows][H_kv][d] bytes, boxes of up to 128 rows, always 128 bytes wide: one
  // head, and TMA fills the rest of each row with zeros.  A tile's cost is nearly
  // the same for every d, so for d = 32 a CTA takes the four heads that share 128
  // bytes of a row, where their query rows fit and the heads by themselves are more
  // CTAs than two on each SM: 4K tokens, 8 KV heads of 8 rows, batch 64, 33.8 instead of
  // 44.7 us (of 16 rows 50 instead of 76); a smaller grid is better kept as it is
  // (batch 32 22.4 us, packed 32.5; of 16 rows 38.9 and 49.9).  Groups that are not full
  // lose (2 heads 44.6 us, packed 63.6), and so do the pairs of d = 64 (48.7, packed
  // 50.9; ragged lengths 34.8 and 38.1).
  const int head_rows = (T_q * G + 7) / 8 * 8;
  const long long head_ctas = (long long)n_split * c.H_kv * c.B;
  const bool packed = c.d == 32 && c.H_kv % 4 == 0 && 4 * head_rows <= 64 &&
                      head_ctas > 2LL * num_sms_current_device();
  const long long rows = (long long)c.units * c.per;
  const int box_rows = c.block_table && c.page_size < 128 ? c.page_size : 128;
  const uint64_t width = (uint64_t)c.H_kv * c.d;
  const uint64_t dims[3] = {packed ? width : (uint64_t)c.d, packed ? 1u : (uint64_t)c.H_kv,
                            (uint64_t)rows};
  const uint64_t strides[2] = {packed ? width : (uint64_t)c.d, width};
  const uint32_t box[3] = {128u, 1u, (uint32_t)box_rows};
  CUtensorMap tm_k, tm_v;
  unsigned* err = nullptr;
  gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;
  if ((st = encode_map(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.k_cache, 3, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B)) != GQA_OK)
    return st;
  if ((st = encode_map(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.v_cache, 3, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B)) != GQA_OK)
    return st;
  gqa::DecodeBlockParams p{};
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.block_log2 = c.block_log2;
  p.page_log2 = c.page_log2;
  p.per_blk = c.per_blk;
  p.heads = packed ? 4 : 1;
  p.head_rows = head_rows;
  p.pieces = n_split == 1 ? 0
                          : length_pieces(c.B, c.H_kv / p.heads, packed ? 4 * head_rows : T_q * G,
                                          c.S_max);
  gqa::DecodeParams& dp = p.dec;
  dp.q = static_cast<const __nv_bfloat16*>(q);
  dp.seq_lens = c.seq_lens;
  dp.B = c.B;
  dp.S_max = c.S_max;
  dp.H_q = H_q;
  dp.H_kv = c.H_kv;
  dp.G = G;
  dp.d = c.d;
  dp.T_q = T_q;
  dp.n_rg = 1;
  dp.n_split = n_split;
  const long long per = ((long long)c.S_max + n_split - 1) / n_split;
  dp.chunk = (int)((per + 127) / 128 * 128);  // (S_max is below 2^31 - 2^15)
  dp.scale_log2 = scale * 1.4426950408889634f;
  dp.ws_ml = static_cast<float2*>(workspace);
  dp.ws_O = workspace ? reinterpret_cast<float*>(
                            static_cast<char*>(workspace) +
                            gqa::decode_ws_O_offset(c.B * T_q, H_q, n_split))
                      : nullptr;
  dp.out = static_cast<__nv_bfloat16*>(out);
  dp.lse = lse;
  dp.err = err;
  dp.wait_ns = g_wait_ns.load();
  dp.block_table = c.block_table;
  dp.max_blocks = c.max_blocks;
  dp.page_size = c.page_size;
  dp.num_pages = c.num_pages;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = cuda_status(gqa::launch_decode_fp8_block(p, tm_k, tm_v, num_sms_current_device(), s));
  if (st != GQA_OK || n_split == 1) return st;
  gqa::CombineParams m;
  m.ws_ml = dp.ws_ml;
  m.ws_O = dp.ws_O;
  m.B = c.B * T_q;
  m.H_q = H_q;
  m.d = c.d;
  m.n_split = n_split;
  m.out = dp.out;
  m.lse = lse;
  m.err = err;
  return cuda_status(gqa::launch_decode_combine(m, s));
}

}  // namespace

extern "C" {

gqa_status gqa_kv_append_fp8_block(const void* k_new, const void* v_new, int64_t new_stride,
                                   const int32_t* n_new, const int32_t* seq_lens, int B, int T,
                                   int S_max, int H_kv, int d, int block, void* k_cache,
                                   void* v_cache, float* k_scale, float* v_scale,
                                   gqa_stream_t stream) {
  gqa::KvBlockParams p;
  const gqa_status st = kv_block_layout(k_cache, v_cache, k_scale, v_scale, nullptr, seq_lens, B,
                                        S_max, false, 0, 0, 0, H_kv, d, block, &p);
  if (st != GQA_OK) return st;
  return run_kv_append(&p, k_new, v_new, new_stride, n_new, T, stream);
}

gqa_status gqa_kv_append_paged_fp8_block(const void* k_new, const void* v_new, int64_t new_stride,
                                         const int32_t* n_new, const int32_t* block_table,
                                         const int32_t* seq_lens, int B, int T, int num_pages,
                                         int page_size, int max_blocks, int H_kv, int d, int block,
                                         void* k_pool, void* v_pool, float* k_scale,
                                         float* v_scale, gqa_stream_t stream) {
  gqa::KvBlockParams p;
  const gqa_status st = kv_block_layout(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, B,
                                        0, true, num_pages, page_size, max_blocks, H_kv, d, block,
                                        &p);
  if (st != GQA_OK) return st;
  return run_kv_append(&p, k_new, v_new, new_stride, n_new, T, stream);
}

gqa_status gqa_kv_read_fp8_block(const void* k_cache, const void* v_cache, const float* k_scale,
                                 const float* v_scale, const int32_t* seq_lens, int B, int S_max,
                                 int H_kv, int d, int block, int start, int S_out, void* k_out,
                                 void* v_out, gqa_stream_t stream) {
  gqa::KvBlockParams p;
  const gqa_status st = kv_block_layout(k_cache, v_cache, k_scale, v_scale, nullptr, seq_lens, B,
                                        S_max, false, 0, 0, 0, H_kv, d, block, &p);
  if (st != GQA_OK) return st;
  return run_kv_read(&p, start, S_out, k_out, v_out, stream);
}

gqa_status gqa_kv_read_paged_fp8_block(const void* k_pool, const void* v_pool,
                                       const float* k_scale, const float* v_scale,
                                       const int32_t* block_table, const int32_t* seq_lens, int B,
                                       int num_pages, int page_size, int max_blocks, int H_kv,
                                       int d, int block, int start, int S_out, void* k_out,
                                       void* v_out, gqa_stream_t stream) {
  gqa::KvBlockParams p;
  const gqa_status st = kv_block_layout(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, B,
                                        0, true, num_pages, page_size, max_blocks, H_kv, d, block,
                                        &p);
  if (st != GQA_OK) return st;
  return run_kv_read(&p, start, S_out, k_out, v_out, stream);
}

gqa_status gqa_attn_decode_fp8_block(const void* q, const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* seq_lens, int B, int T_q, int S_max, int H_q,
                                     int H_kv, int d, int block, float scale, int n_split,
                                     void* workspace, void* out, float* lse,
                                     gqa_stream_t stream) {
  gqa::KvBlockParams c;
  const gqa_status st = kv_block_layout(k_cache, v_cache, k_scale, v_scale, nullptr, seq_lens, B,
                                        S_max, false, 0, 0, 0, H_kv, d, block, &c);
  if (st != GQA_OK) return st;
  return run_decode_fp8_block(c, q, T_q, H_q, scale, n_split, workspace, out, lse, stream);
}

gqa_status gqa_attn_decode_paged_fp8_block(const void* q, const void* k_pool, const void* v_pool,
                                           const float* k_scale, const float* v_scale,
                                           const int32_t* block_table, const int32_t* seq_lens,
                                           int B, int T_q, int num_pages, int page_size,
                                           int max_blocks, int H_q, int H_kv, int d, int block,
                                           float scale, int n_split, void* workspace, void* out,
                                           float* lse, gqa_stream_t stream) {
  gqa::KvBlockParams c;
  const gqa_status st = kv_block_layout(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, B,
                                        0, true, num_pages, page_size, max_blocks, H_kv, d, block,
                                        &c);
  if (st != GQA_OK) return st;
  return run_decode_fp8_block(c, q, T_q, H_q, scale, n_split, workspace, out, lse, stream);
}

int gqa_attn_decode_fp8_block_default_splits(int B, int T_q, int H_q, int H_kv, int S_max) {
  if (B < 1 || T_q < 1 || H_q < 1 || H_kv < 1 || S_max < 1 || H_q % H_kv != 0) return 1;
  const long long groups = (long long)B * H_kv;
  const int rows = (int)std::min<long long>((long long)T_q * (H_q / H_kv), 1 << 20);
  long long n = num_sms_current_device() / groups;
  // Cut by the lengths: room for twice as many pieces of a sequence as they have on average.
  const int pieces = length_pieces(B, H_kv, rows, S_max);
  if (pieces > 0) return 2 * ((pieces + B - 1) / B);
  // Up to 1024 tokens one launch, as gqa_attn_decode_default_splits, but for more than 32
  // rows: a tile of theirs takes 1.8 us, the merge 2.5 (512 tokens, 64 rows: 13.0 us in
  // one split, 11.1 in four).
  const long long tiles = ((long long)S_max + 127) / 128;
  if (S_max <= 1024) return rows > 32 && n >= 4 && tiles >= 4 ? (int)std::min(n, tiles) : 1;
  // Up to 16 query rows a split streams at the HBM rate, and from eight on a multiple
  // of four splits measured best (Llama3-70B heads, 16 against 19 splits: 7.2 / 8.1 us at
  // 4K, 10.1 / 10.4 at 16K; two sequences, 8 against 9: 8.1 / 8.6); more rows are bound
  // by the softmax and want every SM (8 tokens at 32K, 16 / 19: 40.3 / 37.6 us).
  if (rows <= 16 && n >= 8) n -= n % 4;
  n = std::max(1LL, std::min(n, (tiles + 1) / 2));  // at least two tiles each
  // Grids that fill the GPU without splits are split all the same where sequences are
  // long, since several are seldom equally long (8 x 100 to 10K: 24.6 us in three splits,
  // 22.4 in four; 8 x 10K 31.5 and 32.3).  With more than 8 rows an SM holds one CTA
  // instead of two, and what a second wave of them costs weighs more (16 x 16K, 32 rows: 87
  // us in one split, 106 in two), so they are split later.  Of the counts from there on,
  // the one whose last wave leaves the fewest SMs idle is taken (64 rows, 24 x 24K, 4 KV heads:
  // 178 us in three splits, 220 in one, 240 in two).
  const int longest = rows > 8 ? 32768 : B > 1 && S_max > 8192 ? 4096 : 8192;
  const long long fill = ((long long)S_max + longest - 1) / longest;
  const long long least = std::max(n, fill);
  long long last = fill > n ? fill + fill / 2 : n;
  if (rows > 8) last = std::max(last, std::min(3LL, tiles / 20));
  const long long sms = num_sms_current_device();
  double best = 0;
  for (long long c = least; c <= last; ++c) {
    const long long ctas = c * groups, wave = rows > 8 || ctas <= sms ? sms : 2 * sms;
    const double used = (double)ctas / (double)((ctas + wave - 1) / wave * wave);
    if (used > best + 0.01) {
      best = used;
      n = c;
    }
  }
  return (int)n;
}

gqa_status gqa_attn_decode_combine(const void* workspace, int B, int H_q, int d, int n_split,
                                   void* out, float* lse, gqa_stream_t stream) {
  if (!workspace || !out || !lse) return GQA_ERR_INVALID_ARG;
  if (B < 1 || H_q < 1 || n_split < 1 || B > 65535 || H_q > 65535) return GQA_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return GQA_ERR_UNSUPPORTED;
  if (!aligned(workspace, 256) || !aligned(out, 16) || !aligned(lse, 4)) return GQA_ERR_INVALID_ARG;
  unsigned* err = nullptr;
  const gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;
  gqa::CombineParams p;
  p.ws_ml = static_cast<const float2*>(workspace);
  p.ws_O = reinterpret_cast<const float*>(static_cast<const char*>(workspace) +
                                          gqa::decode_ws_O_offset(B, H_q, n_split));
  p.B = B;
  p.H_q = H_q;
  p.d = d;
  p.n_split = n_split;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = err;
  return cuda_status(gqa::launch_decode_combine(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Shared checks and launch of the causal prefill kernel: S query rows per
// sequence against S_kv key rows (chunk: the queries end each sequence).  With `diff`, H_q
// counts the maps of differential attention, two per head.
gqa_status run_prefill(bool chunk, const void* q, const void* k, const void* v,
                       const int32_t* seq_lens, int B, int S, int S_kv, int H_q, int H_kv, int d,
                       float scale, int window, int n_part, void* workspace, void* out, float* lse,
                       gqa_stream_t stream, const gqa::DiffParams* diff = nullptr) {
  if (!q || !k || !v || !out || !lse) return GQA_ERR_INVALID_ARG;
  if (n_part < 1 || n_part > 8 || (n_part > 1 && (!chunk || !workspace))) return GQA_ERR_INVALID_ARG;
  if (workspace && !aligned(workspace, 256)) return GQA_ERR_INVALID_ARG;
  if (B < 1 || S < 1 || S_kv < S || H_q < 1 || H_kv < 1 || H_q % H_kv != 0)
    return GQA_ERR_INVALID_ARG;
  if (B > 65535 || H_q > 65535 || !std::isfinite(scale) || !(scale > 0.f))
    return GQA_ERR_INVALID_ARG;
  if ((long long)B * S * H_q > 0x7fffffffLL || (long long)B * S_kv > 0x7fffffffLL)
    return GQA_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return GQA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || (seq_lens && !aligned(seq_lens, 4)))
    return GQA_ERR_INVALID_ARG;
  unsigned* err = nullptr;
  gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;

  // Q viewed as [B][S][H_q][d] with boxes of 128 rows of one head, 64 elements
  // wide (two boxes per 128-wide row), 128-byte swizzle; K and V likewise.  For
  // d = 32 the 64-element box is wider than the tensor: TMA fills elements
  // 32..63 with zeros, the padding the kernel's 64-wide tiles expect.
  const uint64_t rows_q = diff && diff->split_keys ? H_q / 2 : H_q;
  const uint64_t dq[4] = {(uint64_t)d, rows_q, (uint64_t)S, (uint64_t)B};
  const uint64_t sq[3] = {(uint64_t)d * 2, rows_q * d * 2, (uint64_t)S * rows_q * d * 2};
  const uint64_t dk[4] = {(uint64_t)d, (uint64_t)H_kv, (uint64_t)S_kv, (uint64_t)B};
  const uint64_t sk[3] = {(uint64_t)d * 2, (uint64_t)H_kv * d * 2, (uint64_t)S_kv * H_kv * d * 2};
  const uint32_t box[4] = {64u, 1u, 128u, 1u};
  CUtensorMap tm_q, tm_k, tm_v;
  if ((st = encode_bf16(&tm_q, q, 4, dq, sq, box, CU_TENSOR_MAP_SWIZZLE_128B)) != GQA_OK) return st;
  if ((st = encode_bf16(&tm_k, k, 4, dk, sk, box, CU_TENSOR_MAP_SWIZZLE_128B)) != GQA_OK) return st;
  if ((st = encode_bf16(&tm_v, v, 4, dk, sk, box, CU_TENSOR_MAP_SWIZZLE_128B)) != GQA_OK) return st;

  gqa::PrefillParams p;
  p.B = B;
  p.S = S;
  p.S_kv = S_kv;
  p.seq_lens = seq_lens;
  p.window = window < 0 ? -1 : window;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.G = H_q / H_kv;
  p.d = d;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = err;
  p.wait_ns = g_wait_ns.load();
  p.n_part = n_part;
  p.ws_ml = n_part > 1 ? static_cast<float2*>(workspace) : nullptr;
  p.ws_O = n_part > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                                 gqa::prefill_ws_O_offset((size_t)B * S * H_q, n_part))
                      : nullptr;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = num_sms_current_device();
  if (diff) {
    const gqa::PrefillDiffParams pd{p, *diff};
    st = cuda_status(gqa::launch_prefill_diff(pd, chunk, tm_q, tm_k, tm_v, sms, s));
    if (st != GQA_OK || n_part == 1) return st;
    gqa::DiffMergeParams m{};
    m.diff = *diff;
    m.ws_ml = p.ws_ml;
    m.ws_O = p.ws_O;
    m.m_log2 = 1.f;
    m.B = B;
    m.T = S;
    m.H_maps = H_q;
    m.d = d;
    m.n_part = n_part;
    m.out = p.out;
    m.lse = lse;
    m.lse_b = (long long)H_q * S;
    m.lse_t = 1;
    m.lse_m = S;
    m.err = err;
    return cuda_status(gqa::launch_diff_merge(m, s));
  }
  if (!chunk) return cuda_status(gqa::launch_prefill_causal(p, tm_q, tm_k, tm_v, sms, s));
  st = cuda_status(gqa::launch_prefill_chunk(p, tm_q, tm_k, tm_v, sms, s));
  if (st != GQA_OK || n_part == 1) return st;
  return cuda_status(gqa::launch_prefill_merge(p, s));
}

}  // namespace

extern "C" {

gqa_status gqa_attn_prefill_causal(const void* q, const void* k, const void* v, int B, int S,
                                   int H_q, int H_kv, int d, float scale, void* out, float* lse,
                                   gqa_stream_t stream) {
  return run_prefill(false, q, k, v, nullptr, B, S, S, H_q, H_kv, d, scale, -1, 1, nullptr, out, lse,
                     stream);
}

gqa_status gqa_attn_prefill_chunk(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* seq_lens, int B, int T_q, int S_max, int H_q,
                                  int H_kv, int d, float scale, int window, void* out, float* lse,
                                  gqa_stream_t stream) {
  return run_prefill(true, q, k_cache, v_cache, seq_lens, B, T_q, S_max, H_q, H_kv, d, scale,
                     window, 1, nullptr, out, lse, stream);
}

size_t gqa_attn_prefill_chunk_workspace_bytes(int B, int T_q, int H_q, int d, int n_part) {
  if (B < 1 || T_q < 1 || H_q < 1 || d < 1 || n_part <= 1) return 0;
  const size_t rows = (size_t)B * T_q * H_q;
  return gqa::prefill_ws_O_offset(rows, n_part) + rows * n_part * d * sizeof(float);
}

int gqa_attn_prefill_chunk_default_parts(int B, int T_q, int S_max, int H_q, int H_kv) {
  if (B < 1 || T_q < 1 || S_max < T_q || H_q < 1 || H_kv < 1 || H_q % H_kv != 0) return 1;
  // Split only long items (>= 16 key tiles if the chunk ends the cache), and
  // only when it evens out the last round of the persistent grid: the part
  // count P in 1..4 maximising x / ceil(x), x = items * P / SMs, must beat
  // P = 1 by at least 5% (a split costs a partial write, read and merge).
  if (S_max / 128 < 16) return 1;
  const long long items = (long long)((T_q + 127) / 128) * B * H_kv * ((H_q / H_kv + 1) / 2);
  const int sms = num_sms_current_device();
  auto eff = [&](int P) {
    const double x = (double)items * P / sms;
    return x / std::ceil(x);
  };
  int best = 1;
  for (int P = 2; P <= 4; ++P)
    if (eff(P) > eff(best) + 1e-9) best = P;
  return eff(best) >= eff(1) + 0.05 ? best : 1;
}

gqa_status gqa_attn_prefill_chunk_split(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* seq_lens, int B, int T_q, int S_max,
                                        int H_q, int H_kv, int d, float scale, int window,
                                        int n_part, void* workspace, void* out, float* lse,
                                        gqa_stream_t stream) {
  return run_prefill(true, q, k_cache, v_cache, seq_lens, B, T_q, S_max, H_q, H_kv, d, scale,
                     window, n_part, workspace, out, lse, stream);
}

int gqa_attn_prefill_diff_default_parts(int B, int T_q, int S_max, int H, int H_kv, int window) {
  if (B < 1 || T_q < 1 || S_max < T_q || H < 1 || H > 32767 || H_kv < 1 || H % H_kv != 0) return 1;
  // Parts are for few queries over long keys, whose few work items leave SMs idle: as many as
  // fill them, of two key tiles or more, since a tile takes an item 1.4 us and the partials
  // and their merge 3 to 5.  100 queries of 32 maps of 128: 1K keys 19.2 / 15.1 us in one /
  // four parts (8 maps 19.2 / 12.5), 2K 32.8 / 18 in seven, 4K 56 / 18.9 in eight; 768
  // keys 16.1 / 14.8 in three, but 512 13.0 / 14.4 in two.  Two parts do not pay for short keys (1099
  // queries at 1.6K, 16 maps of 64: 25.5 and 25.9; 1024 at 2K, of 128, 32.0 and 30.3; a
  // prompt of 4K, 4 maps, 53 and 43), nor do more than fill the SMs (512 queries at 2K, 16
  // maps: 31.6 in one, 21.6 in four, 28.8 in six).
  const long long keys = window < 0 ? S_max : std::min<long long>(S_max, (long long)window + 128);
  const long long tiles = keys / 128;
  const long long items = std::min(((long long)T_q + 127) / 128 * B, 1LL << 40) * H;
  const long long n = std::min({8LL, num_sms_current_device() / items, tiles / 2});
  return n < 2 || tiles < (n == 2 ? 16 : 6) ? 1 : (int)n;
}

gqa_status gqa_attn_prefill_diff(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* seq_lens, const float* lam, int64_t lam_stride_b,
                                 int64_t lam_stride_t, int64_t lam_stride_h, int B, int T_q,
                                 int S_max, int H, int H_kv, int d, int split_keys, float scale,
                                 int window, const float* norm_weight, float norm_eps,
                                 float out_scale, int n_part, void* workspace, void* out,
                                 float* lse, gqa_stream_t stream) {
  gqa::DiffParams diff;
  const gqa_status st = diff_params(lam, lam_stride_b, lam_stride_t, lam_stride_h, H, H_kv,
                                    split_keys, norm_weight, norm_eps, out_scale, &diff);
  if (st != GQA_OK) return st;
  // Whole prompts, also given with lengths (all of them S_max, or bad), take the causal kernel
  // (8K tokens, 64 maps of 128: 700 us, 752 as a chunk).
  const int back = window < S_max ? window : -1;
  const bool chunk = T_q != S_max || back >= 0 || n_part > 1;
  return run_prefill(chunk, q, k_cache, v_cache, seq_lens, B, T_q, S_max, 2 * H, H_kv, d, scale,
                     back, n_part, workspace, out, lse, stream, &diff);
}

gqa_status gqa_last_device_error(gqa_stream_t stream) {
  unsigned* err = nullptr;
  gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return GQA_ERR_CUDA;
  unsigned word = 0;
  if (cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost) != cudaSuccess)
    return GQA_ERR_CUDA;
  if (word) {
    const unsigned zero = 0;
    if (cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
      return GQA_ERR_CUDA;
  }
  if (word & gqa::kErrBounds) return GQA_ERR_CUDA;  // bounds-checking builds: an internal fault
  if (word & gqa::kErrTimeout) return GQA_ERR_TIMEOUT;
  if (word & (gqa::kErrBadSeqLen | gqa::kErrBadPage)) return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

uint64_t gqa_set_wait_limit_ns(uint64_t limit_ns) {
  if (limit_ns < 1000) limit_ns = 1000;
  return g_wait_ns.exchange(limit_ns);
}

gqa_status gqa_selftest_wait_timeout(uint64_t limit_ns, gqa_stream_t stream) {
  unsigned* err = nullptr;
  gqa_status st = error_word(&err);
  if (st != GQA_OK) return st;
  if (limit_ns < 1000) limit_ns = 1000;
  return cuda_status(gqa::launch_wait_selftest(err, limit_ns, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
