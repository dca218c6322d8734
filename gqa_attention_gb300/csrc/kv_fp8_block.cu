// kv_fp8_block.cu -- the block-scaled E4M3 cache: quantising new tokens into it
// and reading it back as bf16.
//
// The cache holds E4M3 codes and one fp32 scale for every BLK consecutive
// tokens of a KV head (K and V apart).  Scales written here are powers of two:
// for a block whose largest magnitude is a = m 2^e (1 <= m < 2),
//   s = 2^(e - 8) if m <= 1.75, else 2^(e - 7):  the smallest with a / s <= 448,
// and never below 2^-100.  E4M3 is a floating-point format, so a power of two
// costs no precision against a / 448 above its subnormals, and x / s and the
// re-encoding of older codes are exact before their one rounding.
#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kMinScaleExp = -100;

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the block scale for a largest magnitude given as bf16 bits
// (sign cleared, finite): 1.75 is mantissa 96 of 128.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 127u) > 96u ? 1 : 0);
  return max(e, kMinScaleExp);
}

// Two fp32 values to two E4M3 codes (lo in the low byte): round to nearest
// even, magnitudes above 448 clamp, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ---------------------------------------------------------------- append ----
// One CTA per (touched block, KV head, K or V, sequence): it alone writes that
// block's codes and scale, so nothing is atomic and the result does not depend
// on timing.  The block's new rows are held in registers between the maximum
// and the rounding, so they are read once.
template <int D, int BLK>
struct AppendShape {
  static constexpr int kVecRow = D / 8;            // 16-byte vectors of a bf16 row
  static constexpr int kVecs = BLK * kVecRow;      // of the whole block
  static constexpr int kThreads = kVecs < 256 ? kVecs : 256;
  static constexpr int kPer = kVecs / kThreads;    // per thread
};

template <int D, int BLK, bool PAGED>
__global__ void __launch_bounds__(AppendShape<D, BLK>::kThreads)
    gqa_kv_append_kernel(const KvBlockParams p) {
  using Sh = AppendShape<D, BLK>;
  __shared__ uint32_t s_max[Sh::kThreads / 32];
  const int b = blockIdx.z, kv = blockIdx.y >> 1, is_v = blockIdx.y & 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = p.seq_lens[b];
  const int n = p.n_new ? p.n_new[b] : p.T;
  if (L < n || L > p.S_max || n < 0 || n > p.T) {  // (also L < 0, as n >= 0 > L then)
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, kErrBadSeqLen);
    return;
  }
  const int first_new = L - n;
  const int t0 = (first_new / BLK + static_cast<int>(blockIdx.x)) * BLK;  // the block's first token
  if (n == 0 || t0 >= L) return;
  int unit = b, at = t0;
  if constexpr (PAGED) {
    unit = p.block_table[(size_t)b * p.max_blocks + t0 / p.page_size];
    at = t0 % p.page_size;
    if (unit < 0 || unit >= p.num_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrBadPage);
      return;
    }
  }
  const size_t row0 = (size_t)unit * p.per + at;
  const size_t sidx = ((size_t)unit * p.per_blk + at / BLK) * p.H_kv + kv;
  uint8_t* const cache = is_v ? p.v_cache : p.k_cache;
  float* const scales = is_v ? p.v_scale : p.k_scale;
  const __nv_bfloat16* const src = (is_v ? p.v_new : p.k_new) + (size_t)b * p.T * p.new_stride +
                                   (size_t)kv * D;
  const size_t extent = (size_t)p.units * p.per * p.H_kv * D;

  uint4 x[Sh::kPer];
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < Sh::kPer; ++j) {
    const int v = threadIdx.x + j * Sh::kThreads;
    const int t = t0 + v / Sh::kVecRow, c = v % Sh::kVecRow;
    x[j] = make_uint4(0u, 0u, 0u, 0u);
    if (t >= first_new && t < L)
      x[j] = *reinterpret_cast<const uint4*>(src + (size_t)(t - first_new) * p.new_stride + c * 8);
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
  }
  const bool has_old = t0 < first_new;
  const float s_old = has_old ? scales[sidx] : 0.f;

  auto block_max = [&](uint32_t v) -> uint32_t {  // largest of both halves over the CTA
    v = max(v & 0xffffu, v >> 16);
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (Sh::kThreads > 32) {
      if (lane == 0) s_max[warp] = v;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < Sh::kThreads / 32; ++w) v = max(v, s_max[w]);
    }
    return v;
  };
  uint32_t amax = block_max(mx);
  if (amax >= 0x7f80u) {
    // An infinity or NaN among the new values (the same branch in every
    // thread): all become NaN and stay out of the maximum.
    mx = 0;
#pragma unroll
    for (int j = 0; j < Sh::kPer; ++j) {
      uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] |= 0x7fffu;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] |= 0x7fff0000u;
        const uint32_t a = w[i] & 0x7fff7fffu;
        mx = __vmaxu2(mx, ((a & 0xffffu) >= 0x7f80u ? 0u : a & 0xffffu) |
                              (a >= 0x7f800000u ? 0u : a & 0xffff0000u));
      }
      x[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();  // (s_max is read above)
    amax = block_max(mx);
  }
  const int e_new = scale_exp(amax);
  const float s_new = pow2f(e_new);
  const float s = has_old && s_old >= s_new ? s_old : s_new;
  // x / s: a product where s is the power of two just computed
  const float inv = s == s_new ? pow2f(-e_new) : 1.f / s;
  const bool exact_inv = s == s_new || (__float_as_uint(s) & 0x7fffffu) == 0u;

#pragma unroll
  for (int j = 0; j < Sh::kPer; ++j) {
    const int v = threadIdx.x + j * Sh::kThreads;
    const int t = t0 + v / Sh::kVecRow, c = v % Sh::kVecRow;
    const size_t at_code = ((row0 + v / Sh::kVecRow) * p.H_kv + kv) * D + c * 8;
    uint8_t* const dst = cache + at_code;
    if (t >= first_new && t < L) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        q[i] = exact_inv ? e4m3x2(lo * inv, hi * inv) : e4m3x2(lo / s, hi / s);
      }
      if (in_bounds(at_code, 8, extent, p.err))
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    } else if (t < first_new && s > s_old) {
      // An older row under a scale that grew: its codes are rounded again.
      const float ratio = s_old / s;
      const uint2 old = *reinterpret_cast<const uint2*>(dst);
      const uint32_t w[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu, old.y >> 16};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3x2_to_float2(w[i]);
        q[i] = e4m3x2(f.x * ratio, f.y * ratio);
      }
      if (in_bounds(at_code, 8, extent, p.err))
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    }
  }
  // (every thread's read of the old scale precedes the barrier in block_max or,
  // for a one-warp CTA, the warp reduction)
  if (threadIdx.x == 0 && in_bounds(sidx, 1, (size_t)p.units * p.per_blk * p.H_kv, p.err))
    scales[sidx] = s;
}

// ------------------------------------------------------------------ read ----
// A thread turns 16 codes (one 16-byte load) into 16 bf16 values (two 16-byte
// stores); consecutive threads take consecutive 16-code pieces of a token's
// H_kv x D codes, which lie together in the cache and in the output.
constexpr int kReadThreads = 256;

template <bool PAGED>
__global__ void __launch_bounds__(kReadThreads) gqa_kv_read_kernel(const KvBlockParams p) {
  const int b = blockIdx.z, is_v = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint8_t* const cache = is_v ? p.v_cache : p.k_cache;
  const float* const scales = is_v ? p.v_scale : p.k_scale;
  __nv_bfloat16* const out = is_v ? p.v_out : p.k_out;
  const int L = p.seq_lens[b];
  const bool bad = L < 0 || L > p.S_max;
  if (bad && blockIdx.x == 0 && is_v == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadSeqLen);
  const int row_vecs = p.H_kv * p.d / 16;  // 16-code pieces of a token
  const int head_vecs = p.d / 16;
  const int rows = bad ? p.S_out : min(p.S_out, L - p.start);  // (rows past L are left alone)
  const long long total = (long long)max(rows, 0) * row_vecs;
  const size_t extent = (size_t)p.B * p.S_out * p.H_kv * p.d;
  for (long long v = (long long)blockIdx.x * kReadThreads + threadIdx.x; v < total;
       v += (long long)gridDim.x * kReadThreads) {
    const int i = static_cast<int>(v / row_vecs), c = static_cast<int>(v - (long long)i * row_vecs);
    const int t = p.start + i;
    int unit = b, at = t;
    bool ok = !bad;
    if constexpr (PAGED) {
      if (ok) {
        unit = p.block_table[(size_t)b * p.max_blocks + t / p.page_size];
        at = t % p.page_size;
        if (unit < 0 || unit >= p.num_pages) {
          ok = false;
          atomicOr(p.err, kErrBadPage);
        }
      }
    }
    uint32_t o[8];
    if (ok) {
      const size_t code = (((size_t)unit * p.per + at) * row_vecs + c) * 16;
      const float s = scales[((size_t)unit * p.per_blk + at / p.block) * p.H_kv + c / head_vecs];
      const uint4 w4 = *reinterpret_cast<const uint4*>(cache + code);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f0 = e4m3x2_to_float2(w[k]), f1 = e4m3x2_to_float2(w[k] >> 16);
        o[2 * k] = pack_bf16x2(f0.x * s, f0.y * s);
        o[2 * k + 1] = pack_bf16x2(f1.x * s, f1.y * s);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = 0x7fc07fc0u;  // NaN
    }
    const size_t dst = (((size_t)b * p.S_out + i) * row_vecs + c) * 16;
    if (in_bounds(dst, 16, extent, p.err)) {
      uint4* d4 = reinterpret_cast<uint4*>(out + dst);
      d4[0] = make_uint4(o[0], o[1], o[2], o[3]);
      d4[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <typename K>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, const KvBlockParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int BLK>
cudaError_t launch_append(const KvBlockParams& p, cudaStream_t stream) {
  // T tokens touch at most this many blocks, wherever they start
  const long long slots = ((long long)p.T + BLK - 2) / BLK + 1;
  const dim3 grid(static_cast<unsigned>(slots), 2 * p.H_kv, p.B);
  constexpr int threads = AppendShape<D, BLK>::kThreads;
  return p.block_table ? launch_pdl(gqa_kv_append_kernel<D, BLK, true>, grid, threads, p, stream)
                       : launch_pdl(gqa_kv_append_kernel<D, BLK, false>, grid, threads, p, stream);
}

template <int D>
cudaError_t launch_append_d(const KvBlockParams& p, cudaStream_t stream) {
  switch (p.block) {
    case 16: return launch_append<D, 16>(p, stream);
    case 32: return launch_append<D, 32>(p, stream);
    case 64: return launch_append<D, 64>(p, stream);
    case 128: return launch_append<D, 128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvBlockParams& p, cudaStream_t stream) {
  switch (p.d) {
    case 32: return launch_append_d<32>(p, stream);
    case 64: return launch_append_d<64>(p, stream);
    case 128: return launch_append_d<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv_read(const KvBlockParams& p, int num_sms, cudaStream_t stream) {
  const long long vecs = (long long)p.S_out * p.H_kv * p.d / 16;
  long long x = (vecs + kReadThreads - 1) / kReadThreads;
  const long long most = 64LL * num_sms;
  const dim3 grid(static_cast<unsigned>(x < most ? x : most), 2, p.B);
  return p.block_table ? launch_pdl(gqa_kv_read_kernel<true>, grid, kReadThreads, p, stream)
                       : launch_pdl(gqa_kv_read_kernel<false>, grid, kReadThreads, p, stream);
}

}  // namespace gqa
