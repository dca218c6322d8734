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
#include "kv_blocks.h"
#include "tcgen05.cuh"

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
// One CTA per (touched block, K or V, KV head, sequence): it alone writes that
// block's codes and scale, so nothing is atomic and the result does not depend on
// timing.  The block's new rows are held in registers between the maximum and the
// rounding, so they are read once.  Neighbouring CTAs take the heads of one block
// of tokens, whose pieces of a row lie together, in the new rows (strided by a
// fused projection's width) and in the cache.
//
// Bound by HBM for prompts (each new value read once, each code written once): 32K
// tokens of 8 heads of 128, blocks of 64, 201 MB in 33.1 us, 6.08 TB/s.  That took
// few instructions per value: rows by added strides and 32-bit comparisons, the
// product on fp32 pairs, and the two rare cases (a scale that grew over older
// codes, a present scale that is no power of two) in loops of their own; with all of it
// in one loop 84% of the issue slots were in use and the same prompt took 37.1 us (8
// prompts of 256 to 1K tokens 5.8 us, now 4.4).  Eight vectors a thread, where the
// block has them, halve a thread's share of the set-up (four: 33.9 us).  Single tokens
// are bound by a chain of latencies (length, page, new row and scale, block maximum,
// store): 1.8 us for one sequence, 3.1 for 128.
template <int D, int BLK>
struct AppendShape {
  static constexpr int kVecRow = D / 8;            // 16-byte vectors of a bf16 row
  static constexpr int kVecs = BLK * kVecRow;      // of the whole block
  static constexpr int kThreads = kVecs <= 512 ? 64 : kVecs <= 1024 ? 128 : 256;
  static constexpr int kPer = kVecs / kThreads;    // per thread: 1, 2, 4 or 8
  static constexpr int kStep = kThreads / kVecRow; // rows between a thread's vectors
  static constexpr int kCtas = (kPer <= 4 ? 1536 : 1024) / kThreads;  // of an SM
};

template <int D, int BLK, bool PAGED>
__global__ void __launch_bounds__(AppendShape<D, BLK>::kThreads, AppendShape<D, BLK>::kCtas)
    gqa_kv_append_kernel(const KvBlockParams p) {
  using Sh = AppendShape<D, BLK>;
  __shared__ uint32_t s_max[2][Sh::kThreads / 32];
  const int b = blockIdx.z;
  const int slot = blockIdx.x / (2u * p.H_kv), head = blockIdx.x - slot * 2 * p.H_kv;
  const int is_v = head >= p.H_kv, kv = head - (is_v ? p.H_kv : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = p.seq_lens[b];
  const int n = p.n_new ? p.n_new[b] : p.T;
  if (L < n || L > p.S_max || n < 0 || n > p.T) {  // (also L < 0, as n >= 0 > L then)
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.err, kErrBadSeqLen);
    return;
  }
  const int first_new = L - n;
  const int t0 = append_block_start(L, n, slot, BLK);  // the block's first token
  if (t0 < 0) return;
  // The new rows first: they do not depend on where the block lies.
  const __nv_bfloat16* const src = (is_v ? p.v_new : p.k_new) + (size_t)b * p.T * p.new_stride +
                                   (size_t)kv * D;
  const int r0 = threadIdx.x / Sh::kVecRow, c = threadIdx.x % Sh::kVecRow;
  const int i0 = t0 + r0 - first_new;  // new row of the thread's first vector (negative: an older row)
  uint4 x[Sh::kPer];
  {
    const __nv_bfloat16* px = src + (long long)i0 * p.new_stride + c * 8;
    const long long step = Sh::kStep * p.new_stride;
#pragma unroll
    for (int j = 0; j < Sh::kPer; ++j, px += step) {
      x[j] = make_uint4(0u, 0u, 0u, 0u);
      if (static_cast<unsigned>(i0 + j * Sh::kStep) < static_cast<unsigned>(n))
        x[j] = *reinterpret_cast<const uint4*>(px);
    }
  }
  int unit = b, at = t0;
  if constexpr (PAGED) {
    unit = p.block_table[(size_t)b * p.max_blocks + (t0 >> p.page_log2)];
    at = t0 & (p.page_size - 1);
    if (unit < 0 || unit >= p.num_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrBadPage);
      return;
    }
  }
  const size_t row0 = (size_t)unit * p.per + at;
  const size_t sidx = ((size_t)unit * p.per_blk + at / BLK) * p.H_kv + kv;
  uint8_t* const cache = is_v ? p.v_cache : p.k_cache;
  float* const scales = is_v ? p.v_scale : p.k_scale;
  const size_t extent = (size_t)p.units * p.per * p.H_kv * D;
  const bool has_old = t0 < first_new;
  // (read by every thread before the barrier of the maximum, written after it)
  const float s_old = has_old ? scales[sidx] : 0.f;

  auto block_max = [&](uint32_t v, int turn) -> uint32_t {  // largest of both halves over the CTA
    v = max(v & 0xffffu, v >> 16);
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) s_max[turn][warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < Sh::kThreads / 32; ++w) v = max(v, s_max[turn][w]);
    return v;
  };
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < Sh::kPer; ++j) {
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
  }
  uint32_t amax = block_max(mx, 0);
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
    amax = block_max(mx, 1);
  }
  const int e_new = scale_exp(amax);
  const float s_new = pow2f(e_new);
  // (by magnitude: a negative scale of the caller's, and a NaN one, is replaced)
  const float s = has_old && fabsf(s_old) >= s_new ? fabsf(s_old) : s_new;
  const size_t code0 = ((row0 + r0) * p.H_kv + kv) * D + c * 8;  // of the first vector
  const size_t code_step = (size_t)Sh::kStep * p.H_kv * D;
  auto store = [&](int j, const uint32_t (&q)[4]) {
    const size_t code = code0 + j * code_step;
    if (in_bounds(code, 8, extent, p.err))
      *reinterpret_cast<uint2*>(cache + code) =
          make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
  };
  if (has_old && s != s_old) {
    // The older rows, under a scale that grew (or lost its sign, or was NaN and leaves NaN
    // codes): their codes are rounded again.
    const float ratio = s_old / s;
#pragma unroll
    for (int j = 0; j < Sh::kPer; ++j) {
      if (i0 + j * Sh::kStep >= 0) continue;
      const uint2 old = *reinterpret_cast<const uint2*>(cache + code0 + j * code_step);
      const uint32_t w[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu, old.y >> 16};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3x2_to_float2(w[i]);
        q[i] = e4m3x2(f.x * ratio, f.y * ratio);
      }
      store(j, q);
    }
  }
  // x / s: a product where s is a power of two, as it is unless the caller filled
  // the scales with others.
  if (s == s_new || (__float_as_uint(s) & 0x7fffffu) == 0u) {
    const float inv = s == s_new ? pow2f(-e_new) : 1.f / s;
#pragma unroll
    for (int j = 0; j < Sh::kPer; ++j) {
      if (static_cast<unsigned>(i0 + j * Sh::kStep) >= static_cast<unsigned>(n)) continue;
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        fmul2(lo, hi, __uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u), inv, inv);
        q[i] = e4m3x2(lo, hi);
      }
      store(j, q);
    }
  } else {
#pragma unroll 1
    for (int j = 0; j < Sh::kPer; ++j) {
      if (static_cast<unsigned>(i0 + j * Sh::kStep) >= static_cast<unsigned>(n)) continue;
      uint4 v = x[0];
#pragma unroll
      for (int k = 1; k < Sh::kPer; ++k)
        if (j == k) v = x[k];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = e4m3x2(__uint_as_float(w[i] << 16) / s, __uint_as_float(w[i] & 0xffff0000u) / s);
      store(j, q);
    }
  }
  if (threadIdx.x == 0 && in_bounds(sidx, 1, (size_t)p.units * p.per_blk * p.H_kv, p.err))
    scales[sidx] = s;
}

// ------------------------------------------------------------------ read ----
// A thread turns pieces of 16 codes (a 16-byte load) into 16 bf16 values (a 32-byte
// store), kReadPer of them in flight; consecutive threads take consecutive pieces
// of a token's H_kv x D codes, which lie together in the cache and in the output.
// Bound by HBM: 32K tokens of 8 heads of 128 in pages of 64, 201 MB in 32.0 us, 6.3
// TB/s (pieces of 8 codes: 35.2 us with 78% of the issue slots in use; one piece in
// flight 33.2, four 32.0).
constexpr int kReadThreads = 256, kReadPer = 2;
constexpr int kReadChunk = kReadThreads * kReadPer;  // pieces of a CTA

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
  const uint32_t row_vecs = p.H_kv * p.d / 16;  // pieces of a token
  const int rows = bad ? p.S_out : min(p.S_out, L - p.start);  // (rows past L are left alone)
  const long long first = (long long)blockIdx.x * kReadChunk;
  const int i0 = static_cast<int>(first / row_vecs);
  if (i0 >= rows) return;
  const uint32_t w0 = static_cast<uint32_t>(first - (long long)i0 * row_vecs);
  const size_t extent = (size_t)p.B * p.S_out * p.H_kv * p.d;
  const int head_shift = p.d == 128 ? 3 : p.d == 64 ? 2 : 1;  // pieces of a head
  // piece u of this thread in the output, and in a sequence of a contiguous cache
  const size_t dst0 = ((size_t)b * p.S_out * row_vecs + first + threadIdx.x) * 16;
  const size_t src0 = (((size_t)b * p.per + p.start) * row_vecs + first + threadIdx.x) * 16;

  uint4 w[kReadPer];
  float s[kReadPer];  // (NaN for a row that cannot be read)
  bool live[kReadPer];
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    // piece w0 + threadIdx.x + u * 256 from row i0 on: its row by a multiplication
    // (exact: both factors of the quotient are below 2^11), or by a comparison
    // where a row is longer than the chunk
    const uint32_t x = w0 + threadIdx.x + u * kReadThreads;
    const uint32_t q = row_vecs > kReadChunk ? (x >= row_vecs ? 1u : 0u) : __umulhi(x, p.row_magic);
    const uint32_t piece = x - q * row_vecs;
    const int i = i0 + static_cast<int>(q);
    live[u] = i < rows;
    w[u] = make_uint4(0u, 0u, 0u, 0u);
    s[u] = NAN;
    if (!live[u] || bad) continue;
    int unit = b, at = p.start + i;
    size_t src = src0 + u * kReadThreads * 16;
    if constexpr (PAGED) {
      unit = p.block_table[(size_t)b * p.max_blocks + (at >> p.page_log2)];
      at &= p.page_size - 1;
      if (unit < 0 || unit >= p.num_pages) {
        atomicOr(p.err, kErrBadPage);
        continue;
      }
      src = (((size_t)unit * p.per + at) * row_vecs + piece) * 16;
    }
    w[u] = *reinterpret_cast<const uint4*>(cache + src);
    s[u] = scales[((size_t)unit * p.per_blk + (at >> p.block_log2)) * p.H_kv +
                  (piece >> head_shift)];
  }
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    if (!live[u]) continue;
    const uint32_t c[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = e4m3x2_to_float2(i & 1 ? c[i / 2] >> 16 : c[i / 2]);
      float lo, hi;
      fmul2(lo, hi, f.x, f.y, s[u], s[u]);
      o[i] = pack_bf16x2(lo, hi);
    }
    const size_t dst = dst0 + u * kReadThreads * 16;
    if (!in_bounds(dst, 16, extent, p.err)) continue;
    if (wide) {
      st_global_v8(out + dst, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    } else {
      *reinterpret_cast<uint4*>(out + dst) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(out + dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
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
  const long long slots = append_slots(p.T, p.S_max, BLK);
  if (slots * 2 * p.H_kv > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(slots * 2 * p.H_kv), 1, p.B);
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

cudaError_t launch_kv_read(const KvBlockParams& p_in, cudaStream_t stream) {
  KvBlockParams p = p_in;
  const int row_vecs = p.H_kv * p.d / 16;
  p.row_magic = static_cast<uint32_t>((0x100000000ull + row_vecs - 1) / row_vecs);
  const long long chunks = ((long long)p.S_out * row_vecs + kReadChunk - 1) / kReadChunk;
  if (chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(chunks), 2, p.B);
  return p.block_table ? launch_pdl(gqa_kv_read_kernel<true>, grid, kReadThreads, p, stream)
                       : launch_pdl(gqa_kv_read_kernel<false>, grid, kReadThreads, p, stream);
}

}  // namespace gqa
