// kv_append.cu -- appending keys and values to a bf16 or per-token E4M3 cache, contiguous or
// paged, the keys (and the step's queries) turned by their positions on the way.
//
// The rotation of a pair (x, y) of channels with frequency f at position p:
//   (x cos a - y sin a, x sin a + y cos a),  a = p f.
// The product p f in fp32 would be off by p f 2^-24 (0.008 radians at 128K); instead the
// frequency is held as turns, f / 2 pi modulo 1, in 64 bits of fixed point: the
// integer product with p, modulo 2^64, is the angle's fraction of a turn, off by p 2^-54
// turns at most (the division by 2 pi is in fp64).  Its upper 32 bits become
// an fp32 angle in half turns for sincospif.
//
// A CTA takes some tokens: their rows in the cache (lengths, pages) and the sines and
// cosines of every pair go to shared memory once and serve all heads.  A thread then
// takes 16 channels of a row at a time, the two 16-byte pieces that hold 8 pairs, so the
// turned values leave in the pieces that they came in.
#include "common.cuh"
#include "kv_append.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;  // tokens of a CTA, at most
constexpr int kUnroll = 4;   // rows whose pieces a thread loads at once
constexpr int kHold = 4;     // E4M3: slots a lane keeps between the maximum and the rounding

// 2^64 f / 2 pi modulo 2^64.
__device__ __forceinline__ uint64_t turns_of(float f) {
  double t = static_cast<double>(f) * 0.15915494309189533577;  // 1 / 2 pi
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// Two fp32 values to two E4M3 codes (lo in the low byte), to nearest even; what is not
// finite becomes NaN (the conversion alone would clamp an infinity to 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  lo = isfinite(lo) ? lo : NAN;
  hi = isfinite(hi) ? hi : NAN;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Exponent of the smallest power of two s >= 2^-100 with a / s <= 448 = 1.75 * 2^8, for
// a finite a >= 0 (1.75 is mantissa 0x600000).
__device__ __forceinline__ int scale_exp(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -100);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// 16 channels of a row: the pieces from off0 and off1 (8 channels each).
struct Slot {
  int off0, off1;
  bool turned;
};
// Slot c of a row of d channels.  Pairs (i, i + rot / 2): pieces 8c and rot / 2 + 8c;
// pairs (2i, 2i + 1), and channels from rot on: 16 neighbouring channels.
__device__ __forceinline__ Slot slot_of(int c, int rot, bool interleaved) {
  Slot s;
  s.turned = c < rot / 16;
  const bool apart = s.turned && !interleaved;
  s.off0 = apart ? 8 * c : 16 * c;
  s.off1 = apart ? rot / 2 + 8 * c : 16 * c + 8;
  return s;
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Turns the 8 pairs of a slot: a, b the two pieces, cs the pairs' (cos, sin, cos, sin).
__device__ __forceinline__ void turn(const uint4& a, const uint4& b, const float4 (&cs)[4],
                                     bool interleaved, float (&x)[8], float (&y)[8]) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
  if (!interleaved) {  // pair j: channel j of a and of b
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = unpack_bf16(aw[j]), v = unpack_bf16(bw[j]);
      x[2 * j] = u.x * cs[j].x - v.x * cs[j].y;
      y[2 * j] = u.x * cs[j].y + v.x * cs[j].x;
      x[2 * j + 1] = u.y * cs[j].z - v.y * cs[j].w;
      y[2 * j + 1] = u.y * cs[j].w + v.y * cs[j].z;
    }
  } else {  // pair j: channels 2j and 2j + 1 of the 16; x, y are the pieces again
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 u = unpack_bf16(j < 4 ? aw[j] : bw[j - 4]);
      const float c = j & 1 ? cs[j / 2].z : cs[j / 2].x, s = j & 1 ? cs[j / 2].w : cs[j / 2].y;
      const float p = u.x * c - u.y * s, q = u.x * s + u.y * c;
      if (j < 4) {
        x[2 * j] = p;
        x[2 * j + 1] = q;
      } else {
        y[2 * j - 8] = p;
        y[2 * j - 7] = q;
      }
    }
  }
}
__device__ __forceinline__ void widen(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = unpack_bf16(w[j]);
    x[2 * j] = u.x;
    x[2 * j + 1] = u.y;
  }
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

constexpr long long kSkip = -1;    // a token past the new ones of its sequence
constexpr long long kBad = -2;     // of a sequence with a bad length: its query rows become NaN
constexpr long long kNoPage = -3;  // of a bad page: its query rows are turned all the same

// FP8 = false: rows (queries, keys, values) of all tokens are one list.  FP8 = true: the
// list holds the queries alone, and each warp takes the keys or the values of a token
// whole, for the maximum over its heads.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) gqa_kv_append_rot_kernel(const KvAppendParams p,
                                                                     int tok_per) {
  constexpr int kSlots = D / 16;
  constexpr int kRowStep = kThreads / kSlots;  // rows that the CTA takes at a time
  __shared__ float4 cs_sm[kMaxTok][4][kSlots];
  __shared__ uint64_t turns_sm[D / 2];
  __shared__ long long dst_sm[kMaxTok];  // row of the cache, kSkip or kBad
  __shared__ int pos_sm[kMaxTok];
  const int tid = threadIdx.x;
  const long long tok0 = static_cast<long long>(blockIdx.x) * tok_per;
  const int n_tok = static_cast<int>(min(static_cast<long long>(tok_per),
                                         static_cast<long long>(p.B) * p.T - tok0));
  const bool inter = p.interleaved != 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Where the tokens go.
  if (tid < n_tok) {
    const long long g = tok0 + tid;
    const int b = static_cast<int>(g / p.T), i = static_cast<int>(g - static_cast<long long>(b) * p.T);
    const int L = p.seq_lens[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    long long dst = kSkip;
    int pos = 0;
    if (n < 0 || n > p.T || L < n || L > p.S_max) {
      dst = kBad;
      if (blockIdx.y == 0 && i == 0) atomicOr(p.err, kErrBadSeqLen);
    } else if (i < n) {
      const int at = L - n + i;
      pos = p.positions ? p.positions[g] : at;
      if (p.block_table) {
        const int page = p.block_table[static_cast<long long>(b) * p.max_blocks + at / p.page_size];
        if (page >= 0 && page < p.num_pages)
          dst = static_cast<long long>(page) * p.page_size + at % p.page_size;
        else
          atomicOr(p.err, kErrBadPage);
      } else {
        dst = static_cast<long long>(b) * p.S_max + at;
      }
      if (dst == kSkip) dst = kNoPage;
    }
    dst_sm[tid] = dst;
    pos_sm[tid] = pos;
  }
  if (tid >= 64 && tid - 64 < p.rot / 2) turns_sm[tid - 64] = turns_of(p.freqs[tid - 64]);
  __syncthreads();
  for (int e = tid; e < n_tok * (p.rot / 2); e += kThreads) {
    const int k = e / (p.rot / 2), i = e - k * (p.rot / 2);
    const uint64_t a = static_cast<uint64_t>(static_cast<long long>(pos_sm[k])) * turns_sm[i];
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * (1.f / 2147483648.f), &sn, &cn);
    float2* at = reinterpret_cast<float2*>(&cs_sm[k][(i % 8) / 2][i / 8]) + (i & 1);
    *at = make_float2(cn, sn);
  }
  __syncthreads();

  const size_t hq = static_cast<size_t>(p.H_q) * D, hkv = static_cast<size_t>(p.H_kv) * D;
  const size_t n_cache = (p.block_table ? static_cast<size_t>(p.num_pages) * p.page_size
                                        : static_cast<size_t>(p.B) * p.S_max) * hkv;
  const size_t n_q = static_cast<size_t>(p.B) * p.T * hq;
  const int rows = (p.q ? p.H_q : 0) + (FP8 ? 0 : 2 * p.H_kv);
  const int q_rows = p.q ? p.H_q : 0;
  const Slot sl = slot_of(tid % kSlots, p.rot, inter);
  {
    // (token, row) pairs, kRowStep * gridDim.y apart
    const int step = kRowStep * gridDim.y;
    int k = 0, r = tid / kSlots + kRowStep * blockIdx.y;
    while (rows > 0) {
      uint4 a[kUnroll], c[kUnroll];
      int kk[kUnroll], rr[kUnroll];
      bool any = false;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        while (r >= rows && k < n_tok) {
          r -= rows;
          ++k;
        }
        kk[u] = k;
        rr[u] = r;
        if (k < n_tok && dst_sm[k] != kSkip) {
          const long long g = tok0 + k;
          const __nv_bfloat16* src =
              r < q_rows ? p.q + g * p.q_stride + r * D
              : r < q_rows + p.H_kv ? p.k + g * p.kv_stride + (r - q_rows) * D
                                    : p.v + g * p.kv_stride + (r - q_rows - p.H_kv) * D;
          a[u] = *reinterpret_cast<const uint4*>(src + sl.off0);
          c[u] = *reinterpret_cast<const uint4*>(src + sl.off1);
        } else {
          kk[u] = n_tok;
        }
        any |= k < n_tok;
        r += step;
      }
      if (!any) break;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (kk[u] >= n_tok) continue;
        const long long dst = dst_sm[kk[u]];
        const bool is_q = rr[u] < q_rows, is_v = rr[u] >= q_rows + p.H_kv;
        __nv_bfloat16* out;
        size_t at, extent;
        if (is_q) {
          out = p.q_out;
          at = static_cast<size_t>(tok0 + kk[u]) * hq + static_cast<size_t>(rr[u]) * D;
          extent = n_q;
        } else {
          if (dst < 0) continue;
          out = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache);
          at = static_cast<size_t>(dst) * hkv +
               static_cast<size_t>(rr[u] - q_rows - (is_v ? p.H_kv : 0)) * D;
          extent = n_cache;
        }
        if (sl.turned && !is_v) {
          float4 cs[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) cs[j] = cs_sm[kk[u]][j][tid % kSlots];
          float x[8], y[8];
          turn(a[u], c[u], cs, inter, x, y);
          a[u] = narrow(x);
          c[u] = narrow(y);
        }
        if (dst == kBad) a[u] = c[u] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (in_bounds(at + sl.off0, 8, extent, p.err))
          *reinterpret_cast<uint4*>(out + at + sl.off0) = a[u];
        if (in_bounds(at + sl.off1, 8, extent, p.err))
          *reinterpret_cast<uint4*>(out + at + sl.off1) = c[u];
      }
    }
  }

  if constexpr (FP8) {
    const int warp = tid >> 5, lane = tid & 31;
    const int n_slots = p.H_kv * kSlots;  // of a token's keys or values
    const Slot ls = slot_of(lane % kSlots, p.rot, inter);
    for (int unit = warp + 8 * blockIdx.y; unit < 2 * n_tok; unit += 8 * gridDim.y) {
      const int k = unit >> 1;
      const bool is_v = unit & 1;
      const long long dst = dst_sm[k];
      if (dst < 0) continue;
      const __nv_bfloat16* src = (is_v ? p.v : p.k) + (tok0 + k) * p.kv_stride;
      float4 cs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cs[j] = cs_sm[k][j][lane % kSlots];
      const bool turned = ls.turned && !is_v;
      auto values = [&](const uint4& a, const uint4& c, float (&x)[8], float (&y)[8]) {
        if (turned) {
          turn(a, c, cs, inter, x, y);
        } else {
          widen(a, x);
          widen(c, y);
        }
      };
      uint4 a[kHold], c[kHold];
#pragma unroll
      for (int h = 0; h < kHold; ++h) {
        const int s = lane + 32 * h;
        if (s < n_slots) {
          a[h] = *reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off0);
          c[h] = *reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off1);
        }
      }
      float amax = 0.f;
      auto widest = [&](const uint4& va, const uint4& vc) {
        float x[8], y[8];
        values(va, vc, x, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (isfinite(x[j])) amax = fmaxf(amax, fabsf(x[j]));
          if (isfinite(y[j])) amax = fmaxf(amax, fabsf(y[j]));
        }
      };
#pragma unroll
      for (int h = 0; h < kHold; ++h)
        if (lane + 32 * h < n_slots) widest(a[h], c[h]);
      for (int s = lane + 32 * kHold; s < n_slots; s += 32)
        widest(*reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off0),
               *reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off1));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = scale_exp(amax);
      const float inv = pow2f(-e);
      uint8_t* codes = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
      auto put = [&](int s, const uint4& va, const uint4& vc) {
        float x[8], y[8];
        values(va, vc, x, y);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] = e4m3x2(x[4 * j] * inv, x[4 * j + 1] * inv) |
                 e4m3x2(x[4 * j + 2] * inv, x[4 * j + 3] * inv) << 16;
          w[2 + j] = e4m3x2(y[4 * j] * inv, y[4 * j + 1] * inv) |
                     e4m3x2(y[4 * j + 2] * inv, y[4 * j + 3] * inv) << 16;
        }
        const size_t at = static_cast<size_t>(dst) * hkv + static_cast<size_t>(s / kSlots) * D;
        if (in_bounds(at + ls.off0, 8, n_cache, p.err))
          *reinterpret_cast<uint2*>(codes + at + ls.off0) = make_uint2(w[0], w[1]);
        if (in_bounds(at + ls.off1, 8, n_cache, p.err))
          *reinterpret_cast<uint2*>(codes + at + ls.off1) = make_uint2(w[2], w[3]);
      };
#pragma unroll
      for (int h = 0; h < kHold; ++h)
        if (lane + 32 * h < n_slots) put(lane + 32 * h, a[h], c[h]);
      for (int s = lane + 32 * kHold; s < n_slots; s += 32)
        put(s, *reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off0),
            *reinterpret_cast<const uint4*>(src + (s / kSlots) * D + ls.off1));
      if (lane == 0 && in_bounds(dst, 1, n_cache / hkv, p.err))
        (is_v ? p.v_scale : p.k_scale)[dst] = pow2f(e);
    }
  }
}

template <int D, bool FP8>
cudaError_t launch(const KvAppendParams& p, int sms, cudaStream_t stream) {
  // Tokens to a CTA: enough CTAs for eight on every SM, then as many tokens as share the
  // set-up.  Few tokens: their rows are divided among CTAs.
  const long long tokens = (long long)p.B * p.T;
  long long tok_per = tokens / (16LL * sms);
  tok_per = tok_per < 1 ? 1 : tok_per > kMaxTok ? kMaxTok : tok_per;
  const long long x = (tokens + tok_per - 1) / tok_per;
  if (x > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int rows = (p.q ? p.H_q : 0) + (FP8 ? 0 : 2 * p.H_kv);
  const int passes = (rows * (D / 16) + kThreads - 1) / kThreads;
  long long y = 2LL * sms / x;
  y = y < 1 ? 1 : y > passes ? (passes < 1 ? 1 : passes) : y;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, gqa_kv_append_rot_kernel<D, FP8>, p, static_cast<int>(tok_per));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_rot(const KvAppendParams& p, int sms, cudaStream_t stream) {
  const bool fp8 = p.k_scale != nullptr;
  switch (p.d) {
    case 16: return fp8 ? launch<16, true>(p, sms, stream) : launch<16, false>(p, sms, stream);
    case 32: return fp8 ? launch<32, true>(p, sms, stream) : launch<32, false>(p, sms, stream);
    case 64: return fp8 ? launch<64, true>(p, sms, stream) : launch<64, false>(p, sms, stream);
    case 128: return fp8 ? launch<128, true>(p, sms, stream) : launch<128, false>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gqa
