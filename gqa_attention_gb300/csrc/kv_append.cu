// kv_append.cu -- appending keys and values to a bf16 or per-token E4M3 cache, contiguous or
// paged, the keys (and the step's queries) turned by their positions on the way.
//
// The rotation of a pair (x, y) of channels with frequency f at position p:
//   (x cos a - y sin a, x sin a + y cos a),  a = p f.
// The product p f in fp32 would be off by p f 2^-24 (0.008 radians at 128K); instead the
// frequency is held as turns, f / 2 pi modulo 1, in 64 bits of fixed point: the
// integer product with p, modulo 2^64, is the angle's fraction of a turn.  The division by
// 2 pi is in fp64, constant and product rounded to 2^-53 of themselves, so the angle is
// off by |p f| 2^-52 radians, and the fixed point adds |p| 2^-65 turns.  Its upper 32
// bits become an fp32 angle in half turns for sincospif.
//
// A CTA takes some tokens: their rows in the cache (lengths, pages) and the sines and
// cosines of every pair go to shared memory once and serve all heads.  A thread then
// takes 16 channels of a row at a time, the two 16-byte pieces that hold 8 pairs, so the
// turned values leave in the pieces that they came in.
//
// Bound by HBM for long prompts (32K tokens, 64 / 8 heads of 128: 201 us, 98% of the
// copy's rate; to E4M3 198, 95%), by instructions where keys and values alone go to
// E4M3 (8 heads, 42 us, floor 30), by a chain of latencies for single tokens (length,
// page, angles, store: 2.5 us).
#include <algorithm>

#include "kv_append.h"
#include "tcgen05.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;  // tokens of a CTA, at most
constexpr int kUnroll = 4;   // rows whose pieces a thread loads at once
constexpr int kRing = 2;     // E4M3: tiles that a thread has copies in flight or waiting for

__device__ __forceinline__ void copy_async_16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// 2^64 f / 2 pi modulo 2^64.  (The sign is taken in integers: 1 - t would round to 2^-54,
// 2^-20 radians at position 2^31.)
__device__ __forceinline__ uint64_t turns_of(float f) {
  double t = fabs(static_cast<double>(f)) * 0.15915494309189533577;  // 1 / 2 pi
  t -= floor(t);
  const uint64_t turns = __double2ull_rn(t * 18446744073709551616.0);
  return f < 0.f ? 0 - turns : turns;
}

// Two fp32 values to two E4M3 codes (lo in the low byte), to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
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

// Turns the 8 pairs of a slot: a, b the two pieces, cs[j] the cosines and the sines of pairs
// 2j and 2j + 1.
__device__ __forceinline__ void turn(const uint4& a, const uint4& b, const float4 (&cs)[4],
                                     bool interleaved, float (&x)[8], float (&y)[8]) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
  if (!interleaved) {  // pair j: channel j of a and of b
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = unpack_bf16(aw[j]), v = unpack_bf16(bw[j]);
      float t0, t1;
      fmul2(t0, t1, v.x, v.y, cs[j].z, cs[j].w);
      ffma2(x[2 * j], x[2 * j + 1], u.x, u.y, cs[j].x, cs[j].y, -t0, -t1);
      fmul2(t0, t1, v.x, v.y, cs[j].x, cs[j].y);
      ffma2(y[2 * j], y[2 * j + 1], u.x, u.y, cs[j].z, cs[j].w, t0, t1);
    }
  } else {  // pair j: channels 2j and 2j + 1 of the 16; x, y are the pieces again
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 u = unpack_bf16(j < 4 ? aw[j] : bw[j - 4]);
      const float c = j & 1 ? cs[j / 2].y : cs[j / 2].x, s = j & 1 ? cs[j / 2].w : cs[j / 2].z;
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

// HOLD = 0 (bf16): rows (queries, keys, values) of all tokens are one list.  HOLD > 0 (E4M3):
// the list holds the queries alone, and the CTAs of the last grid row take the keys
// and values.  A token's keys, or its values, are a unit that `width` lanes take whole, for
// the maximum over its heads: a part of a warp, a warp, or several warps, which meet at a
// barrier.  HOLD slots of a lane stay in registers between the maximum and the rounding.  A
// lane copies its own pieces of the next units to shared memory meanwhile, where they
// cost no registers and no barrier.
// EARLY: the CTA's list is one round, whose rows are loaded before the angles are worked
// out.  (With several rounds that is slower: 32K tokens of 80 heads of 128 232 us, 201 if
// each round is loaded when its turn comes.)
template <int D, int HOLD, bool EARLY>
__global__ void __launch_bounds__(kThreads, HOLD == 2 ? 2 : HOLD == 0 && EARLY ? 4 : 3)
    gqa_kv_append_rot_kernel(const KvAppendParams p, int tok_per, int width) {
  constexpr bool FP8 = HOLD > 0;
  constexpr int kSlots = D / 16;
  constexpr int kRowStep = kThreads / kSlots;  // rows that the CTA takes at a time
  __shared__ float4 cs_sm[kMaxTok][4][kSlots];
  __shared__ uint64_t turns_sm[D / 2];
  __shared__ long long dst_sm[kMaxTok];  // row of the cache, kSkip or kBad
  __shared__ int pos_sm[kMaxTok];
  __shared__ uint32_t max_sm[FP8 ? 3 : 1][kThreads / 32];  // E4M3: a warp's share of a maximum
  __shared__ uint4 ring_sm[FP8 ? kRing : 1][FP8 ? 2 * HOLD : 1][FP8 ? kThreads : 1];
  const int tid = threadIdx.x;
  const long long tok0 = static_cast<long long>(blockIdx.x) * tok_per;
  const int n_tok = static_cast<int>(min(static_cast<long long>(tok_per),
                                         static_cast<long long>(p.B) * p.T - tok0));
  const bool inter = p.interleaved != 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const bool kv_role = FP8 && blockIdx.y == gridDim.y - 1;
  const size_t hq = static_cast<size_t>(p.H_q) * D, hkv = static_cast<size_t>(p.H_kv) * D;
  const int q_rows = p.q ? p.H_q : 0;
  const int rows = q_rows + (FP8 ? 0 : 2 * p.H_kv);
  const bool list_role = !FP8 || (rows && (!kv_role || gridDim.y == 1));
  const Slot sl = slot_of(tid % kSlots, p.rot, inter);
  // The list's (token, row) pairs, from this thread's first on.
  const int step = kRowStep * (FP8 && gridDim.y > 1 ? gridDim.y - 1 : gridDim.y);
  int k = 0, r = tid / kSlots + kRowStep * blockIdx.y;
  uint4 a[kUnroll], c[kUnroll];
  int kk[kUnroll], rr[kUnroll];
  auto load_round = [&]() {
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
      } else if (k < n_tok) {
        kk[u] = kMaxTok + 1;  // not a row to write, nor (n_tok) the list's end
      }
      r += step;
    }
  };
  // Tile i of the units: the keys (i even) or values of the `many` tokens from (i / 2) many on,
  // a token to each `width` lanes.  This lane's slots are `at0`, at0 + width, ..
  constexpr int kKeep = FP8 ? HOLD : 1;
  const int warp = tid >> 5, lane = tid & 31;
  const int n_slots = p.H_kv * kSlots;
  const int many = width < 32 ? 32 / width : 1, mine = width < 32 ? lane / width : 0;
  const int at0 = tid % width;
  const int n_teams = width < 32 ? kThreads / 32 : kThreads / width;
  const int my_team = width < 32 ? warp : tid / width;
  const int n_tiles = 2 * ((n_tok + many - 1) / many);
  const Slot ls = slot_of(at0 % kSlots, p.rot, inter);
  auto token_of = [&](int tile) { return (tile >> 1) * many + mine; };
  auto unit_rows = [&](int tile) {
    return ((tile & 1) ? p.v : p.k) + (tok0 + token_of(tile)) * p.kv_stride;
  };
  auto copy_tile = [&](int tile, int stage) {
    const int t = token_of(tile);
    if (tile < n_tiles && t < n_tok && dst_sm[t] >= 0) {
      const __nv_bfloat16* src = unit_rows(tile);
#pragma unroll
      for (int h = 0; h < kKeep; ++h) {
        const int s = at0 + width * h;
        if (s >= n_slots) continue;
        const __nv_bfloat16* row = src + (s / kSlots) * D;
        copy_async_16(&ring_sm[stage][2 * h][tid], row + ls.off0);
        copy_async_16(&ring_sm[stage][2 * h + 1][tid], row + ls.off1);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // Where the tokens go.
  bool wanted = false;
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
    wanted = dst != kSkip;
  }
  if (tid >= 64 && tid - 64 < p.rot / 2) turns_sm[tid - 64] = turns_of(p.freqs[tid - 64]);
  if (!__syncthreads_or(wanted)) return;  // (all of them padding)
  // (the first rows travel while the angles are worked out)
  if (kv_role) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) copy_tile(my_team + i * n_teams, i);
    }
  }
  if constexpr (EARLY) {
    if (list_role) load_round();
  }
  for (int t = tid / (D / 2), i = tid % (D / 2); t < n_tok && i < p.rot / 2; t += kThreads / (D / 2)) {
    if (dst_sm[t] == kSkip) continue;
    const uint64_t angle = static_cast<uint64_t>(static_cast<long long>(pos_sm[t])) * turns_sm[i];
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * (1.f / 2147483648.f), &sn, &cn);
    float* at = reinterpret_cast<float*>(&cs_sm[t][(i % 8) / 2][i / 8]) + (i & 1);
    at[0] = cn;
    at[2] = sn;
  }
  __syncthreads();

  const size_t n_cache = (p.block_table ? static_cast<size_t>(p.num_pages) * p.page_size
                                        : static_cast<size_t>(p.B) * p.S_max) * hkv;
  const size_t n_q = static_cast<size_t>(p.B) * p.T * hq;
  if (list_role) {
    for (;;) {
      if constexpr (!EARLY) {
        load_round();
        bool any = false;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) any |= kk[u] != n_tok;
        if (!any) break;
      }
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
      if constexpr (EARLY) break;
    }
  }

  if constexpr (FP8) {
    // The largest of a unit's values, given as bits (positive floats compare as those).  Of
    // several warps at one barrier: the buffers are taken in turn.
    int buffer = 0;
    auto unit_max = [&](uint32_t v) -> uint32_t {
      if (width < 32) {
        for (int m = width / 2; m; m /= 2) v = max(v, __shfl_xor_sync(0xffffffffu, v, m));
        return v;
      }
      v = __reduce_max_sync(0xffffffffu, v);
      if (width == 32) return v;
      if (lane == 0) max_sm[buffer][warp] = v;
      named_bar_sync(1 + my_team, width);
      const uint32_t got = lane < width / 32 ? max_sm[buffer][my_team * (width / 32) + lane] : 0u;
      buffer = buffer == 2 ? 0 : buffer + 1;
      return __reduce_max_sync(0xffffffffu, got);
    };
    int stage = 0;
    for (int tile = my_team; kv_role && tile < n_tiles; tile += n_teams) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      uint4 va[kKeep], vc[kKeep];
#pragma unroll
      for (int h = 0; h < kKeep; ++h) {
        va[h] = ring_sm[stage][2 * h][tid];
        vc[h] = ring_sm[stage][2 * h + 1][tid];
      }
      const int t = min(token_of(tile), n_tok - 1);
      const bool is_v = tile & 1;
      const long long dst = token_of(tile) < n_tok ? dst_sm[t] : kSkip;
      const bool live = dst >= 0;
      const int own = live ? n_slots : 0;  // slots of this lane's unit
      const __nv_bfloat16* src = unit_rows(tile);
      float4 cs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cs[j] = cs_sm[t][j][at0 % kSlots];
      const bool turned = ls.turned && !is_v;
      auto values = [&](const uint4& u, const uint4& w, float (&x)[8], float (&y)[8]) {
        if (turned) {
          turn(u, w, cs, inter, x, y);
        } else {
          widen(u, x);
          widen(w, y);
        }
      };
      auto values_of = [&](int s, float (&x)[8], float (&y)[8]) {
        const __nv_bfloat16* row = src + (s / kSlots) * D;
        values(*reinterpret_cast<const uint4*>(row + ls.off0),
               *reinterpret_cast<const uint4*>(row + ls.off1), x, y);
      };
      float x[kKeep][8], y[kKeep][8];
      float amax = 0.f;
      auto widest = [&](const float (&v)[8]) {  // (fmaxf passes over NaN)
        float m[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) m[j] = fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1]));
        amax = fmax3(amax, fmax3(m[0], m[1], m[2]), fmaxf(fabsf(v[6]), fabsf(v[7])));
      };
#pragma unroll
      for (int h = 0; h < kKeep; ++h) {
        if (at0 + width * h >= own) continue;
        values(va[h], vc[h], x[h], y[h]);
        widest(x[h]);
        widest(y[h]);
      }
      for (int s = at0 + width * kKeep; s < own; s += width) {
        float u[8], w[8];
        values_of(s, u, w);
        widest(u);
        widest(w);
      }
      // (the pieces have been read: their places take the tile after the next)
      copy_tile(tile + kRing * n_teams, stage);
      stage = stage == kRing - 1 ? 0 : stage + 1;
      amax = __uint_as_float(unit_max(__float_as_uint(amax)));
      auto widest_finite = [&](float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = isfinite(v[j]) ? v[j] : NAN;  // (an infinity would be clamped to 448)
          amax = fmaxf(amax, fabsf(v[j]));
        }
      };
      // Rare: the maximum again, of what is finite.  (Lanes of one warp go together.)
      const bool infinite = amax > 3.4028235e38f;
      if (__any_sync(0xffffffffu, infinite)) {
        amax = 0.f;
#pragma unroll
        for (int h = 0; h < kKeep; ++h) {
          if (at0 + width * h >= own) continue;
          widest_finite(x[h]);
          widest_finite(y[h]);
        }
        for (int s = at0 + width * kKeep; s < own; s += width) {
          float u[8], w[8];
          values_of(s, u, w);
          widest_finite(u);
          widest_finite(w);
        }
        amax = __uint_as_float(unit_max(__float_as_uint(amax)));
      }
      const int e = scale_exp(amax);
      const float inv = pow2f(-e);
      uint8_t* codes = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
      auto coded = [&](float (&v)[8]) -> uint2 {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          fmul2(lo, hi, v[2 * j], v[2 * j + 1], inv, inv);
          w[j] = e4m3x2(lo, hi);
        }
        return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      };
      const size_t row = static_cast<size_t>(dst) * hkv;
      auto put = [&](int s, float (&u)[8], float (&w)[8]) {
        const size_t at = row + (s / kSlots) * D;
        if (in_bounds(at + ls.off0, 8, n_cache, p.err))
          *reinterpret_cast<uint2*>(codes + at + ls.off0) = coded(u);
        if (in_bounds(at + ls.off1, 8, n_cache, p.err))
          *reinterpret_cast<uint2*>(codes + at + ls.off1) = coded(w);
      };
#pragma unroll
      for (int h = 0; h < kKeep; ++h)
        if (at0 + width * h < own) put(at0 + width * h, x[h], y[h]);
      for (int s = at0 + width * kKeep; s < own; s += width) {
        float u[8], w[8];
        values_of(s, u, w);
        if (infinite) {
          widest_finite(u);
          widest_finite(w);
        }
        put(s, u, w);
      }
      if (live && at0 == 0 && in_bounds(dst, 1, n_cache / hkv, p.err))
        (is_v ? p.v_scale : p.k_scale)[dst] = pow2f(e);
    }
  }
}

template <int D, int HOLD>
cudaError_t launch(const KvAppendParams& p, int sms, int width, cudaStream_t stream) {
  constexpr bool FP8 = HOLD > 0;
  // Tokens to a CTA.  bf16: of few rows (half of a round to a token or less) as many as leave
  // one wave of four CTAs to an SM, but no more than one round takes (20 / 5 heads of 64:
  // 1000 tokens 3.2 us, 4.3 with a second wave of 392 CTAs; 4096 6.3 and 7.7); of many rows
  // at least four CTAs to an SM, then as many tokens as share the set-up.  E4M3: whole
  // waves of the two or three CTAs that an SM holds; the same CTA turns the queries and
  // then takes the keys and values, whose copies travel meanwhile, and only where CTAs are
  // few do those go to CTAs of their own (32 / 8 heads of 128: 1000 tokens 5.1 us, 13.3 with
  // four CTAs to an SM and the keys and values always apart; 32K 120 and 130, 95% of the copy
  // rate with 64 query heads).  Few tokens: their rows are divided among CTAs.
  const long long tokens = (long long)p.B * p.T;
  const int rows = (p.q ? p.H_q : 0) + (FP8 ? 0 : 2 * p.H_kv);
  const int pieces = rows * (D / 16);  // of a token in the list
  const bool light = !FP8 && pieces <= kUnroll * kThreads / 2;
  const long long ctas = (!FP8 ? 4 : HOLD == 1 ? 3 : 2) * (long long)sms;
  long long tok_per;
  if (FP8) {
    const long long slots = ctas * ((tokens + ctas * kMaxTok - 1) / (ctas * kMaxTok));
    tok_per = (tokens + slots - 1) / slots;
  } else if (light) {
    tok_per = std::min((tokens + ctas - 1) / ctas, (long long)kUnroll * kThreads / pieces);
  } else {
    tok_per = std::max(1LL, tokens / ctas);
  }
  tok_per = std::min(tok_per, (long long)kMaxTok);
  const long long x = (tokens + tok_per - 1) / tok_per;
  if (x > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int passes = (pieces + kThreads - 1) / kThreads;
  const long long y = std::min((long long)passes, std::max(1LL, 2LL * sms / x));  // (0: no list)
  const bool apart = FP8 && (y != 1 || x <= sms);
  const bool early = tok_per * pieces <= kUnroll * kThreads * y;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(y + (apart ? 1 : 0)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, early ? gqa_kv_append_rot_kernel<D, HOLD, true> : gqa_kv_append_rot_kernel<D, HOLD, false>,
      p, static_cast<int>(tok_per), width);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const KvAppendParams& p, int sms, cudaStream_t stream) {
  if (!p.k_scale) return launch<D, 0>(p, sms, 32, stream);
  const int slots = p.H_kv * (D / 16);
  // A lane holds one slot, or two where that makes one warp of more (32K tokens, K and V
  // alone: 8 heads of 128 41.7 us, 51.6 with two warps to a unit, which meet at a barrier for
  // each maximum; 8 heads of 64, which one warp holds either way, 28.9 and 27.4) and
  // there are tokens to fill the GPU.
  const bool two = slots > 32 && (long long)p.B * p.T > 4LL * sms;
  int width = D / 16;
  while (width < kThreads && slots > (two ? 2 : 1) * width) width *= 2;
  return two ? launch<D, 2>(p, sms, width, stream) : launch<D, 1>(p, sms, width, stream);
}

}  // namespace

cudaError_t launch_kv_append_rot(const KvAppendParams& p, int sms, cudaStream_t stream) {
  switch (p.d) {
    case 16: return launch_d<16>(p, sms, stream);
    case 32: return launch_d<32>(p, sms, stream);
    case 64: return launch_d<64>(p, sms, stream);
    case 128: return launch_d<128>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gqa
