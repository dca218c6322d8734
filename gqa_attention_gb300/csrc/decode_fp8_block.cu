// decode_fp8_block.cu -- split-KV decode over the block-scaled E4M3 cache on the
// fifth-generation tensor cores, the codes taken as they lie in memory.
//
// What it computes, for the T_q last positions of each sequence (row r of a KV
// head is query t = r / G of head kv G + r % G and sees keys below L - T_q + 1 + t):
//   x_j = tau ks_j (q . kc_j),  O = sum_j softmax(x)_j vs_j vc_j,  LSE = ln sum_j e^x_j
// with kc, vc the E4M3 values and ks_j, vs_j the scales of key j's block of
// tokens.  One CTA per (split, KV head, sequence) leaves the partial (m, l, O)
// of decode.cu's layout for the combine kernel, or writes O and LSE (one split).
//
// Keys sit in the M rows of the MMA, query rows in N:
//   S_j = K_j Q^T   (M = 128 keys, N = 2R, K = d; both operands in shared memory)
//   O^T = V_j^T P   (M = d, N = 2R, K = 128 keys; V^T and P are MN-major views)
// so that a thread owns one key: its scales are one register each, its exponents
// R, and a padded row costs no softmax work.  With the rows in M, as decode_tc.cu
// has them, 8 query rows would leave 120 of 128 lanes idle and one warp with all
// 128 exponentials of each row.
//
// kind::f8f6f4 wants both operands in 8 bits, so Q and P are split in two E4M3
// terms, side by side in N:
//   q 2^k = hi + lo / 32.  bf16 carries 8 significant bits and E4M3 four, so the
//     split is exact down to 2^-21 of the row's largest |q| (hi <= 256, so the
//     remainder is at most 8 and 32 times it at most 256).
//   p in (0, 256] = hi + lo / 32, within 2^-9 of p above 2^-6 as bf16 would be,
//     with a smallest step of 2^-14.
// The codes need no conversion, which is what bounds the mma.sync sweep over
// E4M3 codes.
//
// The value scale rides on the exponent: y_j = x_j log2 e + log2 vs_j, P = 2^(y - m + 7)
// with m a running reference within 1 of the largest y since it last fell, and l sums
// P / vs_j in fp32.  So the range of P adapts to vs as well as to the scores.  m is
// raised only when some y exceeds it by more than 1 (P stays below 2^8): a tile
// costs one barrier that ORs that condition, and the row maxima are worked out
// only when it holds.  The merge of the partials holds for any reference.
//
// Two E4M3 terms end at steps of 2^-14, which is 2^-22 of what the reference may be below the
// largest y, and a first token that takes most of the weight (often with a value near
// zero) would leave the rest of the row nothing but roundings: with 1% left to 32K
// tokens of mean-zero values, O was off by 3.5% in 128 splits and by 24% in three.  So m
// also falls: the stream's next tile after a rise of 2^12 or more (the first one among
// them) is looked at, and if its largest y is 2^12 below m, m becomes that y, though not
// less than 2^-24 of its highest, so that O and l keep clear of fp32's end (l also holds
// 1 / vs: m stays where a value scale below 2^-60 has been seen).  Then only the tokens that
// share a tile with such a first token have its rounding (2.1% either way; their values' own
// rounding to E4M3 is as large).  Looking costs 0.15 us in a CTA of eight tiles and up to 2%
// elsewhere; falls of 2^8, looked for at every update, took up to 9%.
//
// O^T stays in tensor memory and is rescaled there when m moves (thread = row d).
//
// What bounds it (device time with the merge, 8 KV heads of 128, 32K tokens): 8 query rows
// 14.6 us for 67 MB, the tiles at HBM's rate after about 5 us of start and merge; 16
// rows 16.7, 32 rows 20.4, 64 rows 30.5, the softmax of R weights a key in two terms.
// One CTA takes 0.35 us a tile with 8 rows, 1.8 us with 64.
//
// Roles: warps 0 and 3 TMA producers of K and V (and two more at the end, for small
// pages), warp 1 issuer of S (and tensor memory), warp 2 issuer of O, the others Q
// split, softmax, rescaling and epilogue.
#include "tcgen05.cuh"

namespace gqa {
namespace {

constexpr int kFbKeys = 128;                // keys per tile
constexpr uint32_t kFbTile = 128u * 128u;   // 128 rows of 128 bytes
constexpr float kLoStep = 1.f / 32.f;       // weight of the low term
constexpr float kPScaleLog2 = 7.f;          // P is held times 2^7
constexpr float kPMaxLog2 = 8.f;            // and must not pass 2^8
constexpr float kFall = 12.f;               // references fall where a tile lies 2^12 below, and
constexpr float kFallMost = 24.f;           // by 2^24 from their highest at most (see above)
constexpr float kFallScale = 8.6736174e-19f;  // 2^-60: not behind a smaller value scale
constexpr float kMinVScale = 7.888609052210118e-31f;  // 2^-100: smaller ones count as zero

// A CTA's share of a batch whose splits follow the sequences' lengths: piece `split` of
// `count` of sequence b, each of `tiles` tiles (b < 0: none).
struct Piece {
  int b, split, count, tiles;
};
// The batch is cut into pieces of as many tiles as are needed for at most `pieces` of them
// (and n_split of a sequence; every sequence has one, also one of a bad length), and
// this CTA takes piece `index` in the order of the sequences.  One warp, lane i with
// the tiles of sequences i, 32 + i and 64 + i (0: a bad length); every warp of the
// grid finds the same cut.
constexpr int kMaxCut = 96;  // sequences
__device__ __noinline__ Piece find_piece(int t0, int t1, int t2, int B, int n_split, int pieces,
                                         int index, int lane) {
  const int total = t0 + t1 + t2;  // (each below 2^24)
  const long long all = static_cast<long long>(__reduce_add_sync(0xffffffffu, total >> 12)) * 4096 +
                        __reduce_add_sync(0xffffffffu, total & 4095);
  const int most = max(1, __reduce_max_sync(0xffffffffu, max(max(t0, t1), t2)));
  auto cuts = [&](int t, int k, int c) {  // pieces of sequence 32 k + lane
    return 32 * k + lane < B ? max(1, (t + c - 1) / c) : 0;
  };
  int lo = max(1, static_cast<int>(max((all + pieces - 1) / pieces,
                                       (most + n_split - 1LL) / n_split)));
  // sum of ceil(t / c) <= all / c + B
  int hi = static_cast<int>(min((long long)most, max((long long)lo, all / (pieces - B) + 1)));
  while (lo < hi) {
    const int c = (lo + hi) / 2;
    const int need = cuts(t0, 0, c) + cuts(t1, 1, c) + cuts(t2, 2, c);
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, need)) <= pieces) hi = c;
    else lo = c + 1;
  }
  int left = index;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int mine = cuts(k == 0 ? t0 : k == 1 ? t1 : t2, k, hi);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, upto > left);
    if (past != 0) {
      const int who = __ffs(past) - 1;
      const int count = __shfl_sync(0xffffffffu, mine, who);
      return {32 * k + who, left - (__shfl_sync(0xffffffffu, upto, who) - count), count, hi};
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return {-1, 0, 0, hi};
}

// How the codes of a tile are loaded: one box of a contiguous cache, a box for each
// page, or, for pages of 16 tokens and up to 32 query rows, such boxes by two warps each
// for K and V.  A warp takes about 150 cycles to issue a box, so the eight of a tile
// take longer than its softmax: batch 16 of 4K to 60K tokens, two queries, 249 us with
// one warp, 215 with two; 64 x 4K, d = 64, 28.4 and 26.9.  At 32 tokens the four boxes fit
// (23.8 us, and 24.7 with the registers of two more warps), as they do beside 64
// rows' softmax (32K, eight queries: 31.6 and 34.4) and in batches cut by their lengths (32
// rows, 8 x 100 to 10K: 31.9 and 32.4).
enum class Load { kTile, kPages, kSmallPages };
constexpr int kSmallPage = 16;

// Compile-time shape of one variant.  R query rows (padded), NS slots per ring,
// NT streams of tiles (stream s takes tiles s, s + NT, ..) and NG groups of rows:
// the 4 NT NG softmax warps share the work of a tile by rows and alternate tiles.
template <int R_, int NS_, int NT_, int NG_>
struct FbShape {
  static constexpr int R = R_, NS = NS_, NT = NT_, NG = NG_;
  static constexpr int RW = R / NG;                 // rows of a warp
  static constexpr int NSB = 2 * NT;                // S buffers
  static constexpr int kWarps = 4 * NT * NG;        // softmax warps
  static constexpr int kRowsQ = R / kWarps;         // rows of Q a warp splits
  static constexpr int threads(Load load) {
    return 128 + 32 * kWarps + (load == Load::kSmallPages ? 64 : 0);
  }
  static constexpr uint32_t kRowP = 2 * R;          // bytes of a key's row of P
  static constexpr uint32_t kOffV = NS * kFbTile;
  static constexpr uint32_t kOffQ = 2 * NS * kFbTile;
  static constexpr uint32_t kOffP = kOffQ + 2 * R * 128;
  static constexpr uint32_t kTileP = 128 * kRowP;
  static constexpr uint32_t kBytes = kOffP + NT * kTileP + 1024;  // + alignment slack
  // tensor memory: the S buffers, then NT accumulators, 2R columns each
  static constexpr uint32_t kColO = NSB * 2 * R;
  static constexpr uint32_t kUsed = (NSB + NT) * 2 * R;
  static constexpr uint32_t kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  // CTAs an SM holds: shared memory (8 KB of it for the static part and the
  // driver's), tensor memory and 24 warps at 80 registers (28 at 72)
  static constexpr int kPerSM =
      2 * (kBytes + 8192) <= 228 * 1024 && threads(Load::kPages) <= 384 && kCols <= 256 ? 2 : 1;
  static_assert(kUsed <= 512 && kRowsQ >= 1, "tensor memory; a row of Q for every warp");
  static_assert(NT * R * 512 <= NS * (int)kFbTile, "the accumulators reuse the K ring");
};

// Instruction descriptor of tcgen05.mma.kind::f8f6f4 with E4M3 operands and fp32
// accumulation: bits 4-5 D format (1 = f32), 7-9 and 10-12 the A and B formats
// (0 = E4M3), 15 and 16 A and B major (1 = MN), 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t instr_desc_e4m3_f32(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor of an MN-major 8-bit operand whose whole N extent is one
// row of SPAN bytes (16, 32, 64 or 128), one row per k, swizzled over the row;
// groups of 8 rows follow one another.  Layout field (bits 61-63): 0 none, 6 32-byte,
// 4 64-byte, 2 128-byte swizzle.  Without a swizzle the leading offset strides the
// groups, with one the stride offset does: both are given.
template <int SPAN>
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  constexpr uint64_t layout = SPAN == 128 ? 2 : SPAN == 64 ? 4 : SPAN == 32 ? 6 : 0;
  constexpr uint64_t stride = (8 * SPAN) >> 4;
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (stride << 16) | (stride << 32) |
         (1ull << 46) | (layout << 61);
}
// Offset of byte `at` in such an operand: 16-byte pieces of a row are swizzled.
template <int SPAN>
__device__ __forceinline__ uint32_t swz_row(uint32_t at) {
  if constexpr (SPAN == 16) return at;
  else return swizzle<SPAN>(at);
}

// Issued by one lane (the caller's): D[tmem] (+)= A[smem] * B[smem], and the arrival
// on `bar` once everything this lane has issued is complete.
__device__ __forceinline__ void tc_mma_f8_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void tc_commit_one(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(e));
  return e != 0;
}

// 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[16]) {
  tmem_st16(taddr, r);
}
// Orders later uses of registers written by tmem_ld_cols after tmem_wait_ld.
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// (lo, hi) fp32 to two E4M3 codes, lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two f16 values to two E4M3 codes.
__device__ __forceinline__ uint32_t pack_e4m3x2(uint32_t f16x2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
  return r;
}

// Sums v[0..N-1] over the 32 lanes, N a power of two: each step halves the
// values a lane holds.  Lane l ends with the total of value l >> (5 - log2 N)
// (the steps take the lane bits from the highest down).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  int off = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
    off >>= 1;
  }
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}
// Whether the phase of `bar` has completed, for the whole (converged) warp: one
// elected lane waits (as long as the hardware lets it), since the lanes' tests of
// one barrier run one after another, and a vote hands on what it has acquired.
__device__ __forceinline__ bool warp_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t"
      "setp.ne.u32 p, %1, %1;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.any.pred q, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) __syncwarp();
  return ok != 0;
}
// One elected lane of the (converged) warp arms a barrier, or issues a copy.
__device__ __forceinline__ void expect_tx_elect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_elect(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                  int c0, int c1, int c2, uint64_t pol) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
      : "memory");
}
// Barrier `id` over `count` threads that returns whether any of them gave true.
__device__ __forceinline__ bool named_bar_any(int id, int count, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "bar.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The terms of a block's scales: the key scale; log2 of the value scale and its
// inverse (value scales below 2^-100 count as zero: a log2 of -100, and the weights'
// bytes masked away; negative ones are NaN).
struct __align__(16) ScaleTerms {
  float ks, lv, ivs;
  uint32_t p_mask;
};
__device__ __forceinline__ ScaleTerms scale_terms(float ks, float vs) {
  ScaleTerms s;
  const bool live = vs >= kMinVScale;
  s.ks = ks;
  float lg;  // (to 2^-22; exact for powers of two)
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(vs));
  s.lv = live ? lg : (vs >= 0.f ? -100.f : NAN);
  // 1 / vs, of the same logarithm. Where lv is NaN the weights carry it to the rows that see
  // the block; those that do not have weights of zero, which a NaN here would make NaN.
  // (Not ex2_approx, which flushes: the inverse of a scale above 2^126 is subnormal.)
  s.ivs = 1.f;
  if (vs >= 0.f) asm("ex2.approx.f32 %0, %1;" : "=f"(s.ivs) : "f"(-s.lv));
  s.p_mask = vs >= 0.f && !live ? 0u : 0xffffffffu;
  return s;
}

template <typename Sh, Load LOAD, bool CUT>
__global__ void __launch_bounds__(Sh::threads(LOAD), Sh::kPerSM)
    gqa_decode_fp8_block_kernel(const __grid_constant__ CUtensorMap tm_k,
                                const __grid_constant__ CUtensorMap tm_v,
                                const DecodeBlockParams pb) {
  constexpr int R = Sh::R, NS = Sh::NS, NT = Sh::NT, NG = Sh::NG, RW = Sh::RW, NSB = Sh::NSB;
  constexpr bool PAGED = LOAD != Load::kTile;
  const DecodeParams& p = pb.dec;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  __shared__ __align__(8) uint64_t s_full[NSB], s_empty[NSB], q_ready, p_ready[NT], o_full[NT],
      drain[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag, bad_page, nan_seen;
  // NaN codes in V of the keys that only some queries see (at most T_q - 1 <= 63), a
  // bit for each byte of the row
  __shared__ __align__(16) uint32_t nan_v[64][4];
  __shared__ __align__(16) float cq[R];         // tau log2(e) 2^-k of each row's query
  __shared__ __align__(16) int lim_sm[R];       // keys below it are visible
  __shared__ uint32_t row_sm[R];                // row of out, lse and the workspace
  __shared__ __align__(16) float red[NT][R][4]; // by stream: maxima of four warps
  // each softmax warp's own copy: its rows' changes of reference and factors
  __shared__ __align__(16) float move_sm[Sh::kWarps][RW], alpha_sm[Sh::kWarps][RW];
  __shared__ __align__(16) float off_sm[Sh::kWarps][RW];  // 7 less each row's reference
  // final sums of l (of four warps) and references
  __shared__ __align__(16) float l_end[NT][R][4];
  __shared__ float m_end[NT][R];
  // What the softmax needs of the scales: a ring of 8 rounds of 32 terms, by tile, head
  // and block of tokens of the tile.
  constexpr int kScRounds = 8, kScRing = 32 * kScRounds;
  __shared__ ScaleTerms sc_sm[kScRing];
  __shared__ __align__(8) uint64_t sc_full[kScRounds];
  __shared__ float fall_sm[kScRounds];  // how far a reference may fall, by round
  __shared__ float most_sm[Sh::kWarps][RW];  // a row's highest reference before it fell

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int split = blockIdx.x, b = blockIdx.z, chunk = p.chunk;
  // KV heads hc blockIdx.y + 0 .. hc - 1 share the 128-byte rows of a tile (hc = 4 packed
  // heads of d = 32, or 1).  Head hl has the query rows r = hl rp + q, q < T_q * G.
  const int hc = pb.heads, rp = pb.head_rows, kv0 = blockIdx.y * hc;
  // first key of the split (rows of a cache are below 2^31 - 256, so keys of a
  // tile past its end still fit)
  int t0 = static_cast<int>(min((long long)split * chunk, (long long)p.S_max));
  const int G = p.G, rows = p.T_q * G;  // of a head
  const int D = p.d;
  // Head of row r (rows past the last head's count as its padding).
  auto head_of = [&](int r) {
    return hc == 1 ? 0 : (r >= rp) + (r >= 2 * rp) + (r >= 3 * rp);
  };
  auto live_row = [&](int r) {
    return r - head_of(r) * rp < rows;
  };
  // r / G without an integer division, as in decode.cu
  const float inv_g = 1.f / static_cast<float>(G);
  auto query_of = [&](int r) {
    return static_cast<int>((static_cast<float>(r - head_of(r) * rp) + 0.5f) * inv_g);
  };
  auto out_row = [&](int r) -> uint32_t {  // of a live row (B * T_q and H_q are below 2^16)
    const int hl = head_of(r), t = query_of(r);
    return static_cast<uint32_t>(b * p.T_q + t) * p.H_q + (kv0 + hl) * G + (r - hl * rp - t * G);
  };
  const size_t n_rows = (size_t)p.B * p.T_q * p.H_q;

  // Tile coordinates: packed heads are 128 bytes of the whole row of H_kv d codes,
  // a head by itself is an index (the map then fills its 128-byte rows with zeros).
  const int tx = hc == 1 ? 0 : static_cast<int>(blockIdx.y) * 128, ty = hc == 1 ? kv0 : 0;

  // Set-up that touches no global memory runs before the dependency wait.
  volatile int* abort_v = &abort_flag;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int s = 0; s < NSB; ++s) {
      mbar_init(smem_u32(&s_full[s]), 1);
      mbar_init(smem_u32(&s_empty[s]), 4 * NG);
    }
    mbar_init(smem_u32(&q_ready), Sh::kWarps);
    for (int s = 0; s < NT; ++s) {
      mbar_init(smem_u32(&p_ready[s]), 4 * NG);
      mbar_init(smem_u32(&o_full[s]), 1);
    }
    for (int s = 0; s < kScRounds; ++s) mbar_init(smem_u32(&sc_full[s]), 1);
    mbar_init(smem_u32(&drain[0]), 1);
    mbar_init(smem_u32(&drain[1]), 1);
    abort_flag = 0;
    bad_page = 0;
    nan_seen = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), Sh::kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  // CUT, a batch cut by its lengths (a variant of its own, since what it keeps in registers
  // costs the others 1 us in 30): the cut is worked out while the previous kernel finishes,
  // from relaxed loads, and again after the dependency wait if a length has changed.
  Piece piece{0, 0, 0, 0};
  int cut_tiles[3] = {0, 0, 0};
  auto take_piece = [&]() {
    piece = find_piece(cut_tiles[0], cut_tiles[1], cut_tiles[2], p.B, p.n_split, pb.pieces,
                       blockIdx.x, lane);
    b = max(piece.b, 0);
    split = piece.split;
    chunk = piece.tiles * kFbKeys;
    t0 = split * chunk;
  };
  auto tiles_of = [&](int L) {
    return L < p.T_q || L > p.S_max ? 0 : (L + kFbKeys - 1) / kFbKeys;
  };
  if constexpr (CUT) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int L = 0;
      if (32 * k + lane < p.B)
        asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];"
                     : "=r"(L)
                     : "l"(p.seq_lens + 32 * k + lane));
      cut_tiles[k] = tiles_of(L);
    }
    take_piece();
  }
  // While the previous kernel finishes, the producer warp prefetches the split's
  // first tiles into L2, one box per lane (see decode.cu: the extent comes from
  // relaxed loads that only aim the prefetch; a prefetch hands over no data).
  if (warp == 0 && p.prefetch_tiles > 0) {
    const int h = PAGED ? min(p.page_size, kFbKeys) : kFbKeys;
    const int nb = kFbKeys / h;
    const int i = lane / nb, sub = lane % nb;
    int L_hint;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(L_hint) : "l"(p.seq_lens + b));
    const int tk = t0 + i * kFbKeys + sub * h;
    if (i < p.prefetch_tiles && tk < min(min(p.S_max, L_hint), t0 + min(chunk, p.S_max - t0))) {
      int row = b * p.S_max + tk;
      bool ok = true;
      if constexpr (PAGED) {
        int pg;
        asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];"
                     : "=r"(pg)
                     : "l"(p.block_table + (size_t)b * p.max_blocks + (tk >> pb.page_log2)));
        ok = pg >= 0 && pg < p.num_pages;
        row = pg * p.page_size + (tk & (p.page_size - 1));
      }
      if (ok) {
        tma_prefetch_l2_3d(&tm_k, tx, ty, row);
        tma_prefetch_l2_3d(&tm_v, tx, ty, row);
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (CUT) {
    bool changed = false;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int t = 32 * k + lane < p.B ? tiles_of(p.seq_lens[32 * k + lane]) : 0;
      changed |= t != cut_tiles[k];
      cut_tiles[k] = t;
    }
    if (__any_sync(0xffffffffu, changed)) take_piece();
    // the slots of the workspace that the sequence has no pieces for: the merge identity
    if (piece.b >= 0 && split == piece.count - 1)
      for (int r = warp; r < R; r += Sh::threads(LOAD) / 32)
        for (int i = piece.count + lane; live_row(r) && i < p.n_split; i += 32) {
          const size_t at = (size_t)out_row(r) * p.n_split + i;
          if (in_bounds(at, 1, n_rows * p.n_split, p.err))
            p.ws_ml[at] = make_float2(-INFINITY, 0.f);
        }
  }
  const bool none = piece.b < 0;  // a CTA past the batch's last piece
  // The softmax warps' rows of Q travel together with the length: row sw, sw +
  // kWarps, ..; lane takes columns 4 lane .. 4 lane + 3.
  const int sw = warp - 4;
  uint2 qw[Sh::kRowsQ];
  if (sw >= 0 && sw < Sh::kWarps) {
#pragma unroll
    for (int i = 0; i < Sh::kRowsQ; ++i) {
      const int r = sw + i * Sh::kWarps;
      qw[i] = make_uint2(0u, 0u);
      if (lane * 4 < D && live_row(r))
        qw[i] = *reinterpret_cast<const uint2*>(p.q + (size_t)out_row(r) * D + lane * 4);
    }
  }
  const int L = p.seq_lens[b];
  const bool bad = L < p.T_q || L > p.S_max;  // (L >= T_q >= 1 otherwise)
  const int t_end = bad || none ? 0 : min(t0 + min(chunk, p.S_max - t0), L);
  const int n = t_end > t0 ? (t_end - t0 + kFbKeys - 1) / kFbKeys : 0;
  if (bad || n == 0) {
    // A bad length: NaN outputs and the error bit.  An empty split: the merge
    // identity (-inf, 0); its O is not written.  (One split is never empty.)
    if (bad && threadIdx.x == 0 && split == 0 && kv0 == 0) atomicOr(p.err, kErrBadSeqLen);
    for (int r = threadIdx.x; r < R; r += Sh::threads(LOAD)) {
      if (none || !live_row(r)) continue;
      const size_t row = out_row(r);
      if (p.n_split == 1) {
        if (in_bounds(row * D, D, n_rows * D, p.err))
          for (int c = 0; c < D; ++c) p.out[row * D + c] = __float2bfloat16(NAN);
        if (in_bounds(row, 1, n_rows, p.err)) p.lse[row] = NAN;
      } else if (in_bounds(row * p.n_split + split, 1, n_rows * p.n_split, p.err)) {
        p.ws_ml[row * p.n_split + split] =
            bad ? make_float2(NAN, NAN) : make_float2(-INFINITY, 0.f);
      }
    }
    if (warp == 1) tmem_dealloc(tmem, Sh::kCols);
    return;
  }

  // A bounded wait of a whole warp that also gives up once another role has
  // aborted.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t addr = smem_u32(bar);
    if (warp_try_wait(addr, parity)) return true;
    const uint64_t since = globaltimer_ns();
#pragma unroll 1
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 32; ++i)
        if (warp_try_wait(addr, parity)) return true;
      const bool late = globaltimer_ns() - since > p.wait_ns;
      if (__any_sync(0xffffffffu, late || *abort_v != 0)) {
        if (lane == 0 && *abort_v == 0) atomicOr(p.err, kErrTimeout);
        __syncwarp();
        *abort_v = 1;
        return false;
      }
    }
  };

  // The same for the one lane that runs an issuer.
  auto wait_one = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t addr = smem_u32(bar);
    if (mbar_try_wait(addr, parity)) return true;
    const uint64_t since = globaltimer_ns();
#pragma unroll 1
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(addr, parity)) return true;
      if (*abort_v != 0) return false;
      if (globaltimer_ns() - since > p.wait_ns) {
        atomicOr(p.err, kErrTimeout);
        *abort_v = 1;
        return false;
      }
    }
  };
  // Rounds of the scales' terms: per_tile of them belong to a tile (a power of two),
  // so a round covers 1 << round_log2 tiles.
  const int sub_log2 = 7 - pb.block_log2;
  const int per_tile_log2 = sub_log2 + (hc == 1 ? 0 : 2);
  const int round_log2 = 5 - per_tile_log2;

  constexpr int kSecond = 4 + Sh::kWarps;  // second producers, of small pages
  if (warp == 0 || warp == 3 || (LOAD == Load::kSmallPages && warp >= kSecond)) {
    // ---------------------------------------------- TMA producers of K and V --
    const bool is_k = warp == 0 || warp == kSecond;
    const bool second = LOAD == Load::kSmallPages && warp >= kSecond;
    const CUtensorMap* const map = is_k ? &tm_k : &tm_v;
    uint64_t* const full = is_k ? k_full : v_full;
    uint64_t* const empty = is_k ? k_empty : v_empty;
    const uint32_t ring = sb + (is_k ? 0u : Sh::kOffV);
    if (lane == 0) tma_prefetch_map(map);
    const int h = PAGED ? min(p.page_size, kFbKeys) : kFbKeys;
    const int nb = kFbKeys / h;  // boxes of a tile, <= 8 (page_size >= 16)
    // Rows of 32 boxes at a time, one per lane, their pages loaded a round before
    // they are used (a round is 4 to 32 tiles).  A box past the end of the split, or
    // of a page outside the pool, reads rows past the pool, which TMA fills with
    // zeros, so that every tile receives its bytes; a bad index is recorded before
    // the barrier of any of its boxes is armed.
    auto fetch = [&](int tile) -> int {  // this lane's page, -1 for none
      const int tok = t0 + tile * kFbKeys + lane * h;
      return PAGED && tok < t_end
                 ? p.block_table[(size_t)b * p.max_blocks + (tok >> pb.page_log2)] : -1;
    };
    auto row_of = [&](int tile, int pg) -> int {
      const int tok = t0 + tile * kFbKeys + lane * h;
      const bool in = pg >= 0 && pg < p.num_pages;
      if (__any_sync(0xffffffffu, tok < t_end && !in) && lane == 0) {
        if (!*reinterpret_cast<volatile int*>(&bad_page)) atomicOr(p.err, kErrBadPage);
        *reinterpret_cast<volatile int*>(&bad_page) = 1;
      }
      __syncwarp();
      return tok < t_end && in ? pg * p.page_size + (tok & (p.page_size - 1))
                               : p.num_pages * p.page_size;
    };
    // V's producer works out the scales' terms of a round at a time, one per lane: lane
    // is tile, then head, then block of the tile.  Pages are loaded two rounds
    // ahead, scales one (terms of one tile at a time take a warp longer than a tile).
    const int sc_tile = lane >> per_tile_log2;
    const int sc_in = lane & ((1 << per_tile_log2) - 1);
    const int sc_kv = kv0 + (sc_in >> sub_log2);
    auto sc_tok = [&](int tile) {
      return t0 + (tile + sc_tile) * kFbKeys + ((sc_in & ((1 << sub_log2) - 1)) << pb.block_log2);
    };
    auto sc_unit = [&](int tile) -> int {  // its page (or sequence), -1 for none
      if (is_k || second || tile + sc_tile >= n) return -1;
      const int tok = sc_tok(tile);
      if (tok >= t_end) return -1;
      if (!PAGED) return b;
      const int pg = p.block_table[(size_t)b * p.max_blocks + (tok >> pb.page_log2)];
      return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    auto sc_load = [&](int tile, int unit) -> float2 {
      if (unit < 0) return make_float2(1.f, 1.f);
      const int tok = sc_tok(tile), in = PAGED ? tok & (p.page_size - 1) : tok;
      const size_t i = ((size_t)unit * pb.per_blk + (in >> pb.block_log2)) * p.H_kv + sc_kv;
      return make_float2(pb.k_scale[i], pb.v_scale[i]);
    };
    float2 scales = sc_load(0, sc_unit(0));
    int sc_u = sc_unit(1 << round_log2);
    const uint64_t pol = l2_policy_evict_first();  // every tile is read once
    const int box0 = second ? nb / 2 : 0;
    const int box1 = LOAD == Load::kSmallPages && !second ? nb / 2 : nb;
    int pages = fetch(32 / nb), rows_l = PAGED ? row_of(0, fetch(0)) : 0, at = 0, slot = 0;
    uint32_t parity = 0;  // of the slot's present use
    int issued = 0;
    float fall_most = kFallMost;  // (V's producer)
    for (int j = 0; j < n; ++j) {
      if (PAGED && at == 32) {  // a round has passed
        rows_l = row_of(j, pages);
        pages = fetch(j + 32 / nb);
        at = 0;
      }
      if (j >= NS && !wait_all(&empty[slot], parity ^ 1)) break;
      const uint32_t fb = smem_u32(&full[slot]), dst = ring + slot * kFbTile;
      // The whole warp runs the copies and one elected lane issues them, which keeps
      // their operands uniform (box i from lane i took a diverged warp's branches:
      // 16-token pages of a 64 x 4K batch 37.6 instead of 33.1 us).
      // The first of two producers arms the barrier; bytes may arrive before that.
      if (!second) expect_tx_elect(fb, kFbTile);
      if constexpr (!PAGED) {
        tma_load_3d_elect(dst, map, fb, tx, ty, b * p.S_max + t0 + j * kFbKeys, pol);
      } else {
#pragma unroll 1
        for (int i = box0; i < box1; ++i)
          tma_load_3d_elect(dst + i * h * 128, map, fb, tx, ty,
                            __shfl_sync(0xffffffffu, rows_l, at + i), pol);
      }
      issued = j + 1;
      if (!is_k && !second && (j & ((1 << round_log2) - 1)) == 0) {
        // A round of terms.  What lies in its place belongs to tiles before j - 7
        // rounds, which the softmax is done with: V's slot of tile j - NS is empty.
        const int round = j >> round_log2;
        sc_sm[(round % kScRounds) * 32 + lane] = scale_terms(scales.x, scales.y);
        if (__any_sync(0xffffffffu, scales.y < kFallScale)) fall_most = 0.f;
        if (lane == 0) fall_sm[round % kScRounds] = fall_most;
        scales = sc_load(j + (1 << round_log2), sc_u);
        sc_u = sc_unit(j + (2 << round_log2));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sc_full[round % kScRounds]));
      }
      at += nb;
      if (++slot == NS) {
        slot = 0;
        parity ^= 1;
      }
    }
    if (lane == 0) {
      // The next kernel may be scheduled; it waits for this grid before it reads.
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // No copy may still target shared memory when the CTA exits.
      for (int j = max(0, issued - NS); j < issued; ++j)
        mbar_wait(smem_u32(&full[j % NS]), (j / NS) & 1, p.wait_ns, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ S issuer --
    // S_j = K_j Q^T into buffer j % NSB, once K_j is there and S_{j - NSB} was read.
    // Packed heads: head hl's columns of K against its rows of Q, into its columns.
    const uint64_t dk = smem_desc_sw128(sb, 16, 1024);  // slot 0; an offset adds to the address
    const uint64_t dq = smem_desc_sw128(sb + Sh::kOffQ, 16, 1024);
    const int ksteps = D / 32;  // of a head: 32 columns of d each
    const uint32_t id = instr_desc_e4m3_f32(128, hc == 1 ? 2 * R : 2 * rp, false, false);
    const uint32_t id_last = instr_desc_e4m3_f32(128, 2 * (R - (hc - 1) * rp), false, false);
    if (elect_one()) {
      bool ok = wait_one(&q_ready, 0);
      int slot = 0, buf = 0;
      uint32_t parity = 0, bparity = 0;
      for (int j = 0; ok && j < n; ++j) {
        ok = wait_one(&k_full[slot], parity) &&
             (j < NSB || wait_one(&s_empty[buf], bparity ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t dkj = dk + slot * (kFbTile >> 4);
        const uint32_t ts = tmem + 2 * R * buf;
        if (hc == 1) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < ksteps) tc_mma_f8_one(ts, dkj + kk * 2, dq + kk * 2, id, kk > 0);
        } else {
#pragma unroll 1
          for (int hl = 0; hl < 4; ++hl)
            tc_mma_f8_one(ts + hl * 2 * rp, dkj + hl * 2, dq + hl * (2 * rp * 128 >> 4),
                          hl == 3 ? id_last : id, false);
        }
        tc_commit_one(smem_u32(&s_full[buf]));
        tc_commit_one(smem_u32(&k_empty[slot]));
        if (++slot == NS) {
          slot = 0;
          parity ^= 1;
        }
        if (++buf == NSB) {
          buf = 0;
          bparity ^= 1;
        }
      }
      // Every MMA issued here has completed before tensor memory is released.
      tc_commit_one(smem_u32(&drain[0]));
      mbar_wait(smem_u32(&drain[0]), 0, p.wait_ns, p.err);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ O issuer --
    // O^T (+)= V_j^T P_j in accumulator j % NT, once both are there (P_j is written
    // after the softmax has rescaled the accumulator, where it does).
    constexpr uint32_t idO = instr_desc_e4m3_f32(128, 2 * R, true, true);
    const uint64_t dv = smem_desc_sw128(sb + Sh::kOffV, kFbTile, 1024);
    const uint64_t dp = smem_desc_mn<Sh::kRowP>(sb + Sh::kOffP);
    if (elect_one()) {
      bool ok = true;
      int slot = 0, s = 0;
      uint32_t parity = 0, sparity = 0;
      for (int j = 0; ok && j < n; ++j) {
        ok = wait_one(&v_full[slot], parity) && wait_one(&p_ready[s], sparity);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dvj = dv + slot * (kFbTile >> 4), dpj = dp + s * (Sh::kTileP >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 keys each: four groups of 8 rows
          tc_mma_f8_one(tmem + Sh::kColO + 2 * R * s, dvj + kk * (4096 >> 4),
                        dpj + kk * (32 * Sh::kRowP >> 4), idO, kk > 0 || j >= NT);
        tc_commit_one(smem_u32(&o_full[s]));
        tc_commit_one(smem_u32(&v_empty[slot]));
        if (++slot == NS) {
          slot = 0;
          parity ^= 1;
        }
        if (++s == NT) {
          s = 0;
          sparity ^= 1;
        }
      }
      tc_commit_one(smem_u32(&drain[1]));
      mbar_wait(smem_u32(&drain[1]), 0, p.wait_ns, p.err);
    }
    __syncwarp();
  } else {
    // ------------------------------------------- softmax, accumulation, end --
    const int quarter = warp & 3;                // tensor-memory lanes 32 * quarter ..
    const int kl = quarter * 32 + lane;          // key of a tile; later, row d of O^T
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int gi = sw >> 2;                      // group of four warps
    const int st = gi / NG, r0 = (gi % NG) * RW;  // stream of tiles, first row
    // Column (and byte of P, and row of Q) of row r's high term; the low term's
    // is 8 further: eight rows' 16 columns are neighbours.
    auto col = [](int r) { return r / 8 * 16 + r % 8; };

    // Q as two E4M3 terms.
#pragma unroll
    for (int i = 0; i < Sh::kRowsQ; ++i) {
      const int r = sw + i * Sh::kWarps;
      const uint2 w = qw[i];
      const float f[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                          __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
      // the exponent of the largest |q| (bf16 bits); an infinity or NaN makes the row NaN
      uint32_t a = max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu),
                       max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
      a = __reduce_max_sync(0xffffffffu, a);
      // |q| 2^k < 256: k = 7 - exponent, kept within the range of normal fp32
      const int k = max(-120, min(120, 7 - (static_cast<int>(a >> 7) - 127)));
      const float up = __int_as_float((k + 127) << 23);
      float lo[4];
      uint32_t hi[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float u = f[2 * e] * up, v = f[2 * e + 1] * up;
        hi[e] = pack_e4m3x2(u, v);
        const float2 g = unpack_e4m3x2(hi[e]);
        lo[2 * e] = (u - g.x) * 32.f;
        lo[2 * e + 1] = (v - g.y) * 32.f;
      }
      const int nh = col(r), nl = nh + 8, c = lane >> 2, in = (lane & 3) * 4;
      st_shared_u32(sb + Sh::kOffQ + nh * 128 + ((c ^ (nh & 7)) << 4) + in, hi[0] | (hi[1] << 16));
      st_shared_u32(sb + Sh::kOffQ + nl * 128 + ((c ^ (nl & 7)) << 4) + in,
                    pack_e4m3x2(lo[0], lo[1]) | (pack_e4m3x2(lo[2], lo[3]) << 16));
      if (lane == 0) {
        cq[r] = a >= 0x7f80u ? NAN : p.scale_log2 * __int_as_float((127 - k) << 23);
        const bool live = live_row(r);
        lim_sm[r] = live ? min(t_end, L - p.T_q + 1 + query_of(r)) : t_end;
        row_sm[r] = live ? out_row(r) : 0xffffffffu;  // (no row of an output: H_q is below 2^16)
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&q_ready));

    // Where the scales' terms of this thread's key lie among a tile's, for each eight
    // rows (one head's).
    constexpr int RU = RW / 8;
    int sc_at[RU];
#pragma unroll
    for (int c = 0; c < RU; ++c)
      sc_at[c] = (head_of(r0 + 8 * c) << sub_log2) + (kl >> pb.block_log2);
    float l[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) l[i] = 0.f;
    float m_mine = -INFINITY;  // reference of row r0 + lane (lanes below RW)
    if (lane < RW) {
      off_sm[sw][lane] = kPScaleLog2;  // (0 for a row without one)
      most_sm[sw][lane] = -INFINITY;
    }
    bool look = true;          // some row has no reference yet, or one that has just risen far
    const int lim_lo = min(t_end, L - p.T_q + 1);  // keys below it: visible from every row
    bool alive = true;
    const uint32_t tO = tmem + lane_base + Sh::kColO + 2 * R * st + 2 * r0;
    const uint32_t prow = sb + Sh::kOffP + st * Sh::kTileP;
    named_bar_sync(5, 32 * Sh::kWarps);  // cq, lim_sm, row_sm

    int turn = 0;  // tiles of this stream so far
    for (int j = st; j < n; j += NT, ++turn) {
      const int key = t0 + j * kFbKeys + kl;
      // (a warp whose wait failed keeps to the barriers of the others)
      if ((j & ((1 << round_log2) - 1)) < NT) {  // the stream's first tile of a round
        const int round = j >> round_log2;
        alive = alive && wait_all(&sc_full[round % kScRounds], (round / kScRounds) & 1);
      }
      alive = alive && wait_all(&s_full[j % NSB], (j / NSB) & 1);
      tc_fence_after();
      const ScaleTerms* const sc = sc_sm + (j << per_tile_log2) % kScRing;
      float y[RW];  // exponents of P: y - m + 7
      float top = -INFINITY;
      {
#pragma unroll
        for (int c0 = 0; c0 < RW; c0 += 8) {
          uint32_t s[16];
          tmem_ld_cols(tmem + lane_base + 2 * R * (j % NSB) + 2 * (r0 + c0), s);
          tmem_wait_ld();
          reg_fence(s);
          const float2 kl2 = *reinterpret_cast<const float2*>(&sc[sc_at[c0 / 8]]);  // ks, lv
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(&cq[r0 + c0 + i]);
            const float4 f4 = *reinterpret_cast<const float4*>(&off_sm[sw][c0 + i]);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              const int e = i + u, r = c0 + e;
              float a0, a1, b0, b1, d0, d1;
              ffma2(a0, a1, __uint_as_float(s[8 + e]), __uint_as_float(s[9 + e]), kLoStep, kLoStep,
                    __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
              fmul2(b0, b1, c[u], c[u + 1], kl2.x, kl2.x);
              fadd2(d0, d1, f[u], f[u + 1], kl2.y, kl2.y);
              ffma2(y[r], y[r + 1], a0, a1, b0, b1, d0, d1);
            }
          }
        }
        if (t0 + (j + 1) * kFbKeys > lim_lo) {
#pragma unroll
          for (int i = 0; i < RW; ++i)
            if (key >= lim_sm[r0 + i]) y[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < RW; i += 2) top = fmax3(top, y[i], y[i + 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (alive && lane == 0) mbar_arrive(smem_u32(&s_empty[j % NSB]));
      const bool update = named_bar_any(1 + gi, 128, look || top > kPMaxLog2);
      if (update) {
        // The rows' maxima over the 128 keys become references where they are
        // larger, or far smaller; lane i works out row r0 + i for its warp.
        float mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float m = warp_max(y[i]);
          if (lane == i) mine = m;
        }
        if (lane < RW) red[st][r0 + lane][quarter] = mine - off_sm[sw][lane];
        named_bar_sync(1 + gi, 128);
        bool rose = false;
        if (lane < RW) {
          const float4 mx = *reinterpret_cast<const float4*>(red[st][r0 + lane]);
          float m_new = fmax3(fmaxf(mx.x, mx.y), fmaxf(mx.z, mx.w), m_mine);
          if (look) {
            const float m_tile = fmaxf(fmaxf(mx.x, mx.y), fmaxf(mx.z, mx.w));
            const float most = fmaxf(most_sm[sw][lane], m_new);
            most_sm[sw][lane] = most;
            if (m_tile < m_mine - kFall && m_tile > -INFINITY)
              m_new = fminf(m_new, fmaxf(m_tile, most - fall_sm[(j >> round_log2) % kScRounds]));
          }
          rose = m_new > m_mine + kFall;
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // no (-inf) - (-inf)
          move_sm[sw][lane] = (m_mine == -INFINITY ? 0.f : m_mine) - ref;
          alpha_sm[sw][lane] = ex2_approx(m_mine - ref);
          off_sm[sw][lane] = kPScaleLog2 - ref;
          m_mine = m_new;
        }
        look = __any_sync(0xffffffffu, lane < RW && (rose || m_mine == -INFINITY));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < RW; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&move_sm[sw][i]);
          const float4 a = *reinterpret_cast<const float4*>(&alpha_sm[sw][i]);
          fadd2(y[i], y[i + 1], y[i], y[i + 1], f.x, f.y);
          fadd2(y[i + 2], y[i + 3], y[i + 2], y[i + 3], f.z, f.w);
          fmul2(l[i], l[i + 1], l[i], l[i + 1], a.x, a.y);
          fmul2(l[i + 2], l[i + 3], l[i + 2], l[i + 3], a.z, a.w);
        }
      }

      // The stream's previous O is complete: its P may be overwritten, and O rescaled
      // (row d = kl of O^T, both terms' columns).
      alive = alive && (turn == 0 || wait_all(&o_full[st], (turn - 1) & 1));
      tc_fence_after();
      if (update && turn > 0) {
#pragma unroll 1
        for (int c = 0; c < RW; c += 8) {
          uint32_t o[16];
          tmem_ld_cols(tO + 2 * c, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = alpha_sm[sw][c + i];
            o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            o[8 + i] = __float_as_uint(__uint_as_float(o[8 + i]) * a);
          }
          tmem_st_cols(tO + 2 * c, o);
        }
        tmem_wait_st();
      }
      // P as two E4M3 terms, rounded to f16 on the way (2^-12 of itself, and
      // steps of 2^-24 below 2^-14, both below what the terms hold).
      // Eight rows' two terms are 16 bytes of this key's row of P, swizzled over it.
#pragma unroll
      for (int c0 = 0; c0 < RW; c0 += 8) {
        uint32_t hi[2], lo[2];
        const float iv = sc[sc_at[c0 / 8]].ivs;
        const uint32_t mask = sc[sc_at[c0 / 8]].p_mask;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const int r = c0 + i;
          const float e0 = ex2_approx(y[r]), e1 = ex2_approx(y[r + 1]);
          const float e2 = ex2_approx(y[r + 2]), e3 = ex2_approx(y[r + 3]);
          ffma2(l[r], l[r + 1], e0, e1, iv, iv, l[r], l[r + 1]);
          ffma2(l[r + 2], l[r + 3], e2, e3, iv, iv, l[r + 2], l[r + 3]);
          uint32_t h[2], d[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = pack_f16x2(u ? e2 : e0, u ? e3 : e1);
            h[u] = pack_e4m3x2(x);
            const uint32_t g = e4m3x2_to_f16x2(h[u]);
            const __half2 q = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x),
                                              *reinterpret_cast<const __half2*>(&g)),
                                      __float2half2_rn(32.f));
            d[u] = pack_e4m3x2(*reinterpret_cast<const uint32_t*>(&q));
          }
          hi[i / 4] = (h[0] | (h[1] << 16)) & mask;
          lo[i / 4] = (d[0] | (d[1] << 16)) & mask;
        }
        st_shared_v4(prow + swz_row<Sh::kRowP>(kl * Sh::kRowP + 2 * (r0 + c0)), hi[0], hi[1], lo[0],
                     lo[1]);
      }
      // Cache rows past the end of the split may hold anything (even NaN codes),
      // and 0 * NaN would reach O: they are zeroed once the tile has landed (by
      // the stream's first row group).  So are the NaN codes of keys that only the
      // later queries see; the end of the kernel puts them into those queries' rows.
      if (t0 + (j + 1) * kFbKeys > lim_lo && r0 == 0) {
        alive = alive && wait_all(&v_full[j % NS], (j / NS) & 1);
        if (alive && key >= lim_lo) {
          uint4* const vrow = reinterpret_cast<uint4*>(smem + Sh::kOffV + (j % NS) * kFbTile + kl * 128);
          const bool past = key >= t_end;
          uint32_t any = 0;
#pragma unroll 1
          for (int c = 0; c < 4 && !past; ++c) {  // 32 bytes: two swizzled pieces
            uint32_t bits = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4* const at = vrow + ((2 * c + h) ^ (kl & 7));
              const uint4 w = *at;
              uint32_t x[4] = {w.x, w.y, w.z, w.w}, here = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t is = __vcmpeq4(x[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                x[i] &= ~is;
                // a bit of each byte of the mask, added up in the top byte
                here |= ((is & 0x08040201u) * 0x01010101u >> 24 & 15u) << (4 * i);
              }
              if (here != 0) *at = make_uint4(x[0], x[1], x[2], x[3]);
              bits |= here << (16 * h);
            }
            nan_v[key - (L - p.T_q + 1)][c] = bits;
            any |= bits;
          }
          if (any != 0) *reinterpret_cast<volatile int*>(&nan_seen) = 1;
          if (past) {
#pragma unroll
            for (int c16 = 0; c16 < 8; ++c16) vrow[c16] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (alive && lane == 0) mbar_arrive(smem_u32(&p_ready[st]));
    }

    // l over the keys, while the last O is worked out; then the stream's O.  It goes
    // through the K ring, so that a warp merges and stores whole rows: free once the
    // last S is complete (or the CTA has failed and writes NaN).
    {
      const float s = warp_sums(l, lane);
      if (lane % (32 / RW) == 0) l_end[st][r0 + lane / (32 / RW)][quarter] = s;
      if (quarter == 0 && lane < RW) m_end[st][r0 + lane] = m_mine;
    }
    alive = alive && wait_all(&s_full[(n - 1) % NSB], ((n - 1) / NSB) & 1) &&
            (turn == 0 || wait_all(&o_full[st], (turn - 1) & 1));
    if (PAGED && alive) {
      // (a bad index is recorded before the barrier of the last V tile is armed)
      alive = wait_all(&v_full[(n - 1) % NS], ((n - 1) / NS) & 1) &&
              *reinterpret_cast<volatile int*>(&bad_page) == 0;
    }
    if (!alive) *abort_v = 1;
    tc_fence_after();
    float* const part = reinterpret_cast<float*>(smem);  // [NT][R][128]
#pragma unroll 1
    for (int c = 0; c < RW; c += 8) {
      uint32_t o[16] = {};
      if (turn > 0) {
        tmem_ld_cols(tO + 2 * c, o);
        tmem_wait_ld();
        reg_fence(o);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[(st * R + r0 + c + i) * 128 + kl] =
            fmaf(__uint_as_float(o[8 + i]), kLoStep, __uint_as_float(o[i]));
    }
    named_bar_sync(5, 32 * Sh::kWarps);
    const bool failed = *abort_v != 0;
    constexpr float kUnscale = 1.f / 128.f;  // P carried 2^7
    for (int r = sw; r < R; r += Sh::kWarps) {
      if (row_sm[r] == 0xffffffffu) continue;
      // (head hl's O lies in rows hl D .. of O^T)
      const int at = r * 128 + min(head_of(r) * D + lane * 4, 124);
      const float4 ls = *reinterpret_cast<const float4*>(l_end[0][r]);
      float m = m_end[0][r], lr = (ls.x + ls.y) + (ls.z + ls.w);
      float4 o = *reinterpret_cast<const float4*>(part + at);
      if constexpr (NT == 2) {  // the merge of two partials
        const float4 l2 = *reinterpret_cast<const float4*>(l_end[1][r]);
        const float m1 = m_end[1][r], M = fmaxf(m, m1), ref = M == -INFINITY ? 0.f : M;
        const float a0 = ex2_approx(m - ref), a1 = ex2_approx(m1 - ref);
        const float4 o1 = *reinterpret_cast<const float4*>(part + R * 128 + at);
        lr = lr * a0 + ((l2.x + l2.y) + (l2.z + l2.w)) * a1;
        o = make_float4(o.x * a0 + o1.x * a1, o.y * a0 + o1.y * a1, o.z * a0 + o1.z * a1,
                        o.w * a0 + o1.w * a1);
        m = M;
      }
      if (*reinterpret_cast<volatile int*>(&nan_seen) != 0) {
        const int dim = at - r * 128;  // of four
        uint32_t bits = 0;
        for (int key = max(t0, lim_lo); key < lim_sm[r]; ++key)
          bits |= nan_v[key - (L - p.T_q + 1)][dim / 32];
        bits >>= dim % 32;
        if (bits & 1u) o.x = NAN;
        if (bits & 2u) o.y = NAN;
        if (bits & 4u) o.z = NAN;
        if (bits & 8u) o.w = NAN;
      }
      const size_t row = row_sm[r];
      if (p.n_split == 1) {
        const float inv = failed ? NAN : 1.f / lr;
        if (lane * 4 < D && in_bounds(row * D + lane * 4, 4, n_rows * D, p.err))
          *reinterpret_cast<uint2*>(p.out + row * D + lane * 4) =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (lane == 0 && in_bounds(row, 1, n_rows, p.err))
          p.lse[row] = failed ? NAN : (m + log2f(lr * kUnscale)) * kLn2;
      } else {
        const size_t idx = row * p.n_split + split;
        if (lane * 4 < D && in_bounds(idx * D + lane * 4, 4, n_rows * p.n_split * D, p.err))
          *reinterpret_cast<float4*>(p.ws_O + idx * D + lane * 4) =
              make_float4(o.x * kUnscale, o.y * kUnscale, o.z * kUnscale, o.w * kUnscale);
        // m in natural-log units; a row with no visible key: (-inf, 0)
        if (lane == 0 && in_bounds(idx, 1, n_rows * p.n_split, p.err))
          p.ws_ml[idx] =
              failed ? make_float2(NAN, NAN) : make_float2(m * kLn2, lr * kUnscale);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kCols);
  }
}

template <typename Sh, Load LOAD, bool CUT = false>
cudaError_t launch_fb(const DecodeBlockParams& p_in, const CUtensorMap& tm_k,
                      const CUtensorMap& tm_v, bool prefetch, cudaStream_t stream) {
  auto kern = gqa_decode_fp8_block_kernel<Sh, LOAD, CUT>;
  constexpr int smem = Sh::kBytes;
  static unsigned char done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {  // benign race: idempotent
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  DecodeBlockParams p = p_in;
  p.dec.prefetch_tiles = prefetch ? 3 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.pieces > 0 ? dim3(p.pieces, p.dec.H_kv / p.heads)
                             : dim3(p.dec.n_split, p.dec.H_kv / p.heads, p.dec.B);
  cfg.blockDim = dim3(Sh::threads(LOAD));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename Deep, typename Shallow>
cudaError_t launch_fb_r(const DecodeBlockParams& p, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, int sms, cudaStream_t stream) {
  // One CTA per SM at most: a deep ring, and the first tiles prefetched into L2 while
  // the previous kernel ends.  More CTAs than SMs: two shallow rings on each SM (8 rows;
  // the larger shapes hold one CTA per SM either way).
  const bool one_wave = (long long)p.dec.n_split * p.dec.B * (p.dec.H_kv / p.heads) <= sms;
  if constexpr (Deep::R > 16) {
    if (p.pieces > 0) {  // at most one CTA per SM
      return p.dec.block_table == nullptr
                 ? launch_fb<Deep, Load::kTile, true>(p, tm_k, tm_v, true, stream)
                 : launch_fb<Deep, Load::kPages, true>(p, tm_k, tm_v, true, stream);
    }
  }
  if (p.dec.block_table == nullptr)
    return one_wave ? launch_fb<Deep, Load::kTile>(p, tm_k, tm_v, true, stream)
                    : launch_fb<Shallow, Load::kTile>(p, tm_k, tm_v, false, stream);
  if constexpr (Deep::R <= 32) {
    if (p.dec.page_size == kSmallPage)
      return one_wave ? launch_fb<Deep, Load::kSmallPages>(p, tm_k, tm_v, true, stream)
                      : launch_fb<Shallow, Load::kSmallPages>(p, tm_k, tm_v, false, stream);
  }
  return one_wave ? launch_fb<Deep, Load::kPages>(p, tm_k, tm_v, true, stream)
                  : launch_fb<Shallow, Load::kPages>(p, tm_k, tm_v, false, stream);
}

}  // namespace

cudaError_t launch_decode_fp8_block(const DecodeBlockParams& p, const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, int sms, cudaStream_t stream) {
  const int rows = p.heads == 1 ? p.dec.T_q * p.dec.G : p.heads * p.head_rows;
  if (rows < 1 || rows > 64 || p.dec.chunk % kFbKeys != 0) return cudaErrorInvalidValue;
  if (p.pieces > 0 && (rows <= 16 || p.pieces <= p.dec.B || p.dec.B > kMaxCut))
    return cudaErrorInvalidValue;
  if (rows <= 8)
    return launch_fb_r<FbShape<8, 6, 2, 1>, FbShape<8, 3, 2, 1>>(p, tm_k, tm_v, sms, stream);
  if (rows <= 16)
    return launch_fb_r<FbShape<16, 6, 2, 2>, FbShape<16, 6, 2, 2>>(p, tm_k, tm_v, sms, stream);
  if (rows <= 32)
    return launch_fb_r<FbShape<32, 5, 2, 2>, FbShape<32, 5, 2, 2>>(p, tm_k, tm_v, sms, stream);
  return launch_fb_r<FbShape<64, 5, 1, 4>, FbShape<64, 5, 1, 4>>(p, tm_k, tm_v, sms, stream);
}

}  // namespace gqa
