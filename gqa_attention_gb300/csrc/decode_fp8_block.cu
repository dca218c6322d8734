// decode_fp8_block.cu -- split-KV decode over the block-scaled E4M3 cache on the
// fifth-generation tensor cores, the codes taken as they lie in memory.
//
// What it computes, for the T_q last positions of each sequence (row r of a KV
// head is query t = r / G of head kv G + r % G and sees keys below L - T_q + 1 + t):
//   x_j = tau ks_j (q . kc_j),  O = sum_j 2^.. softmax(x)_j vs_j vc_j,  LSE = ln sum_j e^x_j
// with kc, vc the E4M3 values and ks_j, vs_j the scales of key j's block of
// tokens.  One CTA per (split, KV head, sequence) leaves the partial (m, l, O)
// of decode.cu's layout for the combine kernel, or writes O and LSE (one split).
//
// Keys sit in the M rows of the MMA, query rows in N:
//   S_j = K_j Q^T   (M = 128 keys, N = 2R, K = d; both operands in shared memory)
//   O^T = V_j^T P   (M = d, N = 2R, K = 128 keys; V^T is the MN-major view of V)
// so that a thread owns one key: its scales are one register each, its exponents
// R, and a padded row costs no softmax work.  With the rows in M, as decode_tc.cu
// has them, 8 query rows would leave 120 of 128 lanes idle and one warp with all
// 128 exponentials of each row.
//
// kind::f8f6f4 wants both operands in 8 bits, so Q and P are split in two E4M3
// terms, side by side in N (rows 0..R-1 the high terms, R..2R-1 the low):
//   q 2^k = hi + lo / 32.  bf16 carries 8 significant bits and E4M3 four, so the
//     split is exact down to 2^-21 of the row's largest |q| (hi <= 256, so the
//     remainder is at most 8 and 32 times it at most 256).
//   p in (0, 256] = hi + lo / 32, within 2^-9 of p above 2^-6 as bf16 would be,
//     with a smallest step of 2^-14: 2^-22 of the reference weight.
// The codes need no conversion, which is what bounds the mma.sync sweep over
// E4M3 codes.
//
// The value scale rides on the exponent: y_j = x_j log2 e + log2 vs_j, P = 2^(y - m + 8)
// with m the running maximum of y over the split, and l sums P / vs_j in fp32.  So
// the range of P adapts to vs as well as to the scores.  m is a reference, not
// the maximum of x; the merge of the partials holds for any reference.
//
// Each P V starts a fresh accumulator that the softmax threads (now thread = row
// d of O^T) add to fp32 registers, rescaled by 2^(m_old - m_new): no
// rescaling pass through tensor memory, and the sum over tiles is fp32.
//
// Roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer (and tensor
// memory), warps 2-5 Q split, softmax, accumulation and epilogue.
#include "tcgen05.cuh"

namespace gqa {
namespace {

constexpr int kFbThreads = 192;
constexpr int kFbKeys = 128;                // keys per tile
constexpr uint32_t kFbTile = 128u * 128u;   // 128 rows of 128 bytes
constexpr float kLoStep = 1.f / 32.f;       // weight of the low term
constexpr float kPScaleLog2 = 8.f;          // P is held times 2^8
constexpr float kMinVScale = 7.888609052210118e-31f;  // 2^-100

template <int R, int NS>
struct FbLayout {
  static constexpr uint32_t kOffV = NS * kFbTile;
  static constexpr uint32_t kOffQ = 2 * NS * kFbTile;
  static constexpr uint32_t kOffP = kOffQ + 2 * R * 128;
  static constexpr uint32_t kBytes = kOffP + 2 * R * 128 + 1024;  // + alignment slack
  static constexpr uint32_t kCols = R == 8 ? 64 : R == 16 ? 128 : R == 32 ? 256 : 512;
  static constexpr uint32_t kColO = 4 * R;  // S_0, S_1 (2R columns each), then O
  static constexpr int kChunk = R < 16 ? R : 16;  // rows handled at once
  static constexpr int kPerSM = 2 * (kBytes + 2048) <= 227 * 1024 ? 2 : 1;
};

// Instruction descriptor of tcgen05.mma.kind::f8f6f4 with E4M3 operands and fp32
// accumulation: bits 4-5 D format (1 = f32), 7-9 and 10-12 the A and B formats
// (0 = E4M3), 15 A major (1 = MN), 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t instr_desc_e4m3_f32(int M, int N, bool a_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 8 or 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
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
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int R, int NS, bool PAGED>
__global__ void __launch_bounds__(kFbThreads, FbLayout<R, NS>::kPerSM)
    gqa_decode_fp8_block_kernel(const __grid_constant__ CUtensorMap tm_k,
                                const __grid_constant__ CUtensorMap tm_v,
                                const DecodeBlockParams pb) {
  using Lay = FbLayout<R, NS>;
  constexpr int RC = Lay::kChunk;
  constexpr int NC = R / RC;
  const DecodeParams& p = pb.dec;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  __shared__ __align__(8) uint64_t s_full[2], q_ready, p_ready, o_full, drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag, bad_page;
  __shared__ float cq[R];                       // tau log2(e) 2^-k of each row's query
  __shared__ int lim_sm[R];                     // keys below it are visible
  __shared__ __align__(16) float red[2][R][4];  // maxima of the four warps, by tile parity
  __shared__ float m_run[2][R];                 // running references, by tile parity

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, kv = blockIdx.y, b = blockIdx.z;
  // first key of the split (rows of a cache are below 2^31 - 256, so keys of a
  // tile past its end still fit)
  const int t0 = static_cast<int>(min((long long)split * p.chunk, (long long)p.S_max));
  const int G = p.G, rows = p.T_q * G;  // <= R
  const int D = p.d;
  auto out_row = [&](int r) -> size_t {
    return ((size_t)b * p.T_q + r / G) * p.H_q + kv * G + r % G;
  };
  const size_t n_rows = (size_t)p.B * p.T_q * p.H_q;
  // NaN outputs of a row (one split), or its partial (m, l) alone
  auto write_nan_or_ml = [&](size_t row, float2 ml) {
    if (p.n_split == 1) {
      if (in_bounds(row * D, D, n_rows * D, p.err))
        for (int c = 0; c < D; ++c) p.out[row * D + c] = __float2bfloat16(NAN);
      if (in_bounds(row, 1, n_rows, p.err)) p.lse[row] = NAN;
    } else if (in_bounds(row * p.n_split + split, 1, n_rows * p.n_split, p.err)) {
      p.ws_ml[row * p.n_split + split] = ml;
    }
  };

  // Set-up that touches no global memory runs before the dependency wait.
  volatile int* abort_v = &abort_flag;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    mbar_init(smem_u32(&s_full[0]), 1);
    mbar_init(smem_u32(&s_full[1]), 1);
    mbar_init(smem_u32(&q_ready), 4);
    mbar_init(smem_u32(&p_ready), 4);
    mbar_init(smem_u32(&o_full), 1);
    mbar_init(smem_u32(&drain), 1);
    abort_flag = 0;
    bad_page = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), Lay::kCols);
    tmem_relinquish();
    tc_fence_before();
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
    if (i < p.prefetch_tiles && tk < min(min(p.S_max, L_hint), t0 + min(p.chunk, p.S_max - t0))) {
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
        tma_prefetch_l2_3d(&tm_k, 0, kv, row);
        tma_prefetch_l2_3d(&tm_v, 0, kv, row);
      }
    }
  }

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = p.seq_lens[b];
  const bool bad = L < p.T_q || L > p.S_max;  // (L >= T_q >= 1 otherwise)
  const int t_end = bad ? 0 : min(t0 + min(p.chunk, p.S_max - t0), L);
  const int n = t_end > t0 ? (t_end - t0 + kFbKeys - 1) / kFbKeys : 0;
  if (threadIdx.x >= 64) {
    for (int r = threadIdx.x - 64; r < R; r += 128) {
      lim_sm[r] = r < rows ? min(t_end, L - p.T_q + 1 + r / G) : t_end;
      m_run[0][r] = -INFINITY;
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  if (bad || n == 0) {
    // A bad length: NaN outputs and the error bit.  An empty split: the merge
    // identity (-inf, 0); its O is not written.  (One split is never empty.)
    if (bad && threadIdx.x == 0 && split == 0 && kv == 0) atomicOr(p.err, kErrBadSeqLen);
    for (int r = threadIdx.x; r < rows; r += kFbThreads)
      write_nan_or_ml(out_row(r), bad ? make_float2(NAN, NAN) : make_float2(-INFINITY, 0.f));
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, Lay::kCols);
    }
    return;
  }

  // A bounded wait that also gives up once another role has aborted, taken by
  // every lane of a warp with one agreed result.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = mbar_try_wait(smem_u32(bar), parity);
    if (!ok && !*abort_v) {
      ok = mbar_wait(smem_u32(bar), parity, p.wait_ns, p.err);
      if (!ok) *abort_v = 1;
    }
    return __all_sync(0xffffffffu, ok);
  };

  if (warp == 0) {
    // ----------------------------------------------------------- TMA producer --
    // The whole warp runs the loop so that a tile's page indices are read in
    // parallel, one box per lane; lane 0 arms each barrier before any copy.
    if (lane == 0) {
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
    }
    const int h = PAGED ? min(p.page_size, kFbKeys) : kFbKeys;
    const int nb = kFbKeys / h;  // <= 8 (page_size >= 16)
    int issued_k = 0, issued_v = 0;
    auto fetch = [&](int j) -> int {  // this lane's page of tile j, -1 for none
      const int tok = t0 + j * kFbKeys + lane * h;
      if (!PAGED || lane >= nb || j >= n || tok >= t_end) return -1;
      const int pg = p.block_table[(size_t)b * p.max_blocks + (tok >> pb.page_log2)];
      return pg >= 0 && pg < p.num_pages ? pg : -2;  // -2: outside the pool
    };
    const uint64_t pol = l2_policy_evict_first();  // every tile is read once
    auto issue = [&](bool is_k, int j, int pg) -> bool {
      const int slot = j % NS;
      if (j >= NS && !wait_all(is_k ? &k_empty[slot] : &v_empty[slot], ((j / NS) - 1) & 1))
        return false;
      const uint32_t fb = smem_u32(is_k ? &k_full[slot] : &v_full[slot]);
      const uint32_t dst = sb + (is_k ? 0u : Lay::kOffV) + slot * kFbTile;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      const int tok0 = t0 + j * kFbKeys;
      if constexpr (!PAGED) {
        if (lane == 0) {
          mbar_arrive_expect_tx(fb, kFbTile);
          tma_load_3d(dst, map, fb, 0, kv, b * p.S_max + tok0, pol);
        }
      } else {
        // A box wholly past the end of the split reads rows past the pool,
        // which TMA fills with zeros, so that every tile receives its bytes; a
        // bad page index is recorded before lane 0's arrive releases it.
        const bool wrong = pg == -2;
        const int row = pg >= 0 ? pg * p.page_size + ((tok0 + lane * h) & (p.page_size - 1))
                                : p.num_pages * p.page_size;
        if (__any_sync(0xffffffffu, wrong) && lane == 0) {
          if (!*reinterpret_cast<volatile int*>(&bad_page)) atomicOr(p.err, kErrBadPage);
          *reinterpret_cast<volatile int*>(&bad_page) = 1;
        }
        if (lane == 0) mbar_arrive_expect_tx(fb, kFbTile);
        __syncwarp();
        if (lane < nb) tma_load_3d(dst + lane * h * 128, map, fb, 0, kv, row, pol);
      }
      return true;
    };
    int pg0 = fetch(0), pg1 = fetch(1);
    bool ok = true;
    for (int j = 0; ok && j < n; ++j) {
      const int pg2 = fetch(j + 2);
      ok = issue(true, j, pg0);
      if (ok) issued_k = j + 1;
      ok = ok && issue(false, j, pg0);
      if (ok) issued_v = j + 1;
      pg0 = pg1;
      pg1 = pg2;
    }
    if (lane == 0) {
      // The next kernel may be scheduled; it waits for this grid before it reads.
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // No copy may still target shared memory when the CTA exits.
      for (int j = max(0, issued_k - NS); j < issued_k; ++j)
        mbar_wait(smem_u32(&k_full[j % NS]), (j / NS) & 1, p.wait_ns, p.err);
      for (int j = max(0, issued_v - NS); j < issued_v; ++j)
        mbar_wait(smem_u32(&v_full[j % NS]), (j / NS) & 1, p.wait_ns, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer --
    constexpr uint32_t idS = instr_desc_e4m3_f32(128, 2 * R, false);
    constexpr uint32_t idO = instr_desc_e4m3_f32(128, 2 * R, true);
    const uint32_t qb = sb + Lay::kOffQ, ppb = sb + Lay::kOffP;
    const int ksteps = D / 32;
    auto issue_s = [&](int j) {  // S_j = K_j Q^T
      const uint32_t kb = sb + (j % NS) * kFbTile;
      for (int kk = 0; kk < ksteps; ++kk)
        tc_mma_f8_ss(tmem + 2 * R * (j & 1), smem_desc_sw128(kb + kk * 32, 16, 1024),
                     smem_desc_sw128(qb + kk * 32, 16, 1024), idS, kk > 0);
    };
    auto finish = [&](int j) -> bool {  // O = V_j^T P_j, once both are there
      if (!wait_all(&v_full[j % NS], (j / NS) & 1)) return false;
      if (!wait_all(&p_ready, j & 1)) return false;
      tc_fence_after();
      const uint32_t vb = sb + Lay::kOffV + (j % NS) * kFbTile;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)  // 32 keys each: four groups of 8 rows of V
        tc_mma_f8_ss(tmem + Lay::kColO, smem_desc_sw128(vb + kk * 4096, kFbTile, 1024),
                     smem_desc_sw128(ppb + kk * 32, 16, 1024), idO, kk > 0);
      tc_commit(smem_u32(&o_full));
      tc_commit(smem_u32(&v_empty[j % NS]));
      return true;
    };
    bool ok = wait_all(&q_ready, 0);
    // Order S_0, S_1, O_0, S_2, O_1, ...: S_{j+1} runs while the softmax works on
    // S_j.  S_j overwrites S_{j-2}, which was read before p_ready(j - 2).
    for (int j = 0; ok && j < n; ++j) {
      ok = wait_all(&k_full[j % NS], (j / NS) & 1);
      if (!ok) break;
      tc_fence_after();
      issue_s(j);
      tc_commit(smem_u32(&s_full[j & 1]));
      tc_commit(smem_u32(&k_empty[j % NS]));
      if (j > 0) ok = finish(j - 1);
    }
    if (ok) finish(n - 1);
    // Every MMA issued here has completed before tensor memory is released.
    tc_commit(smem_u32(&drain));
    mbar_wait(smem_u32(&drain), 0, p.wait_ns, p.err);
    __syncwarp();
  } else {
    // ------------------------------------------- softmax, accumulation, end --
    const int quarter = warp & 3;                // tensor-memory lanes 32 * quarter ..
    const int kl = quarter * 32 + lane;          // key of a tile; later, row d of O^T
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;

    // Q as two E4M3 terms, one row per warp and turn: lane takes columns
    // 4 lane .. 4 lane + 3.
    for (int r = quarter; r < R; r += 4) {
      uint2 w = make_uint2(0u, 0u);
      if (r < rows && lane * 4 < D)
        w = *reinterpret_cast<const uint2*>(p.q + out_row(r) * D + lane * 4);
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
      for (int i = 0; i < 2; ++i) {
        const float u = f[2 * i] * up, v = f[2 * i + 1] * up;
        hi[i] = pack_e4m3x2(u, v);
        const float2 g = unpack_e4m3x2(hi[i]);
        lo[2 * i] = (u - g.x) * 32.f;
        lo[2 * i + 1] = (v - g.y) * 32.f;
      }
      const uint32_t at = (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
      st_shared_u32(sb + Lay::kOffQ + r * 128 + at, hi[0] | (hi[1] << 16));
      st_shared_u32(sb + Lay::kOffQ + (R + r) * 128 + at,
                    pack_e4m3x2(lo[0], lo[1]) | (pack_e4m3x2(lo[2], lo[3]) << 16));
      if (lane == 0) cq[r] = a >= 0x7f80u ? NAN : p.scale_log2 * __int_as_float((127 - k) << 23);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&q_ready));
    named_bar_sync(1, 128);  // cq

    // Scales of this thread's key, one tile ahead; its page, two tiles ahead.
    auto page_of = [&](int j) -> int {
      const int tok = t0 + j * kFbKeys + kl;
      if (j >= n || tok >= t_end) return -1;
      if (!PAGED) return b;
      const int pg = p.block_table[(size_t)b * p.max_blocks + (tok >> pb.page_log2)];
      return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    auto scale_of = [&](int j, int unit, float& ks, float& vs) {
      ks = 1.f;
      vs = 1.f;
      if (unit < 0) return;
      const int tok = t0 + j * kFbKeys + kl;
      const int at = PAGED ? tok & (p.page_size - 1) : tok;
      const size_t i = ((size_t)unit * pb.per_blk + (at >> pb.block_log2)) * p.H_kv + kv;
      ks = pb.k_scale[i];
      vs = pb.v_scale[i];
    };
    float acc[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = l[r] = 0.f;
    const int lim_lo = min(t_end, L - p.T_q + 1);  // keys below it: visible from every row
    int unit1 = page_of(1);
    float ks, vs, ks1, vs1;
    scale_of(0, page_of(0), ks, vs);
    bool alive = true;

    for (int j = 0; j < n; ++j) {
      scale_of(j + 1, unit1, ks1, vs1);
      unit1 = page_of(j + 2);
      // log2 vs and 1 / vs; scales below 2^-100 count as zero, negative ones are NaN
      const bool v_live = vs >= kMinVScale;
      const float lv = v_live ? __log2f(vs) : (vs >= 0.f ? -100.f : NAN);
      const float ivs = v_live ? 1.f / vs : 1.f / kMinVScale;
      const int key = t0 + j * kFbKeys + kl;
      const bool edge = t0 + (j + 1) * kFbKeys > lim_lo;
      const uint32_t tS = tmem + lane_base + 2 * R * (j & 1);
      // (a warp whose wait failed keeps to the barriers of the others)
      alive = alive && wait_all(&s_full[j & 1], (j >> 1) & 1);
      tc_fence_after();
      // y of RC rows from column c0 on
      auto scores = [&](int c0, float (&y)[RC]) {
        uint32_t sh[RC], sl[RC];
        tmem_ld_cols(tS + c0, sh);
        tmem_ld_cols(tS + R + c0, sl);
        tmem_wait_ld();
        reg_fence(sh);
        reg_fence(sl);
#pragma unroll
        for (int i = 0; i < RC; ++i) {
          const float s = fmaf(__uint_as_float(sl[i]), kLoStep, __uint_as_float(sh[i]));
          y[i] = fmaf(s, cq[c0 + i] * ks, lv);
          if (edge && key >= lim_sm[c0 + i]) y[i] = -INFINITY;
        }
      };
      float y[RC];
#pragma unroll
      for (int c = 0; alive && c < NC; ++c) {
        scores(c * RC, y);
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < RC; ++i) {
          const float m = warp_max(y[i]);
          if (lane == i) mine = m;
        }
        if (lane < RC) red[j & 1][c * RC + lane][quarter] = mine;
      }
      named_bar_sync(1, 128);

      // O of the previous tile is complete: its P may be overwritten.
      alive = alive && (j == 0 || wait_all(&o_full, (j - 1) & 1));
      tc_fence_after();
#pragma unroll
      for (int c = 0; alive && c < NC; ++c) {
        const int c0 = c * RC;
        if (NC > 1) scores(c0, y);
        uint32_t oh[RC], ol[RC];
        if (j > 0) {
          tmem_ld_cols(tmem + lane_base + Lay::kColO + c0, oh);
          tmem_ld_cols(tmem + lane_base + Lay::kColO + R + c0, ol);
          tmem_wait_ld();
          reg_fence(oh);
          reg_fence(ol);
        } else {
#pragma unroll
          for (int i = 0; i < RC; ++i) oh[i] = ol[i] = 0u;
        }
        float pr[RC];
#pragma unroll
        for (int i = 0; i < RC; ++i) {
          const int r = c0 + i;
          const float4 mx = *reinterpret_cast<const float4*>(red[j & 1][r]);
          const float m_old = m_run[j & 1][r];
          const float m_new = fmax3(fmaxf(mx.x, mx.y), fmaxf(mx.z, mx.w), m_old);
          if (kl == r) m_run[(j + 1) & 1][r] = m_new;
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // no (-inf) - (-inf)
          const float alpha = ex2_approx(m_old - ref);
          acc[r] = (acc[r] + fmaf(__uint_as_float(ol[i]), kLoStep, __uint_as_float(oh[i]))) * alpha;
          const float e = ex2_approx(y[i] - ref + kPScaleLog2);
          l[r] = fmaf(e, ivs, l[r] * alpha);
          pr[i] = v_live || lv != lv ? e : 0.f;
        }
        // P as two E4M3 terms: byte kl of rows r and R + r, 128-byte swizzled
        // (8-row groups of 1024 bytes).
        const uint32_t pbase = sb + Lay::kOffP + (kl & 15);
        const int chunk = kl >> 4;
#pragma unroll
        for (int i = 0; i < RC; i += 2) {
          const uint32_t hi = pack_e4m3x2(pr[i], pr[i + 1]);
          const float2 g = unpack_e4m3x2(hi);
          const uint32_t lo = pack_e4m3x2((pr[i] - g.x) * 32.f, (pr[i + 1] - g.y) * 32.f);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = c0 + i + u;
            const uint32_t at = pbase + r * 128 + ((chunk ^ (r & 7)) << 4);
            st_shared_u8(at, u ? hi >> 8 : hi);
            st_shared_u8(at + R * 128, u ? lo >> 8 : lo);
          }
        }
      }
      // Cache rows past the end of the split may hold anything (even NaN codes),
      // and 0 * NaN would reach O: they are zeroed once the tile has landed.
      if (t0 + (j + 1) * kFbKeys > t_end) {
        alive = alive && wait_all(&v_full[j % NS], (j / NS) & 1);
        if (alive && key >= t_end) {
          const uint32_t vrow = sb + Lay::kOffV + (j % NS) * kFbTile + kl * 128;
#pragma unroll
          for (int c16 = 0; c16 < 8; ++c16) st_shared_v4(vrow + c16 * 16, 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (alive && lane == 0) mbar_arrive(smem_u32(&p_ready));
      ks = ks1;
      vs = vs1;
    }

    // The last O; l over the 128 keys' threads; then O / l and LSE, or the partial.
    bool page_ok = true;
    if (PAGED && alive) {
      // (a bad index is recorded before the arrive on the last V tile)
      if (wait_all(&v_full[(n - 1) % NS], ((n - 1) / NS) & 1))
        page_ok = *reinterpret_cast<volatile int*>(&bad_page) == 0;
      else
        alive = false;
    }
    alive = alive && wait_all(&o_full, (n - 1) & 1);
    if (alive) {
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t oh[RC], ol[RC];
        tmem_ld_cols(tmem + lane_base + Lay::kColO + c * RC, oh);
        tmem_ld_cols(tmem + lane_base + Lay::kColO + R + c * RC, ol);
        tmem_wait_ld();
        reg_fence(oh);
        reg_fence(ol);
#pragma unroll
        for (int i = 0; i < RC; ++i)
          acc[c * RC + i] += fmaf(__uint_as_float(ol[i]), kLoStep, __uint_as_float(oh[i]));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float s = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) red[n & 1][r][quarter] = s;
      }
    }
    // All four warps reach this barrier, also after a failed wait.
    named_bar_sync(1, 128);
    const bool failed = *abort_v != 0 || !alive || !page_ok;
    constexpr float kUnscale = 1.f / 256.f;  // P carried 2^8
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const size_t row = out_row(r);
      const float4 ls = *reinterpret_cast<const float4*>(red[n & 1][r]);
      const float lr = failed ? NAN : ((ls.x + ls.y) + (ls.z + ls.w)) * kUnscale;
      const float o = acc[r] * kUnscale;
      const float m = m_run[n & 1][r];
      if (p.n_split == 1) {
        if (kl < D && in_bounds(row * D + kl, 1, n_rows * D, p.err))
          p.out[row * D + kl] = __float2bfloat16(failed ? NAN : o / lr);
        if (kl == 0 && in_bounds(row, 1, n_rows, p.err))
          p.lse[row] = failed ? NAN : (m + log2f(lr)) * kLn2;
      } else {
        const size_t idx = row * p.n_split + split;
        if (kl < D && !failed && in_bounds(idx * D + kl, 1, n_rows * p.n_split * D, p.err))
          p.ws_O[idx * D + kl] = o;
        // m in natural-log units; a row with no visible key: (-inf, 0)
        if (kl == 0 && in_bounds(idx, 1, n_rows * p.n_split, p.err))
          p.ws_ml[idx] = failed ? make_float2(NAN, NAN) : make_float2(m * kLn2, lr);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kCols);
  }
}

template <int R, int NS, bool PAGED>
cudaError_t launch_fb(const DecodeBlockParams& p_in, const CUtensorMap& tm_k,
                      const CUtensorMap& tm_v, bool prefetch, cudaStream_t stream) {
  auto kern = gqa_decode_fp8_block_kernel<R, NS, PAGED>;
  constexpr int smem = FbLayout<R, NS>::kBytes;
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
  cfg.gridDim = dim3(p.dec.n_split, p.dec.H_kv, p.dec.B);
  cfg.blockDim = dim3(kFbThreads);
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

template <int R, int DEEP, int SHALLOW>
cudaError_t launch_fb_r(const DecodeBlockParams& p, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, int sms, cudaStream_t stream) {
  // One CTA per SM at most: a deep ring.  More CTAs than SMs: two shallow rings
  // on each SM, where they fit.
  const bool one_wave = (long long)p.dec.n_split * p.dec.H_kv * p.dec.B <= sms;
  const bool paged = p.dec.block_table != nullptr;
  if (one_wave || DEEP == SHALLOW)
    return paged ? launch_fb<R, DEEP, true>(p, tm_k, tm_v, one_wave, stream)
                 : launch_fb<R, DEEP, false>(p, tm_k, tm_v, one_wave, stream);
  return paged ? launch_fb<R, SHALLOW, true>(p, tm_k, tm_v, false, stream)
               : launch_fb<R, SHALLOW, false>(p, tm_k, tm_v, false, stream);
}

}  // namespace

cudaError_t launch_decode_fp8_block(const DecodeBlockParams& p, const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, int sms, cudaStream_t stream) {
  const int rows = p.dec.T_q * p.dec.G;
  if (rows < 1 || rows > 64 || p.dec.chunk % kFbKeys != 0) return cudaErrorInvalidValue;
  if (rows <= 8) return launch_fb_r<8, 6, 3>(p, tm_k, tm_v, sms, stream);
  if (rows <= 16) return launch_fb_r<16, 6, 3>(p, tm_k, tm_v, sms, stream);
  if (rows <= 32) return launch_fb_r<32, 6, 6>(p, tm_k, tm_v, sms, stream);
  return launch_fb_r<64, 5, 5>(p, tm_k, tm_v, sms, stream);
}

}  // namespace gqa
