// decode_diff.cu -- split-KV decode of differential attention, and the merge of its
// partials (also those of a split chunk prefill).
//
// A head h has two maps over the keys of its KV head:
//   O_u = softmax(tau q_u K_u^T) V  (u = 1, 2),   O = O_1 - lam O_2,
// then optionally O / sqrt(mean(O^2) + eps) * w, times a constant.  Both maps read the same
// V rows, and their keys are the same K rows (shared keys: q_1, q_2 are two query
// heads) or the two halves of them (split keys: q_1, q_2 are the halves of one query
// head).  So both sit in the M rows of the grouped-query decode: with shared keys as
// two rows, with split keys as the rows (q_1, 0) and (0, q_2), whose products with whole
// key rows are the two halves' products.  K and V are read once for all maps of a
// KV head, and a row's softmax is the streaming (m, l, O) update of the other decodes.
// The difference needs both maps' final sums, so it is taken where they are known: in the
// epilogue with one split, in the merge with several.
//
// One CTA per (split, 32 query rows, KV head, sequence): two producer warps, one for K and one
// for V, fill a ring of 64-token stages by TMA (a warp takes about 150 cycles to issue a
// box, and a stage of 16-token pages has 8 to 16 of them), and each group of four warps
// takes 16 query rows (one m16n8k16 tile), a warp a 16-token slice of every stage.  Rows
// are ordered (query, map), the maps of a head side by side, so a head's rows never part.
//
// Bound by HBM up to 16 rows: 8 sequences of 1K to 64K, 8 KV heads of 128, 125 us, 6.8
// TB/s; one of 32K 22.4 us, 6.0 TB/s, of which about 4.5 are the start and the merge's
// launch.  Short sequences are a chain of latencies: 1024 tokens of 2 KV heads of 32,
// 3.4 us.  From 17 rows on, without the tensor-core tile of decode_tc.cu, by mma.sync and the
// softmax (20 sequences of 2.5K, 6 KV heads of 64, 64 rows: 36 us, floor 10.5).
#include <type_traits>

#include "decode_common.cuh"
#include "decode_cut.cuh"
#include "diff.h"

namespace gqa {
namespace {

constexpr int kTile = kDecodeTile;
constexpr int kProducers = 2;   // warps: K, V
constexpr int kMaxCluster = 8;  // CTAs of a cluster (the portable size)
constexpr int kGroupWarps = 4;  // warps of a row group: 16 tokens of a stage each

// The epilogue's last step on one head's row: each of `LANES` neighbouring lanes holds
// 4 columns of O_1 and O_2 (divided by their sums); all of them call it together.
template <int LANES>
__device__ __forceinline__ float4 diff_row(const DiffParams& p, float4 a, float4 b, float lam, int c4) {
  float4 y = make_float4(a.x - lam * b.x, a.y - lam * b.y, a.z - lam * b.z, a.w - lam * b.w);
  float f = p.out_scale;
  if (p.norm_eps >= 0.f) {
    float ss = (y.x * y.x + y.y * y.y) + (y.z * y.z + y.w * y.w);
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    f *= rsqrtf(ss * (1.f / (4 * LANES)) + p.norm_eps);
    if (p.norm_weight) {
      const float* w = p.norm_weight + 4 * c4;
      y = make_float4(y.x * w[0], y.y * w[1], y.z * w[2], y.w * w[3]);
    }
  }
  return make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
}

// Stages of a CTA that has an SM to itself, and of one that shares it.  (d = 64 and 32: 96 and
// 48 KB, two and three CTAs of one row group on an SM.  Registers for a third and a
// fourth slowed every CTA down: 1024 tokens by 0.8 us, 8 x 8K of 64 in eight splits
// 13.9 -> 15.5.  Two row groups: 96 registers for a second CTA slow each down, too (5 sequences
// of up to 5K, 30 rows, d = 64: 10.5 -> 12.7 us), but pay where there are more KV heads and
// sequences than SMs (60 x 1K, 5 KV heads, 64 rows: 52 -> 37; 40 x 2.5K, 5 of 32, 24 rows
// 27.0 -> 20.7; 10 x 2.5K, 6 of 64, 64 rows 21 and 29), for d = 32, which loses little,
// where splits do (26 x 5K-9K, one KV head, 42 rows, in five: 25.8 -> 19.2), and for
// clusters of eight that would otherwise want nearly every SM, of which the GPU's parts
// hold few whole ones (4 x 900, 4 KV heads, 24 rows: 11.0 -> 7.7).)
template <int D>
struct Ring {
  static constexpr int kDeep = 6;
  static constexpr int kShallow = D == 128 ? 3 : 6;
  static constexpr int kPair = 5;  // two row groups, in 96 registers for two CTAs on an SM
};

template <int D, int NRG>
constexpr int merge_bytes() {
  return NRG * kGroupWarps * 16 * (D * 4 + 8);
}

// NRG: row groups of 16 of a CTA.  ROWS16 = false: one group of at most 8 rows.
// CLUSTER: p.n_split CTAs (8 at most) of one KV head and sequence are a thread-block cluster that
// merges its partials itself: each leaves its (m, l, O) in its shared memory, and CTA `rank`
// finishes heads rank, rank + n_split, .. from all of them, through distributed shared
// memory.  One launch, no workspace.
// CUT: the batch is cut by its lengths (decode_cut.cuh) and grid x is the piece.
template <int D, int NRG, bool ROWS16, int NSTAGE, bool PAGED, bool CLUSTER, bool CUT>
__global__ void __launch_bounds__((kGroupWarps * NRG + kProducers) * 32,
                                  NSTAGE == Ring<D>::kDeep ? 1 : 2)
    gqa_decode_diff_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const DecodeDiffParams pp) {
  static_assert(ROWS16 || NRG == 1, "fewer than nine rows are one group");
  static_assert(!(CLUSTER && CUT), "a cluster's splits are even");
  using Lay = DecodeLayout<D>;
  constexpr int kCW = kGroupWarps * NRG;  // consumer warps
  constexpr int kStageBytes = Lay::kStageBytes;
  static_assert(merge_bytes<D, NRG>() + (CLUSTER ? 16 * NRG * (D * 4 + 8) : 0) <= NSTAGE * kStageBytes,
                "the partials reuse the ring");
  const DecodeParams& p = pp.dec;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE];
  __shared__ int abort_flag, bad_page;

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem_base = smem_u32(smem);
  volatile int* const abort_v = &abort_flag;
  volatile int* const bad_v = &bad_page;

  // (the row groups of one split are neighbours in launch order, so that their reads of
  // the same K/V tiles meet in L2)
  const int row0 = (blockIdx.x % p.n_rg) * (16 * NRG);  // first query row of this CTA
  const int kv = blockIdx.y;
  int split = blockIdx.x / p.n_rg, b = CUT ? 0 : blockIdx.z, chunk = p.chunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G, h0 = kv * G;
  const int R = min(16 * NRG, p.T_q * G - row0);  // live rows (even)
  // Row x of the KV head is map h0 + x % G of query x / G; x / G without a division: (x +
  // 1/2) / G lies at least 1/32 from the nearest integer, far above the float error.
  const float inv_g = 1.f / static_cast<float>(G);
  auto query_of = [&](int x) { return static_cast<int>((static_cast<float>(x) + 0.5f) * inv_g); };
  auto out_row = [&](int r) -> size_t {  // row of lse and the workspace
    const int x = row0 + r, tq = query_of(x);
    return ((size_t)b * p.T_q + tq) * p.H_q + h0 + (x - tq * G);
  };
  const size_t n_rows = (size_t)p.B * p.T_q * p.H_q;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(smem_u32(&full_bar[s]), kProducers);
      mbar_init(smem_u32(&empty_bar[s]), kCW);
    }
    abort_flag = 0;
    bad_page = 0;
    fence_barrier_init();
  }
  // A batch cut by its lengths: the cut is worked out while the previous kernel
  // finishes, from relaxed loads, and again after the dependency wait if a length has
  // changed.
  Piece piece{0, 0, 0, 0};
  int cut_tiles[3] = {0, 0, 0};
  auto tiles_of = [&](int L) {
    return L < p.T_q || L > p.S_max ? 0 : (L + kTile - 1) / kTile;
  };
  auto take_piece = [&]() {
    piece = find_piece(cut_tiles[0], cut_tiles[1], cut_tiles[2], p.B, p.n_split, pp.pieces,
                       blockIdx.x / p.n_rg, lane);
    b = max(piece.b, 0);
    split = piece.split;
    chunk = piece.tiles * kTile;
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
  // While the previous kernel finishes, the producer warps prefetch the split's first
  // tiles into L2, one (tile, page segment) per lane.  The lengths and pages come
  // from relaxed loads that may see values from before the previous kernel's writes;
  // they only aim the prefetch, which hands no data to the kernel.
  const int box = PAGED ? min(p.page_size, kTile) : kTile;  // rows per box
  const int subs = kTile / box;
  const bool is_v = warp == kCW + 1;  // the second producer
  const CUtensorMap* const tm = is_v ? &tm_v : &tm_k;
  if (p.prefetch_tiles > 0 && warp >= kCW && row0 == 0) {
    int L_hint;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(L_hint) : "l"(p.seq_lens + b));
    const int i = lane / subs, sub = lane % subs;
    const int ahead = i * kTile + sub * box, tk = split * chunk + ahead;
    if (i < p.prefetch_tiles && ahead < chunk && tk < min(p.S_max, L_hint)) {
      int row = b * p.S_max + tk;
      bool ok = true;
      if constexpr (PAGED) {
        int pg;
        asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];"
                     : "=r"(pg)
                     : "l"(p.block_table + (size_t)b * p.max_blocks + tk / p.page_size));
        ok = pg >= 0 && pg < p.num_pages;
        row = pg * p.page_size + tk % p.page_size;
      }
      if (ok) {
#pragma unroll
        for (int blk = 0; blk < Lay::kBlocks; ++blk)
          tma_prefetch_l2_3d(tm, blk * Lay::kBox, kv, row);
      }
    }
  }
  __syncthreads();
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
    if (piece.b < 0) return;  // a CTA past the batch's last piece
    // the slots of the workspace that the sequence has no pieces for: the merge identity
    if (split == piece.count - 1)
      for (int r = warp; r < R; r += kCW + kProducers)
        for (int i = piece.count + lane; i < p.n_split; i += 32) {
          const size_t at = out_row(r) * p.n_split + i;
          if (in_bounds(at, 1, n_rows * p.n_split, p.err))
            p.ws_ml[at] = make_float2(-INFINITY, 0.f);
        }
  }
  const int L = p.seq_lens[b];

  // A bad length: NaN outputs (with several splits a NaN partial).  An empty split: the
  // merge identity (-inf, 0), its O is not written.
  const bool bad_len = L < p.T_q || L > p.S_max || L < 1;
  const long long t_first = static_cast<long long>(split) * chunk;
  // (A cluster's CTAs all see the same length; its empty splits take part in the merge.)
  if (bad_len || (!CLUSTER && t_first >= L)) {
    if (bad_len && threadIdx.x == 0 && split == 0 && kv == 0 && row0 == 0)
      atomicOr(p.err, kErrBadSeqLen);
    const float2 ml = bad_len ? make_float2(NAN, NAN) : make_float2(-INFINITY, 0.f);
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
      const size_t row = out_row(r);
      if (!CLUSTER && p.n_split > 1) {
        if (in_bounds(row * p.n_split + split, 1, n_rows * p.n_split, p.err))
          p.ws_ml[row * p.n_split + split] = ml;
      } else if (split == 0) {
        if (in_bounds(row, 1, n_rows, p.err)) p.lse[row] = NAN;
      }
    }
    if (split == 0 && (CLUSTER || p.n_split == 1))
      for (int e = threadIdx.x; e < R / 2 * D; e += blockDim.x) {
        const size_t row = out_row(2 * (e / D)) / 2;
        if (in_bounds(row * D + e % D, 1, n_rows / 2 * D, p.err))
          p.out[row * D + e % D] = __float2bfloat16(NAN);
      }
    return;
  }
  const int t0 = static_cast<int>(min(t_first, static_cast<long long>(L)));
  const int t_end = min(chunk, L - t0) + t0;
  const int n_tiles = (t_end - t0 + kTile - 1) / kTile;

  // ------------------------------------------------------------ producer ----
  if (warp >= kCW) {
    if (lane == 0) tma_prefetch_map(tm);
    // Lane 0 takes the slot and arms its barrier; box `sub` of a tile is issued by lane
    // `sub` (one box for a contiguous cache).  A page's index is read one tile ahead, so
    // that the read is in flight while the producer waits for a slot.
    const uint64_t pol = p.n_rg == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
    auto page_of = [&](int i) -> int {
      const int tok = t0 + i * kTile + lane * box;
      if (!PAGED || lane >= subs || tok >= t_end) return -1;
      return p.block_table[(size_t)b * p.max_blocks + tok / p.page_size];
    };
    int page = page_of(0);
    int issued = 0;
    bool told = false;  // of a page outside the pool
    for (int i = 0; i < n_tiles; ++i) {
      const int st = i % NSTAGE;
      const int next = page_of(i + 1);
      bool go = true;
      if (lane == 0 && i >= NSTAGE) {
        const uint32_t eb = smem_u32(&empty_bar[st]), par = ((i / NSTAGE) - 1) & 1;
        if (!mbar_try_wait(eb, par) && (*abort_v || !mbar_wait(eb, par, p.wait_ns, p.err))) {
          *abort_v = 1;
          go = false;
        }
      }
      const int tok = t0 + i * kTile + lane * box;
      int row;
      if constexpr (PAGED) {
        // A box wholly past the split's end reads rows past the pool, which arrive as zeros.
        const bool has = lane < subs && tok < t_end;
        const bool bad = has && (page < 0 || page >= p.num_pages);
        row = !has ? p.num_pages * p.page_size
                   : (bad ? 0 : page) * p.page_size + tok % p.page_size;
        // (recorded before lane 0's arrive releases it to the consumers)
        if (__any_sync(0xffffffffu, bad) && lane == 0) {
          if (!is_v && !told) atomicOr(p.err, kErrBadPage);
          told = true;
          *bad_v = 1;
        }
      } else {
        row = b * p.S_max + tok;
      }
      if (lane == 0 && go) mbar_arrive_expect_tx(smem_u32(&full_bar[st]), Lay::kTileBytes);
      if (!__shfl_sync(0xffffffffu, go, 0)) break;
      const uint32_t fb = smem_u32(&full_bar[st]);
      if (lane < subs) {
        const uint32_t dst = smem_base + st * kStageBytes + (is_v ? Lay::kTileBytes : 0) +
                             lane * box * Lay::kSpan;
#pragma unroll
        for (int blk = 0; blk < Lay::kBlocks; ++blk)
          tma_load_3d(dst + blk * Lay::kBlockBytes, tm, fb, blk * Lay::kBox, kv, row, pol);
      }
      page = next;
      issued = i + 1;
    }
    __syncwarp();
    if (lane == 0) {
      // The next kernel may be scheduled now; it waits for this grid before it reads.
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // No copy may still target this CTA's shared memory when it exits.  (After an abort the
      // other producer may not have armed the last stages; the waits are bounded.)
      for (int i = max(0, issued - NSTAGE); i < issued; ++i)
        mbar_wait(smem_u32(&full_bar[i % NSTAGE]), (i / NSTAGE) & 1, p.wait_ns, p.err);
    }
    __syncwarp();
    if constexpr (CLUSTER) {  // the consumers' two cluster barriers
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ------------------------------------------------------------ consumers ---
  const int g = lane >> 2, t = lane & 3;
  const int ws = warp % kGroupWarps, grp = warp / kGroupWarps;
  const int rb = row0 + 16 * grp;  // first row of this warp's group
  // Q as the A operand; rows past T_q * G are zero, and with split keys the half of a row
  // that is its head's other map (rows g and g + 8 have one parity, G being even).
  uint32_t qa[D / 16][4];
  {
    const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q);
    auto word = [&](int x, int kk, int c) -> uint32_t {
      if (x >= p.T_q * G) return 0u;
      const int tq = query_of(x);
      size_t row = ((size_t)b * p.T_q + tq) * p.H_q + h0 + (x - tq * G);
      if (pp.diff.split_keys) {
        if ((kk >= D / 32 ? 1 : 0) != (x & 1)) return 0u;
        row >>= 1;
      }
      return q32[row * (D / 2) + c];
    };
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = word(rb + g, kk, kk * 8 + t);
      qa[kk][1] = ROWS16 ? word(rb + g + 8, kk, kk * 8 + t) : 0u;
      qa[kk][2] = word(rb + g, kk, kk * 8 + t + 4);
      qa[kk][3] = ROWS16 ? word(rb + g + 8, kk, kk * 8 + t + 4) : 0u;
    }
  }
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m0 = -INFINITY, l0 = 0.f, m1 = -INFINITY, l1 = 0.f;
  // ldmatrix lane roles.  K (non-transposed): matrix mi = lane / 8 covers tokens
  // (mi / 2) * 8.. and d-chunk (mi % 2); V (transposed): tokens (mi % 2) * 8.., chunk mi / 2.
  const int k_row = ws * 16 + ((lane >> 4) << 3) + (lane & 7), k_chk = (lane >> 3) & 1;
  const int v_row = ws * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), v_chk = lane >> 4;
  // Query t sees keys below L - T_q + 1 + t.
  const int lim0 = min(t_end, L - p.T_q + 1 + query_of(rb + g));
  const int lim1 = min(t_end, L - p.T_q + 1 + query_of(rb + g + 8));
  const int lim_lo = min(t_end, L - p.T_q + 1 + query_of(rb));

  for (int i = 0; i < n_tiles; ++i) {
    const int st = i % NSTAGE;
    const uint32_t fb = smem_u32(&full_bar[st]), par = (i / NSTAGE) & 1;
    bool ok = mbar_try_wait(fb, par);
    if (!ok) ok = *abort_v == 0 && mbar_wait(fb, par, p.wait_ns, p.err);
    if (!__all_sync(0xffffffffu, ok)) {  // (the warp stays converged for ldmatrix and mma)
      *abort_v = 1;
      break;
    }
    const uint32_t kbase = smem_base + st * kStageBytes, vbase = kbase + Lay::kTileBytes;
    const int tok0 = t0 + i * kTile + ws * 16;  // first token of this warp's slice
    float sacc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t b00, b01, b10, b11;
      ldsm_x4(kbase + Lay::offset(k_row, kk * 2 + k_chk), b00, b01, b10, b11);
      mma_bf16_16816(sacc[0], qa[kk], b00, b01);
      mma_bf16_16816(sacc[1], qa[kk], b10, b11);
    }
    if (pp.diff.split_keys) {
      // A key's half that is not finite makes NaN of the other map's zeros: then the product of
      // each half for itself, of which a row takes its own.  (20 sequences of 1K to 2.5K, 6 KV
      // heads of 64, 64 rows: 31.8 us without the check, 32.9 with it, 34.9 with the two products
      // always, which took 33.3 to 35.7 with shared keys, too.)
      const float sum = ((sacc[0][0] + sacc[0][1]) + (sacc[0][2] + sacc[0][3])) +
                        ((sacc[1][0] + sacc[1][1]) + (sacc[1][2] + sacc[1][3]));
      if (__any_sync(0xffffffffu, isnan(sum))) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = half * (D / 32); kk < (half + 1) * (D / 32); ++kk) {
            uint32_t b00, b01, b10, b11;
            ldsm_x4(kbase + Lay::offset(k_row, kk * 2 + k_chk), b00, b01, b10, b11);
            mma_bf16_16816(x[0], qa[kk], b00, b01);
            mma_bf16_16816(x[1], qa[kk], b10, b11);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((g & 1) == half) sacc[e / 4][e % 4] = x[e / 4][e % 4];
        }
      }
    }
    const bool partial = tok0 + 16 > lim_lo;
    float x0[4], x1[4];  // rows g and g + 8, tokens tok0 + 8 nt + 2 t + c
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int tk = tok0 + nt * 8 + 2 * t + c;
        x0[nt * 2 + c] = !partial || tk < lim0 ? sacc[nt][c] * p.scale_log2 : -INFINITY;
        x1[nt * 2 + c] = !partial || tk < lim1 ? sacc[nt][2 + c] * p.scale_log2 : -INFINITY;
      }
    float p0[4], p1[4] = {0.f, 0.f, 0.f, 0.f};
    const float a0 = online_update(x0, m0, l0, p0);
    float a1 = 1.f;
    if (ROWS16) a1 = online_update(x1, m1, l1, p1);
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      o[n][0] *= a0;
      o[n][1] *= a0;
      if (ROWS16) {
        o[n][2] *= a1;
        o[n][3] *= a1;
      }
    }
    // (the weights in bf16, 2^-8 of each, as mma takes them with V; their sums are fp32)
    const uint32_t pa[4] = {pack_bf16x2(p0[0], p0[1]), pack_bf16x2(p1[0], p1[1]),
                            pack_bf16x2(p0[2], p0[3]), pack_bf16x2(p1[2], p1[3])};
    // O += P V with V's elements under the masks; of the accumulators, rows g and g + 8
    // are kept as they were unless `in0`, `in1`.
    auto pv = [&](uint32_t vm0, uint32_t vm1, auto some, bool in0, bool in1) {
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        uint32_t v[4];
        ldsm_x4_trans(vbase + Lay::offset(v_row, jj * 2 + v_chk), v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float(&acc)[4] = o[2 * jj + u];
          if constexpr (decltype(some)::value) {
            float x[4] = {acc[0], acc[1], acc[2], acc[3]};
            mma_bf16_16816(x, pa, v[2 * u] & vm0, v[2 * u + 1] & vm1);
            acc[0] = in0 ? x[0] : acc[0];
            acc[1] = in0 ? x[1] : acc[1];
            acc[2] = in1 ? x[2] : acc[2];
            acc[3] = in1 ? x[3] : acc[3];
          } else {
            mma_bf16_16816(acc, pa, v[2 * u] & vm0, v[2 * u + 1] & vm1);
          }
        }
      }
    };
    if (!partial) {
      pv(0xffffffffu, 0xffffffffu, std::false_type{}, true, true);
    } else {
      // Rows of V that a query does not see may hold anything, and 0 * NaN is NaN: those
      // at or past a limit are zero in the product.
      const int ta = tok0 + 2 * t, tc = ta + 8;
      auto mask = [](int tk, int lim) {
        return (tk < lim ? 0x0000ffffu : 0u) | (tk + 1 < lim ? 0xffff0000u : 0u);
      };
      bool odd = false;  // an infinity or NaN that only some of several queries see?
      if (p.T_q > 1) {
#pragma unroll
        for (int jj = 0; jj < D / 16; ++jj) {
          uint32_t v[4];
          ldsm_x4_trans(vbase + Lay::offset(v_row, jj * 2 + v_chk), v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = v[e] & mask(e & 1 ? tc : ta, t_end);
            odd |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
          }
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      if (!odd) {
        pv(mask(ta, t_end), mask(tc, t_end), std::false_type{}, true, true);
      } else {  // one query's rows at a time, with that query's limit
        const int q_end = query_of(min(rb + 16, p.T_q * G) - 1);
        const int q0 = query_of(rb + g), q1 = query_of(rb + g + 8);
#pragma unroll 1
        for (int tq = query_of(rb); tq <= q_end; ++tq) {
          const int lim = min(t_end, L - p.T_q + 1 + tq);
          pv(mask(ta, lim), mask(tc, lim), std::true_type{}, q0 == tq, q1 == tq);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty_bar[st]));
  }
  l0 = quad_sum(l0);
  if (ROWS16) l1 = quad_sum(l1);

  // ------------------------------------------- merge the four warp partials --
  named_bar_sync(1, kCW * 32);
  const bool failed = *abort_v != 0 || (PAGED && *bad_v != 0);
  float* mO = reinterpret_cast<float*>(smem);                                  // [kCW][16][D]
  float2* mML = reinterpret_cast<float2*>(smem + kCW * 16 * D * 4);            // [kCW][16]
  if (!failed) {
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      const int col = n * 8 + 2 * t;
      *reinterpret_cast<float2*>(&mO[(warp * 16 + g) * D + col]) = make_float2(o[n][0], o[n][1]);
      if (ROWS16)
        *reinterpret_cast<float2*>(&mO[(warp * 16 + g + 8) * D + col]) =
            make_float2(o[n][2], o[n][3]);
    }
    if (t == 0) {
      mML[warp * 16 + g] = make_float2(m0, l0);
      if (ROWS16) mML[warp * 16 + g + 8] = make_float2(m1, l1);
    }
  }
  named_bar_sync(1, kCW * 32);

  constexpr int V4 = D / 4;                        // lanes of a row, 4 columns each
  constexpr int kRows = ROWS16 ? 16 * NRG : 8;     // rows in shared memory
  auto merged = [&](int r, int c4, float& M, float& Ls) -> float4 {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    M = -INFINITY;
    Ls = 0.f;
    if (failed) {
      M = Ls = NAN;
      return make_float4(NAN, NAN, NAN, NAN);
    }
    const int at = (r / 16) * (kGroupWarps * 16) + r % 16;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) M = fmaxf(M, mML[at + w * 16].x);
    const float ref = (M == -INFINITY) ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) {
      const float2 ml = mML[at + w * 16];
      const float a = ex2_approx(ml.x - ref);
      Ls += a * ml.y;
      const float4 ow = *reinterpret_cast<const float4*>(&mO[(at + w * 16) * D + c4 * 4]);
      acc.x += a * ow.x;
      acc.y += a * ow.y;
      acc.z += a * ow.z;
      acc.w += a * ow.w;
    }
    return acc;
  };
  if (!CLUSTER && p.n_split > 1) {
    for (int e = threadIdx.x; e < kRows * V4; e += kCW * 32) {
      const int r = e / V4, c4 = e % V4;
      if (r >= R) break;
      float M, Ls;
      const float4 acc = merged(r, c4, M, Ls);
      const size_t idx = out_row(r) * p.n_split + split;
      if (in_bounds(idx * D + c4 * 4, 4, n_rows * p.n_split * D, p.err))
        *reinterpret_cast<float4*>(&p.ws_O[idx * D + c4 * 4]) = acc;
      if (c4 == 0 && in_bounds(idx, 1, n_rows * p.n_split, p.err))
        p.ws_ml[idx] = make_float2(M * kLn2, Ls);
    }
    return;
  }
  // Columns 4 c4 .. of rows r and r + 1, the maps of a head: divided by their sums, and
  // the difference.  A warp holds whole rows (V4 divides 32) and calls this converged.
  auto finish = [&](int r, int c4, float4 a, float Ma, float La, float4 c, float Mb, float Lb) {
    const float ia = 1.f / La, ic = 1.f / Lb;
    // (each map rounded before the difference, so that equal maps leave exactly nothing at
    // lam = 1)
    a = make_float4(__fmul_rn(a.x, ia), __fmul_rn(a.y, ia), __fmul_rn(a.z, ia), __fmul_rn(a.w, ia));
    c = make_float4(__fmul_rn(c.x, ic), __fmul_rn(c.y, ic), __fmul_rn(c.z, ic), __fmul_rn(c.w, ic));
    const bool live = r < R;
    const int x = row0 + r, tq = query_of(x), h = (h0 + (x - tq * G)) >> 1;
    const float lam = live ? pp.diff.lam[(long long)b * pp.diff.lam_b + tq * pp.diff.lam_t +
                                         h * pp.diff.lam_h]
                           : 0.f;
    const float4 y = diff_row<V4>(pp.diff, a, c, lam, c4);
    if (!live) return;
    const size_t row = out_row(r);
    const size_t orow = row / 2;
    if (in_bounds(orow * D + c4 * 4, 4, n_rows / 2 * D, p.err))
      *reinterpret_cast<uint2*>(&p.out[orow * D + c4 * 4]) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    if (c4 == 0 && in_bounds(row, 2, n_rows, p.err))
      *reinterpret_cast<float2*>(&p.lse[row]) =
          make_float2((Ma + log2f(La)) * kLn2, (Mb + log2f(Lb)) * kLn2);
  };
  if constexpr (!CLUSTER) {  // one split; whole warps take part or not
    for (int e = threadIdx.x; e < kRows / 2 * V4; e += kCW * 32) {
      const int r = 2 * (e / V4), c4 = e % V4;
      float Ma, La, Mb, Lb;
      const float4 a = merged(r, c4, Ma, La), c = merged(r + 1, c4, Mb, Lb);
      finish(r, c4, a, Ma, La, c, Mb, Lb);
    }
  } else {
    float* cO = reinterpret_cast<float*>(smem + merge_bytes<D, NRG>());  // [kRows][D]
    float2* cML = reinterpret_cast<float2*>(cO + kRows * D);             // [kRows]
#pragma unroll
    for (int it = 0; it < (kRows * V4 + kCW * 32 - 1) / (kCW * 32); ++it) {
      const int e = threadIdx.x + it * kCW * 32, r = e / V4, c4 = e % V4;
      if (r >= kRows) break;
      float M, Ls;
      const float4 acc = merged(r, c4, M, Ls);
      *reinterpret_cast<float4*>(&cO[r * D + c4 * 4]) = acc;
      if (c4 == 0) cML[r] = make_float2(M, Ls);
    }
    __syncwarp();
    cluster_sync();  // every partial of the cluster is in place
    const int C = p.n_split;
    const uint32_t sO = smem_u32(cO), sML = smem_u32(cML);
    // One row folded over the cluster; an empty split has weight 0 (and O = 0).
    auto folded = [&](int r, int c4, float& M, float& Ls) -> float4 {
      float2 ml[kMaxCluster];
      float4 ov[kMaxCluster];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        ov[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q < C) {
          ml[q] = ld_dsmem_f32x2(mapa_shared(sML + r * 8, q));
          ov[q] = ld_dsmem_f32x4(mapa_shared(sO + (r * D + c4 * 4) * 4, q));
        }
      }
      M = -INFINITY;
      bool bad = false;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        bad |= isnan(ml[q].x) || isnan(ml[q].y);
        M = fmaxf(M, ml[q].x);
      }
      const float ref = (M == -INFINITY) ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      Ls = 0.f;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        // (no key of such a split is seen: 0 * NaN must not come of its O)
        if (ml[q].x == -INFINITY) continue;
        const float w = ex2_approx(ml[q].x - ref);
        Ls += w * ml[q].y;
        acc.x += w * ov[q].x;
        acc.y += w * ov[q].y;
        acc.z += w * ov[q].z;
        acc.w += w * ov[q].w;
      }
      if (bad) M = Ls = NAN;
      return acc;
    };
    constexpr int kAtOnce = kCW * 32 / V4;  // heads that the CTA takes at a time
    const int rank = static_cast<int>(cluster_ctarank());
    for (int i = threadIdx.x / V4; 2 * (rank + C * (i - (i % (32 / V4)))) < kRows; i += kAtOnce) {
      // (a warp's lanes stay together: heads past the last are folded from the last's rows)
      const int r = 2 * (rank + C * i), c4 = threadIdx.x % V4, rr = min(r, kRows - 2);
      float Ma, La, Mb, Lb;
      const float4 a = folded(rr, c4, Ma, La), c = folded(rr + 1, c4, Mb, Lb);
      finish(r, c4, a, Ma, La, c, Mb, Lb);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another may still read its partial
  }
}

// ---------------------------------------------------------------- merge ----
// One CTA per head row: 2 D threads, the first D for the first map's columns, the others for
// the second's.  A thread folds the parts of its column, CHUNK to a round of loads; lane i
// of its warp works out the weight of part i of the round and hands it round.  The
// second map's columns then cross through shared memory.  A chain of latencies (the
// partials, the exchange, the store), with lam and the weight loaded beside the
// partials.  Registers are kept few: the CTAs are to be resident beside those of the
// decode, waiting (8K tokens, 19 splits, every thread holding all (m, l) pairs in 128
// registers: 9.4 us a step).
template <int D, int CHUNK>
__global__ void __launch_bounds__(2 * D, 1024 / (2 * D)) gqa_diff_merge_kernel(const DiffMergeParams p) {
  static_assert(CHUNK <= 32, "a lane for each part of a round");
  __shared__ float s_o[D], s_ss[D / 32];
  const int col = threadIdx.x % D, u = threadIdx.x / D, lane = threadIdx.x & 31;
  const int H = p.H_maps / 2;
  const unsigned bt = blockIdx.x / static_cast<unsigned>(H);  // b * T + t
  const int h = blockIdx.x - bt * H;
  const int b = bt / static_cast<unsigned>(p.T), t = bt - b * p.T;
  const size_t row = static_cast<size_t>(bt) * p.H_maps + 2 * h + u;
  const float2* ml = p.ws_ml + row * p.n_part;
  const float* O = p.ws_O + row * p.n_part * D + col;
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float M = -INFINITY, L = 0.f, acc = 0.f;
  bool bad = false;
  const float lam = p.diff.lam[b * p.diff.lam_b + t * p.diff.lam_t + h * p.diff.lam_h];
  const float weight = p.diff.norm_weight ? p.diff.norm_weight[col] : 1.f;
  for (int s0 = 0; s0 < p.n_part; s0 += CHUNK) {
    const bool mine = lane < CHUNK && s0 + lane < p.n_part;
    float2 part = mine ? ml[s0 + lane] : make_float2(-INFINITY, 0.f);
    float ov[CHUNK];
#pragma unroll
    for (int s = 0; s < CHUNK; ++s) ov[s] = s0 + s < p.n_part ? O[(size_t)(s0 + s) * D] : 0.f;
    part.x *= p.m_log2;
    bad |= __any_sync(0xffffffffu, isnan(part.x) || isnan(part.y));
    float cm = part.x;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, k));
    cm = fmaxf(cm, M);
    const float ref = (cm == -INFINITY) ? 0.f : cm;
    const float a = ex2_approx(M - ref);
    // an empty part (m = -inf) has weight 0 and its O (never written) is not used
    const bool live = part.x != -INFINITY;
    const float w = live ? ex2_approx(part.x - ref) : 0.f;
    const unsigned alive = __ballot_sync(0xffffffffu, live);
    float lsum = live ? w * part.y : 0.f;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, k);
    L = L * a + lsum;
    acc *= a;
#pragma unroll
    for (int s = 0; s < CHUNK; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      acc += (alive >> s & 1) ? ws * ov[s] : 0.f;
    }
    M = cm;
  }
  const bool poisoned = bad || !(L > 0.f);
  const size_t n_rows = (size_t)p.B * p.T * p.H_maps;
  float o = poisoned ? NAN : acc / L;
  if (u == 1) s_o[col] = o;
  const long long lse_at = b * p.lse_b + t * p.lse_t + (2 * h + u) * p.lse_m;
  if (col == 0 && in_bounds(lse_at, 1, n_rows, p.err))
    p.lse[lse_at] = poisoned ? NAN : (M + log2f(L)) * kLn2;
  __syncthreads();
  float f = p.diff.out_scale;
  if (u == 0) o = fmaf(-lam, s_o[col], o);
  if (p.diff.norm_eps >= 0.f) {
    if (u == 0) {
      float ss = o * o;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
      if ((col & 31) == 0) s_ss[col / 32] = ss;
    }
    __syncthreads();
    float ss = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) ss += s_ss[w];
    f *= rsqrtf(ss * (1.f / D) + p.diff.norm_eps);
  }
  const size_t at = (static_cast<size_t>(bt) * H + h) * D + col;
  if (u == 0 && in_bounds(at, 1, n_rows / 2 * D, p.err)) p.out[at] = __float2bfloat16(o * weight * f);
}

// The same merge for many rows (a chunk prefill's): one warp per head row, a lane with
// D / 32 columns of both maps, no exchange through shared memory.
constexpr int kRowWarps = 8;

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) gqa_diff_merge_rows_kernel(const DiffMergeParams p) {
  constexpr int VEC = D / 32;
  using Vec = std::conditional_t<VEC == 4, float4, std::conditional_t<VEC == 2, float2, float>>;
  const int lane = threadIdx.x & 31;
  const unsigned H = p.H_maps / 2;
  const size_t item = static_cast<size_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (item >= static_cast<size_t>(p.B) * p.T * H) return;
  const unsigned bt = static_cast<unsigned>(item / H);
  const int h = static_cast<int>(item - static_cast<size_t>(bt) * H);
  const int b = bt / static_cast<unsigned>(p.T), t = bt - b * p.T;
  const float lam = p.diff.lam[b * p.diff.lam_b + t * p.diff.lam_t + h * p.diff.lam_h];
  const size_t row = static_cast<size_t>(bt) * p.H_maps + 2 * h;
  const size_t n_rows = (size_t)p.B * p.T * p.H_maps;
  float o[2][VEC];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float2* ml = p.ws_ml + (row + u) * p.n_part;
    const Vec* O = reinterpret_cast<const Vec*>(p.ws_O + (row + u) * p.n_part * D) + lane;
    float M = -INFINITY, L = 0.f;
    bool bad = false;
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
    for (int s0 = 0; s0 < p.n_part; s0 += 8) {
      const bool mine = lane < 8 && s0 + lane < p.n_part;
      float2 part = mine ? ml[s0 + lane] : make_float2(-INFINITY, 0.f);
      Vec ov[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) ov[s] = s0 + s < p.n_part ? O[(size_t)(s0 + s) * 32] : Vec{};
      part.x *= p.m_log2;
      bad |= __any_sync(0xffffffffu, isnan(part.x) || isnan(part.y));
      float cm = part.x;
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, k));
      cm = fmaxf(__shfl_sync(0xffffffffu, cm, 0), M);
      const float ref = (cm == -INFINITY) ? 0.f : cm;
      const float a = ex2_approx(M - ref);
      // an empty part (m = -inf) has weight 0 and its O (never written) is not used
      const bool live = part.x != -INFINITY;
      const float w = live ? ex2_approx(part.x - ref) : 0.f;
      const unsigned alive = __ballot_sync(0xffffffffu, live);
      const float wl = live ? w * part.y : 0.f;
      L *= a;
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[v] *= a;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        L += __shfl_sync(0xffffffffu, wl, s);
        if (!(alive >> s & 1)) continue;
        const float* x = reinterpret_cast<const float*>(&ov[s]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[v] = fmaf(ws, x[v], acc[v]);
      }
      M = cm;
    }
    const bool poisoned = bad || !(L > 0.f);
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[u][v] = poisoned ? NAN : acc[v] / L;
    const long long at = b * p.lse_b + t * p.lse_t + (2 * h + u) * p.lse_m;
    if (lane == 0 && in_bounds(at, 1, n_rows, p.err))
      p.lse[at] = poisoned ? NAN : (M + log2f(L)) * kLn2;
  }
  float y[VEC], f = p.diff.out_scale, ss = 0.f;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    y[v] = fmaf(-lam, o[1][v], o[0][v]);
    ss += y[v] * y[v];
  }
  if (p.diff.norm_eps >= 0.f) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
    f *= rsqrtf(ss * (1.f / D) + p.diff.norm_eps);
  }
  const int col = lane * VEC;
  const size_t at = item * D + col;
  if (!in_bounds(at, VEC, n_rows / 2 * D, p.err)) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float w = p.diff.norm_weight ? p.diff.norm_weight[col + v] : 1.f;
    y[v] *= w * f;
  }
  if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(p.out + at) = pack_bf16x2(y[0], y[1]);
  else
    p.out[at] = __float2bfloat16(y[0]);
}

template <int D, int NRG, bool ROWS16, int NSTAGE, bool PAGED, bool CLUSTER = false, bool CUT = false>
cudaError_t launch(const DecodeDiffParams& p_in, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                   cudaStream_t stream) {
  constexpr int smem = NSTAGE * DecodeLayout<D>::kStageBytes + 1024;
  constexpr int threads = (kGroupWarps * NRG + kProducers) * 32;
  auto kern = gqa_decode_diff_kernel<D, NRG, ROWS16, NSTAGE, PAGED, CLUSTER, CUT>;
  static unsigned char done[64];
  static int resident[64];
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  int fit = 0;
  e = resident_ctas(reinterpret_cast<const void*>(kern), threads, smem, resident, &fit);
  if (e != cudaSuccess) return e;
  DecodeDiffParams p = p_in;
  // The L2 prefetch pays only when every CTA is resident while the previous kernel drains.
  const long long ctas = (CUT ? (long long)p.pieces : (long long)p.dec.n_split * p.dec.B) *
                         p.dec.n_rg * p.dec.H_kv;
  constexpr int kBytes = 98304 / DecodeLayout<D>::kStageBytes;
  p.dec.prefetch_tiles = ctas <= fit ? (kBytes < 6 ? kBytes : 6) : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = CUT ? dim3(p.pieces * p.dec.n_rg, p.dec.H_kv)
                    : dim3(p.dec.n_split * p.dec.n_rg, p.dec.H_kv, p.dec.B);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.dec.n_split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool PAGED>
cudaError_t launch_rows(const DecodeDiffParams& p_in, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, cudaStream_t stream) {
  DecodeDiffParams p = p_in;
  const int rows = p.dec.T_q * p.dec.G;
  p.dec.n_rg = rows <= 16 ? 1 : (rows + 31) / 32;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  constexpr int kShallow = Ring<D>::kShallow, kDeep = Ring<D>::kDeep, kPair = Ring<D>::kPair;
  // One split of a grid that leaves SMs idle: a cluster for each KV head and sequence (8
  // maps on 2 KV heads of 32, 1024 tokens: 3.4 us, one CTA each 6.4; 32 KV heads' worth of
  // 64 maps of 128, 1024 tokens: 6.8 and 9.6), but for short caches (128 tokens, d = 128: 4.4
  // and 3.5 us; 256 tokens, d = 32: 3.2 and 3.0).
  const long long groups = (long long)p.dec.n_rg * p.dec.H_kv * p.dec.B;
  if (p.dec.n_split == 1 && p.dec.n_rg == 1 && p.dec.S_max > 256) {
    int c = kMaxCluster;
    while (c > 1 && (c * groups > sms || (c - 1) * 64 >= p.dec.S_max)) c /= 2;
    if (c > 1) {
      p.dec.n_split = c;
      const int per = (p.dec.S_max + c - 1) / c;
      p.dec.chunk = (per + kTile - 1) / kTile * kTile;
      if constexpr (D < 128)  // (d = 128 takes the tensor-core tile, decode_tc.cu)
        if (rows > 16)
          return c == kMaxCluster && 2 * c * groups > sms
                     ? launch<D, 2, true, kPair, PAGED, true>(p, tm_k, tm_v, stream)
                     : launch<D, 2, true, kDeep, PAGED, true>(p, tm_k, tm_v, stream);
      if (rows > 8) return launch<D, 1, true, kShallow, PAGED, true>(p, tm_k, tm_v, stream);
      return launch<D, 1, false, kShallow, PAGED, true>(p, tm_k, tm_v, stream);
    }
  }
  if (p.pieces > 0) {
    if (p.dec.n_split < 2 || p.pieces <= p.dec.B || p.dec.B > kMaxCut) return cudaErrorInvalidValue;
    if constexpr (D < 128)
      if (rows > 16) return launch<D, 2, true, kDeep, PAGED, false, true>(p, tm_k, tm_v, stream);
    if (rows > 16) return cudaErrorInvalidValue;
    return rows > 8 ? launch<D, 1, true, kShallow, PAGED, false, true>(p, tm_k, tm_v, stream)
                    : launch<D, 1, false, kShallow, PAGED, false, true>(p, tm_k, tm_v, stream);
  }
  // A grid of at most one CTA per SM takes a deeper ring in the room of a second CTA.
  const bool one = p.dec.n_split * groups <= sms;
  if constexpr (D < 128)
    if (rows > 16)
      return (D == 32 ? p.dec.n_split : 1) * groups > sms
                 ? launch<D, 2, true, kPair, PAGED>(p, tm_k, tm_v, stream)
                 : launch<D, 2, true, kDeep, PAGED>(p, tm_k, tm_v, stream);
  if (rows > 16) return cudaErrorInvalidValue;
  if (rows > 8)
    return one ? launch<D, 1, true, kDeep, PAGED>(p, tm_k, tm_v, stream)
               : launch<D, 1, true, kShallow, PAGED>(p, tm_k, tm_v, stream);
  return one ? launch<D, 1, false, kDeep, PAGED>(p, tm_k, tm_v, stream)
             : launch<D, 1, false, kShallow, PAGED>(p, tm_k, tm_v, stream);
}

cudaError_t launch_merge(void (*kern)(const DiffMergeParams), long long ctas, int threads,
                         const DiffMergeParams& p, cudaStream_t stream) {
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
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

template <int D>
cudaError_t launch_merge_d(const DiffMergeParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.T * (p.H_maps / 2);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // A CTA per row finishes soonest while all of them are on the GPU at once; a warp per row
  // has less to do for each.
  if (rows > 8LL * sms)
    return launch_merge(gqa_diff_merge_rows_kernel<D>, (rows + kRowWarps - 1) / kRowWarps,
                        kRowWarps * 32, p, stream);
  return launch_merge(p.n_part <= 8    ? gqa_diff_merge_kernel<D, 8>
                      : p.n_part <= 16 ? gqa_diff_merge_kernel<D, 16>
                                       : gqa_diff_merge_kernel<D, 32>,
                      rows, 2 * D, p, stream);
}

}  // namespace

cudaError_t launch_decode_diff(const DecodeDiffParams& p, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, cudaStream_t stream) {
  const bool paged = p.dec.block_table != nullptr;
  switch (p.dec.d) {
    case 32: return paged ? launch_rows<32, true>(p, tm_k, tm_v, stream)
                          : launch_rows<32, false>(p, tm_k, tm_v, stream);
    case 64: return paged ? launch_rows<64, true>(p, tm_k, tm_v, stream)
                          : launch_rows<64, false>(p, tm_k, tm_v, stream);
    case 128: return paged ? launch_rows<128, true>(p, tm_k, tm_v, stream)
                           : launch_rows<128, false>(p, tm_k, tm_v, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_diff_merge(const DiffMergeParams& p, cudaStream_t stream) {
  switch (p.d) {
    case 32: return launch_merge_d<32>(p, stream);
    case 64: return launch_merge_d<64>(p, stream);
    case 128: return launch_merge_d<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gqa
