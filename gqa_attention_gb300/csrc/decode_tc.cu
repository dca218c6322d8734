// decode_tc.cu -- split-KV decode of many query rows per KV head on the
// fifth-generation tensor cores.
//
// What it computes: the multi-token decode of decode.cu.  The queries are the
// last T_q positions L - T_q .. L - 1 of each sequence (L = seq_lens[b]),
// query t sees keys 0 .. L - T_q + t, and the G query heads of a KV head read
// that head's K and V ("Attention Kernel 계보" p.2 §1, p.15 §2/§4; the chunk
// alignment of ADR-0060 §0.5.3 for short chunks).  The split-K decode of p.18
// §4: one CTA per (split, KV head, sequence) streams its split's keys once and
// leaves an unnormalised partial (m, l, O) per query row for the log-sum-exp
// merge of the combine kernel (p.4); with one split it writes O and LSE.
//
// Where decode.cu folds the T_q * G rows of a KV head into 16-row mma.sync
// tiles (one CTA per 16 rows, each re-reading K and V), this kernel puts all
// of them (up to 128) in the M rows of one tcgen05.mma tile, so every K/V
// tile is read once per split however many rows there are:
//   S_j = Q K_j^T       (M = 128 rows, N = 128 keys, K = d = 128; SS form)
//   O  += P_j V_j       (P_j bf16 in tensor memory; TS form)
// with FA2's loop order (p.8-p.9): Q stays in shared memory, K and V tiles of
// 128 keys stream through two three-slot rings, loaded in the order the tensor
// core consumes them (K_0, then K_{j+1}, V_j), so a K slot is refilled as soon
// as its S has been computed; (m, l, O) are updated online.  S is
// double-buffered in tensor memory: the tensor core computes S_{j+1} while the
// softmax warps turn S_j into P_j.
//
// Roles (192 threads):
//   warp 0      TMA producer: Q once, then the K and V tiles.
//   warp 1      allocates tensor memory and issues every tcgen05.mma.
//   warps 2-5   softmax + epilogue, thread = query row r = 32 (warp % 4) + lane
//               (tensor-memory lane r).
// Query row r of the tile is query t = r / G of head kv * G + r % G, the order
// in which the TMA box {d/2, G, T_q} of Q lands; rows r >= T_q * G are zero.
// Tensor memory (512 columns x 128 lanes, fp32): S_0 | S_1 | O; P_j (bf16, two
// per column) overwrites the first 64 columns of S_(j%2) once it has been read.
//
// O is rescaled only when a row's running maximum grows by more than 2^8
// (base 2), as in prefill.cu: l and O share one reference, so O / l holds.
//
// PAGED = true: the cache is a pool of fixed-size pages reached through a
// block table (p.17 §2-§4, p.18 §5); each 128-key tile arrives as boxes of
// min(page_size, 128) rows, one page each.  A page index outside the pool is
// reported and replaced by page 0, and the CTA's outputs become NaN.
//
// Differential attention (DIFF; decode_diff.cu says what it is): the rows are the maps of
// the heads, two neighbours each.  With several splits only the merge differs; with one
// the two lanes of a head exchange halves of their columns in the epilogue.  DIFF = 2, split
// keys: the tile of Q is 64 wide, row r being its map's half of a query row, and S takes the
// products with the first half of the keys into the even lanes and with the second half
// into the odd ones.  Batches of several sequences are cut by their
// lengths (decode_cut.cuh), and a row of V among the last T_q tokens that holds an
// infinity or NaN reaches the queries that see it and no others.  4 sequences of 2K to 16K, 4
// tokens of 8 maps each, 8 KV heads, pages of 64: 27 us with the merge, 4.9 TB/s.
#include <type_traits>

#include "decode_cut.cuh"
#include "diff.h"
#include "tcgen05.cuh"

namespace gqa {
namespace {

constexpr int kTcThreads = 192;
constexpr int kTcSlots = 3;                     // slots per ring (K and V)
#ifndef GQA_TC_PREFETCH_TILES
#define GQA_TC_PREFETCH_TILES 3  // 128-key tiles a CTA may warm in L2 before its dependency wait
#endif
static_assert(GQA_TC_PREFETCH_TILES >= 0 && GQA_TC_PREFETCH_TILES <= 32, "one tile per lane");
constexpr int kTcKeys = 128;                    // keys per ring stage
constexpr uint32_t kTileB = 128u * 128u * 2u;   // one 128 x 128 bf16 tile
constexpr uint32_t kHalfB = kTileB / 2;         // 128 rows x 128 bytes
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kTileB;              // K ring after Q
constexpr uint32_t kOffV = kOffK + kTcSlots * kTileB;  // then the V ring
constexpr uint32_t kTcSmem = kOffV + kTcSlots * kTileB + 1024;
constexpr uint32_t kColO = 256;                 // O after S_0, S_1
constexpr float kRescaleLog2 = 8.f;

__host__ __device__ __forceinline__ const DecodeParams& base_params(const DecodeParams& p) {
  return p;
}
__host__ __device__ __forceinline__ const DecodeParams& base_params(const DecodeDiffParams& p) {
  return p.dec;
}
// D[tmem] (+)= A[smem] * B[smem] as tc_mma_ss, without the lanes of D whose bit in `skip` is set,
// the same 32 bits for each 32 lanes: what those hold stays.
__device__ __forceinline__ void tc_mma_ss_lanes(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate, uint32_t skip) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(skip)
      : "memory");
}

template <int DIFF>
using TcParamsOf = std::conditional_t<DIFF != 0, DecodeDiffParams, DecodeParams>;

// CUT = true: the batch is cut by its lengths.  A variant of its own, so that the others'
// splits stay plainly the block's index.
template <bool PAGED, int DIFF, bool CUT>
__global__ void __launch_bounds__(kTcThreads, 1)
    gqa_decode_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const TcParamsOf<DIFF> pp) {
  const DecodeParams& p = base_params(pp);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full, drain;
  __shared__ __align__(8) uint64_t k_full[kTcSlots], k_empty[kTcSlots], v_full[kTcSlots],
      v_empty[kTcSlots];
  __shared__ __align__(8) uint64_t s_full[2], p_ready[2], pv_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int bad_page;
  // differential: per column of V, the first of the last T_q tokens that holds an infinity or
  // NaN there
  __shared__ int odd_from[DIFF ? 128 : 1], odd_seen;

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int split = blockIdx.x, b = CUT ? 0 : blockIdx.z, chunk = p.chunk;
  const int kv = blockIdx.y;
  const int G = p.G, rows = p.T_q * G;  // rows <= 128 (checked on the host)
  auto out_row = [&](int r) -> size_t {
    return ((size_t)b * p.T_q + r / G) * p.H_q + kv * G + r % G;
  };
  const size_t n_rows = (size_t)p.B * p.T_q * p.H_q;  // rows of out, lse and the workspace
  // NaN outputs of a row (one split), or its partial (m, l) alone (O is not read)
  auto write_nan_or_ml = [&](size_t row, float2 ml) {
    if (p.n_split == 1) {
      if (DIFF && (row & 1)) {
        // (the head's output row is its first map's to write)
      } else if (const size_t at = (DIFF ? row / 2 : row) * 128;
                 in_bounds(at, 128, (DIFF ? n_rows / 2 : n_rows) * 128, p.err)) {
        for (int c = 0; c < 128; ++c) p.out[at + c] = __float2bfloat16(NAN);
      }
      if (in_bounds(row, 1, n_rows, p.err)) p.lse[row] = NAN;
    } else if (in_bounds(row * p.n_split + split, 1, n_rows * p.n_split, p.err)) {
      p.ws_ml[row * p.n_split + split] = ml;
    }
  };

  // Set-up that touches no global memory runs before the dependency wait.
  volatile int* abort_v = &abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&drain), 1);
    for (int s = 0; s < kTcSlots; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&s_full[x]), 1);
      mbar_init(smem_u32(&p_ready[x]), 4);
    }
    mbar_init(smem_u32(&pv_done), 1);
    if (DIFF) odd_seen = 0;
    abort_flag = 0;
    bad_page = 0;
    fence_barrier_init();
  }
  if (DIFF && threadIdx.x < 128) odd_from[threadIdx.x] = 0x7fffffff;
  // Q rows past T_q * G are zero (their S, P and O rows are never stored, but
  // stay finite); the TMA box fills rows 0 .. rows - 1 only.
  for (int i = threadIdx.x; i < (128 - rows) * 16; i += kTcThreads) {
    const int r = rows + i / 16, c = i % 16;
    st_shared_v4(sb + kOffQ + (c >> 3) * kHalfB + r * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  // A batch cut by its lengths: the cut is worked out while the previous kernel
  // finishes, from relaxed loads, and again after the dependency wait if a length has
  // changed.
  Piece piece{0, 0, 0, 0};
  int cut_tiles[3] = {0, 0, 0};
  auto tiles_of = [&](int L) {
    return L < p.T_q || L > p.S_max ? 0 : (L + kTcKeys - 1) / kTcKeys;
  };
  auto take_piece = [&]() {
    if constexpr (CUT) {
      piece = find_piece(cut_tiles[0], cut_tiles[1], cut_tiles[2], p.B, p.n_split, pp.pieces,
                         blockIdx.x, lane);
      // (the same in every lane; a reduction's result is known to be)
      piece.b = __reduce_max_sync(0xffffffffu, piece.b);
      piece.split = __reduce_max_sync(0xffffffffu, piece.split);
      piece.count = __reduce_max_sync(0xffffffffu, piece.count);
      piece.tiles = __reduce_max_sync(0xffffffffu, piece.tiles);
      b = max(piece.b, 0);
      split = piece.split;
      chunk = piece.tiles * kTcKeys;
    }
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
  // While the previous kernel finishes, the producer warp prefetches this
  // split's first K/V tiles into L2, one tile (paged: one page segment of a
  // tile) per lane; the launcher enables it when the whole grid is resident at
  // once.  The extent comes from a relaxed load of seq_lens[b] and, for a
  // paged cache, the rows from relaxed loads of the block table; they may see
  // values from before the previous kernel's writes and only aim the prefetch
  // (an index outside the pool is skipped).  A prefetch hands no data to the
  // kernel and L2 is where writes become coherent.
  if (warp == 0 && p.prefetch_tiles > 0) {
    const int h = PAGED ? min(p.page_size, kTcKeys) : kTcKeys;  // rows per box
    const int nb = kTcKeys / h;
    const int i = lane / nb, sub = lane % nb;
    int L_hint;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(L_hint) : "l"(p.seq_lens + b));
    const int ahead = i * kTcKeys + sub * h, tk = split * chunk + ahead;
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
      if (ok)
        for (int dh = 0; dh < 2; ++dh) {
          tma_prefetch_l2_3d(&tm_k, dh * 64, kv, row);
          tma_prefetch_l2_3d(&tm_v, dh * 64, kv, row);
        }
    }
  }

  // Launched as a programmatic dependent of the previous kernel in the
  // stream: nothing is read or written before that kernel has completed.
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
      for (int r = warp; r < rows; r += kTcThreads / 32)
        for (int i = piece.count + lane; i < p.n_split; i += 32) {
          const size_t at = out_row(r) * p.n_split + i;
          if (in_bounds(at, 1, n_rows * p.n_split, p.err))
            p.ws_ml[at] = make_float2(-INFINITY, 0.f);
        }
  }
  const bool none = CUT && piece.b < 0;  // a CTA past the batch's last piece
  const int L = p.seq_lens[b];
  const bool bad = L < p.T_q || L > p.S_max;  // (L >= T_q >= 1 otherwise)
  const int t0 = split * chunk;
  // (t0 + chunk may pass 2^31 for a sequence's last piece)
  const int t_end = bad || none ? 0 : t0 + min(chunk, L - t0);
  const int n = t_end > t0 ? (t_end - t0 + kTcKeys - 1) / kTcKeys : 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  if (bad || n == 0) {
    // A bad length: NaN outputs and the error bit.  An empty split: the merge
    // identity (-inf, 0); its O is not written.  (One split is never empty.)
    if (bad && threadIdx.x == 0 && split == 0 && kv == 0) atomicOr(p.err, kErrBadSeqLen);
    for (int r = threadIdx.x; r < rows && !none; r += kTcThreads)
      write_nan_or_ml(out_row(r), bad ? make_float2(NAN, NAN) : make_float2(-INFINITY, 0.f));
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
    return;
  }

  // A bounded wait that also gives up once another role has aborted.  A phase
  // that has already completed passes at once: the abort flag is read only on
  // the slow path, since a shared-memory load in front of every wait delays
  // the MMA warp's next issue (the tensor core queues about one instruction).
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(smem_u32(bar), parity)) return true;
    if (*abort_v) return false;
    if (mbar_wait(smem_u32(bar), parity, p.wait_ns, p.err)) return true;
    *abort_v = 1;
    return false;
  };
  // The same, taken by every lane of a warp, with one agreed result.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    const bool ok = wait(bar, parity);
    return __all_sync(0xffffffffu, ok);
  };

  if (warp == 0) {
    // ----------------------------------------------------------- TMA producer --
    // The whole warp runs the loop (so that the page indices of a tile are
    // read in parallel, one per lane); lane 0 arms each barrier before any
    // copy of its tile is issued.
    const uint32_t qb = smem_u32(&q_full);
    if (lane == 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      mbar_arrive_expect_tx(qb, static_cast<uint32_t>(rows) * (DIFF == 2 ? 128u : 256u));
      if constexpr (DIFF == 2) {  // all half rows, in the order of the maps
        tma_load_4d(sb + kOffQ, &tm_q, qb, 0, 0, kv * (G / 2), b * p.T_q);
      } else {
        for (int dh = 0; dh < 2; ++dh)
          tma_load_3d(sb + kOffQ + dh * kHalfB, &tm_q, qb, dh * 64, kv * G, b * p.T_q);
      }
    }
    // K_0, then K_{j+1} and V_j: the order in which the tensor core reads
    // them.  A tile's slot is refilled once the MMA that read it completed.
    int k_issued = 0, v_issued = 0;
    // Paged: boxes of h rows, one page each (h = page_size up to 128), box i
    // of a tile issued by lane i.  Each tile's page indices are read once,
    // two tiles ahead, so the reads are in flight while the producer waits for
    // a slot; K_j and V_j use the same boxes.  A box wholly past the split end
    // reads rows past the pool, which TMA fills with zeros, so that every tile
    // still receives its full bytes.
    const int h = PAGED ? min(p.page_size, kTcKeys) : kTcKeys;
    const int nb = kTcKeys / h;  // <= 8 (page_size >= 16)
    struct Box {
      int pg;
      bool has;
    };
    auto fetch = [&](int j) -> Box {  // this lane's page of tile j
      Box x;
      const int tok = t0 + j * kTcKeys + lane * h;
      x.has = PAGED && lane < nb && j < n && tok < t_end;
      x.pg = x.has ? p.block_table[(size_t)b * p.max_blocks + tok / p.page_size] : 0;
      return x;
    };
    // every K/V tile is read by this CTA alone, once: evict-first in L2
    const uint64_t kv_pol = l2_policy_evict_first();
    auto issue = [&](bool is_k, int j, Box x) -> bool {
      const int slot = j % kTcSlots;
      uint64_t* empty = is_k ? &k_empty[slot] : &v_empty[slot];
      if (j >= kTcSlots && !wait_all(empty, ((j / kTcSlots) - 1) & 1)) return false;
      const uint32_t fb = smem_u32(is_k ? &k_full[slot] : &v_full[slot]);
      const uint32_t dst = sb + (is_k ? kOffK : kOffV) + slot * kTileB;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      const int tok0 = t0 + j * kTcKeys;
      if constexpr (!PAGED) {
        if (lane == 0) {
          mbar_arrive_expect_tx(fb, kTileB);
          for (int dh = 0; dh < 2; ++dh)
            tma_load_3d(dst + dh * kHalfB, map, fb, dh * 64, kv, b * p.S_max + tok0, kv_pol);
        }
      } else {
        const bool bad = x.has && (x.pg < 0 || x.pg >= p.num_pages);
        const int row = x.has ? (bad ? 0 : x.pg) * p.page_size + (tok0 + lane * h) % p.page_size
                              : p.num_pages * p.page_size;
        // a bad index is recorded before lane 0's arrive releases it
        if (__any_sync(0xffffffffu, bad) && lane == 0) {
          if (!*reinterpret_cast<volatile int*>(&bad_page)) atomicOr(p.err, kErrBadPage);
          *reinterpret_cast<volatile int*>(&bad_page) = 1;
        }
        if (lane == 0) mbar_arrive_expect_tx(fb, kTileB);
        __syncwarp();
        if (lane < nb)
          for (int dh = 0; dh < 2; ++dh)
            tma_load_3d(dst + dh * kHalfB + lane * h * 128, map, fb, dh * 64, kv, row, kv_pol);
      }
      return true;
    };
    Box box_j = fetch(0), box_j1 = fetch(1);  // tiles j and j + 1
    bool ok = issue(true, 0, box_j);
    if (ok) k_issued = 1;
    for (int j = 0; ok && j < n; ++j) {
      const Box box_j2 = fetch(j + 2);
      if (j + 1 < n) {
        ok = issue(true, j + 1, box_j1);
        if (!ok) break;
        k_issued = j + 2;
      }
      ok = issue(false, j, box_j);
      if (ok) v_issued = j + 1;
      box_j = box_j1;
      box_j1 = box_j2;
    }
    if (lane == 0) {
      // The next kernel in the stream may be scheduled now; it waits for this
      // grid before it reads anything.
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // No copy may still target shared memory when the CTA exits.
      for (int j = max(0, k_issued - kTcSlots); j < k_issued; ++j)
        mbar_wait(smem_u32(&k_full[j % kTcSlots]), (j / kTcSlots) & 1, p.wait_ns, p.err);
      for (int j = max(0, v_issued - kTcSlots); j < v_issued; ++j)
        mbar_wait(smem_u32(&v_full[j % kTcSlots]), (j / kTcSlots) & 1, p.wait_ns, p.err);
      mbar_wait(qb, 0, p.wait_ns, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer --
    constexpr uint32_t idS = instr_desc_bf16_f32(128, 128, false);
    constexpr uint32_t idPV = instr_desc_bf16_f32(128, 128, true);
    auto issue_s = [&](int x, int slot) {  // S_x = Q K^T
      const uint32_t kb = sb + kOffK + slot * kTileB;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * kHalfB + (kk & 3) * 32;
        if constexpr (DIFF == 2)
          tc_mma_ss_lanes(tmem + 128 * x, smem_desc_sw128(sb + kOffQ + (kk & 3) * 32, 16, 1024),
                          smem_desc_sw128(kb + off, 16, 1024), idS, (kk & 3) > 0,
                          kk < 4 ? 0xaaaaaaaau : 0x55555555u);
        else
          tc_mma_ss(tmem + 128 * x, smem_desc_sw128(sb + kOffQ + off, 16, 1024),
                    smem_desc_sw128(kb + off, 16, 1024), idS, kk > 0);
      }
    };
    auto issue_pv = [&](int x, int slot, bool acc) {  // O (+)= P_x V, P_x in tensor memory
      const uint32_t vb = sb + kOffV + slot * kTileB;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        tc_mma_ts(tmem + kColO, tmem + 128 * x + 8 * kk, smem_desc_sw128(vb + kk * 2048, kHalfB, 1024),
                  idPV, (acc || kk > 0) ? 1 : 0);
    };
    // P_j V_j once V_j has landed and the softmax has written P_j; then V_j's
    // slot is free.
    auto finish_tile = [&](int j) -> bool {
      if (!wait_all(&v_full[j % kTcSlots], (j / kTcSlots) & 1)) return false;
      if (!wait_all(&p_ready[j & 1], (j >> 1) & 1)) return false;
      tc_fence_after();
      issue_pv(j & 1, j % kTcSlots, j > 0);
      tc_commit(smem_u32(&pv_done));
      tc_commit(smem_u32(&v_empty[j % kTcSlots]));
      return true;
    };
    bool ok = wait_all(&q_full, 0);
    // Tensor-pipe order S_0, S_1, P_0 V_0, S_2, P_1 V_1, ...: S_{j+1} runs while
    // the softmax works on S_j.  S_j overwrites P_{j-2}, whose P V was issued
    // before it (the MMAs of one thread execute in issue order).
    for (int j = 0; ok && j < n; ++j) {
      const int slot = j % kTcSlots;
      if (!wait_all(&k_full[slot], (j / kTcSlots) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      issue_s(j & 1, slot);
      tc_commit(smem_u32(&s_full[j & 1]));
      tc_commit(smem_u32(&k_empty[slot]));
      if (j > 0 && !finish_tile(j - 1)) ok = false;
    }
    if (ok) finish_tile(n - 1);
    // Every MMA issued here has completed (and every commit has landed)
    // before tensor memory is released.
    tc_commit(smem_u32(&drain));
    mbar_wait(smem_u32(&drain), 0, p.wait_ns, p.err);
    __syncwarp();
  } else {
    // ------------------------------------------------- softmax + epilogue --
    const int quarter = warp & 3;  // tensor-memory lanes 32 * quarter ..
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_base + kColO;
    const float c2 = p.scale_log2;
    // Keys below `lim` are visible from this row: query t = r / G sees keys up
    // to L - T_q + t, and this split ends at t_end.  The bound shared by every
    // real row is lim_lo; tiles wholly below it need no mask.
    const int lim = r < rows ? min(t_end, L - p.T_q + 1 + r / G) : t_end;
    const int lim_lo = min(t_end, L - p.T_q + 1);
    float m_ref = -INFINITY, l = 0.f;
    bool alive = true;
    for (int j = 0; j < n; ++j) {
      const int x = j & 1;
      const uint32_t tS = tmem + lane_base + 128 * x;
      if (!wait_all(&s_full[x], (j >> 1) & 1)) {
        alive = false;
        break;
      }
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));

      const int tb = t0 + j * kTcKeys;  // key of column 0
      if (tb + kTcKeys > lim_lo) {
        const int vis = lim - tb;  // columns c < vis are visible
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= vis) sr[c] = __float_as_uint(-INFINITY);
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 8) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          m4[u] = fmax3(m4[u], __uint_as_float(sr[c + 2 * u]), __uint_as_float(sr[c + 2 * u + 1]));
      }
      const float m_tile = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * c2;  // c2 > 0
      float alpha = 1.f;
      bool rescale = false;
      // No visible key in this row so far: l and O are 0, nothing to rescale.
      if (m_ref == -INFINITY) {
        m_ref = m_tile;
      } else if (m_tile > m_ref + kRescaleLog2) {
        alpha = ex2_approx(m_ref - m_tile);
        m_ref = m_tile;
        rescale = true;
      }
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;

      // P = 2^(x c2 - m_ref), summed in fp32, written as packed bf16 over the
      // first 64 columns of S_x: the A operand of P_j V_j.
      float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 16) {
        uint32_t pk[8];
#pragma unroll
        for (int g8 = 0; g8 < 16; g8 += 8) {
          float e[8];
#pragma unroll
          for (int u = 0; u < 8; u += 2)
            ffma2(e[u], e[u + 1], __uint_as_float(sr[c0 + g8 + u]), __uint_as_float(sr[c0 + g8 + u + 1]),
                  c2, c2, neg, neg);
#pragma unroll
          for (int u = 0; u < 8; ++u) e[u] = ex2_approx(e[u]);
          fadd2(sa0, sa1, sa0, sa1, e[0], e[1]);
          fadd2(sb0, sb1, sb0, sb1, e[2], e[3]);
          fadd2(sa0, sa1, sa0, sa1, e[4], e[5]);
          fadd2(sb0, sb1, sb0, sb1, e[6], e[7]);
#pragma unroll
          for (int u = 0; u < 4; ++u) pk[g8 / 2 + u] = pack_bf16x2(e[2 * u], e[2 * u + 1]);
        }
        tmem_st8(tS + c0 / 2, pk);
      }
      l = l * alpha + ((sa0 + sa1) + (sb0 + sb1));

      // P_{j-1} V_{j-1} has completed, so O is stable (P_j V_j is issued only
      // after p_ready below).  Every tile takes this wait, so the completions
      // of pv_done are consumed strictly in order.
      if (j > 0) {
        if (!wait_all(&pv_done, (j - 1) & 1)) {
          alive = false;
          break;
        }
        tc_fence_after();
      }
      // O rows of this warp whose reference moved: O *= alpha (never on the
      // first tile, where m_ref starts from -inf).
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
          reg_fence32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(tO + 32 * c, o);
        }
      }

      // Cache rows at or past the split end may hold anything (even NaN: the
      // padding of a sequence, or the next sequence's rows), and 0 * NaN would
      // reach O through P V, so row r of this V tile is zeroed if it lies past
      // the end, once the tile has landed (it is refilled only after P_j V_j).
      // (Differential: nor may what the last T_q tokens hold reach the queries before
      // them.  Elements that are not finite become zeros, and the epilogue gives NaN in
      // their columns to the rows that see them.)
      if (tb + kTcKeys > (DIFF ? lim_lo : t_end)) {
        if (!wait_all(&v_full[j % kTcSlots], (j / kTcSlots) & 1)) {
          alive = false;
          break;
        }
        if (tb + r >= t_end) {
          const uint32_t vrow = sb + kOffV + (j % kTcSlots) * kTileB + r * 128;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int c16 = 0; c16 < 8; ++c16)
              st_shared_v4(vrow + hh * kHalfB + c16 * 16, 0u, 0u, 0u, 0u);
        }
        if constexpr (DIFF != 0) {
          // (16-byte pieces of those rows, shared out among the threads: a row's thread
          // looking through its row alone took 4 us)
          const int first = max(lim_lo - tb, 0), pieces = (min(t_end - tb, kTcKeys) - first) * 16;
          for (int e = threadIdx.x - 64; e < pieces; e += 128) {
            const int row = first + (e >> 4), u = e & 15;
            const uint32_t at = sb + kOffV + (j % kTcSlots) * kTileB + (u >> 3) * kHalfB + row * 128 +
                                (u & 7) * 16;
            uint4 w = ld_shared_v4(at);
            auto odd = [](uint32_t x) {
              return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
            };
            if (odd(w.x) || odd(w.y) || odd(w.z) || odd(w.w)) {
              // piece u of its half is logical piece (u ^ row) % 8 (128-byte swizzle)
              const int col0 = (u >> 3) * 64 + ((u ^ row) & 7) * 8;
              uint32_t* const wp = &w.x;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t ex = i & 1 ? 0x7f800000u : 0x7f80u;
                if ((wp[i / 2] & ex) != ex) continue;
                wp[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                atomicMin(&odd_from[col0 + i], tb + row);
              }
              st_shared_v4(at, w.x, w.y, w.z, w.w);
              odd_seen = 1;
            }
          }
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_ready[x]));
    }

    // Epilogue: the last P V, then O / l and LSE, or this split's partial.
    // Paged: a bad page index (recorded before the producer's arrive on the
    // last V tile, which this wait acquires) makes the outputs NaN.
    bool page_ok = true;
    // (every warp comes here; what the others found in V is in place behind this)
    if constexpr (DIFF != 0) named_bar_sync(1, 128);
    if (PAGED && alive) {
      if (wait_all(&v_full[(n - 1) % kTcSlots], ((n - 1) / kTcSlots) & 1))
        page_ok = *reinterpret_cast<volatile int*>(&bad_page) == 0;
      else
        alive = false;
    }
    if (alive && page_ok && wait_all(&pv_done, (n - 1) & 1)) {
      tc_fence_after();
      const bool store = r < rows;
      const size_t row = store ? out_row(r) : 0;
      const bool one = p.n_split == 1;
      const float inv = 1.f / l;
      if constexpr (DIFF != 0) {
        if (odd_seen) {  // NaN where this row sees what was not finite in V
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (odd_from[32 * c + i] < lim) o[i] = __float_as_uint(NAN);
            tmem_st32(tO + 32 * c, o);
          }
          tmem_wait_st();
        }
      }
      auto load_o = [&](int c, uint32_t (&o)[32]) {  // 32 columns of this row's O
        tmem_ld32(tO + 32 * c, o);
        tmem_wait_ld();
        reg_fence32(o);
      };
      if constexpr (DIFF != 0) {
        if (one) {
          // Lanes 2h and 2h + 1 hold the maps of a head: of each chunk the even lane takes
          // columns 0 .. 15 of both, the odd one the others.
          const DiffParams& df = pp.diff;
          const bool second = lane & 1;
          const float inv_a = __shfl_sync(0xffffffffu, inv, lane & ~1);
          const float inv_b = __shfl_sync(0xffffffffu, inv, lane | 1);
          const int tq = r / G, head = (kv * G + r % G) >> 1;
          const float lam = store ? df.lam[b * df.lam_b + tq * df.lam_t + head * df.lam_h] : 0.f;
          auto difference = [&](int c, float (&y)[16]) {
            uint32_t o[32];
            load_o(c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? o[i] : o[16 + i], 1);
              const float a = __uint_as_float(second ? got : o[i]);
              const float z = __uint_as_float(second ? o[16 + i] : got);
              y[i] = fmaf(-lam, __fmul_rn(z, inv_b), __fmul_rn(a, inv_a));
            }
          };
          float f = df.out_scale;
          if (df.norm_eps >= 0.f) {
            float ss = 0.f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float y[16];
              difference(c, y);
#pragma unroll
              for (int i = 0; i < 16; ++i) ss += y[i] * y[i];
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            f *= rsqrtf(ss * (1.f / 128.f) + df.norm_eps);
          }
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float y[16];
            difference(c, y);
            const int col = 32 * c + (second ? 16 : 0);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float w0 = df.norm_weight ? df.norm_weight[col + 2 * i] : 1.f;
              const float w1 = df.norm_weight ? df.norm_weight[col + 2 * i + 1] : 1.f;
              w[i] = pack_bf16x2(y[2 * i] * w0 * f, y[2 * i + 1] * w1 * f);
            }
            const size_t at = row / 2 * 128 + col;
            if (store && in_bounds(at, 16, n_rows / 2 * 128, p.err)) {
              *reinterpret_cast<uint4*>(p.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(p.out + at + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
#pragma unroll 1
      for (int c = 0; c < (DIFF && one ? 0 : 4); ++c) {
        uint32_t o[32];
        load_o(c, o);
        if (!store) continue;
        const size_t at = (one ? row : row * p.n_split + split) * 128 + 32 * c;
        if (!in_bounds(at, 32, n_rows * (one ? 1 : p.n_split) * 128, p.err)) continue;
        if (one) {
          uint4* d4 = reinterpret_cast<uint4*>(p.out + row * 128 + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[8 * v + 0]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
            d4[v] = w;
          }
        } else {
          // (the workspace is 256-byte aligned, a partial row 512 bytes)
          float* d = p.ws_O + (row * p.n_split + split) * 128 + 32 * c;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            st_global_v8(d + 8 * v, o[8 * v], o[8 * v + 1], o[8 * v + 2], o[8 * v + 3], o[8 * v + 4],
                         o[8 * v + 5], o[8 * v + 6], o[8 * v + 7]);
        }
      }
      if (store) {
        if (one && in_bounds(row, 1, n_rows, p.err))
          p.lse[row] = (m_ref + log2f(l)) * kLn2;
        else if (!one && in_bounds(row * p.n_split + split, 1, n_rows * p.n_split, p.err))
          // m in natural-log units; a row with no visible key: (-inf, 0)
          p.ws_ml[row * p.n_split + split] = make_float2(m_ref * kLn2, l);
      }
    } else if (r < rows) {  // a wait gave up, or a bad page: this row's outputs are NaN
      write_nan_or_ml(out_row(r), make_float2(NAN, NAN));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

namespace {

template <bool PAGED, int DIFF, bool CUT = false>
cudaError_t launch_tc(const TcParamsOf<DIFF>& p_in, int pieces, const CUtensorMap& tm_q,
                      const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
  auto kern = gqa_decode_tc_kernel<PAGED, DIFF, CUT>;
  static unsigned char attr_done[64];
  static int sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) {
      sm_count[dev] = sms;
      attr_done[dev] = 1;
    }
  }
  TcParamsOf<DIFF> pp = p_in;
  DecodeParams& p = const_cast<DecodeParams&>(base_params(pp));
  // One CTA per SM: the L2 prefetch pays only when every CTA is resident
  // while the previous kernel drains, and for a paged cache only with pages
  // of at least 64 tokens (T_q = 8, Llama3-70B 32K: 28.9 -> 26.5 us at page
  // 128, but 32.8 -> 34.3 us at page 16, whose 24 small boxes per CTA cost
  // more than they hide).
  const long long ctas = pieces > 0 ? (long long)pieces * p.H_kv : (long long)p.n_split * p.H_kv * p.B;
  const int sms = (dev >= 0 && dev < 64) ? sm_count[dev] : 0;
  const bool small_pages = PAGED && p.page_size < 64;
  p.prefetch_tiles = (ctas <= sms && !small_pages) ? GQA_TC_PREFETCH_TILES : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = pieces > 0 ? dim3(pieces, p.H_kv) : dim3(p.n_split, p.H_kv, p.B);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_q, tm_k, tm_v, pp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

bool tc_shape_ok(const DecodeParams& p) {
  return p.d == 128 && p.T_q * p.G <= 128 && p.chunk % kTcKeys == 0;
}

}  // namespace

cudaError_t launch_decode_tc(const DecodeParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, cudaStream_t stream) {
  if (!tc_shape_ok(p)) return cudaErrorInvalidValue;
  return p.block_table ? launch_tc<true, 0>(p, 0, tm_q, tm_k, tm_v, stream)
                       : launch_tc<false, 0>(p, 0, tm_q, tm_k, tm_v, stream);
}

cudaError_t launch_decode_diff_tc(const DecodeDiffParams& p, const CUtensorMap& tm_q,
                                  const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                  cudaStream_t stream) {
  if (!tc_shape_ok(p.dec)) return cudaErrorInvalidValue;
  if (p.pieces > 0 && (p.dec.n_split < 2 || p.pieces <= p.dec.B || p.dec.B > kMaxCut))
    return cudaErrorInvalidValue;
  auto go = [&](auto paged, auto form, auto cut) {
    return launch_tc<decltype(paged)::value, decltype(form)::value, decltype(cut)::value>(
        p, p.pieces, tm_q, tm_k, tm_v, stream);
  };
  auto with_form = [&](auto paged, auto form) {
    return p.pieces > 0 ? go(paged, form, std::true_type{}) : go(paged, form, std::false_type{});
  };
  auto with_page = [&](auto paged) {
    return p.diff.split_keys ? with_form(paged, std::integral_constant<int, 2>{})
                             : with_form(paged, std::integral_constant<int, 1>{});
  };
  return p.dec.block_table ? with_page(std::true_type{}) : with_page(std::false_type{});
}

}  // namespace gqa
