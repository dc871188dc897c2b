// Attention of many query rows over one range of keys, for sm_103a (TMA +
// tcgen05 + TMEM).
//
// The decode kernel (decode_kernel.cuh) serves at most 32 query rows per KV
// head and puts key positions along the MMA's M dimension.  Here the rows are
// many -- a prompt's tokens against an encoder's states, or every sequence of
// a batch against a prefix they share -- and fill M themselves.  Per tile of
// 128 rows and block of 128 keys of one (batch, KV head) pair:
//
//     S[128 x 128] = Q_tile[128 x d] K_blk[128 x d]^T       (TMEM, fp32)
//     P            = exp2(S * scale*log2e - m)              (online softmax)
//     O[128 x d]  += P[128 x 128] V_blk[128 x d]            (TMEM, fp32)
//
// A tile's rows are the G query heads of T = 128 / G consecutive query tokens
// (row t*G + g), so one TMA box brings them and the heads of a KV head share
// its keys.  Tokens past the last one are zeros, rows past T*G whatever was
// there before; a row of the MMA reaches no other row, and neither is ever
// written out.
//
// Warps: 4 softmax warps per tile, then one TMA producer, one MMA issuer and
// one that walks the plan and hands the others their items through a ring in
// shared memory (so that none of them keeps the plan's state in registers).
// A row of S is one TMEM lane, so one softmax thread holds a whole row: its
// max and sum need no exchange, P goes back into the TMEM columns of its S
// (16-bit, the value MMA's A operand) and never passes through shared memory.
//   head_dim 64, 128: two tiles; one's softmax runs under the other's MMAs.
//     They are 256 rows that share each K/V block, or, where few rows are all
//     there are, the same rows with the key blocks dealt to them in turn
//     ("split keys"): each then leaves a partial of its own.
//   head_dim 256: O takes half of TMEM, so there is one tile, with two S
//     slots: the next block's QK runs under this block's softmax.  K and V
//     blocks are two ring tiles each, their 128-element d-halves.
//
// What bounds it, measured on GB300 (bf16): at head_dim 128 a step of two
// tiles takes ~3200 cycles, in which the tensor core works for 2048, the
// exponential units for 1024 and shared memory for ~2048 (Q and K at QK, which
// alone take all of its 128 bytes a clock; V at PV, the next blocks' arrival).
// The two add up rather than overlap: without exponentials, maxima and sums
// (wrong results, to see) the kernel is only 8% faster, since a QK that shares
// shared memory with an arriving block takes 750-950 cycles and not 516.  2048
// tokens of 32 heads against 8192 keys, 4 of them, run at 1.4 PFLOP/s (769-794
// us, by box; 871 a call in a loop long enough for the card's power limit, which
// takes the clock from 2070 to ~1650 MHz).  At head_dim 256 the one tile takes its K and V, 64 bytes a
// clock, from L2, which gives ~50: a block takes ~2600 cycles, 333 tokens of 16
// heads against 5001 keys, 2 of them, 50 us.  Where a section's rows are
// few, a block costs what its chain takes (~1900 cycles, split between two
// tiles) and an item ~4600 more: its QK, softmax, PV and epilogue follow one
// another, with little to run under them.  A CTA starts its first K load after
// ~4 us, most of it code fetched for the first time.
//
// The running max is only replaced when it grows by more than 8 (log2 units),
// as in the decode kernel; a warp whose rows need it rescales its own lanes
// of O, after the value MMA of the block before has landed.  Warps whose rows
// all lie past the tile's last one only keep step.
//
// Work: rows_plan.cuh.  A launch has one section of batch entries (cross
// attention), or two: a prefix that a batch shares, all its rows as one
// entry, and the sequences' own keys.  Triples that are cut, or all of them
// (every_piece), leave fp32 partials (O_s, its maximum and sum) for
// rows_merge.cuh.
//
// Every wait is bounded, as in the decode kernel, with the time that the items
// in the ring may take on top (items_in_ring_ns).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_kernel.cuh"
#include "rows_plan.cuh"
#include "rows_ptx.cuh"

namespace gqa {

constexpr int kTileRows = 128;  // query rows of a tile (the MMA M dimension)

struct RowsSection {
  CUtensorMap tm_q;     // q [B, nq, Hq, d], box {64, G, tokens, 1}
  CUtensorMap tm_k;     // k [B, S_max, Hkv, d], box {64, 1, 128, 1}
  CUtensorMap tm_v;     // v, same
  const int32_t* lens;  // [B] keys of each entry
  long long part_row;   // first of the section's partial rows
  long long rec;        // first of its records (every_piece)
  int nq;               // query tokens of an entry
  int tokens;           // query tokens of a tile: at most 128 / G
  int groups;           // tile groups of an entry: triples are h * groups + group
  int split_keys;       // both tiles hold the same rows
  // TMEM lane of the second tile's first row: 0, or 64 where split tiles have at
  // most 64 rows, whose warps then are not those of the first tile's scheduler
  // (behind a long prefix 189 us, 192 without)
  int shift;
  int causal;           // token t sees keys j <= L - nq + t
};

struct RowsParams {
  RowsSection s[2];
  RowsPlan plan;
  void* out;            // [B, nq, Hq, d] bf16, fp16 or fp32: the rows of uncut triples
  float* lse;           // [B, nq, Hq] or null
  float* o_part;        // partial rows of d; a piece of a section holds kTiles * tokens * G of them, tile by tile
  float2* ml_part;      // its maximum (log2 units) and sum, one per partial row; sum 0: it saw nothing
  // every_piece: rec[triple] = {first piece, pieces} (0 pieces: no keys), the
  // pieces consecutive.  Else rec[CTA] = {triple, pieces} of the cut triple
  // that begins in this CTA (at most one), or {-1, 0}; its pieces are
  // 2 * CTA + 1 and then 2 * c of the CTAs c that follow.
  int2* rec;
  int Hq, G;
  int out_dtype;
  int out_v32;          // out is 32-byte aligned
  int every_piece;      // every triple leaves partials, none writes out / lse
  float scale_log2;
  unsigned long long timeout_ns;  // of a wait: items_in_ring_ns() among it
  unsigned int* err_word;
  // byte extents of the buffers the kernel writes, checked by -DGQA_DEBUG builds
  unsigned long long out_bytes, lse_bytes, o_part_bytes, ml_part_bytes, rec_bytes;
};

// One item of a CTA: a range of key blocks of one triple.
struct RowsItem {
  int section, b, h;
  int tok0;               // the first query token of its tiles
  int blk_begin, blk_end; // blk_begin < 0: no further item
  int turn;               // the first block taken is blk_begin + turn; after the last comes blk_begin
  __device__ __forceinline__ int block(int i) const {  // the i-th taken
    const int b = blk_begin + turn + i;
    return b < blk_end ? b : b - (blk_end - blk_begin);
  }
  int L;                  // keys of entry b
  int piece;              // where its partials go; -1: final output
};
constexpr int kItemRing = 4;
constexpr uint64_t kBlockNs = 20000;  // far more than a key block of an item takes

// A role may have nothing to do while others work through all the items of the
// ring: the plan's warp, when it is full, and the second tile's warps, where a
// last group of rows fills one tile only, which leave the items they have no
// part in at once and then wait for the next one, or for its first scores.  So
// every wait may take as long as that, beside its timeout.
GQA_HD uint64_t items_in_ring_ns(int max_len) {
  return static_cast<uint64_t>(num_blocks(max_len)) * kItemRing * kBlockNs;
}

template <int HEAD_DIM>
struct RowsCfg {
  static constexpr int kTiles = HEAD_DIM == 256 ? 1 : 2;  // row tiles of a CTA
  static constexpr int kChunks = HEAD_DIM / 64;           // 128-byte swizzle atoms along d
  static constexpr int kTileDim = HEAD_DIM < 128 ? HEAD_DIM : 128;
  static constexpr int kTileChunks = kTileDim / 64;
  static constexpr int kTilesPerBlock = HEAD_DIM / kTileDim;  // ring tiles of a K or V block
  static constexpr int kStageBytes = kBlockN * kTileDim * 2;
  static constexpr int kQTileBytes = kTileRows * HEAD_DIM * 2;  // one of kTiles Q slots, taken in turn
  static constexpr int kQBytes = kTiles * kQTileBytes;
  static constexpr int kStagesK = HEAD_DIM == 64 ? 4 : 2;
  static constexpr int kStagesV = kStagesK;
  static constexpr int kSoftmaxWarps = 4 * kTiles;
  // Two tiles: three warpgroups (softmax, softmax, and the other roles with an
  // idle warp), so that registers can move from the third to the softmax
  // warps, which hold a row of 128 scores each: 384 threads x 168 at launch =
  // 256 x 208 + 128 x 88 (with 168 for all and the plan walked by every role,
  // rows spilled: long prompts took 1230 us, 905 since).  One tile: 224 threads have registers enough.
  static constexpr bool kMoveRegs = kTiles == 2;
  static constexpr int kThreads = kMoveRegs ? 384 : 224;
  static constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kControlRegs = 88;
  static_assert(256 * kSoftmaxRegs + 128 * kControlRegs <= 384 * kLaunchRegs, "more registers than the launch has");
  static constexpr int kRingBytes = (kStagesK + kStagesV) * kStageBytes;
  static constexpr int kItemBytes = kItemRing * static_cast<int>(sizeof(RowsItem));
  static constexpr int kPlanBytes = 4 * (kMaxRowsEntries + 1) + 4 * kMaxRowsEntries;
  static constexpr int kMiscBytes = 512 + kItemBytes + kPlanBytes + 12;
  static constexpr int kSmemBytes = 1024 + kQBytes + kRingBytes + kMiscBytes;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kOCol = 256;  // after the two S slots of 128 columns
  static_assert(kSmemBytes <= 227 * 1024, "shared memory over budget");
  static_assert(kOCol + kTiles * HEAD_DIM <= kTmemCols, "TMEM column plan");
  static_assert(kStagesK % kTilesPerBlock == 0, "rings of whole blocks");
};

// IN_F16: q, k, v (and P) are fp16; otherwise bf16.
template <int HEAD_DIM, bool IN_F16>
__global__ void __launch_bounds__(RowsCfg<HEAD_DIM>::kThreads, 1)
gqa_rows_kernel(const __grid_constant__ RowsParams p) {
  using Cfg = RowsCfg<HEAD_DIM>;
  constexpr int NT = Cfg::kTiles, KCH = Cfg::kChunks, TCH = Cfg::kTileChunks, TPB = Cfg::kTilesPerBlock;
  constexpr uint32_t NSK = Cfg::kStagesK, NSV = Cfg::kStagesV;
  constexpr int kProducerWarp = Cfg::kSoftmaxWarps, kMmaWarp = kProducerWarp + 1, kPlanWarp = kProducerWarp + 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;
  uint8_t* kring = qbuf + Cfg::kQBytes;
  uint8_t* vring = kring + NSK * Cfg::kStageBytes;
  uint8_t* misc = vring + NSV * Cfg::kStageBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(misc);
  RowsItem* items_ring = reinterpret_cast<RowsItem*>(misc + 512);
  uint32_t* s_pre = reinterpret_cast<uint32_t*>(misc + 512 + Cfg::kItemBytes);
  int32_t* s_len = reinterpret_cast<int32_t*>(s_pre + kMaxRowsEntries + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_len + kMaxRowsEntries);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t bar_base = ptx::smem_u32(bar);
  auto BAR = [&](int i) -> uint32_t { return bar_base + 8u * static_cast<uint32_t>(i); };
  // The S, P and O barriers are indexed by S slot: the tile, or (one tile) the
  // block's parity.  A parity wait is sound only while the phase before the
  // awaited one is known to be complete; with one tile, QK(g) is issued ahead
  // of PV(g-1), so S(g) complete says that PV(g-2) has landed, no later one.
  constexpr int K_FULL = 0, K_EMPTY = K_FULL + NSK, V_FULL = K_EMPTY + NSK, V_EMPTY = V_FULL + NSV,
                Q_FULL = V_EMPTY + NSV, Q_EMPTY = Q_FULL + NT, S_FULL = Q_EMPTY + NT, P_HALF = S_FULL + 2,
                P_FULL = P_HALF + 2, O_FULL = P_FULL + 2, DRAIN = O_FULL + 2, ITEM_FULL = DRAIN + 1,
                ITEM_EMPTY = ITEM_FULL + kItemRing, N_BARRIERS = ITEM_EMPTY + kItemRing;
  static_assert(N_BARRIERS <= 64, "barrier words");

  // (a shuffle tells the compiler that it is the same in all the warp)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int n0 = p.plan.s[0].batch, n_entries = n0 + p.plan.s[1].batch;

  // ---------------------------------------------------------------- set-up
  if (warp == 0) {
    for (int i = lane; i < N_BARRIERS; i += 32) {
      uint32_t arrivals = 1;
      if (i >= P_HALF && i < P_FULL + 2) arrivals = 4;         // the softmax warps of a tile
      if (i >= ITEM_EMPTY) arrivals = Cfg::kSoftmaxWarps + 2;  // softmax warps, producer, issuer
      ptx::mbar_init(BAR(i), arrivals);
    }
    if (lane == 0) *abort_flag = 0;
    ptx::fence_barrier_init();
  } else if (warp == kProducerWarp && lane < 6 && p.plan.s[lane / 3].batch != 0) {
    const RowsSection& s = p.s[lane / 3];
    ptx::prefetch_tensormap(lane % 3 == 0 ? &s.tm_q : lane % 3 == 1 ? &s.tm_k : &s.tm_v);
  }
  __syncwarp();
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), Cfg::kTmemCols);
    ptx::tmem_relinquish();
  }
  // Lengths may be produced, and outputs still read, by the previous kernel.
  ptx::griddep_wait();
  // The next launch may set itself up; it waits for this grid before it
  // reads or writes anything this grid touches.
  ptx::griddep_launch_dependents();
  for (int i = threadIdx.x; i < n_entries; i += Cfg::kThreads) {
    const int sec = i < n0 ? 0 : 1;
    const int raw = p.s[sec].lens[i - (sec ? n0 : 0)], L = clamp_len(raw, p.plan.s[sec].max_len);
    if (p.plan.dealt == 0) s_len[i] = L;
    if (raw != L && blockIdx.x == 0) detail::set_error(p.err_word, kErrBadSeqlen, nullptr);
    if (p.plan.dealt != 0 && blockIdx.x != 0) break;  // only flagged, by one CTA
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (p.every_piece != 0 && p.plan.dealt == 0) {
    // the records of entries without keys, which the plan does not list: one
    // thread of this kernel, an item at a time, takes ~0.5 us for each
    for (int i = blockIdx.x; i < n_entries; i += p.plan.num_ctas) {  // empty_owner
      if (s_len[i] > 0) continue;
      const int sec = i < n0 ? 0 : 1, heads = p.plan.s[sec].heads;
      int2* rec = p.rec + p.s[sec].rec + static_cast<long long>(i - (sec ? n0 : 0)) * heads;
      for (int hh = threadIdx.x; hh < heads; hh += Cfg::kThreads)
        if (detail::write_ok(p.err_word, p.rec, p.rec_bytes, rec + hh, sizeof(int2))) rec[hh] = make_int2(-1, 0);
    }
  }
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // The next item of this role (one thread, or a whole warp): waits for it,
  // copies it, releases its place.  False at the end of the work, or, with
  // ok = false, when the wait ran out.
  uint32_t n_items = 0;
  auto next_item = [&](RowsItem& it, bool& ok, bool whole_warp) -> bool {
    const int i = static_cast<int>(n_items % kItemRing);
    ok = ok && ptx::mbar_wait_bounded(BAR(ITEM_FULL + i), (n_items / kItemRing) & 1u, abort_flag, p.timeout_ns);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    it = items_ring[i];
    if (whole_warp) __syncwarp();
    if (lane == 0) ptx::mbar_arrive(BAR(ITEM_EMPTY + i));
    ++n_items;
    return it.blk_begin >= 0;
  };
  // Q slots of an item: its row tiles that hold any token (at least one)
  auto slots_of = [&](const RowsItem& w) {
    const RowsSection& s = p.s[w.section];
    return NT == 2 && s.split_keys == 0 && w.tok0 + s.tokens < s.nq ? 2 : 1;
  };

  if (warp >= kProducerWarp) {
  if constexpr (Cfg::kMoveRegs) ptx::regs_dec<Cfg::kControlRegs>();
  if (warp == kProducerWarp) {
    // ============================================================= producer
    if (lane == 0) {
      uint32_t tk = 0, tv = 0, tq = 0;  // ring tiles and Q slots loaded
      bool ok = true;
      auto load_block = [&](bool is_v, const RowsItem& w, int blk) -> bool {
        const RowsSection& s = p.s[w.section];
#pragma unroll
        for (int hf = 0; hf < TPB; ++hf) {
          const uint32_t n = is_v ? tv : tk, ns = is_v ? NSV : NSK, stage = n % ns;
          const uint32_t full = BAR((is_v ? V_FULL : K_FULL) + static_cast<int>(stage));
          const uint32_t empty = BAR((is_v ? V_EMPTY : K_EMPTY) + static_cast<int>(stage));
          // the first pass over a ring needs no wait
          if (n >= ns && !ptx::mbar_wait_bounded(empty, ((n / ns) & 1u) ^ 1u, abort_flag, p.timeout_ns)) return false;
          ptx::mbar_arrive_expect_tx(full, Cfg::kStageBytes);
          detail::check_coord(p.err_word, w.b >= 0 && w.b < p.plan.s[w.section].batch && w.h >= 0 &&
                                              (w.h + 1) * p.G <= p.Hq && blk >= 0 &&
                                              blk * kBlockN < p.plan.s[w.section].max_len);
          uint8_t* dst = (is_v ? vring : kring) + stage * Cfg::kStageBytes;
#pragma unroll
          for (int kc = 0; kc < TCH; ++kc)
            ptx::tma_load_4d(ptx::smem_u32(dst + kc * 16384), is_v ? &s.tm_v : &s.tm_k, full, (hf * TCH + kc) * 64,
                             w.h, blk * kBlockN, w.b);
          if (is_v) ++tv; else ++tk;
        }
        return true;
      };
      RowsItem it;
      while (next_item(it, ok, false)) {
        if (it.blk_begin >= it.blk_end) continue;
        const RowsSection& s = p.s[it.section];
        const int nt = slots_of(it);
        for (int t = 0; t < nt; ++t, ++tq) {
          const int slot = static_cast<int>(tq % NT);
          if (tq >= NT && !ptx::mbar_wait_bounded(BAR(Q_EMPTY + slot), ((tq / NT) & 1u) ^ 1u, abort_flag, p.timeout_ns)) {
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(BAR(Q_FULL + slot), static_cast<uint32_t>(KCH * s.tokens * p.G * 128));
#pragma unroll
          for (int kc = 0; kc < KCH; ++kc)
            ptx::tma_load_4d(ptx::smem_u32(qbuf + slot * Cfg::kQTileBytes + kc * 16384 + s.shift * 128), &s.tm_q,
                             BAR(Q_FULL + slot), kc * 64, it.h * p.G, it.tok0 + t * s.tokens, it.b);
        }
        // K0, then K(i+1), V(i): at most one block of K ahead of its V
        const int n = it.blk_end - it.blk_begin;
        if (ok) ok = load_block(false, it, it.block(0));
        for (int i = 0; i < n && ok; ++i) {
          if (i + 1 < n) ok = load_block(false, it, it.block(i + 1));
          if (ok) ok = load_block(true, it, it.block(i));
        }
        if (!ok) break;
      }
      if (!ok) detail::set_error(p.err_word, kErrTimeout, abort_flag);
      // The copies issued last land before the CTA exits, whether this thread
      // gave up or another role does while they are on their way.
      for (uint32_t u = tk > NSK ? tk - NSK : 0u; u < tk; ++u)
        ptx::mbar_wait_bounded(BAR(K_FULL + static_cast<int>(u % NSK)), (u / NSK) & 1u, nullptr, p.timeout_ns);
      for (uint32_t u = tv > NSV ? tv - NSV : 0u; u < tv; ++u)
        ptx::mbar_wait_bounded(BAR(V_FULL + static_cast<int>(u % NSV)), (u / NSV) & 1u, nullptr, p.timeout_ns);
      for (uint32_t u = tq > NT ? tq - NT : 0u; u < tq; ++u)
        ptx::mbar_wait_bounded(BAR(Q_FULL + static_cast<int>(u % NT)), (u / NT) & 1u, nullptr, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // =========================================================== MMA issuer
    // The whole warp walks the items, converged, and one elected thread issues.
    {
      constexpr uint32_t idesc_qk = ptx::idesc_f16_f32(128, kBlockN, 0, 0, !IN_F16);
      constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, Cfg::kTileDim, 0, 1, !IN_F16);
      const uint64_t q_desc = ptx::smem_desc_sw128(ptx::smem_u32(qbuf), 16, 1024);
      const uint64_t k_desc = ptx::smem_desc_sw128(ptx::smem_u32(kring), 16, 1024);
      // V as the MN-major B operand: 64-element chunks of d 16 KB apart, 8 keys 1 KB
      const uint64_t v_desc = ptx::smem_desc_sw128(ptx::smem_u32(vring), 16384, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(q_desc), k_lo = static_cast<uint32_t>(k_desc),
                     v_lo = static_cast<uint32_t>(v_desc);
      const uint32_t q_hi = static_cast<uint32_t>(q_desc >> 32), k_hi = static_cast<uint32_t>(k_desc >> 32),
                     v_hi = static_cast<uint32_t>(v_desc >> 32);
      const uint32_t leader = ptx::elect_one();
      bool ok = true;
      uint32_t u = 0;            // K/V blocks
      uint32_t uq = 0;           // Q slots
      uint32_t g[2] = {0u, 0u};  // value MMAs of each S slot
      auto wait = [&](int i, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(BAR(i), parity & 1u, abort_flag, p.timeout_ns));
      };
      RowsItem it;
      while (next_item(it, ok, true)) {
        const int n = __shfl_sync(0xffffffffu, it.blk_end - it.blk_begin, 0);
        if (n <= 0) continue;
        const int nt = __shfl_sync(0xffffffffu, slots_of(it), 0);
        for (int t = 0; t < nt; ++t) wait(Q_FULL + static_cast<int>((uq + t) % NT), (uq + t) / NT);
        // The item's steps j, each a QK and a PV of one block: with two tiles
        // of rows, tile j % 2 and block j / 2; with split keys, tile j % 2 and
        // block j; with one tile, block j (in S slot j % 2 where two are free).
        // S slot t holds S and P of tile t, and the MMAs run in issue order:
        // a step's QK may overwrite the P of the step `ahead` before it once
        // that one's PV is issued.  With one tile and two slots QK(j+1) goes
        // first, over P(j-1), whose PV is issued already.
        const bool two = nt == 2;
        const int steps = two ? 2 * n : n;
        const int ahead = NT == 1 ? 1 : (two || __shfl_sync(0xffffffffu, p.s[it.section].split_keys, 0) != 0 ? 2 : 1);
        // (16-byte units)  Shifted rows are at `shift` in their Q slot: the second tile reads it from its start,
        // the first one from there on, each with rows of other data beside its own.
        const uint32_t q_shift = __shfl_sync(0xffffffffu, static_cast<uint32_t>(p.s[it.section].shift), 0) * 8;
        auto slot_of = [&](int j) -> uint32_t {
          return NT == 1 ? (u + static_cast<uint32_t>(j)) & 1u : (ahead == 2 ? static_cast<uint32_t>(j) & 1u : 0u);
        };
        auto block_of = [&](int j) -> uint32_t { return u + static_cast<uint32_t>(two ? j >> 1 : j); };
        auto qk = [&](int j) {
          const uint32_t slot = slot_of(j), blk = block_of(j), qs = (uq + (two ? slot : 0u)) % NT;
#pragma unroll
          for (int hf = 0; hf < TPB; ++hf) {
            const uint32_t m = blk * TPB + hf, stage = m % NSK;
            if (!two || slot == 0u) wait(K_FULL + static_cast<int>(stage), m / NSK);
            if (!ok) return;
            ptx::tc_fence_after();
            const uint32_t qd = q_lo + ((qs * Cfg::kQTileBytes) >> 4) + (slot == 0u ? q_shift : 0u);
            const uint32_t kd = k_lo + ((stage * Cfg::kStageBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < Cfg::kTileDim / 16; ++kk) {
              const int k = hf * (Cfg::kTileDim / 16) + kk;
              ptx::mma_f16_ss_elect(leader, tmem_base + slot * kBlockN, qd + (k >> 2) * 1024 + (k & 3) * 2, q_hi,
                                    kd + (kk >> 2) * 1024 + (kk & 3) * 2, k_hi, idesc_qk, k > 0 ? 1u : 0u);
            }
          }
          ptx::mma_commit_elect(leader, BAR(S_FULL + static_cast<int>(slot)));
          if (!two || slot == 1u) {  // the block's last use
#pragma unroll
            for (int hf = 0; hf < TPB; ++hf)
              ptx::mma_commit_elect(leader, BAR(K_EMPTY + static_cast<int>((blk * TPB + hf) % NSK)));
          }
          if (j + 1 == steps)
            for (int t = 0; t < nt; ++t) ptx::mma_commit_elect(leader, BAR(Q_EMPTY + static_cast<int>((uq + t) % NT)));
        };
        auto pv = [&](int j) {
          const uint32_t slot = slot_of(j), blk = block_of(j);
          const uint32_t o_tmem = tmem_base + Cfg::kOCol + (NT == 1 ? 0u : slot * HEAD_DIM);
          constexpr int KK = kBlockN / 16, PARTS = NT == 1 ? 1 : 2;
          const bool first = j < (NT == 1 ? 1 : ahead);
          // (V first: it has most often arrived, and P is the one waited for)
          if (TPB == 1 && (!two || slot == 0u)) wait(V_FULL + static_cast<int>(blk % NSV), blk / NSV);
          // P comes in two halves, so that the first one's MMAs run under the
          // last exponentials: 4 x 2048 tokens of 32 heads against 8192 keys
          // 766 us and not 797, a batch behind 32768 keys 194 and not 199
          // (thirds at 1/2 and 3/4: 812, 205).  One tile waits for V, not P.
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            wait((part + 1 < PARTS ? P_HALF : P_FULL) + static_cast<int>(slot), g[slot]);
#pragma unroll
            for (int hf = 0; hf < TPB; ++hf) {
              const uint32_t m = blk * TPB + hf, stage = m % NSV;
              if (TPB > 1) wait(V_FULL + static_cast<int>(stage), m / NSV);
              if (!ok) return;
              ptx::tc_fence_after();
              const uint32_t vd = v_lo + ((stage * Cfg::kStageBytes) >> 4);
#pragma unroll
              for (int kk = part * (KK / PARTS); kk < (part + 1) * (KK / PARTS); ++kk)
                ptx::mma_f16_ts_elect(leader, o_tmem + hf * Cfg::kTileDim, tmem_base + slot * kBlockN + kk * 8,
                                      vd + kk * (2048 >> 4), v_hi, idesc_pv, (kk > 0 || !first) ? 1u : 0u);
            }
          }
          ++g[slot];
          ptx::mma_commit_elect(leader, BAR(O_FULL + static_cast<int>(slot)));
          if (!two || slot == 1u) {
#pragma unroll
            for (int hf = 0; hf < TPB; ++hf)
              ptx::mma_commit_elect(leader, BAR(V_EMPTY + static_cast<int>((blk * TPB + hf) % NSV)));
          }
        };
#pragma unroll 1
        for (int j = -ahead; j < steps && ok; ++j) {
          if constexpr (NT == 1) {
            if (j + 1 < steps) qk(j + 1);
            if (j >= 0 && ok) pv(j);
          } else {
            if (j >= 0) pv(j);
            if (ok && j + ahead < steps) qk(j + ahead);
          }
        }
        u += static_cast<uint32_t>(n);
        uq += static_cast<uint32_t>(nt);
      }
      if (!ok && lane == 0) detail::set_error(p.err_word, kErrTimeout, abort_flag);
      // every MMA has completed before TMEM is released
      ptx::mma_commit_elect(leader, BAR(DRAIN));
      ptx::mbar_wait_bounded(BAR(DRAIN), 0, nullptr, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == kPlanWarp) {
    // ========================================================== plan walker
    if (p.plan.dealt == 0) {
      // exclusive prefix sums of the entries' units
      uint32_t run = 0;
      for (int base = 0; base < n_entries; base += 32) {
        const int i = base + lane;
        uint32_t units = 0;
        if (i < n_entries) {
          const RowsPlanSection& s = p.plan.s[i < n0 ? 0 : 1];
          units = static_cast<uint32_t>(s.heads) * static_cast<uint32_t>(rows_units(s, s_len[i]));
        }
        uint32_t incl = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (i < n_entries) s_pre[i] = run + incl - units;
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) s_pre[n_entries] = run;
      __syncwarp();
    }
    if (lane == 0) {
      bool ok = true;
      int2 cut = make_int2(-1, 0);  // the cut triple that begins in this CTA
      RowsPlanIter iter;
      iter.init(&p.plan, p.s[0].lens, p.s[1].lens, s_len, s_pre, static_cast<int>(blockIdx.x));
      for (uint32_t n = 0; ok; ++n) {
        RowsWork w;
        const bool more = iter.next(w);
        RowsItem it;
        it.blk_begin = -1;
        it.blk_end = -1;
        if (more) {
          const RowsSection& s = p.s[w.section];
          const int triple = w.b * p.plan.s[w.section].heads + w.hh;
          const bool partial = p.every_piece != 0 || w.whole == 0, first_piece = w.blk_begin == 0;
          const int n_pieces = w.blk_begin < w.blk_end ? w.n_pieces : 0;
          it.section = w.section;
          it.b = w.b;
          it.h = w.hh / s.groups;
          it.tok0 = (w.hh - it.h * s.groups) * (NT * s.tokens);
          it.blk_begin = w.blk_begin;
          it.blk_end = w.blk_end;
          it.turn = w.turn;
          it.L = w.L;
          it.piece = partial ? rows_piece(p.every_piece != 0, p.plan.dealt != 0, triple, static_cast<int>(blockIdx.x),
                                          first_piece)
                             : -1;
          if (first_piece && partial) {
            if (p.every_piece == 0)
              cut = make_int2(triple, n_pieces);
            else if (detail::write_ok(p.err_word, p.rec, p.rec_bytes, p.rec + s.rec + triple, sizeof(int2)))
              p.rec[s.rec + triple] = make_int2(it.piece, n_pieces);
          }
        }
        const int i = static_cast<int>(n % kItemRing);
        if (n >= kItemRing)
          ok = ptx::mbar_wait_bounded(BAR(ITEM_EMPTY + i), ((n / kItemRing) & 1u) ^ 1u, abort_flag, p.timeout_ns);
        if (!ok) break;
        items_ring[i] = it;
        ptx::mbar_arrive(BAR(ITEM_FULL + i));
        if (!more) break;
      }
      if (!ok) detail::set_error(p.err_word, kErrTimeout, abort_flag);
      // After a timeout too: the merge then finds places within this launch's
      // partials, though what they hold may be an earlier call's.  Where every
      // triple leaves partials it ignores records that name others.  The output
      // is invalid in either case, and the error word says so.
      if (p.every_piece == 0 && p.rec != nullptr &&
          detail::write_ok(p.err_word, p.rec, p.rec_bytes, p.rec + blockIdx.x, sizeof(int2)))
        p.rec[blockIdx.x] = cut;
    }
    __syncwarp();
  }
  } else {
    // ======================================================== softmax warps
    if constexpr (Cfg::kMoveRegs) ptx::regs_inc<Cfg::kSoftmaxRegs>();
    const int t = warp >> 2;                        // this warp's row tile
    const int r = (warp & 3) * 32 + lane;           // its TMEM lane: a row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem_base + lanes + Cfg::kOCol + static_cast<uint32_t>(t * HEAD_DIM);
    const uint64_t scale2 = ptx::pack_f32x2(p.scale_log2, p.scale_log2);
    uint32_t g = 0;  // blocks of this tile
    uint32_t u = 0;  // K/V blocks of the items before
    bool ok = true;
    auto pack16 = [](float lo, float hi) -> uint32_t {
      if constexpr (IN_F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
      }
    };
    auto wait = [&](int i, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && ptx::mbar_wait_bounded(BAR(i), parity & 1u, abort_flag, p.timeout_ns));
      return ok;
    };

    auto wait_pv = [&](uint32_t blk_g) {  // the value MMA of this tile's block blk_g has landed
      return NT == 2 ? wait(O_FULL + t, blk_g) : wait(O_FULL + static_cast<int>(blk_g & 1u), blk_g >> 1);
    };

    RowsItem it;
    while (next_item(it, ok, true)) {
      const int n_blk = it.blk_end - it.blk_begin;
      const uint32_t u0 = u;
      u += static_cast<uint32_t>(n_blk);
      const bool split_keys = NT == 2 && p.s[it.section].split_keys != 0;
      if (!split_keys && t >= slots_of(it)) continue;
      const int rows = p.s[it.section].tokens * p.G;   // of a tile
      const int first_lane = t == 1 ? p.s[it.section].shift : 0;
      const int rr = r - first_lane;                   // the row within the tile
      const bool active = rr >= lane && rr - lane < rows;  // this warp holds any of them
      // the last key this row sees is L - 1, or (causal) L - nq + its token; all
      // tokens of a causal section are in one tile, and both hold that one (check_prefix)
      const int causal_cut = p.s[it.section].causal != 0 ? p.s[it.section].nq - 1 : 0;
      const int sees = it.L - causal_cut + (causal_cut != 0 ? it.tok0 + rr / p.G : 0);
      const int step = split_keys ? 2 : 1, i0 = split_keys ? t : 0;

      float nm = kNoMax, l = 0.f;  // -max (log2 units; kNoMax while it is -inf) and the sum of this row
      for (int i = i0; i < n_blk; i += step, ++g) {
        const int blk = it.block(i);
        const uint32_t slot = NT == 2 ? static_cast<uint32_t>(t) : (g & 1u);
        const uint32_t s_addr = tmem_base + lanes + slot * kBlockN;
        const bool first = i == i0;
        if (!wait(S_FULL + static_cast<int>(slot), NT == 2 ? g : g >> 1)) break;
        const int tail = it.L - blk * kBlockN;  // keys of this block
        if (tail < kBlockN) {
          // V rows past the end hold whatever the buffer holds there; zero
          // them (up to the capacity, past which TMA wrote zeros) so that
          // 0 * garbage cannot reach O.  One tile's warps do it, before their
          // P lets the issuer start on this V; 8 lanes to a row (a row each
          // would have all 32 on the same banks).  The parity wait is sound: a
          // complete S says that every PV issued before it has landed, among
          // them the one that read the stage's V before (one tile: that is
          // PV(g-1), issued after this S, and waited for).
          const int cap = min(p.plan.s[it.section].max_len - blk * kBlockN, kBlockN);
          if ((t == 0 || split_keys) && cap > tail) {
            if constexpr (NT == 1) {
              if (g >= 1 && !wait_pv(g - 1)) break;
            }
#pragma unroll
            for (int hf = 0; hf < TPB; ++hf) {
              const uint32_t n = (u0 + static_cast<uint32_t>(i)) * TPB + hf, stage = n % NSV;
              if (!wait(V_FULL + static_cast<int>(stage), n / NSV)) break;
              uint8_t* z = vring + stage * Cfg::kStageBytes + (lane & 7) * 16;
#pragma unroll 1
              for (int row = tail + (warp & 3) * 4 + (lane >> 3); row < cap; row += 16) {
#pragma unroll
                for (int kc = 0; kc < TCH; ++kc)
                  *reinterpret_cast<uint4*>(z + kc * 16384 + row * 128) = make_uint4(0, 0, 0, 0);
              }
            }
            if (!ok) break;
            ptx::fence_proxy_async_smem();
          }
        }
        if (!active) {  // no row of this warp is read: whatever its lanes hold may stand for P
          __syncwarp();
          if (NT == 2 && lane == 0) ptx::mbar_arrive(BAR(P_HALF + static_cast<int>(slot)));
          if (lane == 0) ptx::mbar_arrive(BAR(P_FULL + static_cast<int>(slot)));
          continue;
        }
        ptx::tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(s_addr + 32 * c, x + 32 * c);
        ptx::tmem_wait_ld();

        if ((blk + 1) * kBlockN > it.L - causal_cut) {
          const int seen = sees - blk * kBlockN < tail ? sees - blk * kBlockN : tail;
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            if (!__any_sync(0xffffffffu, seen < c + 32)) continue;
            // bits, which the hardware moves to predicates several at a time: half the code of comparisons
            const uint32_t vis = seen >= c + 32 ? 0xffffffffu : seen <= c ? 0u : (1u << (seen - c)) - 1u;
#pragma unroll
            for (int j = c; j < c + 32; ++j) x[j] = (vis >> (j - c)) & 1u ? x[j] : 0xff800000u;  // -inf
          }
        }

        float mx[4] = {__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]), __uint_as_float(x[3])};
#pragma unroll
        for (int j = 4; j < 124; j += 8) {
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2)
            mx[i2] = ptx::max3(mx[i2], __uint_as_float(x[j + 2 * i2]), __uint_as_float(x[j + 2 * i2 + 1]));
        }
        mx[0] = ptx::max3(mx[0], __uint_as_float(x[124]), __uint_as_float(x[125]));
        mx[1] = ptx::max3(mx[1], __uint_as_float(x[126]), __uint_as_float(x[127]));
        const float m_blk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;  // the scale is positive
        if (first) {
          nm = m_blk == -INFINITY ? kNoMax : -m_blk;
        } else if (__any_sync(0xffffffffu, rr < rows && m_blk + nm > kRescaleThreshold)) {
          // O may be rescaled once the value MMA of the block before has landed
          if (!wait_pv(g - 1)) break;
          ptx::tc_fence_after();
          const float m_old = nm == kNoMax ? -INFINITY : -nm;
          const float m_new = fmaxf(m_old, m_blk);
          const float alpha = m_new == -INFINITY ? 1.f : ptx::ex2_approx(m_old - m_new);
          nm = m_new == -INFINITY ? kNoMax : -m_new;
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < HEAD_DIM / 16; ++c) {
            float o[16];
            ptx::tmem_ld_32x32b_x16(o_addr + 16 * c, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= alpha;
            ptx::tmem_st_32x32b_x16(o_addr + 16 * c, o);
          }
          ptx::tmem_wait_st();
        }

        // P, in place of the scores: 16-bit, two to a column
        const uint64_t nm2 = ptx::pack_f32x2(nm, nm);
        auto exps = [&](int c) {  // of 16 columns
#pragma unroll
          for (int k = 16 * c; k < 16 * c + 16; k += 2) {
            float a, b;
            ptx::unpack_f32x2(ptx::fma_f32x2(ptx::pack_f32x2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), scale2,
                                             nm2), a, b);
            x[k] = __float_as_uint(ptx::ex2_in_order(a));
            x[k + 1] = __float_as_uint(ptx::ex2_in_order(b));
          }
        };
        auto put_p = [&](int c) {
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[j] = pack16(__uint_as_float(x[16 * c + 2 * j]), __uint_as_float(x[16 * c + 2 * j + 1]));
          ptx::tmem_st_32x32b_x8u(s_addr + 8 * c, w);
        };
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          exps(c);
          if (NT == 2 && c == 6) {  // the first half's stores, up to columns 79 by now, have had time
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(BAR(P_HALF + static_cast<int>(slot)));
          }
          if (c > 0) put_p(c - 1);  // under the next exponentials, whose unit then does not wait for it
        }
        put_p(7);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(BAR(P_FULL + static_cast<int>(slot)));

        // the sum, from the unrounded p, under the value MMA
        uint64_t s2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int j = 0; j < 64; ++j)
          s2[j & 3] = ptx::add_f32x2(s2[j & 3], ptx::pack_f32x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])));
        float a, b;
        ptx::unpack_f32x2(ptx::add_f32x2(ptx::add_f32x2(s2[0], s2[1]), ptx::add_f32x2(s2[2], s2[3])), a, b);
        l += a + b;
      }
      if (!ok) break;

      // ------------------------------------------------------------ epilogue
      const bool partial = it.piece >= 0;
      if (n_blk == 0 && partial) continue;  // 0 pieces: the merge reads nothing of this triple
      const bool empty = i0 >= n_blk;       // this tile had no key
      if (!active) continue;
      if (!empty) {
        if (!wait_pv(g - 1)) break;
        ptx::tc_fence_after();
      }
      const RowsSection& sec = p.s[it.section];
      if (partial) {
        // O as it stands, with its maximum and sum: the merge normalises.  Rows
        // of tokens past the last one have a place too, which nothing reads.
        const long long prow = sec.part_row + (static_cast<long long>(it.piece) * NT + t) * rows + rr;
        float* dst = p.o_part + prow * HEAD_DIM;
        const bool store =
            rr < rows && !empty && detail::write_ok(p.err_word, p.o_part, p.o_part_bytes, dst, HEAD_DIM * 4ull);
        if (rr < rows && detail::write_ok(p.err_word, p.ml_part, p.ml_part_bytes, p.ml_part + prow, sizeof(float2)))
          p.ml_part[prow] = make_float2(-nm, l);
        if (empty) continue;
#pragma unroll 1
        for (int c = 0; c < HEAD_DIM; c += 32) {
          uint32_t o[4][8];
          ptx::tmem_ld_32x32b_x32(o_addr + c, o[0]);
          ptx::tmem_wait_ld();
          if (store) {
#pragma unroll
            for (int q = 0; q < 4; ++q) ptx::st_global_v8(dst + c + 8 * q, o[q]);
          }
          __syncwarp();  // the next TMEM load is the whole warp's
        }
        continue;
      }
      // (final rows are never of split or shifted tiles, which leave partials)
      const int r_tok = r / p.G, tok = it.tok0 + t * sec.tokens + r_tok;
      const bool row_valid = r_tok < sec.tokens && tok < sec.nq;
      const long long row = (static_cast<long long>(it.b) * sec.nq + tok) * p.Hq + it.h * p.G + (r - r_tok * p.G);
      const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;  // a row that saw only -inf scores: 0; NaN stays NaN
      const float lse = l > 0.f || l != l ? 0.69314718055994531f * (__log2f(l) - nm) : -INFINITY;
      const bool out16 = p.out_dtype != kOutF32;
      uint8_t* dst = static_cast<uint8_t*>(p.out) + row * (HEAD_DIM * (out16 ? 2 : 4));
      const bool store =
          row_valid && detail::write_ok(p.err_word, p.out, p.out_bytes, dst, HEAD_DIM * (out16 ? 2ull : 4ull));
      if (row_valid && p.lse != nullptr && detail::write_ok(p.err_word, p.lse, p.lse_bytes, p.lse + row, 4ull))
        p.lse[row] = lse;
      auto put = [&](uint8_t* to, const uint32_t (&v)[8]) {
        if (p.out_v32 != 0) {
          ptx::st_global_v8(to, v);
        } else {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
      };
#pragma unroll 1
      for (int c = 0; c < HEAD_DIM / 16; ++c) {  // 16 columns at a time
        float o[16];
        if (!empty) {
          ptx::tmem_ld_32x32b_x16(o_addr + 16 * c, o);
          ptx::tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = empty || inv == 0.f ? 0.f : o[j] * inv;
        if (store) {
          uint32_t v[8];
          if (out16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = pack16(o[2 * j], o[2 * j + 1]);
            put(dst + 32 * c, v);
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(o[8 * q + j]);
              put(dst + 64 * c + 32 * q, v);
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok) detail::set_error(p.err_word, kErrTimeout, abort_flag);
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();  // every role is done with TMEM and shared memory
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace gqa
