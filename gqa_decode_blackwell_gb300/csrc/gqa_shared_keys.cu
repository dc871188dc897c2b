// Host side of include/gqa_shared_keys.h: argument checks, plans, tensor maps
// and launches of the rows kernel (many query rows over one range of keys)
// and its merges; a cross-attention call of few rows is a decode call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/gqa_shared_keys.h"
#include "host.h"
#include "rows_host.h"
#include "rows_kernel.cuh"
#include "rows_launch.h"
#include "rows_merge.cuh"

namespace gqa {
namespace {

// Units of the plan's line (rows_plan.cuh): a key block against two tiles of
// rows, against one tile alone, at head_dim 256, against few rows (split between
// the tiles); a triple's fixed cost -- Q load, pipeline fill, epilogue -- with
// many rows and with few; the zeros of a triple without keys.  Weights that were
// tuned on whole calls, not times: only the ratios within a launch matter, and a
// launch has blocks of at most two kinds.  (A two-tile block, 14, takes ~1.7 us;
// one at head_dim 256, 8, ~1.4 us: both sections of such a launch have that one.)
// Measured on one GB300, us per call, with the units of a split block and item
// beside (the first line on another: 188, 312, 140, 27.1):
//   7, 16 (here)   128 sequences of up to 2048 keys behind 32768 (64 / 8 heads of
//                  128) 185; 1020 of 200 behind 2000 (32 / 8) 326; 256 of 400
//                  behind 16000 144; 32 of up to 512 behind 4000 28.1
//   8, 32          191, 437, 175, 32.6
//   8, 20          182, 363, 159, 28.2
//   6, 12          203, 293, 162, 27.5
// (a lone tile at 8 units instead of 12: the last of these 37 us, not 31.7, as it
// was then; 64 prompts of 200 tokens, 60 without keys, 35 us, 39 with zeros at 20.)
constexpr int kTwoTileUnits = 14, kLoneTileUnits = 12, kWideUnits = 8, kItemUnits = 32, kZerosUnits = 12;
constexpr int kSplitUnits = 7, kSplitItemUnits = 16;
// An item of the one tile of 128-element heads over pages, against blocks of 8
// (kWideUnits).  The calls above, at 4 / 8 / 12 / 16 / 32 units: 26 tokens 65.9 / 65.3 /
// 65.0 / 65.6 / 66.0 us, 16 tokens 45.7 / 44.3 / 44.0 / 43.8 / 44.4, 1 token 23.4 / 23.2 /
// 23.5 / 23.6 / 24.8.
constexpr int kLoneItemUnits = 12;
// Output elements from which on a merge of all rows costs more than it saves: whole
// triples then write their own.  Measured on GB300 over pages of 500 keys, us a call (all
// partials, whole ones written), 32 / 8 heads: 64 rows of 128 16 sequences 15.3 and
// 16.4, 38 (2.5M elements) 25.4 and 25.0, 76 41.4 and 38.9; 104 rows 10 sequences 14.8
// and 16.5, 19 (2.0M) 19.7 and 19.4, 76 47.3 and 40.4; 32 rows 38 22.5 and 24.0; 120 rows
// of 256 10 (2.5M) 24.3 both ways, 76 90.6 and 68.3; 4 rows of 256 76 58.9 and 60.9.
constexpr long long kWholeElements = 1 << 21;
// Up to this many rows a merge gives each a CTA, whose warps share its pieces;
// beyond, a warp to a row.  Measured on GB300, a whole call: 384 rows of 256
// 28.2 us (33.3 with a warp each), 1024 rows of 128 the same both ways, 2048
// rows of 64 30.9 us (25.8).
constexpr size_t kMergeSharedRows = 1024;

int group_of(const gqa_desc_t* d) { return d->q_heads / d->kv_heads; }

// Few rows fit the decode kernel, which puts the keys along the MMA's M
// dimension and streams them with a 16- or 32-column tile.  Measured on GB300
// (decode kernel, rows kernel): 8 x 8 KV heads of 4096 keys, 4 rows 23.0 and
// 31.4 us, 32 rows 27.1 and 33.6; 8 KV heads of 512 keys, 32 rows 10.8 and
// 10.3; 64 x 8 of 1000 keys, 32 rows 58.1 and 64.6.
bool few_rows(const gqa_desc_t* d) {
  return static_cast<long long>(d->q_tokens) * group_of(d) <= GQA_MAX_QROWS;
}

// Rows that fit one tile are given to both tiles, with the key blocks in turn:
// the softmax of one runs under the other's MMAs.  At head_dim 128 a full tile
// is better left alone, since each piece then writes, and the merge reads, half
// as much, and its blocks come no faster than memory brings them.  Measured on
// GB300 (split, not split): 2 x 8 triples of 128 rows of 128, 4096 keys 23.6
// and 20.8 us, 32768 keys 61.4 and 58.8; of 64 rows 19.6 and 20.4, 56.2 and
// 57.8; 4 x 4 triples of 128 rows of 64, 16384 keys 27.8 and 31.9.
bool split_keys(const gqa_desc_t& d, int tiles) {
  const int G = group_of(&d), tokens = kTileRows / G;
  return tiles == 2 && d.q_tokens <= tokens && (d.head_dim == 64 || d.q_tokens * G <= kTileRows / 2);
}

}  // namespace

RowsLaunch make_launch(const gqa_desc_t* d0, const gqa_desc_t* d1, int sm, bool paged) {
  RowsLaunch r;
  std::memset(&r, 0, sizeof r);
  r.head_dim = d0->head_dim;
  r.q_heads = d0->q_heads;
  r.kv_heads = d0->kv_heads;
  r.in_dtype = d0->in_dtype;
  r.out_dtype = d0->out_dtype;
  r.scale = d0->scale;
  r.status = GQA_ERR_UNSUPPORTED;
  r.n = d1 != nullptr ? 2 : 1;
  r.d[0] = *d0;
  if (d1 != nullptr) r.d[1] = *d1;
  const int G = group_of(d0), most_tokens = kTileRows / G;
  // Rows that fit one tile, over pages: one tile of 128-element heads to a CTA,
  // whose blocks are then deeper in flight and whose items leave one piece, not two.
  // Measured on GB300, us a call (one tile, two): 16 sequences of 1000-8192 keys,
  // 32 / 8 heads, up to 26 tokens 65.0 and 70.1, 8 tokens 57.5 and 60.8; 32 of
  // 300-2048, up to 16 tokens 44.0 and 48.3; 8 of 1000-4096, 1 token 23.4 and 24.6.
  // Batches whose lengths do not fit beside its rings take two.
  const bool lone = paged && d0->head_dim == 128 && d0->q_tokens <= most_tokens && d0->batch <= kMaxLoneEntries;
  const int tiles = d0->head_dim == 256 || lone ? 1 : 2;
  r.tiles = tiles;
  // Triples of rows that fit one tile all leave partials, and so do all triples
  // of a prefix's launch.  But over pages, from kWholeElements on, those that one CTA
  // holds write their rows themselves (of split keys none can).
  const long long elements = static_cast<long long>(d0->batch) * d0->q_tokens * d0->q_heads * d0->head_dim;
  const bool whole = paged && elements >= kWholeElements && !split_keys(*d0, tiles);
  r.every_piece = r.n == 2 || (r.d[0].q_tokens <= most_tokens && !whole);
  long long entries = 0, units = 0;
  for (int i = 0; i < r.n; ++i) {
    const gqa_desc_t& d = r.d[i];
    auto& s = r.s[i];
    s.split_keys = split_keys(d, tiles) ? 1 : 0;
    s.tokens = d.q_tokens < most_tokens ? d.q_tokens : most_tokens;
    s.shift = s.split_keys && s.tokens * G <= kTileRows / 2 ? kTileRows / 2 : 0;
    const int per_group = (s.split_keys ? 1 : tiles) * s.tokens;
    s.groups = (d.q_tokens - 1) / per_group + 1;
    const long long heads = static_cast<long long>(d.kv_heads) * s.groups;
    if (heads * d.batch > INT_MAX / 2) return r;
    s.triples = static_cast<int>(heads * d.batch);
    RowsPlanSection& ps = r.plan.s[i];
    ps.batch = d.batch;
    ps.heads = static_cast<int>(heads);
    ps.groups = s.groups;
    ps.max_len = d.max_seqlen;
    ps.block_units = tiles == 1                  ? kWideUnits
                     : s.split_keys              ? kSplitUnits
                     : d.q_tokens <= most_tokens ? kLoneTileUnits
                                                 : kTwoTileUnits;
    ps.item_units = s.split_keys ? kSplitItemUnits : lone ? kLoneItemUnits : kItemUnits;
    ps.empty_units = r.every_piece ? 0 : kZerosUnits;
    ps.block_div = rows_divisor(ps.block_units);
    entries += d.batch;
    units += static_cast<long long>(s.triples) * rows_units(ps, d.max_seqlen);
  }
  r.plan.dealt = entries > kMaxRowsEntries || units > INT_MAX ? 1 : 0;
  long long ctas = sm;
  if (r.plan.dealt) {
    const long long triples = static_cast<long long>(r.s[0].triples) + r.s[1].triples;
    if (triples < ctas) ctas = triples;
  } else {
    // a CTA per block at most (RowsPlanIter: ranges at least a block long):
    // 4 rows of a 64-element head behind 512 keys take 10.0 us so, and 12.7
    // with half as many
    const int w0 = r.plan.s[0].block_units, w1 = r.plan.s[1].block_units;
    const long long most = units / (w0 > w1 ? w0 : w1);
    if (most < ctas) ctas = most < 1 ? 1 : most;
  }
  r.plan.num_ctas = static_cast<int>(ctas);
  r.plan.ctas_div = rows_divisor(r.plan.num_ctas);
  for (int i = 0; i < r.n; ++i) {
    auto& s = r.s[i];
    if (r.every_piece) s.pieces = r.plan.dealt ? s.triples : s.triples + ctas;
    else s.pieces = r.plan.dealt || ctas == 1 ? 0 : 2 * ctas;
    s.part_row = r.part_rows;
    s.rec = r.records;
    r.part_rows += s.pieces * tiles * s.tokens * G;
    r.records += r.every_piece ? s.triples : (s.pieces > 0 ? ctas : 0);
    if (s.pieces > INT_MAX) return r;
  }
  r.status = GQA_OK;
  return r;
}

RowsWs rows_ws(const RowsLaunch& r) {
  RowsWs w{0, 0, 0};
  if (r.part_rows == 0) return w;
  const size_t rows = static_cast<size_t>(r.part_rows);
  w.ml_off = round_up(rows * r.head_dim * sizeof(float), kWsAlign);
  w.rec_off = w.ml_off + round_up(rows * sizeof(float2), kWsAlign);
  w.total = w.rec_off + round_up(static_cast<size_t>(r.records) * sizeof(int2), kWsAlign);
  return w;
}

bool encode_heads_map(CUtensorMap* m, int in_dtype, const void* base, int head_dim, int heads, int positions,
                      int outer, int64_t head_stride, int64_t pos_stride, int64_t outer_stride, int box_heads,
                      int box_positions, CUtensorMapL2promotion l2) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const CUtensorMapDataType type =
      in_dtype == GQA_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(positions), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[3] = {2 * static_cast<cuuint64_t>(head_stride), 2 * static_cast<cuuint64_t>(pos_stride),
                                 2 * static_cast<cuuint64_t>(outer_stride)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_positions), 1};
  return enc(m, type, 4, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, l2,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

gqa_status_t launch_kernel(const void* fn, dim3 grid, int threads, int smem, void* params, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr = pdl_attr(!env_flag("GQA_DISABLE_PDL"));
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[] = {params};
  return cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status_t run_rows(DeviceState* st, const RowsLaunch& r, const void* q, const Keys* keys, const PagedCall* paged,
                      void* out, float* lse, uint8_t* ws, cudaStream_t stream) {
  RowsParams p;
  std::memset(&p, 0, sizeof p);
  if (encode_fn() == nullptr) return GQA_ERR_CUDA;
  const int G = r.q_heads / r.kv_heads;
  for (int i = 0; i < r.n; ++i) {
    const gqa_desc_t& d = r.d[i];
    RowsSection& s = p.s[i];
    const int64_t D = d.head_dim;
    // dense [B, positions, heads, d]
    auto dense = [&](CUtensorMap* m, const void* base, int heads, int positions, int box_heads, int box_positions) {
      return encode_heads_map(m, d.in_dtype, base, d.head_dim, heads, positions, d.batch, D, D * heads,
                              D * heads * positions, box_heads, box_positions);
    };
    if (!dense(&s.tm_q, q, d.q_heads, d.q_tokens, G, r.s[i].tokens)) return GQA_ERR_INVALID_ARG;
    CUtensorMap* maps[2] = {&s.tm_k, &s.tm_v};
    const void* bases[2] = {keys[i].k, keys[i].v};
    for (int m = 0; m < 2; ++m) {
      bool ok;
      if (paged != nullptr) {
        const gqa_pages_t& g = *paged->geometry;
        // A head's row of 64 elements is 128 bytes, and twice as many would bring
        // another head's, which may be gone before it is asked for (16 sequences of
        // 32768 keys of 8 heads of 64, one loading warp: 248 us with 256-byte fetches, 207 so).
        ok = encode_heads_map(maps[m], d.in_dtype, bases[m], d.head_dim, d.kv_heads, g.page_size, g.num_pages,
                              g.head_stride, g.pos_stride, g.page_stride, 1, 1 << paged->keys.box_shift,
                              d.head_dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
      } else {
        ok = dense(maps[m], bases[m], d.kv_heads, d.max_seqlen, 1, kBlockN);
      }
      if (!ok) return GQA_ERR_INVALID_ARG;
    }
    s.lens = keys[i].lens;
    s.part_row = r.s[i].part_row;
    s.rec = r.s[i].rec;
    s.nq = d.q_tokens;
    s.tokens = r.s[i].tokens;
    s.groups = r.s[i].groups;
    s.split_keys = r.s[i].split_keys;
    s.shift = r.s[i].shift;
    s.causal = d.causal != 0 ? 1 : 0;
  }
  p.plan = r.plan;
  if (paged != nullptr) {
    // Small pages are bound by the warp that issues their boxes.  Measured on GB300, us
    // a call of 16 sequences of 8192 keys, 32 / 8 heads (one loader, two):
    //   64, split keys, 1 token      pages of 16 83 and 56, of 32 60 and 51, of 64 54 and 50
    //   64, split keys, 26 tokens    88 and 62, 64 and 55, 58 and 55
    //   64, 64 tokens                95 and 88, 87 and 88, 87 and 88
    //   128, 64 tokens               116 and 111, 112 and 111, 111 and 111
    // and of 130 sequences of 1024 keys, which at 128 take two tiles however few their rows:
    //   128, split keys, 9 tokens    112 and 112, 105 and 109, 104 and 108
    //   128, 26 tokens               120 and 120, 119 and 120, 119 and 119
    // With pages of 128 split keys of 64 take 97 and 99 (16 sequences of 16384 keys).
    // (One tile has no warp to spare: heads of 128, pages of 16 91 and 87, but 16 trees
    // of 26 tokens in pages of 32 56.5 and 57.6, with either number of loaders, for the
    // warp alone.)
    const int page = paged->geometry->page_size;
    p.pages = paged->keys;
    p.two_loaders = page == 16 || (r.head_dim == 64 && r.s[0].split_keys != 0 && page <= 64) ? 1 : 0;
  }
  const RowsWs w = rows_ws(r);
  if (w.total > 0) {
    p.o_part = reinterpret_cast<float*>(ws);
    p.ml_part = reinterpret_cast<float2*>(ws + w.ml_off);
    p.rec = reinterpret_cast<int2*>(ws + w.rec_off);
    p.o_part_bytes = w.ml_off;
    p.ml_part_bytes = w.rec_off - w.ml_off;
    p.rec_bytes = w.total - w.rec_off;
  }
  const gqa_desc_t& last = r.d[r.n - 1];  // the batch as the caller sees it
  const size_t rows = static_cast<size_t>(last.batch) * last.q_tokens * r.q_heads;
  p.out = out;
  p.lse = lse;
  p.out_bytes = rows * r.head_dim * (r.out_dtype == GQA_DTYPE_FP32 ? 4u : 2u);
  p.lse_bytes = lse != nullptr ? rows * 4u : 0u;
  p.Hq = r.q_heads;
  p.G = G;
  p.out_dtype = r.out_dtype;
  p.out_v32 = aligned(out, 32) ? 1 : 0;
  p.every_piece = r.every_piece ? 1 : 0;
  const float scale = r.scale > 0.f ? r.scale : 1.0f / std::sqrt(static_cast<float>(r.head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  const int longest = r.d[0].max_seqlen > last.max_seqlen ? r.d[0].max_seqlen : last.max_seqlen;
  p.timeout_ns = wait_timeout_ns() + items_in_ring_ns(longest);
  const bool f16 = r.in_dtype == GQA_DTYPE_FP16;
  const int hd = r.head_dim;
  const bool pg = paged != nullptr;
  const KernelRef ref = hd == 64    ? (pg ? rows_kernel_ref_64_1(2, f16) : rows_kernel_ref_64_0(2, f16))
                        : hd == 256 ? (pg ? rows_kernel_ref_256_1(1, f16) : rows_kernel_ref_256_0(1, f16))
                                    : (pg ? rows_kernel_ref_128_1(r.tiles, f16) : rows_kernel_ref_128_0(2, f16));
  const unsigned bit = 24u + (hd == 64 ? 0u : hd == 128 ? 6u : 12u) + (f16 ? 1u : 0u) + (pg ? 2u : 0u) +
                       (hd == 128 && r.tiles == 1 ? 2u : 0u);
  gqa_status_t rc = ensure_smem_attr(st, bit, ref.fn, ref.smem_bytes, ref.regs);
  if (rc != GQA_OK) return rc;
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
  rc = launch_kernel(ref.fn, dim3(static_cast<unsigned>(r.plan.num_ctas)), ref.threads, ref.smem_bytes, &p, stream);
  if (rc != GQA_OK || w.total == 0) return rc;

  RowsMergeParams m;
  std::memset(&m, 0, sizeof m);
  m.o_part = p.o_part;
  m.ml_part = p.ml_part;
  m.rec = p.rec;
  m.n_sections = r.n;
  for (int i = 0; i < r.n; ++i) {
    m.s[i].part_row = r.s[i].part_row;
    m.s[i].rec = r.s[i].rec;
    m.s[i].nq = r.d[i].q_tokens;
    m.s[i].tokens = r.s[i].tokens;
    m.s[i].groups = r.s[i].groups;
    m.s[i].split_keys = r.s[i].split_keys;
    m.s[i].pieces = static_cast<int>(r.s[i].pieces);
  }
  m.out = out;
  m.lse = lse;
  m.out_dtype = r.out_dtype;
  m.batch = last.batch;
  m.nq = last.q_tokens;
  m.Hq = r.q_heads;
  m.G = G;
  m.kv_heads = r.kv_heads;
  m.tiles = r.tiles;
  m.paged = paged != nullptr ? 1 : 0;
  m.err_word = p.err_word;
  m.out_bytes = p.out_bytes;
  m.lse_bytes = p.lse_bytes;
  // Of a paged call's few rows each gets a CTA (below), of more each a place among
  // its tile's.
  if (paged != nullptr && (!r.every_piece || rows > kMergeSharedRows)) {
    const bool cut = !r.every_piece;
    const void* fn = hd == 64    ? (cut ? reinterpret_cast<const void*>(&gqa_tile_merge_kernel<64, true>)
                                        : reinterpret_cast<const void*>(&gqa_tile_merge_kernel<64, false>))
                     : hd == 256 ? (cut ? reinterpret_cast<const void*>(&gqa_tile_merge_kernel<256, true>)
                                        : reinterpret_cast<const void*>(&gqa_tile_merge_kernel<256, false>))
                                 : (cut ? reinterpret_cast<const void*>(&gqa_tile_merge_kernel<128, true>)
                                        : reinterpret_cast<const void*>(&gqa_tile_merge_kernel<128, false>));
    const int per_cta = kTileMergeThreads / 32 * kTileMergeRows;
    const int per_triple = (m.s[0].split_keys ? 1 : m.tiles) * m.s[0].tokens * G;
    return launch_kernel(fn, dim3(static_cast<unsigned>(cut ? r.plan.num_ctas : r.s[0].triples),
                                  (per_triple + per_cta - 1) / per_cta), kTileMergeThreads, 0, &m, stream);
  }
  if (!r.every_piece) {
    const void* fn = hd == 64    ? reinterpret_cast<const void*>(&gqa_rows_merge_kernel<64>)
                     : hd == 256 ? reinterpret_cast<const void*>(&gqa_rows_merge_kernel<256>)
                                 : reinterpret_cast<const void*>(&gqa_rows_merge_kernel<128>);
    const int per_cta = kMergeWarps * (hd == 256 ? kCutRows<256> : kCutRows<128>);
    const int per_triple = m.tiles * m.s[0].tokens * G;
    return launch_kernel(fn, dim3(static_cast<unsigned>(r.plan.num_ctas), (per_triple + per_cta - 1) / per_cta),
                         kMergeThreads, 0, &m, stream);
  }
  const bool share = rows <= kMergeSharedRows;
  const void* fn = hd == 64    ? (share ? reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<64, kMergeWarps>)
                                        : reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<64, 1>))
                   : hd == 256 ? (share ? reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<256, kMergeWarps>)
                                        : reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<256, 1>))
                               : (share ? reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<128, kMergeWarps>)
                                        : reinterpret_cast<const void*>(&gqa_pieces_merge_kernel<128, 1>));
  const size_t want = share ? rows : (rows + kMergeWarps - 1) / kMergeWarps;
  return launch_kernel(fn, dim3(static_cast<unsigned>(want)), kMergeThreads, 0, &m, stream);
}

namespace {

gqa_status_t check_cross(const gqa_desc_t* d) {
  const gqa_status_t rc = check_desc_any_rows(d);
  if (rc != GQA_OK) return rc;
  if (d->causal != 0 || d->reduction != GQA_REDUCE_AUTO || group_of(d) > GQA_MAX_GROUP) return GQA_ERR_UNSUPPORTED;
  // the merge's grid (a row to a quarter of a CTA) and the rows' index arithmetic
  const long long rows = static_cast<long long>(d->batch) * d->q_heads;
  return rows > 0 && d->q_tokens > INT_MAX / rows ? GQA_ERR_UNSUPPORTED : GQA_OK;
}

// The rows of a sequence's own keys, all there are of a causal section, are one
// tile, or the same in both (split_keys): the kernel's causal limit is a row's
// place in its tile.
static_assert(2 * GQA_MAX_QROWS <= kTileRows, "a sequence's own rows are split by keys, never by tokens");

// The prefix as a problem of its own: one entry of B * nq tokens.
gqa_status_t check_prefix(const gqa_desc_t* d, int max_prefix, gqa_desc_t* prefix) {
  const gqa_status_t rc = check_desc(d);
  if (rc != GQA_OK) return rc;
  if (max_prefix < 1) return GQA_ERR_INVALID_ARG;
  if (d->reduction != GQA_REDUCE_AUTO || max_prefix > (1 << 30)) return GQA_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(d->batch) * d->q_tokens * d->q_heads;
  if (rows > INT_MAX) return GQA_ERR_UNSUPPORTED;
  *prefix = *d;
  prefix->batch = 1;
  prefix->q_tokens = d->batch * d->q_tokens;
  prefix->max_seqlen = max_prefix;
  prefix->causal = 0;
  return GQA_OK;
}

}  // namespace

bool output_ok(const void* out, const float* lse) {
  return out != nullptr && aligned(out, 16) && (lse == nullptr || aligned(lse, 4));
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && aligned(ws, kWsAlign));
}

}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_cross_workspace_size(const gqa_desc_t* desc) {
  if (check_cross(desc) != GQA_OK || desc->batch == 0) return 0;
  if (few_rows(desc)) return gqa_decode_workspace_size(desc, 0);
  int dev = 0;
  DeviceState* st = nullptr;
  if (current_device(&dev, &st) != GQA_OK) return 0;
  const RowsLaunch r = make_launch(desc, nullptr, st->sm_count, false);
  return r.status == GQA_OK ? rows_ws(r).total : 0;
}

gqa_status_t gqa_cross_attn(const gqa_desc_t* desc, const void* q, const void* k, const void* v,
                            const int32_t* kv_lens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
  gqa_status_t rc = check_cross(desc);
  if (rc != GQA_OK) return rc;
  if (desc->batch == 0) return GQA_OK;  // nothing to compute; pointers may be null
  if (few_rows(desc))
    return gqa_decode_attn(desc, q, k, v, kv_lens, out, lse, 0, workspace, workspace_bytes, stream);
  if ((rc = check_inputs(q, k, v, kv_lens)) != GQA_OK) return rc;
  if (!output_ok(out, lse)) return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  const RowsLaunch r = make_launch(desc, nullptr, st->sm_count, false);
  if (r.status != GQA_OK) return r.status;
  if (!workspace_ok(workspace, workspace_bytes, rows_ws(r).total)) return GQA_ERR_WORKSPACE;
  const Keys keys[1] = {{k, v, kv_lens}};
  return run_rows(st, r, q, keys, nullptr, out, lse, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

size_t gqa_prefix_workspace_size(const gqa_desc_t* desc, int max_prefix) {
  gqa_desc_t prefix;
  if (check_prefix(desc, max_prefix, &prefix) != GQA_OK || desc->batch == 0) return 0;
  int dev = 0;
  DeviceState* st = nullptr;
  if (current_device(&dev, &st) != GQA_OK) return 0;
  const RowsLaunch r = make_launch(&prefix, desc, st->sm_count, false);
  return r.status == GQA_OK ? rows_ws(r).total : 0;
}

gqa_status_t gqa_prefix_attn(const gqa_desc_t* desc, const void* q, const void* k_prefix, const void* v_prefix,
                             const int32_t* prefix_len, int max_prefix, const void* k_cache, const void* v_cache,
                             const int32_t* seqlens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  gqa_desc_t prefix;
  gqa_status_t rc = check_prefix(desc, max_prefix, &prefix);
  if (rc != GQA_OK) return rc;
  if (desc->batch == 0) return GQA_OK;
  if ((rc = check_inputs(q, k_cache, v_cache, seqlens)) != GQA_OK) return rc;
  if ((rc = check_inputs(q, k_prefix, v_prefix, prefix_len)) != GQA_OK) return rc;
  if (!output_ok(out, lse)) return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  const RowsLaunch r = make_launch(&prefix, desc, st->sm_count, false);
  if (r.status != GQA_OK) return r.status;
  if (!workspace_ok(workspace, workspace_bytes, rows_ws(r).total)) return GQA_ERR_WORKSPACE;
  const Keys keys[2] = {{k_prefix, v_prefix, prefix_len}, {k_cache, v_cache, seqlens}};
  return run_rows(st, r, q, keys, nullptr, out, lse, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_shared_keys_plan(const gqa_desc_t* desc, int prefix_len, int max_prefix, const int32_t* kv_lens_host,
                                  int sm_count, int* num_ctas, int* every_piece, int* info, int32_t* items,
                                  int64_t max_items, int64_t* num_items) {
  gqa_desc_t prefix;
  const bool with_prefix = max_prefix > 0;
  gqa_status_t rc = with_prefix ? check_prefix(desc, max_prefix, &prefix) : check_cross(desc);
  if (rc != GQA_OK) return rc;
  if (desc->batch > 0 && kv_lens_host == nullptr) return GQA_ERR_INVALID_ARG;
  if (sm_count <= 0) {
    int dev = 0;
    DeviceState* st = nullptr;
    if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
    sm_count = st->sm_count;
  }
  if (num_items) *num_items = 0;
  if (desc->batch == 0) return GQA_OK;
  const RowsLaunch r = with_prefix ? make_launch(&prefix, desc, sm_count, false) : make_launch(desc, nullptr, sm_count, false);
  if (r.status != GQA_OK) return r.status;
  if (num_ctas) *num_ctas = r.plan.num_ctas;
  if (every_piece) *every_piece = r.every_piece ? 1 : 0;
  for (int i = 0; i < 2 && info != nullptr; ++i) {
    info[4 * i] = r.s[i].tokens;
    info[4 * i + 1] = r.s[i].groups;
    info[4 * i + 2] = r.s[i].split_keys;
    info[4 * i + 3] = static_cast<int>(r.s[i].pieces);
  }
  const int32_t* raw[2] = {with_prefix ? &prefix_len : kv_lens_host, with_prefix ? kv_lens_host : nullptr};
  // as the kernel stages them (a dealt plan walks the lengths themselves)
  int32_t lens[kMaxRowsEntries];
  uint32_t pre[kMaxRowsEntries + 1] = {0};
  int entries = 0;
  for (int i = 0; i < r.n && !r.plan.dealt; ++i)
    for (int b = 0; b < r.d[i].batch; ++b, ++entries) {
      const RowsPlanSection& s = r.plan.s[i];
      lens[entries] = clamp_len(raw[i][b], s.max_len);
      pre[entries + 1] =
          pre[entries] + static_cast<uint32_t>(s.heads) * static_cast<uint32_t>(rows_units(s, lens[entries]));
    }
  int64_t n = 0;
  auto list = [&](int c, const RowsWork& w) {
    if (items != nullptr && n < max_items) {
      int32_t* o = items + 9 * n;
      const int groups = r.s[w.section].groups, triple = w.b * r.plan.s[w.section].heads + w.hh;
      const bool partial = r.every_piece || w.whole == 0, keys = w.blk_begin < w.blk_end;
      o[0] = c; o[1] = w.section; o[2] = w.b; o[3] = w.hh / groups; o[4] = w.hh % groups;
      o[5] = w.blk_begin; o[6] = w.blk_end;
      o[7] = partial && keys ? rows_piece(r.every_piece, r.plan.dealt != 0, triple, c, w.blk_begin == 0) : -1;
      o[8] = keys ? w.n_pieces : 0;
    }
    ++n;
  };
  for (int c = 0; c < r.plan.num_ctas; ++c) {
    RowsPlanIter it;
    it.init(&r.plan, raw[0], raw[1], lens, pre, c);
    RowsWork w;
    while (it.next(w)) list(c, w);
  }
  for (int e = 0; e < entries && r.every_piece; ++e) {
    RowsWork w;
    std::memset(&w, 0, sizeof w);
    w.section = e < r.plan.s[0].batch ? 0 : 1;
    w.b = e - (w.section ? r.plan.s[0].batch : 0);
    for (; lens[e] == 0 && w.hh < r.plan.s[w.section].heads; ++w.hh) list(empty_owner(r.plan, e), w);
  }
  if (num_items) *num_items = n;
  return GQA_OK;
}

}  // extern "C"
