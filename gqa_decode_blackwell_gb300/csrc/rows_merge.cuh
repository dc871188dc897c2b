// Merge of the partials of rows_kernel.cuh, and of a shared prefix's partials
// with those of each sequence's own keys.  A piece s of a row is O_s, not
// normalised, its maximum m_s (log2 units) and its sum l_s:
//
//   M = max_s m_s;  w_s = 2^(m_s - M);  W = sum_s w_s l_s;
//   O = sum_s w_s O_s / W;  lse = ln 2 (M + log2 W)
//
// in fp32, in a fixed order: the result is bit-identical from run to run.  A
// warp keeps a running maximum and sums over a row's pieces, whose values it
// loads a batch at a time, all of them before the first is used: what bounds
// the merge is how much it has in flight, not its arithmetic (loads of one
// piece at a time: prompts of 256 tokens 115 us a call, not 94; the merge alone
// takes 12 us there for 80 MB of partials).  A lane owns HEAD_DIM / 32
// consecutive elements.  A piece with l_s = 0 saw nothing, and its O_s, which
// may be anything, takes no part.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "combine_kernel.cuh"
#include "rows_kernel.cuh"

namespace gqa {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

struct RowsMergeSection {
  long long part_row;  // as in RowsSection
  long long rec;
  int nq, tokens, groups, split_keys;
  int pieces;          // pieces its part of o_part holds: records that name others are ignored
};

struct RowsMergeParams {
  const float* o_part;
  const float2* ml_part;
  const int2* rec;
  int n_sections;
  RowsMergeSection s[2];
  void* out;
  float* lse;
  int out_dtype;
  int batch, nq, Hq, G, kv_heads;
  int tiles;           // row tiles of a triple
  int paged;           // a tile's partial rows lie 8 elements of all of them after another
  unsigned int* err_word;
  unsigned long long out_bytes, lse_bytes;  // byte extents, checked by -DGQA_DEBUG builds
};

namespace detail {

// n partial rows: `first`, then from `next` on in steps of `stride`.
struct PieceRun {
  long long first, next, stride;
  int n;
  __device__ __forceinline__ long long at(int j) const { return j == 0 ? first : next + (j - 1) * stride; }
};

// A row's merge so far: M = max_s m_s, W = sum_s 2^(m_s - M) l_s, acc = sum_s 2^(m_s - M) O_s.
template <int VEC>
struct RowSum {
  float M, W, acc[VEC];
  __device__ __forceinline__ void clear() {
    M = -INFINITY;
    W = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  }
  // Adds a piece; an empty one leaves everything as it is.
  __device__ __forceinline__ void add(float2 ml, const float (&v)[VEC]) {
    if (ml.y == 0.f) return;
    const float m = fmaxf(M, ml.x);
    const float a = M == -INFINITY ? 0.f : ptx::ex2_approx(M - m), b = ptx::ex2_approx(ml.x - m);
    M = m;
    W = W * a + b * ml.y;  // (a NaN sum stays one)
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = acc[e] * a + b * v[e];
  }
};

// Pieces first, first + step, ... of n (piece j begins at partial row at(j)) into R consecutive rows' sums, NB of
// them in flight.  This lane's elements are `in_row` past a row's beginning.
template <int HEAD_DIM, int R, int NB, typename At>
__device__ __forceinline__ void add_pieces(RowSum<HEAD_DIM / 32> (&sum)[R], const RowsMergeParams& p, const At& at,
                                           int n, int first, int step, int in_row) {
  constexpr int VEC = HEAD_DIM / 32;
  for (int j0 = first; j0 < n; j0 += NB * step) {
    float2 ml[NB][R];
    float v[NB][R][VEC];
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int j = j0 + q * step;
      const long long row = at(j < n ? j : j0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        ml[q][r] = p.ml_part[row + r];
        load_vec<VEC>(p.o_part + (row + r) * HEAD_DIM + in_row, v[q][r]);
      }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      if (j0 + q * step >= n) break;
#pragma unroll
      for (int r = 0; r < R; ++r) sum[r].add(ml[q][r], v[q][r]);
    }
  }
}

// Two elements of a 16-bit output.
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int out_dtype) {
  if (out_dtype == kOutF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int HEAD_DIM>
__device__ __forceinline__ void write_row(const RowSum<HEAD_DIM / 32>& sum, const RowsMergeParams& p, long long row) {
  constexpr int VEC = HEAD_DIM / 32;
  const int lane = threadIdx.x & 31;
  const bool none = sum.W == 0.f;
  const float inv = none ? 0.f : 1.0f / sum.W;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = none ? 0.f : sum.acc[i] * inv;
  if (p.out_dtype == kOutF32) {
    float* dst = static_cast<float*>(p.out) + row * HEAD_DIM + lane * VEC;
    if (!write_ok(p.err_word, p.out, p.out_bytes, dst, VEC * 4)) return;
    if constexpr (VEC == 8) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
      *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
    }
  } else {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = pack_out(acc[2 * i], acc[2 * i + 1], p.out_dtype);
    uint16_t* dst = static_cast<uint16_t*>(p.out) + row * HEAD_DIM + lane * VEC;
    if (!write_ok(p.err_word, p.out, p.out_bytes, dst, VEC * 2)) return;
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
  if (lane == 0 && p.lse != nullptr && write_ok(p.err_word, p.lse, p.lse_bytes, p.lse + row, 4))
    p.lse[row] = none ? -INFINITY : 0.69314718055994531f * (sum.M + __log2f(sum.W));
}

}  // namespace detail

// Rows a warp of the cut triples' merge takes at once: most of those have two
// pieces, and two pieces of one short row are little to have in flight, while
// many rows leave few warps on an SM (prompts, rows of 128: 86.7 us a call with 2,
// 87.3 with 4, 96.5 with 8; wide heads, of 256: 50.1 with 1, 50.7 with 2).
template <int HEAD_DIM>
constexpr int kCutRows = HEAD_DIM == 256 ? 1 : 2;

// The cut triples of a launch of one section: blockIdx.x is the CTA of that
// launch in which a cut triple may begin, blockIdx.y a group of its rows.
template <int HEAD_DIM>
__global__ void __launch_bounds__(kMergeThreads)
gqa_rows_merge_kernel(const RowsMergeParams p) {
  constexpr int R = kCutRows<HEAD_DIM>;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const RowsMergeSection& s = p.s[0];
  const int2 rec = p.rec[blockIdx.x];
  if (rec.x < 0 || rec.y <= 0 || 2 * (static_cast<int>(blockIdx.x) + rec.y) > s.pieces) return;
  const int rows = s.tokens * p.G;  // of a tile
  const long long piece_rows = static_cast<long long>(p.tiles) * rows;
  // rows i .. i + R - 1 of the triple's tiles (past the last one: the last again)
  const int i0 = (static_cast<int>(blockIdx.y) * kMergeWarps + static_cast<int>(threadIdx.x >> 5)) * R;
  if (i0 >= piece_rows) return;
  const int i = i0 + R <= piece_rows ? i0 : static_cast<int>(piece_rows) - R;
  detail::PieceRun run;
  run.first = (2ll * blockIdx.x + 1) * piece_rows + i;
  run.next = 2ll * (blockIdx.x + 1) * piece_rows + i;
  run.stride = 2ll * piece_rows;
  run.n = rec.y;
  detail::RowSum<HEAD_DIM / 32> sum[R];
#pragma unroll
  for (int r = 0; r < R; ++r) sum[r].clear();
  detail::add_pieces<HEAD_DIM, R, 2>(sum, p, [&](int j) { return run.at(j); }, run.n, 0, 1,
                                     static_cast<int>(threadIdx.x & 31) * (HEAD_DIM / 32));
  const int per_batch = p.kv_heads * s.groups;
  const int b = rec.x / per_batch, hg = rec.x - b * per_batch;
  const int h = hg / s.groups, grp = hg - h * s.groups;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = (i + r) / rows, in_tile = i + r - t * rows;
    const int tok = (grp * p.tiles + t) * s.tokens + in_tile / p.G;
    if (tok >= s.nq) continue;
    const long long row = (static_cast<long long>(b) * s.nq + tok) * p.Hq + h * p.G + in_tile % p.G;
    detail::write_row<HEAD_DIM>(sum[r], p, row);
  }
}

// Every row of a batch, from the pieces of one or two sections: its own keys
// (the last section), and before them the prefix, whose one entry holds all
// the batch's tokens.  WARPS = 1: a warp to a row; else (launches of few rows)
// a CTA, whose warps take its pieces in turn and join their sums.
template <int HEAD_DIM, int WARPS>
__global__ void __launch_bounds__(kMergeThreads)
gqa_pieces_merge_kernel(const RowsMergeParams p) {
  constexpr int VEC = HEAD_DIM / 32;
  // More in flight, or, with wider pieces, more warps on an SM: prefix of drafts
  // (64) 23.5 us with 8 and 24.9 with 4, large prefix (128) 189.4 and 186.8.
  constexpr int NB = HEAD_DIM == 64 && WARPS == 1 ? 8 : 4;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rows = static_cast<uint32_t>(p.batch) * static_cast<uint32_t>(p.nq) * static_cast<uint32_t>(p.Hq);
  const uint32_t row = WARPS > 1 ? blockIdx.x : blockIdx.x * kMergeWarps + warp;
  if (row >= rows) return;
  const uint32_t bt = row / static_cast<uint32_t>(p.Hq);  // b * nq + t
  const int hq = static_cast<int>(row - bt * static_cast<uint32_t>(p.Hq)), h = hq / p.G;
  detail::PieceRun run[2];
  int in_row = lane * VEC;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    run[i].n = 0;
    if (i >= p.n_sections) continue;
    const RowsMergeSection& s = p.s[i];
    const int b = static_cast<int>(bt / static_cast<uint32_t>(s.nq));  // the section's entry, the token within it
    const int tok = static_cast<int>(bt) - b * s.nq;
    const int per_group = (s.split_keys ? 1 : p.tiles) * s.tokens;
    const int grp = tok / per_group, in_group = tok - grp * per_group;
    const int t = in_group / s.tokens, r = (in_group - t * s.tokens) * p.G + (hq - h * p.G);
    const int2 rec = p.rec[s.rec + (static_cast<long long>(b) * p.kv_heads + h) * s.groups + grp];
    const long long tile_rows = static_cast<long long>(s.tokens) * p.G;
    run[i].first = s.part_row + (static_cast<long long>(rec.x) * p.tiles + t) * tile_rows + r;
    run[i].stride = s.split_keys ? tile_rows : p.tiles * tile_rows;
    run[i].next = run[i].first + run[i].stride;
    const bool there = rec.x >= 0 && rec.y > 0 && rec.x <= s.pieces - rec.y;
    run[i].n = !there ? 0 : s.split_keys ? rec.y * p.tiles : rec.y;
    if (p.paged != 0 && i == 0)
      in_row = (in_row / 8 * static_cast<int>(tile_rows) + r) * 8 + in_row % 8 - r * HEAD_DIM;
  }
  detail::RowSum<VEC> sum[1];
  sum[0].clear();
  const int n0 = run[0].n;
  detail::add_pieces<HEAD_DIM, 1, NB>(sum, p, [&](int j) { return j < n0 ? run[0].at(j) : run[1].at(j - n0); },
                                      n0 + run[1].n, WARPS > 1 ? warp : 0, WARPS, in_row);
  if constexpr (WARPS > 1) {
    __shared__ float s_acc[WARPS][HEAD_DIM], s_m[WARPS], s_w[WARPS];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s_acc[warp][lane * VEC + e] = sum[0].acc[e];
    if (lane == 0) {
      s_m[warp] = sum[0].M;
      s_w[warp] = sum[0].W;
    }
    __syncthreads();
    if (warp != 0) return;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) M = fmaxf(M, s_m[k]);
    sum[0].clear();
    sum[0].M = M;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      if (s_w[k] == 0.f) continue;
      const float w = ptx::ex2_approx(s_m[k] - M);
      sum[0].W += w * s_w[k];
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[0].acc[e] += w * s_acc[k][lane * VEC + e];
    }
  }
  detail::write_row<HEAD_DIM>(sum[0], p, row);
}

// The rows of a paged launch whose triples hold many, a triple to blockIdx.x
// (CUT: the cut triple, if any, that begins in that CTA of the launch) and a group
// of its rows to blockIdx.y.  A warp takes four rows, which lie side by side in
// each piece: a lane has 8 elements at a time of one of them, and four lanes a line.
// What the kernels above have in flight for a row or two is here for four, and a row's
// weights are computed by 8 lanes, not 32 (whole calls over pages, us, of those kernels
// and, rows lying one after another, of this one: 16 x 8 tiles of 104 rows of 128
// elements 65.6, 63.7; 32 x 8 of 64 rows 43.7, 41.8; 48 of 128 rows of 256 elements
// 60.3, 58.9).
constexpr int kTileMergeThreads = 128, kTileMergeRows = 4;

template <int HEAD_DIM, bool CUT>
__global__ void __launch_bounds__(kTileMergeThreads)
gqa_tile_merge_kernel(const RowsMergeParams p) {
  constexpr int UNITS = HEAD_DIM / 64, VEC = 8 * UNITS;
  // pieces in flight: 4 against 2, 16 trees of 26 tokens 56.4 and 57.1 us (128), 42.0 and
  // 42.7 (64), but of cut triples, 60 tokens, 75.3 and 72.8 (128)
  constexpr int kBatch = CUT || HEAD_DIM == 256 ? 2 : 4;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const RowsMergeSection& s = p.s[0];
  const int lane = threadIdx.x & 31;
  const int2 rec = p.rec[s.rec + blockIdx.x];
  const int tile_rows = s.tokens * p.G, own_tiles = s.split_keys ? 1 : p.tiles;  // tiles with rows of their own
  const long long piece_rows = static_cast<long long>(p.tiles) * tile_rows;
  int triple = static_cast<int>(blockIdx.x), n = 0;
  detail::PieceRun run;
  if constexpr (CUT) {
    triple = rec.x;
    if (rec.x < 0 || rec.y <= 0 || 2 * (static_cast<int>(blockIdx.x) + rec.y) > s.pieces) return;
    n = rec.y;
    run.first = (2ll * blockIdx.x + 1) * piece_rows;
    run.next = 2ll * (blockIdx.x + 1) * piece_rows;
    run.stride = 2ll * piece_rows;
  } else {
    const bool there = rec.x >= 0 && rec.y > 0 && rec.x <= s.pieces - rec.y;
    n = !there ? 0 : s.split_keys ? rec.y * p.tiles : rec.y;
    run.first = s.part_row + rec.x * piece_rows;
    run.stride = s.split_keys ? tile_rows : piece_rows;
    run.next = run.first + run.stride;
  }
  const int rows = own_tiles * tile_rows;
  const int i0 = (static_cast<int>(blockIdx.y) * (kTileMergeThreads / 32) + static_cast<int>(threadIdx.x >> 5)) *
                 kTileMergeRows;
  if (i0 >= rows) return;
  const int i = min(i0 + (lane & 3), rows - 1);  // (past the last row: the last again)
  const int t = i / tile_rows, in_tile = i - t * tile_rows, unit0 = lane >> 2;
  const float* o = p.o_part + static_cast<long long>(t) * tile_rows * HEAD_DIM + (unit0 * tile_rows + in_tile) * 8;
  detail::RowSum<VEC> sum;
  sum.clear();
  for (int j0 = 0; j0 < n; j0 += kBatch) {
    float2 ml[kBatch];
    float v[kBatch][VEC];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (j0 + q >= n) break;
      const long long at = run.at(j0 + q);
      ml[q] = p.ml_part[at + i];
#pragma unroll
      for (int k = 0; k < UNITS; ++k) {
        float x[8];
        detail::load_vec<8>(o + at * HEAD_DIM + k * 64 * tile_rows, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[q][8 * k + e] = x[e];
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (j0 + q >= n) break;
      sum.add(ml[q], v[q]);
    }
  }
  const int per_batch = p.kv_heads * s.groups;
  const int b = triple / per_batch, hg = triple - b * per_batch;
  const int h = hg / s.groups, grp = hg - h * s.groups;
  const int r_tok = in_tile / p.G, tok = (grp * own_tiles + t) * s.tokens + r_tok;
  if (tok >= s.nq) return;
  const long long row = (static_cast<long long>(b) * s.nq + tok) * p.Hq + h * p.G + (in_tile - r_tok * p.G);
  const bool none = sum.W == 0.f;
  const float inv = none ? 0.f : 1.0f / sum.W;
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    const long long to = row * HEAD_DIM + (unit0 + 8 * k) * 8;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = none ? 0.f : sum.acc[8 * k + e] * inv;
    if (p.out_dtype == kOutF32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + to);
      if (!detail::write_ok(p.err_word, p.out, p.out_bytes, dst, 32)) continue;
      dst[0] = make_float4(y[0], y[1], y[2], y[3]);
      dst[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = detail::pack_out(y[2 * e], y[2 * e + 1], p.out_dtype);
      uint16_t* dst = static_cast<uint16_t*>(p.out) + to;
      if (!detail::write_ok(p.err_word, p.out, p.out_bytes, dst, 16)) continue;
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (unit0 == 0 && p.lse != nullptr && detail::write_ok(p.err_word, p.lse, p.lse_bytes, p.lse + row, 4))
    p.lse[row] = none ? -INFINITY : 0.69314718055994531f * (sum.M + __log2f(sum.W));
}

}  // namespace gqa
