// Log-sum-exp merge of the partials of rows_kernel.cuh, and of a shared
// prefix's partials with those of each sequence's own keys:
//
//   M = max_s lse_s;  w_s = exp(lse_s - M);  O = sum_s w_s O_s / sum_s w_s;
//   lse = M + ln(sum_s w_s)
//
// over normalised fp32 partials, pieces with lse_s = -inf skipped (their rows
// are never read), in a fixed order: the result is bit-identical from run to
// run.  One warp per row; a lane owns HEAD_DIM / 32 consecutive elements.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "combine_kernel.cuh"
#include "rows_kernel.cuh"

namespace gqa {

constexpr int kMergeThreads = 128;  // four rows

// Partials [slots][rows][d] as the decode kernel leaves them: n_pieces (one
// 16-byte record per (batch, KV head) pair, or null) says how many slots hold
// pieces of the pair's rows, else all of them do.
struct DecodePartials {
  const float* o;
  const float* lse;
  const int32_t* n_pieces;
  int slots;
};

struct RowsMergeParams {
  // the rows kernel's partials and records
  const float* o_part;
  const float* lse_part;
  const int2* rec;
  int pieces;               // partial tiles o_part holds: records that name others are ignored
  int tiles, tokens;        // row tiles per triple, tokens per tile
  int groups, kv_heads;     // tile groups; KV heads
  void* out;
  float* lse;
  int out_dtype;
  int batch, nq, Hq, G;
  // the shared prefix only
  int prefix_in_rows;       // the prefix's partials are the rows kernel's (else `prefix`)
  DecodePartials prefix, own;
};

namespace detail {

// A run of partial rows: row `first`, then n - 1 more from `next` in steps of `stride`.
struct PieceRun {
  const float* o;
  const float* lse;
  long long first, next, stride;
  int n;
  __device__ __forceinline__ long long at(int j) const { return j == 0 ? first : next + (j - 1) * stride; }
};

__device__ __forceinline__ PieceRun decode_run(const DecodePartials& d, long long rows, long long row, long long pair) {
  PieceRun r;
  r.o = d.o;
  r.lse = d.lse;
  r.first = row;
  r.next = row + rows;
  r.stride = rows;
  r.n = d.slots;
  if (d.n_pieces != nullptr) {
    const int n = d.n_pieces[pair * 4];
    r.n = n < d.slots ? n : d.slots;
  }
  return r;
}

template <int HEAD_DIM, int RUNS>
__device__ __forceinline__ void merge_row(const PieceRun (&runs)[RUNS], void* out, float* lse, int out_dtype,
                                          long long row) {
  constexpr int VEC = HEAD_DIM / 32;
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < RUNS; ++i)
    for (int j = lane; j < runs[i].n; j += 32) {
      const float v = runs[i].lse[runs[i].at(j)];
      M = v != v || M != M ? NAN : fmaxf(M, v);  // a NaN piece makes the row NaN, not disappear
    }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, M, o);
    M = v != v || M != M ? NAN : fmaxf(M, v);
  }
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  float W = 0.f;
  if (M != -INFINITY) {
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      for (int j0 = 0; j0 < runs[i].n; j0 += 32) {
        const float l = j0 + lane < runs[i].n ? runs[i].lse[runs[i].at(j0 + lane)] : -INFINITY;
        const float w = l == -INFINITY ? 0.f : ptx::ex2_approx((l - M) * kLog2e);
        W += w;
        const int cnt = runs[i].n - j0 < 32 ? runs[i].n - j0 : 32;
        constexpr int kBatch = VEC <= 4 ? 4 : 2;  // partial rows in flight
        for (int j = 0; j < cnt; j += kBatch) {
          float v[kBatch][VEC], wb[kBatch];
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const float ws = __shfl_sync(0xffffffffu, w, (j + q) & 31);
            wb[q] = j + q < cnt ? ws : 0.f;
            if (wb[q] != 0.f) {
              load_vec<VEC>(runs[i].o + runs[i].at(j0 + j + q) * HEAD_DIM + lane * VEC, v[q]);
            } else {
#pragma unroll
              for (int e = 0; e < VEC; ++e) v[q][e] = 0.f;
            }
          }
#pragma unroll
          for (int q = 0; q < kBatch; ++q)
            if (wb[q] != 0.f) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) acc[e] += wb[q] * v[q][e];
            }
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
    const float inv = 1.0f / W;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] *= inv;
  }
  if (out_dtype == kOutF32) {
    float* dst = static_cast<float*>(out) + row * HEAD_DIM + lane * VEC;
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
    for (int i = 0; i < VEC / 2; ++i) {
      if (out_dtype == kOutF16) {
        const __half2 h = __floats2half2_rn(acc[2 * i], acc[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint16_t* dst = static_cast<uint16_t*>(out) + row * HEAD_DIM + lane * VEC;
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
  if (lane == 0 && lse != nullptr) lse[row] = M == -INFINITY ? -INFINITY : M + 0.69314718055994531f * __log2f(W);
}

}  // namespace detail

// The cut triples of a rows-kernel launch: blockIdx.x is the CTA of that
// launch in which a cut triple may begin, blockIdx.y a group of its rows.
template <int HEAD_DIM>
__global__ void __launch_bounds__(kMergeThreads)
gqa_rows_merge_kernel(const RowsMergeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int2 rec = p.rec[blockIdx.x];
  if (rec.x < 0 || rec.y <= 0 || 2 * (static_cast<int>(blockIdx.x) + rec.y) > p.pieces) return;
  const int r = static_cast<int>(blockIdx.y) * (kMergeThreads / 32) + (threadIdx.x >> 5);  // row of the triple's tiles
  const int t = r / kTileRows, rt = r - t * kTileRows;
  const int per_batch = p.kv_heads * p.groups;
  const int b = rec.x / per_batch, hg = rec.x - b * per_batch;
  const int h = hg / p.groups, grp = hg - h * p.groups;
  const int tok = (grp * p.tiles + t) * p.tokens + rt / p.G;
  if (t >= p.tiles || rt >= p.tokens * p.G || tok >= p.nq) return;
  const long long tile_rows = static_cast<long long>(p.tiles) * kTileRows;
  detail::PieceRun run[1];
  run[0].o = p.o_part;
  run[0].lse = p.lse_part;
  run[0].first = (2ll * blockIdx.x + 1) * tile_rows + r;
  run[0].next = 2ll * (blockIdx.x + 1) * tile_rows + r;
  run[0].stride = 2ll * tile_rows;
  run[0].n = rec.y;
  const long long row = (static_cast<long long>(b) * p.nq + tok) * p.Hq + h * p.G + rt % p.G;
  detail::merge_row<HEAD_DIM>(run, p.out, p.lse, p.out_dtype, row);
}

// Every row of a batch: the shared prefix's pieces, then its own keys'.
template <int HEAD_DIM>
__global__ void __launch_bounds__(kMergeThreads)
gqa_prefix_merge_kernel(const RowsMergeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long rows = static_cast<long long>(p.batch) * p.nq * p.Hq;
  const long long row = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  const long long tok = row / p.Hq;  // b * nq + t: the token among the prefix's rows
  const int hq = static_cast<int>(row - tok * p.Hq), h = hq / p.G;
  detail::PieceRun run[2];
  if (p.prefix_in_rows != 0) {
    const long long per_triple = static_cast<long long>(p.tiles) * p.tokens;
    const long long grp = tok / per_triple;
    const int in_triple = static_cast<int>(tok - grp * per_triple);
    const int t = in_triple / p.tokens, rt = (in_triple - t * p.tokens) * p.G + (hq - h * p.G);
    const int2 rec = p.rec[static_cast<long long>(h) * p.groups + grp];
    const long long tile_rows = static_cast<long long>(p.tiles) * kTileRows;
    run[0].o = p.o_part;
    run[0].lse = p.lse_part;
    run[0].first = rec.x * tile_rows + t * kTileRows + rt;
    run[0].next = run[0].first + tile_rows;
    run[0].stride = tile_rows;
    run[0].n = rec.x >= 0 && rec.y > 0 && rec.x <= p.pieces - rec.y ? rec.y : 0;
  } else {
    run[0] = detail::decode_run(p.prefix, rows, row, h);
  }
  run[1] = detail::decode_run(p.own, rows, row, (tok / p.nq) * p.kv_heads + h);
  detail::merge_row<HEAD_DIM>(run, p.out, p.lse, p.out_dtype, row);
}

}  // namespace gqa
