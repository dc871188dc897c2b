// Log-sum-exp merge of the partials of rows_kernel.cuh, and of a shared
// prefix's partials with those of each sequence's own keys:
//
//   M = max_s lse_s;  w_s = exp(lse_s - M);  O = sum_s w_s O_s / sum_s w_s;
//   lse = M + ln(sum_s w_s)
//
// over normalised fp32 partials, pieces with lse_s = -inf skipped (their rows
// are never read), in a fixed order: the result is bit-identical from run to
// run.  A lane owns HEAD_DIM / 32 consecutive elements of a row; a row
// is one warp's, or (WARPS > 1, launches of few rows) its pieces are dealt to
// a CTA's warps and their sums joined through shared memory.
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
  const float* lse_part;
  const int2* rec;
  int n_sections;
  RowsMergeSection s[2];
  void* out;
  float* lse;
  int out_dtype;
  int batch, nq, Hq, G, kv_heads;
  int tiles;           // row tiles of a triple
};

namespace detail {

// n partial rows: `first`, then from `next` on in steps of `stride`.
struct PieceRun {
  long long first, next, stride;
  int n;
  __device__ __forceinline__ long long at(int j) const { return j == 0 ? first : next + (j - 1) * stride; }
};

__device__ __forceinline__ float max_or_nan(float a, float b) {  // a NaN piece makes the row NaN
  return a != a || b != b ? NAN : fmaxf(a, b);
}

// Merges runs[0 .. n_runs) into row `row`.  With WARPS > 1 the CTA's warps
// share the row, and every thread of the CTA must call it.
template <int HEAD_DIM, int WARPS>
__device__ __forceinline__ void merge_row(const float* __restrict__ o_part, const float* __restrict__ lse_part,
                                          const PieceRun (&runs)[2], int n_runs, void* out, float* lse, int out_dtype,
                                          long long row) {
  constexpr int VEC = HEAD_DIM / 32;
  constexpr int kBatch = 32 / VEC;  // partial rows in flight
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31, warp = WARPS > 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  float M = -INFINITY;
  for (int i = 0; i < n_runs; ++i)
    for (int j = lane; j < runs[i].n; j += 32) M = max_or_nan(M, lse_part[runs[i].at(j)]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = max_or_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  float W = 0.f;  // the weights of this lane's pieces
  if (M != -INFINITY) {
    for (int i = 0; i < n_runs; ++i) {
      // this warp's pieces: warp, warp + WARPS, ...; 32 of them at a time
      for (int j0 = warp; j0 < runs[i].n; j0 += 32 * WARPS) {
        const int mine = j0 + lane * WARPS;
        const float l = mine < runs[i].n ? lse_part[runs[i].at(mine)] : -INFINITY;
        const float w = l == -INFINITY ? 0.f : ptx::ex2_approx((l - M) * kLog2e);
        W += w;
        const int left = (runs[i].n - j0 + WARPS - 1) / WARPS, cnt = left < 32 ? left : 32;
        for (int j = 0; j < cnt; j += kBatch) {
          float v[kBatch][VEC], wb[kBatch];
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const float ws = __shfl_sync(0xffffffffu, w, (j + q) & 31);
            wb[q] = j + q < cnt ? ws : 0.f;
            if (wb[q] != 0.f) {
              load_vec<VEC>(o_part + runs[i].at(j0 + (j + q) * WARPS) * HEAD_DIM + lane * VEC, v[q]);
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
  }
  if constexpr (WARPS > 1) {
    __shared__ float s_acc[WARPS][HEAD_DIM];
    __shared__ float s_w[WARPS];
    __syncthreads();  // a row before is done with them
#pragma unroll
    for (int i = 0; i < VEC; ++i) s_acc[warp][lane * VEC + i] = acc[i];
    if (lane == 0) s_w[warp] = W;
    __syncthreads();
    if (warp != 0) return;
    W = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      W += s_w[k];
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += s_acc[k][lane * VEC + i];
    }
  }
  if (M != -INFINITY) {
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

// The cut triples of a launch of one section: blockIdx.x is the CTA of that
// launch in which a cut triple may begin, blockIdx.y a group of its rows.
template <int HEAD_DIM>
__global__ void __launch_bounds__(kMergeThreads)
gqa_rows_merge_kernel(const RowsMergeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const RowsMergeSection& s = p.s[0];
  const int2 rec = p.rec[blockIdx.x];
  if (rec.x < 0 || rec.y <= 0 || 2 * (static_cast<int>(blockIdx.x) + rec.y) > s.pieces) return;
  const int rows = s.tokens * p.G;  // of a tile
  const int per_batch = p.kv_heads * s.groups;
  const int b = rec.x / per_batch, hg = rec.x - b * per_batch;
  const int h = hg / s.groups, grp = hg - h * s.groups;
  const long long piece_rows = static_cast<long long>(p.tiles) * rows;
  detail::PieceRun run[2];
  run[0].stride = 2ll * piece_rows;
  run[0].n = rec.y;
  // rows of the triple's tiles
  for (int i = static_cast<int>(blockIdx.y) * kMergeWarps + (threadIdx.x >> 5); i < p.tiles * rows;
       i += static_cast<int>(gridDim.y) * kMergeWarps) {
    const int t = i / rows, r = i - t * rows;
    const int tok = (grp * p.tiles + t) * s.tokens + r / p.G;
    if (tok >= s.nq) break;
    run[0].first = (2ll * blockIdx.x + 1) * piece_rows + i;
    run[0].next = 2ll * (blockIdx.x + 1) * piece_rows + i;
    const long long row = (static_cast<long long>(b) * s.nq + tok) * p.Hq + h * p.G + r % p.G;
    detail::merge_row<HEAD_DIM, 1>(p.o_part, p.lse_part, run, 1, p.out, p.lse, p.out_dtype, row);
  }
}

// Every row of a batch, from the pieces of one or two sections: its own keys
// (the last section), and before them the prefix, whose one entry holds all
// the batch's tokens.
template <int HEAD_DIM, int WARPS>
__global__ void __launch_bounds__(kMergeThreads)
gqa_pieces_merge_kernel(const RowsMergeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long rows = static_cast<long long>(p.batch) * p.nq * p.Hq;
  const int mine = WARPS > 1 ? 0 : static_cast<int>(threadIdx.x >> 5);
  for (long long row = static_cast<long long>(blockIdx.x) * (kMergeWarps / WARPS) + mine; row < rows;
       row += static_cast<long long>(gridDim.x) * (kMergeWarps / WARPS)) {
    const uint32_t bt = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.Hq);  // b * nq + t
    const int hq = static_cast<int>(static_cast<uint32_t>(row) - bt * static_cast<uint32_t>(p.Hq)), h = hq / p.G;
    detail::PieceRun run[2];
    for (int i = 0; i < p.n_sections; ++i) {
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
    }
    detail::merge_row<HEAD_DIM, WARPS>(p.o_part, p.lse_part, run, p.n_sections, p.out, p.lse, p.out_dtype, row);
  }
}

}  // namespace gqa
