// The host side of a rows-kernel launch (gqa_shared_keys.cu), shared with that of
// the paged cache (gqa_paged.cu).
#pragma once
#include "../../include/gqa_paged.h"
#include "host.h"
#include "paged.h"
#include "rows_plan.cuh"

namespace gqa {

// One launch of the rows kernel: its sections, its plan and where each
// section's pieces and records go.
struct RowsLaunch {
  int head_dim, q_heads, kv_heads, in_dtype, out_dtype;
  float scale;
  int n;                  // sections
  int tiles;              // row tiles of a CTA
  gqa_desc_t d[2];        // each section as a problem of its own
  struct { int tokens, groups, split_keys, shift, triples; long long pieces, part_row, rec; } s[2];
  RowsPlan plan;
  bool every_piece;
  long long part_rows, records;
  gqa_status_t status;
};

struct RowsWs {
  size_t ml_off, rec_off, total;
};

struct Keys {  // a section's keys
  const void* k;
  const void* v;
  const int32_t* lens;
};

// Keys in a paged cache (the launch then has one section).
struct PagedCall {
  const gqa_pages_t* geometry;
  PagedKeys keys;
};

// Sections d0 and, for a prefix's launch, d1.  paged: d0's keys are.
RowsLaunch make_launch(const gqa_desc_t* d0, const gqa_desc_t* d1, int sm, bool paged);
RowsWs rows_ws(const RowsLaunch& r);

// The rows kernel and, where it leaves partials, their merge; `ws` holds
// rows_ws() bytes.  paged: null, or where the keys lie.
gqa_status_t run_rows(DeviceState* st, const RowsLaunch& r, const void* q, const Keys* keys, const PagedCall* paged,
                      void* out, float* lse, uint8_t* ws, cudaStream_t stream);

// Tensor map of rank 4 with boxes {64, box_heads, box_positions, 1} over
// [outer, positions, heads, d] with the given strides (in elements).
bool encode_heads_map(CUtensorMap* m, int in_dtype, const void* base, int head_dim, int heads, int positions,
                      int outer, int64_t head_stride, int64_t pos_stride, int64_t outer_stride, int box_heads,
                      int box_positions, CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);

gqa_status_t launch_kernel(const void* fn, dim3 grid, int threads, int smem, void* params, cudaStream_t s);
bool output_ok(const void* out, const float* lse);
bool workspace_ok(const void* ws, size_t bytes, size_t need);

}  // namespace gqa
