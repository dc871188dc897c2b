// Host side of include/gqa_shared_keys.h: argument checks, plans, tensor maps
// and launches of the rows kernel (many query rows over one range of keys)
// and its merges; few rows go to the decode kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/gqa_shared_keys.h"
#include "host.h"
#include "rows_kernel.cuh"
#include "rows_launch.h"
#include "rows_merge.cuh"

namespace gqa {
namespace {

// Item units X of the balanced plan (plan.cuh): a triple's fixed cost -- Q
// load, pipeline fill, epilogue -- in key blocks.
constexpr int kRowsItemUnits = 1;

int group_of(const gqa_desc_t* d) { return d->q_heads / d->kv_heads; }
int tiles_per_triple(int head_dim) { return head_dim == 256 ? 1 : 2; }
int tile_tokens(const gqa_desc_t* d) { return kTileRows / group_of(d); }
int group_tokens_of(const gqa_desc_t* d) { return tiles_per_triple(d->head_dim) * tile_tokens(d); }

// Few rows fit the decode kernel, which puts the keys along the MMA's M
// dimension and streams them faster than a mostly empty 128-row tile would.
bool few_rows(const gqa_desc_t* d) {
  return static_cast<long long>(d->q_tokens) * group_of(d) <= GQA_MAX_QROWS;
}

struct RowsPlan {
  PlanParams pp;
  int groups;         // tile groups per (batch, KV head)
  long long triples;
  long long pieces;   // partial tile groups the workspace holds (0: nothing is cut)
  long long records;
  gqa_status_t status;
};

RowsPlan make_rows_plan(const gqa_desc_t* d, int sm, bool every_piece) {
  RowsPlan rp;
  std::memset(&rp, 0, sizeof rp);
  rp.status = GQA_OK;
  const int gt = group_tokens_of(d);
  rp.groups = (d->q_tokens - 1) / gt + 1;
  const long long heads = static_cast<long long>(d->kv_heads) * rp.groups;  // the plan's "KV heads"
  if (heads > INT_MAX || heads * d->batch > INT_MAX - 65536) {
    rp.status = GQA_ERR_UNSUPPORTED;
    return rp;
  }
  rp.triples = heads * d->batch;
  PlanParams& pp = rp.pp;
  pp.batch = d->batch;
  pp.kv_heads = static_cast<int>(heads);
  pp.max_seqlen = d->max_seqlen;
  pp.min_blocks = 1;
  const int nblk = num_blocks(d->max_seqlen);
  const long long units = static_cast<long long>(d->batch) * pair_units(nblk, kRowsItemUnits);
  if (d->batch <= kMaxSmemB && units <= INT_MAX) {
    pp.mode = PLAN_BALANCED;
    pp.item_units = kRowsItemUnits;
    const long long all = units * heads;
    pp.num_ctas = static_cast<int>(all < sm ? all : sm);
    if (every_piece) {
      rp.pieces = rp.triples + pp.num_ctas;
      rp.records = rp.triples;
    } else if (pp.num_ctas > 1) {
      rp.pieces = 2ll * pp.num_ctas;
      rp.records = pp.num_ctas;
    }
    if (rp.pieces > INT_MAX) rp.status = GQA_ERR_UNSUPPORTED;
    return rp;
  }
  // Batches whose lengths the kernel does not stage: whole triples dealt to
  // the CTAs in turn (there are more of them than SMs).
  pp.mode = PLAN_SPLITS;
  pp.num_splits = 1;
  pp.num_ctas = static_cast<int>(rp.triples < sm ? rp.triples : sm);
  if (every_piece) rp.status = GQA_ERR_UNSUPPORTED;  // not reached: a prefix's plan has one batch entry
  return rp;
}

struct RowsWs {
  size_t o_off, lse_off, rec_off, total;
};

RowsWs rows_ws(const gqa_desc_t* d, const RowsPlan& rp) {
  RowsWs w{0, 0, 0, 0};
  if (rp.pieces == 0) return w;
  const size_t rows = static_cast<size_t>(rp.pieces) * tiles_per_triple(d->head_dim) * kTileRows;
  w.lse_off = round_up(rows * d->head_dim * sizeof(float), kWsAlign);
  w.rec_off = w.lse_off + round_up(rows * sizeof(float), kWsAlign);
  w.total = w.rec_off + round_up(static_cast<size_t>(rp.records) * sizeof(int2), kWsAlign);
  return w;
}

gqa_status_t encode_rows_maps(const gqa_desc_t* d, const void* q, const void* k, const void* v, RowsParams* p) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return GQA_ERR_CUDA;
  const cuuint64_t D = static_cast<cuuint64_t>(d->head_dim);
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      d->in_dtype == GQA_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto encode = [&](CUtensorMap* m, const void* base, int heads, int positions, int box_heads, int box_positions) {
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(positions),
                                static_cast<cuuint64_t>(d->batch)};
    const cuuint64_t strides[3] = {D * 2, D * 2 * dims[1], D * 2 * dims[1] * dims[2]};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_positions), 1};
    return enc(m, type, 4, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const bool ok = encode(&p->tm_q, q, d->q_heads, d->q_tokens, group_of(d), tile_tokens(d)) &&
                  encode(&p->tm_k, k, d->kv_heads, d->max_seqlen, 1, kBlockN) &&
                  encode(&p->tm_v, v, d->kv_heads, d->max_seqlen, 1, kBlockN);
  return ok ? GQA_OK : GQA_ERR_INVALID_ARG;
}

// The rows kernel over desc's rows and keys; `ws` holds rows_ws() bytes.
gqa_status_t launch_rows(DeviceState* st, const gqa_desc_t* d, const RowsPlan& rp, bool every_piece, const void* q,
                         const void* k, const void* v, const int32_t* lens, void* out, float* lse, uint8_t* ws,
                         cudaStream_t s) {
  RowsParams p;
  std::memset(&p, 0, sizeof p);
  gqa_status_t rc = encode_rows_maps(d, q, k, v, &p);
  if (rc != GQA_OK) return rc;
  p.lens = lens;
  p.out = out;
  p.lse = lse;
  const size_t rows = static_cast<size_t>(d->batch) * d->q_tokens * d->q_heads;
  p.out_bytes = out != nullptr ? rows * d->head_dim * (d->out_dtype == GQA_DTYPE_FP32 ? 4u : 2u) : 0u;
  p.lse_bytes = lse != nullptr ? rows * 4u : 0u;
  if (rp.pieces > 0) {
    const RowsWs w = rows_ws(d, rp);
    p.o_part = reinterpret_cast<float*>(ws + w.o_off);
    p.lse_part = reinterpret_cast<float*>(ws + w.lse_off);
    p.rec = reinterpret_cast<int2*>(ws + w.rec_off);
    p.o_part_bytes = w.lse_off;
    p.lse_part_bytes = w.rec_off - w.lse_off;
    p.rec_bytes = w.total - w.rec_off;
  }
  p.plan = rp.pp;
  p.nq = d->q_tokens;
  p.Hq = d->q_heads;
  p.G = group_of(d);
  p.groups = rp.groups;
  p.tokens = tile_tokens(d);
  p.out_dtype = d->out_dtype;
  p.out_v32 = aligned(out, 32) ? 1 : 0;
  p.all_partial = every_piece ? 1 : 0;
  const float scale = d->scale > 0.f ? d->scale : 1.0f / std::sqrt(static_cast<float>(d->head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = wait_timeout_ns();
  const bool f16 = d->in_dtype == GQA_DTYPE_FP16;
  const KernelRef k_ref = d->head_dim == 64    ? rows_kernel_ref_64(f16)
                          : d->head_dim == 256 ? rows_kernel_ref_256(f16)
                                               : rows_kernel_ref_128(f16);
  const unsigned bit = 24u + (d->head_dim == 64 ? 0u : d->head_dim == 128 ? 2u : 4u) + (f16 ? 1u : 0u);
  if ((rc = ensure_smem_attr(st, bit, k_ref.fn, k_ref.smem_bytes, k_ref.regs)) != GQA_OK) return rc;
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(rp.pp.num_ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(k_ref.threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(k_ref.smem_bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr = pdl_attr(!env_flag("GQA_DISABLE_PDL"));
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  return cudaLaunchKernelExC(&cfg, k_ref.fn, args) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status_t launch_merge(const RowsMergeParams& m, int head_dim, bool prefix, dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr = pdl_attr(!env_flag("GQA_DISABLE_PDL"));
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (prefix)
    e = head_dim == 64    ? cudaLaunchKernelEx(&cfg, gqa_prefix_merge_kernel<64>, m)
        : head_dim == 256 ? cudaLaunchKernelEx(&cfg, gqa_prefix_merge_kernel<256>, m)
                          : cudaLaunchKernelEx(&cfg, gqa_prefix_merge_kernel<128>, m);
  else
    e = head_dim == 64    ? cudaLaunchKernelEx(&cfg, gqa_rows_merge_kernel<64>, m)
        : head_dim == 256 ? cudaLaunchKernelEx(&cfg, gqa_rows_merge_kernel<256>, m)
                          : cudaLaunchKernelEx(&cfg, gqa_rows_merge_kernel<128>, m);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

RowsMergeParams merge_params(const gqa_desc_t* d, const RowsPlan& rp, uint8_t* ws) {
  RowsMergeParams m;
  std::memset(&m, 0, sizeof m);
  if (rp.pieces > 0) {
    const RowsWs w = rows_ws(d, rp);
    m.o_part = reinterpret_cast<const float*>(ws + w.o_off);
    m.lse_part = reinterpret_cast<const float*>(ws + w.lse_off);
    m.rec = reinterpret_cast<const int2*>(ws + w.rec_off);
  }
  m.pieces = static_cast<int>(rp.pieces);
  m.tiles = tiles_per_triple(d->head_dim);
  m.tokens = tile_tokens(d);
  m.groups = rp.groups;
  m.kv_heads = d->kv_heads;
  m.out_dtype = d->out_dtype;
  m.batch = d->batch;
  m.nq = d->q_tokens;
  m.Hq = d->q_heads;
  m.G = group_of(d);
  return m;
}

// The decode kernel's side of a merge: a balanced (or, for large batches, a
// fixed-split) launch whose pieces all end up in [slots][rows][d] fp32: rows
// that were not split are its final fp32 output, which goes to slot 0.
struct DecodeSide {
  HostPlan hp;
  int slots;
  size_t rows;
  size_t o_off, lse_off, np_off, total;  // within the side's own part of the workspace
};

gqa_desc_t partial_desc(const gqa_desc_t* d) {
  gqa_desc_t s = *d;
  s.out_dtype = GQA_DTYPE_FP32;
  s.reduction = GQA_REDUCE_COMBINE;
  return s;
}

DecodeSide decode_side(const gqa_desc_t* d, int sm) {
  DecodeSide s;
  const gqa_desc_t pd = partial_desc(d);
  s.hp = make_plan(&pd, 0, sm, false);
  s.slots = s.hp.combine ? s.hp.num_slots : 1;
  s.rows = static_cast<size_t>(d->batch) * d->q_tokens * d->q_heads;
  s.o_off = 0;
  s.lse_off = round_up(s.slots * s.rows * d->head_dim * sizeof(float), kWsAlign);
  s.np_off = s.lse_off + round_up(s.slots * s.rows * sizeof(float), kWsAlign);
  s.total = s.np_off + round_up(static_cast<size_t>(d->batch) * d->kv_heads * 4 * sizeof(int32_t), kWsAlign);
  return s;
}

gqa_status_t launch_decode_side(DeviceState* st, const gqa_desc_t* d, const DecodeSide& ds, const void* q,
                                const void* k, const void* v, const int32_t* lens, uint8_t* ws, cudaStream_t s) {
  const gqa_desc_t pd = partial_desc(d);
  DecodeParams p;
  const gqa_status_t rc = prepare_decode(&pd, q, k, v, lens, ds.hp, &p, false);
  if (rc != GQA_OK) return rc;
  p.o_part = reinterpret_cast<float*>(ws + ds.o_off);
  p.lse_part = reinterpret_cast<float*>(ws + ds.lse_off);
  p.out = p.o_part;
  p.lse = p.lse_part;
  p.out_bytes = ds.rows * d->head_dim * 4u;
  p.lse_bytes = ds.rows * 4u;
  p.o_part_bytes = ds.lse_off - ds.o_off;
  p.lse_part_bytes = ds.np_off - ds.lse_off;
  if (ds.hp.combine && ds.hp.use_n_pieces) {
    p.n_pieces = reinterpret_cast<int32_t*>(ws + ds.np_off);
    p.n_pieces_bytes = ds.total - ds.np_off;
  }
  return launch_decode(st, p, d->in_dtype == GQA_DTYPE_FP16, s);
}

DecodePartials partials_of(const DecodeSide& ds, uint8_t* ws) {
  DecodePartials r;
  r.o = reinterpret_cast<const float*>(ws + ds.o_off);
  r.lse = reinterpret_cast<const float*>(ws + ds.lse_off);
  r.n_pieces = ds.hp.combine && ds.hp.use_n_pieces ? reinterpret_cast<const int32_t*>(ws + ds.np_off) : nullptr;
  r.slots = ds.slots;
  return r;
}

// What the rows kernel asks of a description beyond check_desc_any_rows.
gqa_status_t check_rows(const gqa_desc_t* d) {
  return group_of(d) > GQA_MAX_GROUP ? GQA_ERR_UNSUPPORTED : GQA_OK;
}

gqa_status_t check_cross(const gqa_desc_t* d) {
  const gqa_status_t rc = check_desc_any_rows(d);
  if (rc != GQA_OK) return rc;
  if (d->causal != 0 || d->reduction != GQA_REDUCE_AUTO) return GQA_ERR_UNSUPPORTED;
  return check_rows(d);
}

// The prefix phase as a problem of its own: one batch entry of B * nq tokens.
gqa_status_t check_prefix(const gqa_desc_t* d, int max_prefix, gqa_desc_t* prefix) {
  gqa_status_t rc = check_desc(d);
  if (rc != GQA_OK) return rc;
  if (max_prefix < 1) return GQA_ERR_INVALID_ARG;
  if (d->reduction != GQA_REDUCE_AUTO || max_prefix > (1 << 30)) return GQA_ERR_UNSUPPORTED;
  const long long tokens = static_cast<long long>(d->batch) * d->q_tokens;
  if (tokens > INT_MAX / 2) return GQA_ERR_UNSUPPORTED;
  *prefix = *d;
  prefix->batch = 1;
  prefix->q_tokens = static_cast<int>(tokens);
  prefix->max_seqlen = max_prefix;
  prefix->causal = 0;
  return GQA_OK;
}

bool output_ok(const void* out, const float* lse) {
  return out != nullptr && aligned(out, 16) && (lse == nullptr || aligned(lse, 4));
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && aligned(ws, kWsAlign));
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_cross_workspace_size(const gqa_desc_t* desc) {
  if (check_cross(desc) != GQA_OK || desc->batch == 0) return 0;
  if (few_rows(desc)) return gqa_decode_workspace_size(desc, 0);
  int dev = 0;
  DeviceState* st = nullptr;
  if (current_device(&dev, &st) != GQA_OK) return 0;
  const RowsPlan rp = make_rows_plan(desc, st->sm_count, false);
  return rp.status == GQA_OK ? rows_ws(desc, rp).total : 0;
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
  const RowsPlan rp = make_rows_plan(desc, st->sm_count, false);
  if (rp.status != GQA_OK) return rp.status;
  if (!workspace_ok(workspace, workspace_bytes, rows_ws(desc, rp).total)) return GQA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((rc = launch_rows(st, desc, rp, false, q, k, v, kv_lens, out, lse, ws, s)) != GQA_OK) return rc;
  if (rp.pieces == 0) return GQA_OK;
  RowsMergeParams m = merge_params(desc, rp, ws);
  m.out = out;
  m.lse = lse;
  const unsigned chunks = static_cast<unsigned>(m.tiles * kTileRows / (kMergeThreads / 32));
  return launch_merge(m, desc->head_dim, false, dim3(static_cast<unsigned>(rp.pp.num_ctas), chunks, 1), s);
}

size_t gqa_prefix_workspace_size(const gqa_desc_t* desc, int max_prefix) {
  gqa_desc_t pre;
  if (check_prefix(desc, max_prefix, &pre) != GQA_OK || desc->batch == 0) return 0;
  int dev = 0;
  DeviceState* st = nullptr;
  if (current_device(&dev, &st) != GQA_OK) return 0;
  const size_t own = decode_side(desc, st->sm_count).total;
  if (few_rows(&pre)) return decode_side(&pre, st->sm_count).total + own;
  const RowsPlan rp = make_rows_plan(&pre, st->sm_count, true);
  return rp.status == GQA_OK ? rows_ws(&pre, rp).total + own : 0;
}

gqa_status_t gqa_prefix_attn(const gqa_desc_t* desc, const void* q, const void* k_prefix, const void* v_prefix,
                             const int32_t* prefix_len, int max_prefix, const void* k_cache, const void* v_cache,
                             const int32_t* seqlens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  gqa_desc_t pre;
  gqa_status_t rc = check_prefix(desc, max_prefix, &pre);
  if (rc != GQA_OK) return rc;
  if (desc->batch == 0) return GQA_OK;
  if ((rc = check_inputs(q, k_cache, v_cache, seqlens)) != GQA_OK) return rc;
  if ((rc = check_inputs(q, k_prefix, v_prefix, prefix_len)) != GQA_OK) return rc;
  if (!output_ok(out, lse)) return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  const bool few = few_rows(&pre);
  const DecodeSide own = decode_side(desc, st->sm_count);
  DecodeSide shared;
  RowsPlan rp;
  std::memset(&rp, 0, sizeof rp);
  size_t shared_bytes;
  if (few) {
    shared = decode_side(&pre, st->sm_count);
    shared_bytes = shared.total;
  } else {
    rp = make_rows_plan(&pre, st->sm_count, true);
    if (rp.status != GQA_OK) return rp.status;
    shared_bytes = rows_ws(&pre, rp).total;
  }
  const long long rows = static_cast<long long>(own.rows);
  const long long grid = (rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  if (grid > INT_MAX) return GQA_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, shared_bytes + own.total)) return GQA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* ws_own = ws + shared_bytes;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = few ? launch_decode_side(st, &pre, shared, q, k_prefix, v_prefix, prefix_len, ws, s)
           : launch_rows(st, &pre, rp, true, q, k_prefix, v_prefix, prefix_len, nullptr, nullptr, ws, s);
  if (rc != GQA_OK) return rc;
  if ((rc = launch_decode_side(st, desc, own, q, k_cache, v_cache, seqlens, ws_own, s)) != GQA_OK) return rc;
  RowsMergeParams m = merge_params(&pre, rp, ws);
  m.out = out;
  m.lse = lse;
  m.batch = desc->batch;
  m.nq = desc->q_tokens;
  m.prefix_in_rows = few ? 0 : 1;
  if (few) m.prefix = partials_of(shared, ws);
  m.own = partials_of(own, ws_own);
  return launch_merge(m, desc->head_dim, true, dim3(static_cast<unsigned>(grid), 1, 1), s);
}

gqa_status_t gqa_shared_keys_plan(const gqa_desc_t* desc, int every_piece, const int32_t* kv_lens_host, int sm_count,
                                  int* num_ctas, int* group_tokens, int* num_pieces, int32_t* items,
                                  int64_t max_items, int64_t* num_items) {
  gqa_status_t rc = check_cross(desc);
  if (rc != GQA_OK) return rc;
  if (desc->batch > 0 && kv_lens_host == nullptr) return GQA_ERR_INVALID_ARG;
  if (every_piece != 0 && desc->batch != 1) return GQA_ERR_INVALID_ARG;
  if (sm_count <= 0) {
    int dev = 0;
    DeviceState* st = nullptr;
    if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
    sm_count = st->sm_count;
  }
  const RowsPlan rp = make_rows_plan(desc, sm_count, every_piece != 0);
  if (rp.status != GQA_OK) return rp.status;
  if (num_ctas) *num_ctas = rp.pp.num_ctas;
  if (group_tokens) *group_tokens = group_tokens_of(desc);
  if (num_pieces) *num_pieces = static_cast<int>(rp.pieces);
  const int B = desc->batch;
  std::vector<int32_t> clamped(static_cast<size_t>(B > 0 ? B : 1)), pre(static_cast<size_t>(B) + 1, 0);
  for (int b = 0; b < B; ++b) {
    clamped[b] = clamp_len(kv_lens_host[b], desc->max_seqlen);
    if (rp.pp.mode == PLAN_BALANCED) pre[b + 1] = pre[b] + pair_units(num_blocks(clamped[b]), rp.pp.item_units);
  }
  int64_t n = 0;
  for (int c = 0; c < rp.pp.num_ctas && B > 0; ++c) {
    WorkIter it;
    it.init(rp.pp, kv_lens_host, clamped.data(), pre.data(), c);
    WorkItem w;
    while (it.next(w)) {
      if (items != nullptr && n < max_items) {
        int32_t* r = items + 8 * n;
        const long long triple = static_cast<long long>(w.b) * rp.pp.kv_heads + w.h;
        const bool partial = every_piece != 0 || w.slot >= 0;
        r[0] = c; r[1] = w.b; r[2] = w.h / rp.groups; r[3] = w.h % rp.groups; r[4] = w.blk_begin; r[5] = w.blk_end;
        r[6] = !partial ? -1 : static_cast<int32_t>(every_piece != 0 ? triple + c : 2 * c + (w.first_piece ? 1 : 0));
        r[7] = w.blk_begin < w.blk_end ? w.n_pieces : 0;
      }
      ++n;
    }
  }
  if (num_items) *num_items = n;
  return GQA_OK;
}

}  // extern "C"
