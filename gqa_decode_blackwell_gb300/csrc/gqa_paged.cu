// Host side of include/gqa_paged.h: argument checks, the rotation's table, and
// the launches of the kernels around a paged cache (paged_kernels.cuh) and of the
// rows kernel over one.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/gqa_paged.h"
#include "host.h"
#include "paged_kernels.cuh"
#include "rows_host.h"

namespace gqa {
namespace {

static_assert(kMaxTreeTokens == GQA_MAX_TREE_TOKENS, "the tree kernel's threads");

// A batch of new tokens and the cache they belong to, without the limits of
// attention.
gqa_status_t check_paged(const gqa_desc_t* d, const gqa_pages_t* g) {
  if (d == nullptr || g == nullptr) return GQA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->q_tokens < 1 || d->q_heads < 1 || d->kv_heads < 1 || d->max_seqlen < 1)
    return GQA_ERR_INVALID_ARG;
  if (d->in_dtype != GQA_DTYPE_BF16 && d->in_dtype != GQA_DTYPE_FP16) return GQA_ERR_INVALID_ARG;
  if (g->num_pages < 1 || g->max_pages < 1 || g->page_size < 1) return GQA_ERR_INVALID_ARG;
  if (g->page_stride < 1 || g->pos_stride < 1 || g->head_stride < 1) return GQA_ERR_INVALID_ARG;
  if (g->page_stride % 8 != 0 || g->pos_stride % 8 != 0 || g->head_stride % 8 != 0) return GQA_ERR_INVALID_ARG;
  if (d->max_seqlen > static_cast<long long>(g->max_pages) * g->page_size) return GQA_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return GQA_ERR_UNSUPPORTED;
  if (g->pos_stride < d->head_dim || g->head_stride < d->head_dim || g->page_stride < d->head_dim)
    return GQA_ERR_INVALID_ARG;
  if (g->page_size < 16 || g->page_size > 65536 || (g->page_size & (g->page_size - 1)) != 0)
    return GQA_ERR_UNSUPPORTED;
  // a tensor map's strides are below 2^40 bytes
  constexpr int64_t kMost = (int64_t{1} << 39) - 8;
  if (g->page_stride > kMost || g->pos_stride > kMost || g->head_stride > kMost) return GQA_ERR_UNSUPPORTED;
  if (d->max_seqlen > (1 << 30) || d->q_heads > 65535 || d->kv_heads > 65535) return GQA_ERR_UNSUPPORTED;
  if (static_cast<long long>(d->batch) * d->q_tokens > INT_MAX) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

gqa_status_t check_rope(const gqa_rotary_t* r, int head_dim) {
  if (r->dim < 2 || r->dim % 2 != 0 || r->dim > head_dim) return GQA_ERR_INVALID_ARG;
  if (!(r->magnitude >= 0.f) || std::isinf(r->magnitude)) return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

bool word_ok(const void* p) { return p != nullptr && aligned(p, 4); }
bool index_ok(const void* p) { return p == nullptr || aligned(p, 4); }
bool rows_ok(const void* p) { return p != nullptr && aligned(p, 16); }

PagedKeys paged_keys(const gqa_pages_t& g, const int32_t* table, const int32_t* news) {
  PagedKeys k;
  std::memset(&k, 0, sizeof k);
  k.table = table;
  k.news = news;
  k.cols = g.max_pages;
  k.num_pages = g.num_pages;
  while ((1 << k.page_shift) < g.page_size) ++k.page_shift;
  k.page_mask = g.page_size - 1;
  k.box_shift = k.page_shift < 7 ? k.page_shift : 7;
  return k;
}

// Bytes from a cache's first element to behind its last one.
unsigned long long cache_bytes(const gqa_pages_t& g, int kv_heads, int head_dim) {
  auto last = [](int n, int64_t stride) { return static_cast<unsigned long long>(n - 1) * static_cast<unsigned long long>(stride); };
  return 2 * (last(g.num_pages, g.page_stride) + last(g.page_size, g.pos_stride) + last(kv_heads, g.head_stride) + head_dim);
}

// Elements of the runs that a number of pairs comes apart into.
int run_of(bool interleaved, int pairs) {
  return interleaved || pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : pairs % 2 == 0 ? 2 : 1;
}

template <typename T, bool APPEND, bool INTERLEAVED, int N>
const void* rotary_instance(bool grouped) {
  if constexpr (APPEND)
    return grouped ? reinterpret_cast<const void*>(&gqa_append_kernel<T, INTERLEAVED, N, true>)
                   : reinterpret_cast<const void*>(&gqa_append_kernel<T, INTERLEAVED, N, false>);
  else
    return grouped ? reinterpret_cast<const void*>(&gqa_rotary_kernel<T, INTERLEAVED, N, true>)
                   : reinterpret_cast<const void*>(&gqa_rotary_kernel<T, INTERLEAVED, N, false>);
}

// The rotation kernel for a type, a layout and a run.
template <typename T, bool APPEND>
const void* rotary_fn(bool interleaved, int run, bool grouped) {
  if (interleaved) return rotary_instance<T, APPEND, true, 8>(grouped);
  return run == 8   ? rotary_instance<T, APPEND, false, 8>(grouped)
         : run == 4 ? rotary_instance<T, APPEND, false, 4>(grouped)
         : run == 2 ? rotary_instance<T, APPEND, false, 2>(grouped)
                    : rotary_instance<T, APPEND, false, 1>(grouped);
}

// Few tokens are spread over CTAs of a unit (two runs) a thread, up to a GPU full
// of them; of many each has one CTA, which computes the token's angles once, of
// 256 threads where they have two units or more each or all of them one, and else of
// 128.  Measured on GB300 (128, 256): 8192 places of 384 units 18.5 and 20.4 us, 8192
// of 256 21.1 and 21.0, 2048 of 1280 20.2 and 16.5, 2048 of 512 in fp32 25.5 and 24.2.
// Many tokens of few units share CTAs.
template <bool APPEND>
gqa_status_t launch_rotary(int dtype, bool interleaved, RotaryParams& p, long long tokens, int rows, int sm,
                           cudaStream_t s) {
  const int run = run_of(interleaved, p.pairs);
  const long long units = static_cast<long long>(rows) * (p.head_dim / (2 * run));
  long long threads = 128, parts = (units + threads - 1) / threads;
  const long long spread = 16LL * sm / tokens;
  const bool grouped = spread < 1 && units <= kGroupUnits;
  if (grouped) {
    p.group = static_cast<int>(kGroupThreads / units);
    threads = kGroupThreads;
    parts = 1;
  } else if (spread < parts) {
    threads = units > 2 * kRotaryThreads || units % kRotaryThreads == 0 ? kRotaryThreads : 128;
    parts = spread > 1 ? spread : 1;
  }
  p.tokens = tokens;
  const void* fn;
  if (dtype == GQA_DTYPE_FP16) {
    fn = rotary_fn<__half, APPEND>(interleaved, run, grouped);
  } else if (APPEND || dtype == GQA_DTYPE_BF16) {
    fn = rotary_fn<__nv_bfloat16, APPEND>(interleaved, run, grouped);
  } else {
    if constexpr (!APPEND) fn = rotary_fn<float, APPEND>(interleaved, run, grouped);
  }
  const long long ctas = grouped ? (tokens + p.group - 1) / p.group : tokens;
  return launch_kernel(fn, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(parts < 65535 ? parts : 65535)),
                       static_cast<int>(threads), 0, &p, s);
}

gqa_status_t check_tree(const gqa_desc_t* d, const gqa_pages_t* g) {
  gqa_status_t rc = check_desc_any_rows(d);
  if (rc != GQA_OK) return rc;
  if ((rc = check_paged(d, g)) != GQA_OK) return rc;
  if (d->reduction != GQA_REDUCE_AUTO || d->q_heads / d->kv_heads > 128 || d->q_tokens > GQA_MAX_TREE_TOKENS)
    return GQA_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(d->batch) * d->q_tokens * d->q_heads;
  return rows > INT_MAX ? GQA_ERR_UNSUPPORTED : GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

gqa_status_t gqa_rotary_turns(int dim, double base, int scaling, double factor, int original_length, double slow,
                              double fast, uint64_t* turns) {
  if (dim < 2 || dim % 2 != 0 || dim > 2 * kMaxPairs || turns == nullptr) return GQA_ERR_INVALID_ARG;
  if (!(base > 1.0) || std::isinf(base) || !(factor >= 1.0) || std::isinf(factor)) return GQA_ERR_INVALID_ARG;
  if (scaling < GQA_ROTARY_NONE || scaling > GQA_ROTARY_PARTS) return GQA_ERR_INVALID_ARG;
  if (scaling == GQA_ROTARY_NONE && factor != 1.0) return GQA_ERR_INVALID_ARG;
  if (scaling == GQA_ROTARY_PARTS && (original_length < 1 || !(slow >= 0.0) || !(fast > slow) || std::isinf(fast)))
    return GQA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == GQA_ROTARY_BASE && dim > 2) base *= std::pow(factor, static_cast<double>(dim) / (dim - 2));
  if (std::isinf(base)) return GQA_ERR_INVALID_ARG;
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (scaling == GQA_ROTARY_LINEAR) f /= factor;
    if (scaling == GQA_ROTARY_PARTS) {
      double w = (original_length * f / two_pi - slow) / (fast - slow);
      w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
      f = f / factor * (1.0 - w) + f * w;
    }
    // f <= 1, so this is below 1/6 of a turn; rounded to the nearest step
    turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
  }
  return GQA_OK;
}

gqa_status_t gqa_rotary_apply(const gqa_rotary_t* rope, const uint64_t* turns, const int32_t* positions,
                              int64_t tokens, int heads, int head_dim, int dtype, const void* x, int64_t x_stride,
                              void* out, int64_t out_stride, void* stream) {
  if (rope == nullptr || tokens < 0 || heads < 1) return GQA_ERR_INVALID_ARG;
  if (dtype != GQA_DTYPE_BF16 && dtype != GQA_DTYPE_FP16 && dtype != GQA_DTYPE_FP32) return GQA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return GQA_ERR_UNSUPPORTED;
  gqa_status_t rc = check_rope(rope, head_dim);
  if (rc != GQA_OK) return rc;
  const int64_t dense = static_cast<int64_t>(heads) * head_dim;
  if (heads > 65535 || tokens > INT_MAX) return GQA_ERR_UNSUPPORTED;
  if (x_stride < dense || out_stride < dense || x_stride % 8 != 0 || out_stride % 8 != 0) return GQA_ERR_INVALID_ARG;
  if (x_stride > LLONG_MAX / 8 / (tokens + 1) || out_stride > LLONG_MAX / 8 / (tokens + 1))
    return GQA_ERR_UNSUPPORTED;
  if (tokens == 0) return GQA_OK;  // pointers may be null
  if (turns == nullptr || !aligned(turns, 8) || !word_ok(positions) || !rows_ok(x) || !rows_ok(out))
    return GQA_ERR_INVALID_ARG;
  if (x == out && x_stride != out_stride) return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  RotaryParams p;
  std::memset(&p, 0, sizeof p);
  p.turns = turns;
  p.positions = positions;
  p.x = RotaryPart{x, out, x_stride, out_stride, heads};
  p.head_dim = head_dim;
  p.pairs = rope->dim / 2;
  p.inverse = rope->inverse != 0 ? 1 : 0;
  p.magnitude = rope->magnitude > 0.f ? rope->magnitude : 1.f;
  p.x_bytes = static_cast<unsigned long long>((tokens - 1) * out_stride + dense) * (dtype == GQA_DTYPE_FP32 ? 4 : 2);
#ifdef GQA_DEBUG
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
#endif
  return launch_rotary<false>(dtype, rope->interleaved != 0, p, tokens, heads, st->sm_count,
                              static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_paged_append(const gqa_desc_t* desc, const gqa_pages_t* pages, const gqa_rotary_t* rope,
                              const uint64_t* turns, const int32_t* positions, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                              void* k_cache, void* v_cache, const int32_t* page_table, const int32_t* seqlens,
                              const int32_t* new_lens, void* stream) {
  gqa_status_t rc = check_paged(desc, pages);
  if (rc != GQA_OK) return rc;
  if ((rope == nullptr) != (turns == nullptr)) return GQA_ERR_INVALID_ARG;
  if (rope != nullptr) {
    if ((rc = check_rope(rope, desc->head_dim)) != GQA_OK) return rc;
    if (rope->inverse != 0) return GQA_ERR_INVALID_ARG;
  }
  if ((q == nullptr) != (q_out == nullptr)) return GQA_ERR_INVALID_ARG;
  const int64_t d = desc->head_dim, dense_q = d * desc->q_heads, dense_k = d * desc->kv_heads;
  if (k_stride < dense_k || v_stride < dense_k || k_stride % 8 != 0 || v_stride % 8 != 0) return GQA_ERR_INVALID_ARG;
  if (q != nullptr && (q_stride < dense_q || q_stride % 8 != 0)) return GQA_ERR_INVALID_ARG;
  const int64_t tokens = static_cast<int64_t>(desc->batch) * desc->q_tokens;
  const int64_t most = LLONG_MAX / 8 / (tokens + 1);
  if (k_stride > most || v_stride > most || (q != nullptr && q_stride > most)) return GQA_ERR_UNSUPPORTED;
  if (desc->batch == 0) return GQA_OK;  // pointers may be null
  if (!rows_ok(k) || !rows_ok(v) || !rows_ok(k_cache) || !rows_ok(v_cache)) return GQA_ERR_INVALID_ARG;
  if (q != nullptr && (!aligned(q, 16) || !aligned(q_out, 16))) return GQA_ERR_INVALID_ARG;
  if (q != nullptr && q == q_out && q_stride != dense_q) return GQA_ERR_INVALID_ARG;
  if (!word_ok(page_table) || !word_ok(seqlens) || !index_ok(new_lens) || !index_ok(positions) ||
      (turns != nullptr && !aligned(turns, 8)))
    return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  RotaryParams p;
  std::memset(&p, 0, sizeof p);
  p.turns = turns;
  p.positions = positions;
  p.x = RotaryPart{q, q_out, q_stride, dense_q, q != nullptr ? desc->q_heads : 0};
  p.k = RotaryPart{k, nullptr, k_stride, 0, desc->kv_heads};
  p.v = RotaryPart{v, nullptr, v_stride, 0, desc->kv_heads};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page_stride = pages->page_stride;
  p.pos_stride = pages->pos_stride;
  p.head_stride = pages->head_stride;
  p.pages = paged_keys(*pages, page_table, new_lens);
  p.seqlens = seqlens;
  p.max_seqlen = desc->max_seqlen;
  p.nq = desc->q_tokens;
  p.head_dim = desc->head_dim;
  p.pairs = rope != nullptr ? rope->dim / 2 : 0;
  p.magnitude = rope != nullptr && rope->magnitude > 0.f ? rope->magnitude : 1.f;
  p.x_bytes = q != nullptr ? static_cast<unsigned long long>(tokens * dense_q) * 2 : 0;
  p.cache_bytes = cache_bytes(*pages, desc->kv_heads, desc->head_dim);
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
  return launch_rotary<true>(desc->in_dtype, rope != nullptr && rope->interleaved != 0, p, tokens,
                             p.x.heads + 2 * desc->kv_heads, st->sm_count, static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_tree_from_parents(int batch, int q_tokens, int max_seqlen, const int32_t* parents,
                                   const int32_t* seqlens, const int32_t* new_lens, uint32_t* tree,
                                   int32_t* positions, void* stream) {
  if (batch < 0 || q_tokens < 1 || max_seqlen < 1) return GQA_ERR_INVALID_ARG;
  if (q_tokens > GQA_MAX_TREE_TOKENS || max_seqlen > (1 << 30)) return GQA_ERR_UNSUPPORTED;
  if (batch == 0) return GQA_OK;
  if (!word_ok(parents) || !word_ok(seqlens) || !word_ok(tree) || !index_ok(new_lens) || !index_ok(positions))
    return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  gqa_status_t rc = current_device(&dev, &st);
  if (rc != GQA_OK) return rc;
  TreeParams p;
  std::memset(&p, 0, sizeof p);
  p.parents = parents;
  p.seqlens = seqlens;
  p.news = new_lens;
  p.tree = tree;
  p.positions = positions;
  p.nq = q_tokens;
  p.words = (q_tokens + 31) / 32;
  p.max_seqlen = max_seqlen;
  const unsigned long long rows = static_cast<unsigned long long>(batch) * q_tokens;
  p.tree_bytes = rows * p.words * 4;
  p.positions_bytes = positions != nullptr ? rows * 4 : 0;
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
  return launch_kernel(reinterpret_cast<const void*>(&gqa_tree_kernel), dim3(static_cast<unsigned>(batch)),
                       32 * p.words, 0, &p, static_cast<cudaStream_t>(stream));
}

size_t gqa_tree_workspace_size(const gqa_desc_t* desc, const gqa_pages_t* pages) {
  if (check_tree(desc, pages) != GQA_OK || desc->batch == 0) return 0;
  int dev = 0;
  DeviceState* st = nullptr;
  if (current_device(&dev, &st) != GQA_OK) return 0;
  const RowsLaunch r = make_launch(desc, nullptr, st->sm_count, true);
  return r.status == GQA_OK ? rows_ws(r).total : 0;
}

gqa_status_t gqa_tree_attn(const gqa_desc_t* desc, const gqa_pages_t* pages, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* page_table, const int32_t* seqlens,
                           const int32_t* new_lens, const uint32_t* tree, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  gqa_status_t rc = check_tree(desc, pages);
  if (rc != GQA_OK) return rc;
  if (tree != nullptr && desc->causal != 0) return GQA_ERR_INVALID_ARG;
  if (desc->batch == 0) return GQA_OK;  // nothing to compute; pointers may be null
  if ((rc = check_inputs(q, k_cache, v_cache, seqlens)) != GQA_OK) return rc;
  if (!word_ok(page_table) || !index_ok(new_lens) || !index_ok(tree) || !output_ok(out, lse))
    return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  const RowsLaunch r = make_launch(desc, nullptr, st->sm_count, true);
  if (r.status != GQA_OK) return r.status;
  if (!workspace_ok(workspace, workspace_bytes, rows_ws(r).total)) return GQA_ERR_WORKSPACE;
  PagedCall call;
  call.geometry = pages;
  call.keys = paged_keys(*pages, page_table, new_lens);
  call.keys.tree = tree;
  call.keys.tree_words = (desc->q_tokens + 31) / 32;
  call.keys.chain = tree == nullptr && desc->causal != 0 ? 1 : 0;
  const Keys keys[1] = {{k_cache, v_cache, seqlens}};
  return run_rows(st, r, q, keys, &call, out, lse, static_cast<uint8_t*>(workspace),
                  static_cast<cudaStream_t>(stream));
}

gqa_status_t gqa_paged_keep(const gqa_desc_t* desc, const gqa_pages_t* pages, void* k_cache, void* v_cache,
                            const int32_t* page_table, const int32_t* seqlens, const int32_t* new_lens,
                            const int32_t* path, int max_keep, const int32_t* keep_lens, int32_t* seqlens_out,
                            void* stream) {
  gqa_status_t rc = check_paged(desc, pages);
  if (rc != GQA_OK) return rc;
  if (max_keep < 1) return GQA_ERR_INVALID_ARG;
  if (desc->batch == 0) return GQA_OK;
  if (!rows_ok(k_cache) || !rows_ok(v_cache) || !word_ok(page_table) || !word_ok(seqlens) || !index_ok(new_lens) ||
      !word_ok(path) || !word_ok(keep_lens) || !index_ok(seqlens_out))
    return GQA_ERR_INVALID_ARG;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = current_device(&dev, &st)) != GQA_OK) return rc;
  KeepParams p;
  std::memset(&p, 0, sizeof p);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page_stride = pages->page_stride;
  p.pos_stride = pages->pos_stride;
  p.head_stride = pages->head_stride;
  p.pages = paged_keys(*pages, page_table, new_lens);
  p.seqlens = seqlens;
  p.path = path;
  p.keep_lens = keep_lens;
  p.seqlens_out = seqlens_out;
  p.nq = desc->q_tokens;
  p.max_seqlen = desc->max_seqlen;
  p.max_keep = max_keep;
  p.kv_heads = desc->kv_heads;
  p.head_dim = desc->head_dim;
  p.cache_bytes = cache_bytes(*pages, desc->kv_heads, desc->head_dim);
  p.lens_bytes = seqlens_out != nullptr ? static_cast<unsigned long long>(desc->batch) * 4 : 0;
  if ((rc = error_word(st, &p.err_word)) != GQA_OK) return rc;
  return launch_kernel(reinterpret_cast<const void*>(&gqa_keep_kernel), dim3(static_cast<unsigned>(desc->batch)),
                       kKeepThreads, 0, &p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
