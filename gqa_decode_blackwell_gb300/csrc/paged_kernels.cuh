// Kernels around attention over a paged cache: the position rotation, alone
// (gqa_rotary_kernel) and on the way into the cache (gqa_append_kernel), the
// drafts' tree from their parents, and the accepted branch's move.  All are bound
// by memory, or, for few tokens, by the latency of one launch.
//
// Angles.  A pair that turns f radians a position has turned
// position * f / (2 pi) times, and only the fraction of a turn matters.  With
// f / (2 pi) as a 64-bit fraction u, that is the product position * u modulo 2^64:
// one integer multiplication, exact, where a product in fp32 would lose 2^-24 of
// an angle of 10^5 radians, all of a fast pair's accuracy at position 10^6.  The
// fraction's nearest quarter turn is split off as an integer, and what is left, at
// most an eighth of a turn either way, goes to sinpi and cospi in fp32 with an
// error of 2^-25 of it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_kernel.cuh"
#include "paged.h"

namespace gqa {

constexpr int kRotaryThreads = 128;
constexpr int kMaxPairs = 128;  // of a head: head_dim / 2

// Tokens' heads to rotate or copy: `heads` of each token, dense, `stride`
// elements from token to token.
struct RotaryPart {
  const void* src;
  void* dst;
  long long src_stride, dst_stride;
  int heads;
};

struct RotaryParams {
  const uint64_t* turns;     // [pairs]; null: nothing is rotated
  const int32_t* positions;  // [tokens], or null (append): the token's place in its sequence
  RotaryPart x;              // rotated: the tensor, or the queries
  // append only
  RotaryPart k, v;           // dst is unused: they go to the cache
  void* k_cache;
  void* v_cache;
  long long page_stride, pos_stride, head_stride;
  PagedKeys pages;
  const int32_t* seqlens;
  int max_seqlen, nq;
  int head_dim, pairs;
  int inverse;
  float magnitude;
  unsigned int* err_word;
};

namespace detail {

// (cos, sin) of a whole position's angle, times the magnitude.
__device__ __forceinline__ float2 turn_of(uint64_t turns, int position, int inverse, float magnitude) {
  const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;  // modulo a whole turn
  const uint32_t near = static_cast<uint32_t>(at >> 32) + (1u << 29);
  const uint32_t quarter = near >> 30;  // the nearest one
  const int32_t rest = static_cast<int32_t>(near & 0x3fffffffu) - (1 << 29);
  float s, c;
  sincospif(static_cast<float>(rest) * (1.0f / 2147483648.0f), &s, &c);  // half turns: at most 1/4
  float2 r = make_float2(c, s);
  if (quarter & 1) r = make_float2(-s, c);
  if (quarter & 2) r = make_float2(-r.x, -r.y);
  if (inverse) r.y = -r.y;
  return make_float2(r.x * magnitude, r.y * magnitude);
}

// 8 consecutive elements, as fp32 and as they are in memory.
template <typename T>
struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
  }
  __device__ __forceinline__ float get(int e) const { return to_f32(reinterpret_cast<const T*>(raw)[e]); }
  __device__ __forceinline__ void set(int e, float v) { from_f32(reinterpret_cast<T*>(raw)[e], v); }
  static __device__ __forceinline__ float to_f32(float v) { return v; }
  static __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
  static __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ void from_f32(float& d, float v) { d = v; }
  static __device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }
  static __device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
};

__device__ __forceinline__ void turn(float2 cs, float a, float b, float& ra, float& rb) {
  ra = a * cs.x - b * cs.y;
  rb = a * cs.y + b * cs.x;
}

// Where 16 elements of a head that one thread takes begin: its i-th of
// head_dim / 16.  Pairs of halves: two runs of 8 that are each other's partners
// as long as there are any, then 16 in a row; else 16 in a row.
template <bool INTERLEAVED>
__device__ __forceinline__ int2 runs_of(int i, int pairs) {
  if (!INTERLEAVED && 8 * i < pairs) return make_int2(8 * i, pairs + 8 * i);
  return make_int2(16 * i, 16 * i + 8);
}

template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_runs(Eight<T>& a, Eight<T>& b, const float2* table, int i, int pairs) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      Eight<T>& v = e < 4 ? a : b;
      if (8 * i + e >= pairs) continue;
      float ra, rb;
      turn(table[8 * i + e], v.get(2 * (e & 3)), v.get(2 * (e & 3) + 1), ra, rb);
      v.set(2 * (e & 3), ra);
      v.set(2 * (e & 3) + 1, rb);
    }
  } else {
    if (8 * i >= pairs) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float ra, rb;
      turn(table[8 * i + e], a.get(e), b.get(e), ra, rb);
      a.set(e, ra);
      b.set(e, rb);
    }
  }
}

// The rows of one CTA: head r of them is at src(r) and goes to dst(r); those
// with rotated(r) are rotated by the table, of which `ready` waits once.
// VEC: 16 elements a thread at a time, where partners are whole runs of 8 apart
// (interleaved, or halves of a multiple of 8 pairs); else a pair at a time, which
// takes any even number of rotated elements (20 of 64, 12 heads: as fast at 77
// tokens, a third of the rate at 8192).
template <typename T, bool INTERLEAVED, bool VEC, typename Src, typename Dst, typename Rotated, typename Ready>
__device__ __forceinline__ void turn_heads(int n_rows, int head_dim, int pairs, const float2* table, int part,
                                           int parts, const Src& src, const Dst& dst, const Rotated& rotated,
                                           const Ready& ready) {
  const int per_row = head_dim / (VEC ? 16 : 2), n = n_rows * per_row, step = parts * kRotaryThreads;
  int u = part * kRotaryThreads + static_cast<int>(threadIdx.x);
  if constexpr (VEC) {
    Eight<T> a, b;
    int r = 0, i = 0;
    auto load = [&] {
      r = u / per_row;
      i = u - r * per_row;
      const int2 at = runs_of<INTERLEAVED>(i, rotated(r) ? pairs : 0);
      const T* from = src(r);
      a.load(from + at.x);
      b.load(from + at.y);
    };
    if (u < n) load();
    ready();  // with the first loads under way
    while (u < n) {
      const bool turns = rotated(r);
      if (turns) turn_runs<T, INTERLEAVED>(a, b, table, i, pairs);
      T* to = dst(r);
      if (to != nullptr) {
        const int2 at = runs_of<INTERLEAVED>(i, turns ? pairs : 0);
        a.store(to + at.x);
        b.store(to + at.y);
      }
      if ((u += step) < n) load();
    }
  } else {
    T a, b;
    int r = 0, lo = 0, hi = 0;
    bool turns = false;
    int i = 0;
    auto load = [&] {
      r = u / per_row;
      i = u - r * per_row;
      turns = rotated(r) && i < pairs;  // (else two elements past the pairs, as they are; only halves come here)
      lo = turns ? i : 2 * i;
      hi = turns ? i + pairs : 2 * i + 1;
      a = src(r)[lo];
      b = src(r)[hi];
    };
    if (u < n) load();
    ready();
    while (u < n) {
      if (turns) {
        float ra, rb;
        turn(table[i], Eight<T>::to_f32(a), Eight<T>::to_f32(b), ra, rb);
        Eight<T>::from_f32(a, ra);
        Eight<T>::from_f32(b, rb);
      }
      T* to = dst(r);
      if (to != nullptr) {
        to[lo] = a;
        to[hi] = b;
      }
      if ((u += step) < n) load();
    }
  }
}

}  // namespace detail

// A token to blockIdx.x, of whose heads blockIdx.y takes its part.
template <typename T, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kRotaryThreads)
gqa_rotary_kernel(const RotaryParams p) {
  __shared__ float2 table[kMaxPairs];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long token = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  const int position = p.positions[token];
  const uint64_t turns = tid < p.pairs ? p.turns[tid] : 0;
  const T* src = static_cast<const T*>(p.x.src) + token * p.x.src_stride;
  T* dst = static_cast<T*>(p.x.dst) + token * p.x.dst_stride;
  detail::turn_heads<T, INTERLEAVED, VEC>(
      p.x.heads, p.head_dim, p.pairs, table, static_cast<int>(blockIdx.y), static_cast<int>(gridDim.y),
      [&](int r) { return src + static_cast<long long>(r) * p.head_dim; },
      [&](int r) { return dst + static_cast<long long>(r) * p.head_dim; }, [](int) { return true; },
      [&] {
        if (tid < p.pairs) table[tid] = detail::turn_of(turns, position, p.inverse, p.magnitude);
        __syncthreads();
      });
}

// The same for a batch's new tokens: queries into x.dst, keys and values into
// the page that holds the token's place.
template <typename T, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kRotaryThreads)
gqa_append_kernel(const RotaryParams p) {
  __shared__ float2 table[kMaxPairs];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long token = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.nq));
  const int t = static_cast<int>(blockIdx.x) - b * p.nq;
  const uint64_t turns = tid < p.pairs ? p.turns[tid] : 0;
  const int raw = p.seqlens[b], L = clamp_len(raw, p.max_seqlen);
  if (raw != L && t == 0 && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  const int n = detail::live_tokens(p.pages, p.err_word, b, L, p.nq);
  if (t >= n) return;
  const int place = L - n + t;
  const int position = p.positions != nullptr ? p.positions[token] : place;
  const int page = detail::page_of(p.pages, p.err_word, b, place);
  const bool there = page < p.pages.num_pages;
  const long long at = page * p.page_stride + (place & p.pages.page_mask) * p.pos_stride;
  const T* q = static_cast<const T*>(p.x.src) + token * p.x.src_stride;
  const T* k = static_cast<const T*>(p.k.src) + token * p.k.src_stride;
  const T* v = static_cast<const T*>(p.v.src) + token * p.v.src_stride;
  T* q_out = static_cast<T*>(p.x.dst) + token * p.x.dst_stride;
  T* k_to = static_cast<T*>(p.k_cache) + at;
  T* v_to = static_cast<T*>(p.v_cache) + at;
  const int hq = p.x.heads, hk = p.k.heads;
  detail::turn_heads<T, INTERLEAVED, VEC>(
      hq + 2 * hk, p.head_dim, p.pairs, table, static_cast<int>(blockIdx.y), static_cast<int>(gridDim.y),
      [&](int r) {
        const long long d = p.head_dim;
        return r < hq ? q + r * d : r < hq + hk ? k + (r - hq) * d : v + (r - hq - hk) * d;
      },
      [&](int r) -> T* {
        if (r < hq) return q_out + static_cast<long long>(r) * p.head_dim;
        if (!there) return nullptr;
        return r < hq + hk ? k_to + (r - hq) * p.head_stride : v_to + (r - hq - hk) * p.head_stride;
      },
      [&](int r) { return r < hq + hk && p.pairs > 0; },
      [&] {
        if (tid < p.pairs) table[tid] = detail::turn_of(turns, position, 0, p.magnitude);
        __syncthreads();
      });
}

constexpr int kMaxTreeTokens = 256, kMaxTreeWords = kMaxTreeTokens / 32;

struct TreeParams {
  const int32_t* parents;   // [B, nq]
  const int32_t* seqlens;
  const int32_t* news;
  uint32_t* tree;           // [B, nq, words]
  int32_t* positions;       // [B, nq] or null
  int nq, words, max_seqlen;
  unsigned int* err_word;
};

// A CTA to a sequence, a thread to a token.  Each token holds the bits of the
// ancestors found so far and the one they end at, and takes over that one's in
// turn: the branch it knows doubles every round, so that a chain of 256 drafts is
// done in 8 (following parents one by one would take a round for each).
__global__ void __launch_bounds__(kMaxTreeTokens)
gqa_tree_kernel(const TreeParams p) {
  __shared__ uint32_t bits[kMaxTreeWords][kMaxTreeTokens];
  __shared__ int up[kMaxTreeTokens];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = static_cast<int>(blockIdx.x), t = static_cast<int>(threadIdx.x);
  const int raw = p.seqlens[b], L = clamp_len(raw, p.max_seqlen);
  if (raw != L && t == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  PagedKeys k;
  k.news = p.news;
  const int n = detail::live_tokens(k, p.err_word, b, L, p.nq);
  int above = -1;
  if (t < n) {
    above = p.parents[static_cast<long long>(b) * p.nq + t];
    if (above < -1 || above >= t) {
      atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
      above = -1;
    }
  }
  uint32_t own[kMaxTreeWords];
#pragma unroll
  for (int w = 0; w < kMaxTreeWords; ++w) {
    own[w] = t < n && w == t / 32 ? 1u << (t & 31) : 0u;
    bits[w][t] = own[w];
  }
  up[t] = above;
  while (__syncthreads_or(above >= 0)) {  // an ancestor's index falls every round
    const int next = above >= 0 ? up[above] : -1;
#pragma unroll
    for (int w = 0; w < kMaxTreeWords; ++w)
      if (above >= 0 && w < p.words) own[w] |= bits[w][above];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMaxTreeWords; ++w) bits[w][t] = own[w];
    up[t] = above = next;
  }
  if (t >= p.nq) return;
  const long long row = static_cast<long long>(b) * p.nq + t;
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kMaxTreeWords; ++w) {
    depth += __popc(own[w]);
    if (w < p.words) p.tree[row * p.words + w] = own[w];
  }
  if (p.positions != nullptr) p.positions[row] = t < n ? L - n + depth : 0;
}

constexpr int kKeepThreads = 256;

struct KeepParams {
  void* k_cache;
  void* v_cache;
  long long page_stride, pos_stride, head_stride;
  PagedKeys pages;
  const int32_t* seqlens;
  const int32_t* path;       // [B, max_keep]
  const int32_t* keep_lens;  // [B]
  int32_t* seqlens_out;      // [B] or null; may be seqlens
  int nq, max_seqlen, max_keep, kv_heads, head_dim;
  unsigned int* err_word;
};

// A CTA to a sequence, 8 elements of K or of V to a thread, which moves them
// for all of the branch.  Token path[i] moves to place i <= path[i], and the
// tokens of a branch ascend, so nothing is overwritten that this thread or a later
// batch of it still reads: a batch of rows is loaded whole, then stored.
__global__ void __launch_bounds__(kKeepThreads)
gqa_keep_kernel(const KeepParams p) {
  constexpr int kBatch = 8;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const int raw = p.seqlens[b], L = clamp_len(raw, p.max_seqlen);
  if (raw != L && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  const int n = detail::live_tokens(p.pages, p.err_word, b, L, p.nq), first = L - n;
  const int asked = p.keep_lens[b];
  const int most = asked < 0 ? 0 : (asked > p.max_keep ? p.max_keep : asked);
  if (asked != most && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
  const int32_t* path = p.path + static_cast<long long>(b) * p.max_keep;
  // tokens of the branch that are in range and ascend
  __shared__ int s_bad;
  if (tid == 0) s_bad = most;
  __syncthreads();
  for (int i = tid; i < most; i += kKeepThreads) {
    const int at = path[i], before = i > 0 ? path[i - 1] : -1;
    if (at <= before || at >= n || at < 0) atomicMin(&s_bad, i);
  }
  __syncthreads();
  const int keep = s_bad;
  if (tid == 0) {
    if (keep != most) atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
    if (p.seqlens_out != nullptr) p.seqlens_out[b] = first + keep;
  }
  const int per_head = p.head_dim / 8, per_cache = p.kv_heads * per_head;
  for (int c = tid; c < 2 * per_cache; c += kKeepThreads) {
    const int in = c < per_cache ? c : c - per_cache, head = in / per_head;
    uint16_t* base = static_cast<uint16_t*>(c < per_cache ? p.k_cache : p.v_cache) + head * p.head_stride +
                     (in - head * per_head) * 8;
    for (int i0 = 0; i0 < keep; i0 += kBatch) {
      uint4 row[kBatch];
      uint16_t* to[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        to[j] = nullptr;
        const int i = i0 + j;
        if (i >= keep) continue;
        const int at = path[i];
        if (at == i) continue;  // in its place
        const int from_page = detail::page_of(p.pages, p.err_word, b, first + at);
        const int to_page = detail::page_of(p.pages, p.err_word, b, first + i);
        if (from_page >= p.pages.num_pages || to_page >= p.pages.num_pages) continue;
        row[j] = *reinterpret_cast<const uint4*>(base + from_page * p.page_stride +
                                                 ((first + at) & p.pages.page_mask) * p.pos_stride);
        to[j] = base + to_page * p.page_stride + ((first + i) & p.pages.page_mask) * p.pos_stride;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (to[j] != nullptr) *reinterpret_cast<uint4*>(to[j]) = row[j];
    }
  }
}

}  // namespace gqa
