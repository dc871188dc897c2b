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
#include <type_traits>

#include "decode_kernel.cuh"
#include "paged.h"

namespace gqa {

constexpr int kRotaryThreads = 256;  // of a CTA, at most
constexpr int kMaxPairs = 128;  // of a head: head_dim / 2
// Tokens of at most this many units (two runs of a head) share a CTA of
// kGroupThreads, a unit to a thread.
constexpr int kGroupUnits = 64, kGroupThreads = 2 * kGroupUnits;

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
  int group;                 // tokens of a CTA (kernels of groups)
  long long tokens;
  unsigned int* err_word;
  // byte extents of what is written (x.dst, each cache), checked by -DGQA_DEBUG builds
  unsigned long long x_bytes, cache_bytes;
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

// N consecutive elements (N * sizeof(T) bytes, aligned to as many or to 16), two
// to a word where they are of 16 bits.
template <typename T, int N>
struct Run {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T)), kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 2) {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[e]);
    } else if constexpr (std::is_same<T, __half>::value) {
      return __half2float(__ushort_as_half(static_cast<unsigned short>(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu)));
    } else {
      return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
  }
  // elements e and e + 1 (e even); the second is lost in a run of one
  __device__ __forceinline__ void set2(int e, float lo, float hi) {
    if constexpr (sizeof(T) == 4) {
      w[e] = __float_as_uint(lo);
      if constexpr (N > 1) w[e + 1] = __float_as_uint(hi);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 v = __floats2half2_rn(lo, hi);
      w[e / 2] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
      w[e / 2] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

__device__ __forceinline__ void turn(float c, float s, float a, float b, float& ra, float& rb) {
  ra = a * c - b * s;
  rb = a * s + b * c;
}

// A token's angles in shared memory: two pairs to a word, (cos, cos, sin, sin), in
// the order in which a unit's threads ask for them -- pairs 2 k and 2 k + 1 of all
// units side by side, so that 8 threads read 128 bytes without a bank conflict
// (pairs one after another: 19.4 us a prompt's append, 18.5 so).
template <int N>
__device__ __forceinline__ int angle_at(int i, int k, int pairs) {
  return k * ((pairs + N - 1) / N) + i;
}
template <int N>
__device__ __forceinline__ void put_angle(float4* table, int pair, int pairs, float2 cs) {
  const int i = pair / N, e = pair - i * N;
  float* w = reinterpret_cast<float*>(table + angle_at<N>(i, e / 2, pairs)) + e % 2;
  w[0] = cs.x;
  w[2] = cs.y;
}

// Where the two runs of N elements that one thread takes of a head begin, its
// i-th pair of them.  Pairs of halves: each other's partners as long as there are
// any, then 2 N in a row; else 2 N in a row.
template <bool INTERLEAVED, int N>
__device__ __forceinline__ int2 runs_of(int i, int pairs) {
  if (!INTERLEAVED && N * i < pairs) return make_int2(N * i, pairs + N * i);
  return make_int2(2 * N * i, 2 * N * i + N);
}

template <typename T, bool INTERLEAVED, int N>
__device__ __forceinline__ void turn_runs(Run<T, N>& a, Run<T, N>& b, const float4* table, int i, int pairs) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      Run<T, N>& v = e < N / 2 ? a : b;
      constexpr int H = N / 2;
      if (N * i + e >= pairs) continue;
      const float4 cs = table[angle_at<N>(i, e / 2, pairs)];
      float ra, rb;
      turn(cs.x, cs.z, v.get(2 * (e % H)), v.get(2 * (e % H) + 1), ra, rb);
      v.set2(2 * (e % H), ra, rb);
      if (N * i + e + 1 >= pairs) continue;
      turn(cs.y, cs.w, v.get(2 * (e % H) + 2), v.get(2 * (e % H) + 3), ra, rb);
      v.set2(2 * (e % H) + 2, ra, rb);
    }
  } else {
    if (N * i >= pairs) return;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float4 cs = table[angle_at<N>(i, e / 2, pairs)];
      float ra[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f};
      turn(cs.x, cs.z, a.get(e), b.get(e), ra[0], rb[0]);
      if constexpr (N > 1) turn(cs.y, cs.w, a.get(e + 1), b.get(e + 1), ra[1], rb[1]);
      a.set2(e, ra[0], ra[1]);
      b.set2(e, rb[0], rb[1]);
    }
  }
}

// Stores a run into the head at `to`, from element `at` on.
template <typename T, int N>
__device__ __forceinline__ void put_run(const RotaryParams& p, const Run<T, N>& run, T* to, int at) {
  if (write_ok(p.err_word, to, p.head_dim * sizeof(T), to + at, N * sizeof(T))) run.store(to + at);
}
// `to`, if a head there lies inside the buffer it belongs to.
template <typename T>
__device__ __forceinline__ T* head_in(const RotaryParams& p, const void* base, unsigned long long bytes, T* to) {
  return write_ok(p.err_word, base, bytes, to, p.head_dim * sizeof(T)) ? to : nullptr;
}

// The rows of one CTA: head r of them is at src(r) and goes to dst(r) (nowhere, if
// that is null); those with rotated(r) are rotated by the table, which `ready`
// fills while the first loads are under way.  (The next two runs loaded ahead cost
// registers, and so CTAs: prompts 24.0 us, then 19.7 without.)
template <typename T, bool INTERLEAVED, int N, typename Src, typename Dst, typename Rotated, typename Ready>
__device__ __forceinline__ void turn_heads(const RotaryParams& p, int n_rows, const float4* table, const Src& src,
                                           const Dst& dst, const Rotated& rotated, const Ready& ready) {
  const int head_dim = p.head_dim, pairs = p.pairs;
  // units of a row: a power of two, as head_dim and N are
  const int row_shift = 31 - __clz(head_dim / (2 * N)), n = n_rows << row_shift;
  const int step = static_cast<int>(gridDim.y * blockDim.x);
  int u = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
  Run<T, N> a, b;
  int r = 0, i = 0;
  auto load = [&] {
    r = u >> row_shift;
    i = u - (r << row_shift);
    const int2 at = runs_of<INTERLEAVED, N>(i, rotated(r) ? pairs : 0);
    const T* from = src(r);
    a.load(from + at.x);
    b.load(from + at.y);
  };
  if (u < n) load();
  ready();
  while (u < n) {
    const bool turns = rotated(r);
    if (turns) turn_runs<T, INTERLEAVED, N>(a, b, table, i, pairs);
    T* to = dst(r);
    if (to != nullptr) {
      const int2 at = runs_of<INTERLEAVED, N>(i, turns ? pairs : 0);
      put_run(p, a, to, at.x);
      put_run(p, b, to, at.y);
    }
    if ((u += step) < n) load();
  }
}

// A group's tokens: this thread's among them and its unit, and the tokens there
// are.  Their angles lie one token's behind the other's, 128 threads' units of 8 pairs
// at most: 512 words, for tokens of one head.
constexpr int kGroupAngles = kGroupThreads * 4;
struct Member {
  int sub, unit, count, angles;
  bool here;
};
template <int N>
__device__ __forceinline__ Member member_of(const RotaryParams& p, int n_rows) {
  const int units = n_rows << (31 - __clz(p.head_dim / (2 * N))), tid = static_cast<int>(threadIdx.x);
  Member m;
  m.sub = tid / units;
  m.unit = tid - m.sub * units;
  const long long left = p.tokens - static_cast<long long>(blockIdx.x) * p.group;
  m.count = left < p.group ? static_cast<int>(left) : p.group;
  m.angles = (N > 1 ? N / 2 : 1) * ((p.pairs + N - 1) / N);
  m.here = m.sub < m.count;
  return m;
}

}  // namespace detail

// A token to blockIdx.x, of whose heads blockIdx.y takes its part.  N: the longest
// run, of 8, 4, 2 or 1, that pairs of halves come apart into; 8 where neighbours
// are pairs.  Measured on GB300: 1264 tokens of 36 heads of 64, of which 16, 24, 20 and
// 6 elements turn (runs of 8, 4, 2, 1), 5.3, 6.2, 8.0 and 10.8 us.  32 registers let an
// SM hold 2048 threads (40: 2048 tokens of 80 heads of 256 18.8 us, 16.5 so).
// GROUPED: p.group tokens of few heads to a CTA, a unit to a thread; a CTA to each
// would be bound by the CTAs an SM can start (44931 tokens of 8 heads of 64 45.5 us, 16.0
// so, at HBM rate 13.6; 10935 of them 11.4 and 5.6).
template <typename T, bool INTERLEAVED, int N, bool GROUPED>
__global__ void __launch_bounds__(GROUPED ? kGroupThreads : kRotaryThreads, GROUPED ? 12 : sizeof(T) == 4 ? 6 : 8)
gqa_rotary_kernel(const RotaryParams p) {
  __shared__ float4 table[GROUPED ? detail::kGroupAngles : kMaxPairs];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if constexpr (GROUPED) {
    const detail::Member m = detail::member_of<N>(p, p.x.heads);
    const long long first = static_cast<long long>(blockIdx.x) * p.group;
    const int row_shift = 31 - __clz(p.head_dim / (2 * N)), head = m.unit >> row_shift;
    const int i = m.unit - (head << row_shift);
    const int2 at = detail::runs_of<INTERLEAVED, N>(i, p.pairs);
    const long long in_token = static_cast<long long>(head) * p.head_dim, token = first + m.sub;
    detail::Run<T, N> a, b;
    if (m.here) {
      const T* from = static_cast<const T*>(p.x.src) + token * p.x.src_stride + in_token;
      a.load(from + at.x);
      b.load(from + at.y);
    }
    for (int j = static_cast<int>(threadIdx.x); j < m.count * p.pairs; j += kGroupThreads) {
      const int s = j / p.pairs, pair = j - s * p.pairs;
      detail::put_angle<N>(table + s * m.angles, pair, p.pairs,
                           detail::turn_of(p.turns[pair], p.positions[first + s], p.inverse, p.magnitude));
    }
    __syncthreads();
    if (!m.here) return;
    detail::turn_runs<T, INTERLEAVED, N>(a, b, table + m.sub * m.angles, i, p.pairs);
    T* to = detail::head_in(p, p.x.dst, p.x_bytes, static_cast<T*>(p.x.dst) + token * p.x.dst_stride + in_token);
    if (to == nullptr) return;
    detail::put_run(p, a, to, at.x);
    detail::put_run(p, b, to, at.y);
    return;
  }
  const long long token = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  const int position = p.positions[token];
  const uint64_t turns = tid < p.pairs ? p.turns[tid] : 0;
  const T* src = static_cast<const T*>(p.x.src) + token * p.x.src_stride;
  T* dst = static_cast<T*>(p.x.dst) + token * p.x.dst_stride;
  detail::turn_heads<T, INTERLEAVED, N>(
      p, p.x.heads, table, [&](int r) { return src + static_cast<long long>(r) * p.head_dim; },
      [&](int r) { return detail::head_in(p, p.x.dst, p.x_bytes, dst + static_cast<long long>(r) * p.head_dim); },
      [](int) { return true; },
      [&] {
        for (int i = tid; i < p.pairs; i += static_cast<int>(blockDim.x))
          detail::put_angle<N>(table, i, p.pairs,
                               detail::turn_of(i == tid ? turns : p.turns[i], position, p.inverse, p.magnitude));
        __syncthreads();
      });
}

// The same for a batch's new tokens: queries into x.dst, keys and values into
// the page that holds the token's place.
template <typename T, bool INTERLEAVED, int N, bool GROUPED>
__global__ void __launch_bounds__(GROUPED ? kGroupThreads : kRotaryThreads, GROUPED ? 12 : sizeof(T) == 4 ? 6 : 8)
gqa_append_kernel(const RotaryParams p) {
  __shared__ float4 table[GROUPED ? detail::kGroupAngles : kMaxPairs];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if constexpr (GROUPED) {
    __shared__ int positions[kGroupThreads];
    const int hq = p.x.heads, hk = p.k.heads, d = p.head_dim;
    const detail::Member m = detail::member_of<N>(p, hq + 2 * hk);
    const long long token = static_cast<long long>(blockIdx.x) * p.group + m.sub;
    const int row_shift = 31 - __clz(d / (2 * N)), r = m.unit >> row_shift, i = m.unit - (r << row_shift);
    const int pairs = r < hq + hk ? p.pairs : 0;
    const int2 at = detail::runs_of<INTERLEAVED, N>(i, pairs);
    detail::Run<T, N> a, b;
    bool there = false;
    int place = 0, page = -1;
    if (m.here) {
      const int e = static_cast<int>(static_cast<unsigned>(token) / static_cast<unsigned>(p.nq));
      const int t = static_cast<int>(token) - e * p.nq;
      const int raw = p.seqlens[e], asked = detail::asked_tokens(p.pages, e, p.nq);
      const int given = p.positions != nullptr ? p.positions[token] : 0;
      const int L = clamp_len(raw, p.max_seqlen);
      if (raw != L && t == 0 && m.unit == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
      const int n = detail::live_tokens(asked, p.err_word, L, p.nq);
      there = t < n;
      place = L - n + t;
      if (there) {
        const T* from = r < hq        ? static_cast<const T*>(p.x.src) + token * p.x.src_stride + r * d
                        : r < hq + hk ? static_cast<const T*>(p.k.src) + token * p.k.src_stride + (r - hq) * d
                                      : static_cast<const T*>(p.v.src) + token * p.v.src_stride + (r - hq - hk) * d;
        a.load(from + at.x);
        b.load(from + at.y);
        page = detail::page_number(p.pages, p.err_word, e, place);
      }
      if (m.unit == 0) positions[m.sub] = p.positions != nullptr ? given : place;
    }
    __syncthreads();
    for (int j = static_cast<int>(threadIdx.x); j < m.count * p.pairs; j += kGroupThreads) {
      const int s = j / p.pairs, pair = j - s * p.pairs;
      detail::put_angle<N>(table + s * m.angles, pair, p.pairs,
                           detail::turn_of(p.turns[pair], positions[s], 0, p.magnitude));
    }
    __syncthreads();
    if (!there) return;
    if (pairs > 0) detail::turn_runs<T, INTERLEAVED, N>(a, b, table + m.sub * m.angles, i, pairs);
    T* to;
    if (r < hq) {
      to = detail::head_in(p, p.x.dst, p.x_bytes, static_cast<T*>(p.x.dst) + token * p.x.dst_stride + r * d);
    } else {
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages.num_pages)) {
        atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
        return;
      }
      const int h = r < hq + hk ? r - hq : r - hq - hk;
      T* cache = static_cast<T*>(r < hq + hk ? p.k_cache : p.v_cache);
      to = detail::head_in(p, cache, p.cache_bytes,
                           cache + page * p.page_stride + (place & p.pages.page_mask) * p.pos_stride + h * p.head_stride);
    }
    if (to == nullptr) return;
    detail::put_run(p, a, to, at.x);
    detail::put_run(p, b, to, at.y);
    return;
  }
  const long long token = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.nq));
  const int t = static_cast<int>(blockIdx.x) - b * p.nq;
  const uint64_t turns = tid < p.pairs ? p.turns[tid] : 0;
  const int raw = p.seqlens[b], asked = detail::asked_tokens(p.pages, b, p.nq);
  const int given = p.positions != nullptr ? p.positions[token] : 0;
  const int L = clamp_len(raw, p.max_seqlen);
  if (raw != L && t == 0 && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  const int n = detail::live_tokens(asked, p.err_word, L, p.nq);
  if (t >= n) return;
  const int place = L - n + t;
  const int position = p.positions != nullptr ? given : place;
  const int page = detail::page_number(p.pages, p.err_word, b, place);
  const T* q = static_cast<const T*>(p.x.src) + token * p.x.src_stride;
  const T* k = static_cast<const T*>(p.k.src) + token * p.k.src_stride;
  const T* v = static_cast<const T*>(p.v.src) + token * p.v.src_stride;
  T* q_out = static_cast<T*>(p.x.dst) + token * p.x.dst_stride;
  // (where they go is not known before the page is: the first loads need not wait for it)
  T *k_to = nullptr, *v_to = nullptr;
  const int hq = p.x.heads, hk = p.k.heads;
  detail::turn_heads<T, INTERLEAVED, N>(
      p, hq + 2 * hk, table,
      [&](int r) {
        const long long d = p.head_dim;
        return r < hq ? q + r * d : r < hq + hk ? k + (r - hq) * d : v + (r - hq - hk) * d;
      },
      [&](int r) -> T* {
        if (r < hq) return detail::head_in(p, p.x.dst, p.x_bytes, q_out + static_cast<long long>(r) * p.head_dim);
        if (k_to == nullptr) return nullptr;
        return r < hq + hk ? detail::head_in(p, p.k_cache, p.cache_bytes, k_to + (r - hq) * p.head_stride)
                           : detail::head_in(p, p.v_cache, p.cache_bytes, v_to + (r - hq - hk) * p.head_stride);
      },
      [&](int r) { return r < hq + hk && p.pairs > 0; },
      [&] {
        for (int i = tid; i < p.pairs; i += static_cast<int>(blockDim.x))
          detail::put_angle<N>(table, i, p.pairs,
                               detail::turn_of(i == tid ? turns : p.turns[i], position, 0, p.magnitude));
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pages.num_pages)) {
          const long long at = page * p.page_stride + (place & p.pages.page_mask) * p.pos_stride;
          k_to = static_cast<T*>(p.k_cache) + at;
          v_to = static_cast<T*>(p.v_cache) + at;
        } else if (tid == 0) {
          atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
        }
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
  unsigned long long tree_bytes, positions_bytes;  // byte extents, checked by -DGQA_DEBUG builds
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
  PagedKeys k;
  k.news = p.news;
  const int raw = p.seqlens[b], asked = detail::asked_tokens(k, b, p.nq), L = clamp_len(raw, p.max_seqlen);
  int above = t < p.nq ? p.parents[static_cast<long long>(b) * p.nq + t] : -1;
  if (raw != L && t == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  const int n = detail::live_tokens(asked, p.err_word, L, p.nq);
  if (t >= n) above = -1;
  if (above < -1 || above >= t) {
    atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
    above = -1;
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
    uint32_t* to = p.tree + row * p.words + w;
    if (w < p.words && detail::write_ok(p.err_word, p.tree, p.tree_bytes, to, 4)) *to = own[w];
  }
  if (p.positions != nullptr && detail::write_ok(p.err_word, p.positions, p.positions_bytes, p.positions + row, 4))
    p.positions[row] = t < n ? L - n + depth : 0;
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
  unsigned long long cache_bytes, lens_bytes;  // byte extents, checked by -DGQA_DEBUG builds
};

// A CTA to a sequence, 8 elements of K or of V to a thread, which moves them
// for all of the branch.  Token path[i] moves to place i <= path[i], and the
// tokens of a branch ascend, so nothing is overwritten that this thread or a later
// batch of it still reads: a batch of rows is loaded whole, then stored.
//
// What bounds it is a chain of loads, so a token's are looked up by a thread of its
// own, as soon as they can be: lengths and path, then the pages of a token and of its
// place, then the rows.
__global__ void __launch_bounds__(kKeepThreads)
gqa_keep_kernel(const KeepParams p) {
  constexpr int kBatch = 8;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const int32_t* path = p.path + static_cast<long long>(b) * p.max_keep;
  const int raw = p.seqlens[b], given = detail::asked_tokens(p.pages, b, p.nq), asked = p.keep_lens[b];
  int at = -1, before = -1;  // of token tid of the branch, to begin with
  auto load = [&](int i) {
    at = i < p.max_keep ? path[i] : -1;
    before = i > 0 && i < p.max_keep ? path[i - 1] : -1;
  };
  load(tid);
  const int L = clamp_len(raw, p.max_seqlen);
  if (raw != L && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadSeqlen));
  const int n = detail::live_tokens(given, p.err_word, L, p.nq), first = L - n;
  const int most = asked < 0 ? 0 : (asked > p.max_keep ? p.max_keep : asked);
  if (asked != most && tid == 0) atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
  // the page of the token at `at`, and of place i (a token in range is not before its place)
  int from = 0, to = 0;
  auto look_up = [&](int i) {
    if (i >= most || at < i || at >= n) return;
    from = detail::page_number(p.pages, p.err_word, b, first + at);
    to = detail::page_number(p.pages, p.err_word, b, first + i);
  };
  look_up(tid);
  __shared__ int s_bad;  // the first token of the branch that is out of range or does not ascend
  if (tid == 0) s_bad = most;
  __syncthreads();
  for (int i = tid; i < most; i += kKeepThreads) {
    if (i != tid) load(i);
    if (at <= before || at >= n || at < 0) atomicMin(&s_bad, i);
  }
  __syncthreads();
  const int keep = s_bad;
  if (tid == 0) {
    if (keep != most) atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
    if (p.seqlens_out != nullptr && detail::write_ok(p.err_word, p.seqlens_out, p.lens_bytes, p.seqlens_out + b, 4))
      p.seqlens_out[b] = first + keep;
  }
  __shared__ long long s_from[kKeepThreads], s_to[kKeepThreads];  // below 0: it stays, or is lost
  const int per_head = p.head_dim / 8, per_cache = p.kv_heads * per_head;
  for (int base = 0; base < keep; base += kKeepThreads) {
    const int here = min(keep - base, kKeepThreads), i = base + tid;
    if (i < keep) {
      if (most > kKeepThreads) {
        load(i);
        look_up(i);
      }
      s_from[tid] = -1;
      if (at != i) {
        const unsigned pages = static_cast<unsigned>(p.pages.num_pages);
        if (static_cast<unsigned>(from) < pages && static_cast<unsigned>(to) < pages) {
          s_from[tid] = from * p.page_stride + ((first + at) & p.pages.page_mask) * p.pos_stride;
          s_to[tid] = to * p.page_stride + ((first + i) & p.pages.page_mask) * p.pos_stride;
        } else {
          atomicOr(p.err_word, static_cast<unsigned>(kErrBadIndex));
        }
      }
    }
    __syncthreads();
    for (int c = tid; c < 2 * per_cache; c += kKeepThreads) {
      const int in = c < per_cache ? c : c - per_cache, head = in / per_head;
      uint16_t* base_of = static_cast<uint16_t*>(c < per_cache ? p.k_cache : p.v_cache);
      uint16_t* cache = base_of + head * p.head_stride + (in - head * per_head) * 8;
      for (int i0 = 0; i0 < here; i0 += kBatch) {
        uint4 row[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < here && s_from[i0 + j] >= 0) row[j] = *reinterpret_cast<const uint4*>(cache + s_from[i0 + j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i0 + j < here && s_from[i0 + j] >= 0 &&
              detail::write_ok(p.err_word, base_of, p.cache_bytes, cache + s_to[i0 + j], 16))
            *reinterpret_cast<uint4*>(cache + s_to[i0 + j]) = row[j];
      }
    }
    __syncthreads();
  }
}

}  // namespace gqa
