// A paged cache as the kernels see it, and which of an entry's drafted tokens
// a query token sees.
//
// Positions [0, L) of an entry lie in pages of 2^page_shift positions: position
// j in page table[b][j >> page_shift], at j & page_mask.  TMA fetches boxes of
// 2^box_shift positions: a page, or 128 positions of a larger one.
//
// The last `live` of the L positions are the entry's new tokens.  Every one of
// them sees the positions before the first; of the new ones token t sees
// [0, t] (chain), those whose bit its row of `tree` has set, or (neither) all.
#pragma once
#include <cstdint>

#include "plan.cuh"

namespace gqa {

enum : unsigned { kErrBadIndex = 8u };  // beside kErrTimeout and its like (decode_kernel.cuh)

struct PagedKeys {
  const int32_t* table;   // [B, cols]
  const int32_t* news;    // [B] new tokens of each entry, or null: nq
  const uint32_t* tree;   // [B, nq, tree_words] bits, or null
  int cols, num_pages;
  int page_shift, page_mask, box_shift;
  int tree_words;
  int chain;
};

#ifdef __CUDACC__
namespace detail {

// The page of position pos of entry b.  A number that names no page is flagged
// and replaced by the one past the last, whose box TMA fills with zeros.
__device__ __forceinline__ int page_of(const PagedKeys& k, unsigned int* err_word, int b, int pos) {
  const int page = k.table[static_cast<long long>(b) * k.cols + (pos >> k.page_shift)];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(k.num_pages)) return page;
  atomicOr(err_word, kErrBadIndex);
  return k.num_pages;
}

// New tokens of entry b, which has L positions: at most nq, and at most L.
__device__ __forceinline__ int live_tokens(const PagedKeys& k, unsigned int* err_word, int b, int L, int nq) {
  const int most = L < nq ? L : nq;
  if (k.news == nullptr) return most;
  const int n = k.news[b];
  if (n < 0 || n > nq) atomicOr(err_word, kErrBadIndex);
  return n < 0 ? 0 : (n > most ? most : n);
}

// Token t's row of bits, or null.
__device__ __forceinline__ const uint32_t* branch_of(const PagedKeys& k, int b, int nq, int t) {
  return k.tree == nullptr ? nullptr : k.tree + (static_cast<long long>(b) * nq + t) * k.tree_words;
}

// Bits [0, n) of 32 (n of any sign).
__device__ __forceinline__ uint32_t seen_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Of the 32 positions from `from` new tokens past the first new one on: those
// before the first, and those the row's bits name (every one, without a row).
__device__ __forceinline__ uint32_t branch_bits(const uint32_t* row, int words, int from) {
  if (row == nullptr || from <= -32) return 0xffffffffu;
  const int i = from >> 5, s = from & 31;  // (arithmetic shift: -1 for the 31 positions before)
  const uint32_t lo = i < 0 ? 0xffffffffu : (i < words ? row[i] : 0u), hi = i + 1 < words ? row[i + 1] : 0u;
  return __funnelshift_r(lo, hi, s);
}

}  // namespace detail
#endif

}  // namespace gqa
