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
#ifdef __CUDACC__
#include "decode_kernel.cuh"
#endif

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

// The token whose bits a thread fetches for row rr of its tile, whose token is tok.
// Threads whose rows hold none take token 0's, which are not used: rows behind the
// entry's last token, and the lanes in front of a shifted tile's first row, where rr
// (and with it tok) is below 0.
GQA_HD int bits_token(int rr, int tok, int live) { return rr < 0 || tok >= live ? 0 : tok; }

#ifdef __CUDACC__
namespace detail {

// The table's page number of position pos of entry b.  -DGQA_DEBUG builds record a
// position that the entry's row does not reach, and read none.
__device__ __forceinline__ int page_number(const PagedKeys& k, unsigned int* err_word, int b, int pos) {
#ifdef GQA_DEBUG
  if (b < 0 || pos < 0 || (pos >> k.page_shift) >= k.cols) {
    atomicOr(err_word, kErrBounds);
    return -1;
  }
#else
  (void)err_word;
#endif
  return k.table[static_cast<long long>(b) * k.cols + (pos >> k.page_shift)];
}

// The page of position pos of entry b.  A number that names no page is flagged
// and replaced by the one past the last, whose box TMA fills with zeros.
__device__ __forceinline__ int page_of(const PagedKeys& k, unsigned int* err_word, int b, int pos) {
  const int page = page_number(k, err_word, b, pos);
  if (static_cast<unsigned>(page) < static_cast<unsigned>(k.num_pages)) return page;
  atomicOr(err_word, kErrBadIndex);
  return k.num_pages;
}

// This lane's page of block blk of entry b, which has L positions: that of the
// block's box `lane`, if it has one that holds any.
__device__ __forceinline__ int lane_page(const PagedKeys& k, unsigned int* err_word, int b, int blk, int L, int lane) {
  const int in_block = lane << k.box_shift, pos = blk * kBlockN + in_block;
  return in_block < kBlockN && pos < L ? page_of(k, err_word, b, pos) : 0;
}

// The boxes of block blk of KV head h that hold any of the entry's L positions,
// into a tile at shared address dst: `chunks` of 64 elements, 16 KB apart, from
// element `elem` on.  Their bytes are expected at `bar`.  The whole warp calls it,
// with the block's pages (lane_page), and the thread that `issues` issues.  (Pages
// are handed over four at a time: one by one, boxes of 16 positions bound wide
// heads, 68 us a call of eight trees of 40 tokens, 63 so.)
template <int CHUNKS>
__device__ __forceinline__ void load_pages(const PagedKeys& k, const void* map, uint32_t bar, uint32_t dst, int blk,
                                           int L, int h, int elem, int pages, bool issues, uint64_t policy) {
  const int box = 1 << k.box_shift, first = blk * kBlockN;
  const int held = (min(L - first, kBlockN) + box - 1) >> k.box_shift;
  if (issues) ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(held * box * CHUNKS * 128));
#pragma unroll 1
  for (int i0 = 0; i0 < held; i0 += 4) {
    int page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = __shfl_sync(0xffffffffu, pages, i0 + i);
    if (issues) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= held) break;
        const int at = (i0 + i) << k.box_shift;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
          ptx::tma_load_4d_hint(dst + c * 16384 + at * 128, map, bar, elem + c * 64, h, (first + at) & k.page_mask, page[i],
                                policy);
      }
    }
    __syncwarp();
  }
}

// Warms L2 with one of `ctas` CTAs' share of the page table's lines (as far as a
// warp's lanes reach).  A prefetch returns no data, so it may run before the
// previous kernel has finished.
__device__ __forceinline__ void prefetch_table(const PagedKeys& k, int entries, int ctas, int lane) {
  const long long lines = (static_cast<long long>(entries) * k.cols + 31) / 32;
  const long long line = static_cast<long long>(lane) * ctas + blockIdx.x;
  if (line < lines) ptx::prefetch_l2(k.table + line * 32);
}

// New tokens of entry b as given (loaded together with its length, ahead of
// what may flag either: a load does not move past an atomic).
__device__ __forceinline__ int asked_tokens(const PagedKeys& k, int b, int nq) {
  return k.news == nullptr ? nq : k.news[b];
}
// Those there are of an entry that has L positions: at most nq, and at most L.
__device__ __forceinline__ int live_tokens(int asked, unsigned int* err_word, int L, int nq) {
  const int most = L < nq ? L : nq;
  if (asked < 0 || asked > nq) atomicOr(err_word, kErrBadIndex);
  return asked < 0 ? 0 : (asked > most ? most : asked);
}

// Bits [0, n) of 32 (n of any sign).
__device__ __forceinline__ uint32_t seen_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Words of bits that say which positions token t of entry b sees, of the 128
// from `from` new tokens past the first new one on: bit i of them, shifted right
// by from modulo 32.  Positions before the first are seen, those the tree has no
// bits for are not (and without a tree all are).  -DGQA_DEBUG builds record a token
// that has no row, and read none.
__device__ __forceinline__ void branch_words(uint32_t (&w)[5], const PagedKeys& k, unsigned int* err_word, int b, int nq,
                                             int t, int from) {
  const uint32_t* row = k.tree == nullptr ? nullptr : k.tree + (static_cast<long long>(b) * nq + t) * k.tree_words;
  const bool in_tree = b >= 0 && static_cast<unsigned>(t) < static_cast<unsigned>(nq);
  check_coord(err_word, in_tree);
#ifdef GQA_DEBUG
  if (!in_tree) row = nullptr;
#endif
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int at = (from >> 5) + i;  // (an arithmetic shift: below 0 for what comes before)
    w[i] = row == nullptr || at < 0 ? 0xffffffffu : at < k.tree_words ? row[at] : 0u;
  }
}

}  // namespace detail
#endif

}  // namespace gqa
