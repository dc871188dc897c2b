// Work partition of the rows kernel (rows_kernel.cuh), shared by the kernel
// and the host-side view of it.
//
// A launch has one or two sections: a set of batch entries, each with a
// length, and per entry `heads` triples (KV heads x tile groups) that read
// the entry's key blocks.  The sections' triples, in order, are laid along a
// line of units: a triple with blocks takes item_units for its fixed cost (Q
// load, pipeline fill, epilogue) and then block_units for every block; one
// without takes empty_units for the zeros to write, so that a batch's empty
// entries are spread like its work -- or none and is not listed, where all
// there is to write is a record (empty_owner).  The U units are cut into C
// ranges of equal length (give or take one unit), one per CTA, and a block
// belongs to the CTA in whose range it begins.  A range is never shorter than
// a block, so the CTAs that hold a triple's blocks are consecutive and each
// holds at least one.
//
// The units let blocks of different cost share a launch: compute-bound ones
// of a prefix that many rows share, and memory-bound ones of the sequences'
// own keys, run side by side on different SMs and end together.
//
// Batches with more entries than the kernel stages lengths for (or so much work
// that units would pass 32 bits, in which all of this is computed: emulated
// 64-bit divisions cost a CTA's start-up microseconds) are dealt whole, triple
// by triple, to the CTAs in turn.
#pragma once
#include <cstdint>

#include "plan.cuh"

namespace gqa {

constexpr int kMaxRowsEntries = 4096;  // batch entries whose lengths are staged in shared memory

struct RowsPlanSection {
  int batch;        // entries (0: no such section)
  int heads;        // triples of an entry
  int max_len;      // lengths are clamped to [0, max_len]
  int block_units;  // of a block
  int item_units;
  int empty_units;  // of a triple without blocks; 0: such triples are not listed
  int groups;       // triples that share an entry's keys of one KV head
};

struct RowsPlan {
  RowsPlanSection s[2];
  int num_ctas;
  int dealt;        // whole triples in turn, instead of equal ranges
};

struct RowsWork {
  int section, b, hh;      // triple hh of entry b
  int L;
  int blk_begin, blk_end;  // equal: no keys
  int turn;                // blocks are taken from blk_begin + turn on, and then from blk_begin
  int whole;               // all of the triple's blocks
  int n_pieces;            // of the triple, where blk_begin is its first block
};

GQA_HD int rows_units(const RowsPlanSection& s, int L) {
  const int nblk = num_blocks(L);
  return nblk > 0 ? nblk * s.block_units + s.item_units : s.empty_units;
}

struct RowsPlanIter {
  const RowsPlan* rp;
  const int32_t* lens;     // clamped lengths of both sections' entries (dealt: unused)
  const uint32_t* pre;     // entries + 1 prefix sums of their units
  const int32_t* raw0;     // each section's lengths
  const int32_t* raw1;
  uint32_t U, lo, hi;
  uint32_t q, rem, C;      // ranges: `rem` of q + 1 units, then of q
  int e, hh, cta;
  long long next_triple;

  // First unit of CTA c's range, and the CTA whose range holds unit u.
  GQA_HD uint32_t start(uint32_t c) const { return c * q + (c < rem ? c : rem); }
  GQA_HD int owner(uint32_t u) const {
    const uint32_t split = rem * (q + 1);
    return static_cast<int>(u < split ? u / (q + 1) : rem + (u - split) / q);
  }
  // The first entry from `a` on that holds units past u (the number of entries if none does).
  GQA_HD int reaching(uint32_t u, int a) const {
    int z = rp->s[0].batch + rp->s[1].batch;
    while (a < z) {
      const int mid = (a + z) / 2;
      if (pre[mid + 1] > u) z = mid; else a = mid + 1;
    }
    return a;
  }
  GQA_HD const RowsPlanSection& section(int entry) const { return rp->s[entry < rp->s[0].batch ? 0 : 1]; }

  GQA_HD void init(const RowsPlan* plan, const int32_t* lens0, const int32_t* lens1, const int32_t* clamped,
                   const uint32_t* prefix, int c) {
    rp = plan; lens = clamped; pre = prefix; raw0 = lens0; raw1 = lens1; cta = c;
    next_triple = c;
    if (rp->dealt) return;
    const int E = rp->s[0].batch + rp->s[1].batch;
    U = pre[E];
    const uint32_t w0 = static_cast<uint32_t>(rp->s[0].block_units), w1 = static_cast<uint32_t>(rp->s[1].block_units);
    const uint32_t most = U / (w0 > w1 ? w0 : w1);  // ranges at least a block long
    C = most < 1 ? 1 : (most < static_cast<uint32_t>(rp->num_ctas) ? most : static_cast<uint32_t>(rp->num_ctas));
    q = U / C;
    rem = U - q * C;
    hh = 0;
    if (static_cast<uint32_t>(c) >= C) {  // this CTA owns nothing
      e = E;
      lo = hi = U;
      return;
    }
    lo = start(static_cast<uint32_t>(c));
    hi = start(static_cast<uint32_t>(c) + 1);
    e = reaching(lo, 0);
    if (e < E && pre[e] < lo)
      hh = static_cast<int>((lo - pre[e]) / static_cast<uint32_t>(rows_units(section(e), lens[e])));
  }
  GQA_HD void emit(RowsWork& w, int blk_begin, int blk_end, int whole, int pieces) {
    w.section = e < rp->s[0].batch ? 0 : 1;
    w.b = e - (w.section ? rp->s[0].batch : 0);
    w.hh = hh;
    w.L = lens[e];
    w.blk_begin = blk_begin;
    w.blk_end = blk_end;
    w.turn = 0;
    w.whole = whole;
    w.n_pieces = pieces;
  }
  GQA_HD bool next_dealt(RowsWork& w) {
    const long long n0 = static_cast<long long>(rp->s[0].batch) * rp->s[0].heads;
    const long long n1 = static_cast<long long>(rp->s[1].batch) * rp->s[1].heads;
    if (next_triple >= n0 + n1) return false;
    w.section = next_triple < n0 ? 0 : 1;
    const long long t = next_triple - (w.section ? n0 : 0);
    const RowsPlanSection& s = rp->s[w.section];
    w.b = static_cast<int>(div_nonneg(t, s.heads));
    w.hh = static_cast<int>(t - static_cast<long long>(w.b) * s.heads);
    w.L = clamp_len((w.section ? raw1 : raw0)[w.b], s.max_len);
    w.blk_begin = 0;
    w.blk_end = num_blocks(w.L);
    w.turn = 0;
    w.whole = 1;
    w.n_pieces = 1;
    next_triple += rp->num_ctas;
    return true;
  }
  GQA_HD bool next(RowsWork& w) {
    if (rp->dealt) return next_dealt(w);
    const int E = rp->s[0].batch + rp->s[1].batch;
    while (e < E) {
      const RowsPlanSection& s = section(e);
      const uint32_t u = static_cast<uint32_t>(rows_units(s, lens[e]));
      if (u == 0) {  // a run of these may be long
        e = reaching(pre[e], e + 1);
        continue;
      }
      const uint32_t v = pre[e] + static_cast<uint32_t>(hh) * u;
      if (v >= hi) return false;
      const uint32_t nblk = static_cast<uint32_t>(num_blocks(lens[e]));
      bool mine = false;
      if (nblk == 0) {
        if (v >= lo) {
          emit(w, 0, 0, 1, 1);
          mine = true;
        }
      } else {
        const uint32_t bu = static_cast<uint32_t>(s.block_units);
        const uint32_t first = v + static_cast<uint32_t>(s.item_units);  // where block 0 begins
        const uint32_t last = first + (nblk - 1) * bu;                    // and the last one
        const uint32_t from = lo > first ? (lo - first + bu - 1) / bu : 0;
        const uint32_t upto = hi > last ? nblk : (hi > first ? (hi - first + bu - 1) / bu : 0);
        if (from < upto) {
          const bool whole = from == 0 && upto == nblk;
          emit(w, static_cast<int>(from), static_cast<int>(upto), whole,
               from > 0 ? 0 : (whole ? 1 : owner(last) - cta + 1));
          // Tile groups that share keys are cut at different blocks.  Each
          // range begins with the block whose index is a multiple of a range's
          // blocks, so that all reach a block at the same time, and memory is
          // asked for it once (64 tokens of 64 / 8 heads, two groups, against
          // 131072 keys 201 us, 213 without).
          if (s.groups > 1 && from > 0) {
            const uint32_t every = q / bu, past = from - from / every * every;
            if (past > 0 && every - past < upto - from) w.turn = static_cast<int>(every - past);
          }
          mine = true;
        }
      }
      if (++hh == s.heads) { hh = 0; ++e; }
      if (mine) return true;
    }
    return false;
  }
};

// The CTA that records the triples of entry e (of both sections) that has no
// keys, in launches that do not list those.
GQA_HD int empty_owner(const RowsPlan& p, int e) { return e % p.num_ctas; }

// Where a piece's partials go: indexes of pieces that no two pieces of a
// section share.  every_piece: triple + CTA (both grow along the line, never
// standing still together); else only cut triples have pieces, at most two in
// a CTA: 2 * CTA, + 1 for a triple's first.
GQA_HD int rows_piece(bool every_piece, bool dealt, int triple, int cta, bool first_piece) {
  if (every_piece) return dealt ? triple : triple + cta;
  return 2 * cta + (first_piece ? 1 : 0);
}

}  // namespace gqa
