// Work partition of the rows kernel (rows_kernel.cuh), shared by the kernel
// and the host-side view of it.
//
// A launch has one or two sections: a set of batch entries, each with a
// length, and per entry `heads` triples (KV heads x tile groups) that read
// the entry's key blocks.  The sections' triples, in order, are laid along a
// line of units: a triple with blocks takes item_units for its fixed cost (Q
// load, pipeline fill, epilogue) and then block_units for every block; one
// without takes none.  The U units are cut into C equal ranges, one per CTA,
// and a block belongs to the CTA in whose range it begins.  A range is never
// shorter than a block, so the CTAs that hold a triple's blocks are
// consecutive and each holds at least one.
//
// The units let blocks of different cost share a launch: compute-bound ones
// of a prefix that many rows share, and memory-bound ones of the sequences'
// own keys, run side by side on different SMs and end together.
//
// Batches with more entries than the kernel stages lengths for are dealt
// whole, triple by triple, to the CTAs in turn.
#pragma once
#include <cstdint>

#include "plan.cuh"

namespace gqa {

constexpr int kMaxRowsEntries = 1024;  // batch entries whose lengths are staged in shared memory

struct RowsPlanSection {
  int batch;        // entries (0: no such section)
  int heads;        // triples of an entry
  int max_len;      // lengths are clamped to [0, max_len]
  int block_units, item_units;
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
  int first_piece, n_pieces;
};

GQA_HD int rows_units(const RowsPlanSection& s, int L) {
  const int nblk = num_blocks(L);
  return nblk > 0 ? nblk * s.block_units + s.item_units : 0;
}

struct RowsPlanIter {
  RowsPlan rp;
  const int32_t* lens;    // clamped lengths of both sections' entries (dealt: unused)
  const long long* pre;   // entries + 1 prefix sums of their units
  const int32_t* raw[2];  // each section's lengths
  long long U, lo, hi, next_triple;
  int e, hh, cta, C;

  GQA_HD void init(const RowsPlan& p, const int32_t* raw0, const int32_t* raw1, const int32_t* clamped,
                   const long long* prefix, int c) {
    rp = p; lens = clamped; pre = prefix; raw[0] = raw0; raw[1] = raw1; cta = c;
    next_triple = c;
    if (rp.dealt) return;
    const int E = rp.s[0].batch + rp.s[1].batch;
    U = pre[E];
    int longest = 1;
    for (int i = 0; i < 2; ++i)
      if (rp.s[i].batch > 0 && rp.s[i].block_units > longest) longest = rp.s[i].block_units;
    const long long most = div_nonneg(U, longest);
    C = most < 1 ? 1 : (most < rp.num_ctas ? static_cast<int>(most) : rp.num_ctas);
    hh = 0;
    if (c >= C) {  // this CTA owns nothing
      e = E;
      lo = hi = U;
      return;
    }
    lo = muldiv(c, U, C);
    hi = muldiv(c + 1, U, C);
    int a = 0, z = E;  // the first entry that reaches lo
    while (a < z) {
      const int mid = (a + z) / 2;
      if (pre[mid + 1] > lo || pre[mid] >= lo) z = mid; else a = mid + 1;
    }
    e = a;
    if (e < E && pre[e] < lo) {
      const int u = rows_units(section(e), lens[e]);
      if (u > 0) hh = static_cast<int>(div_nonneg(lo - pre[e], u));
    }
  }
  GQA_HD const RowsPlanSection& section(int entry) const { return rp.s[entry < rp.s[0].batch ? 0 : 1]; }
  GQA_HD int owner(long long u) const { return static_cast<int>(div_nonneg((u + 1) * C - 1, U)); }
  GQA_HD void advance() {
    if (++hh == section(e).heads) { hh = 0; ++e; }
  }
  GQA_HD void emit(RowsWork& w, int blk_begin, int blk_end, int first, int pieces) {
    w.section = e < rp.s[0].batch ? 0 : 1;
    w.b = e - (w.section ? rp.s[0].batch : 0);
    w.hh = hh;
    w.L = lens[e];
    w.blk_begin = blk_begin;
    w.blk_end = blk_end;
    w.first_piece = first;
    w.n_pieces = pieces;
    advance();
  }
  GQA_HD bool next_dealt(RowsWork& w) {
    const long long n0 = static_cast<long long>(rp.s[0].batch) * rp.s[0].heads;
    const long long n1 = static_cast<long long>(rp.s[1].batch) * rp.s[1].heads;
    if (next_triple >= n0 + n1) return false;
    w.section = next_triple < n0 ? 0 : 1;
    const long long t = next_triple - (w.section ? n0 : 0);
    const RowsPlanSection& s = rp.s[w.section];
    w.b = static_cast<int>(div_nonneg(t, s.heads));
    w.hh = static_cast<int>(t - static_cast<long long>(w.b) * s.heads);
    w.L = clamp_len(raw[w.section][w.b], s.max_len);
    w.blk_begin = 0;
    w.blk_end = num_blocks(w.L);
    w.first_piece = 1;
    w.n_pieces = 1;
    next_triple += rp.num_ctas;
    return true;
  }
  GQA_HD bool next(RowsWork& w) {
    if (rp.dealt) return next_dealt(w);
    const int E = rp.s[0].batch + rp.s[1].batch;
    while (e < E) {
      const RowsPlanSection& s = section(e);
      const int u = rows_units(s, lens[e]);
      const long long v = pre[e] + static_cast<long long>(hh) * u;
      if (u == 0) {
        if ((v >= lo && v < hi) || (v == U && cta == C - 1)) {
          emit(w, 0, 0, 1, 1);
          return true;
        }
        if (v >= hi) return false;
        advance();
        continue;
      }
      if (v >= hi) return false;
      const int nblk = num_blocks(lens[e]), bu = s.block_units;
      const long long first = v + s.item_units;  // where block 0 begins
      const long long from = lo > first ? div_nonneg(lo - first + bu - 1, bu) : 0;
      const long long upto = hi > first ? div_nonneg(hi - first + bu - 1, bu) : 0;
      const int blk_begin = static_cast<int>(from < nblk ? from : nblk);
      const int blk_end = static_cast<int>(upto < nblk ? upto : nblk);
      if (blk_begin >= blk_end) {
        advance();
        continue;
      }
      const int pieces = owner(first + static_cast<long long>(nblk - 1) * bu) - owner(first) + 1;
      emit(w, blk_begin, blk_end, blk_begin == 0, pieces);
      return true;
    }
    return false;
  }
};

// Where a piece's partials go: indexes of pieces that no two pieces of a
// section share.  every_piece: triple + CTA (both grow along the line, never
// standing still together); else only cut triples have pieces, at most two in
// a CTA: 2 * CTA, + 1 for a triple's first.
GQA_HD int rows_piece(bool every_piece, bool dealt, int triple, int cta, bool first_piece) {
  if (every_piece) return dealt ? triple : triple + cta;
  return 2 * cta + (first_piece ? 1 : 0);
}

}  // namespace gqa
