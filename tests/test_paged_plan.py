"""The plan of attention over pages, on the host: the launch that the library
describes (make_launch) and the partition that the kernel's plan warp walks
(RowsPlanIterT of one section), every CTA of it, compiled from the kernel's own
headers and linked against the library.

Required of every launch: each block of each triple in one item, pieces that no
two items share, inside the workspace, and as the merges look for them."""
import os

import pytest

from gqa_decode_blackwell_gb300 import build as gbuild
from tests.test_paged_bounds import host_program


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


DIVISIONS = r"""
#include "rows_plan.cuh"
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>

int main() {
  std::mt19937 rng(1);
  long long bad = 0;
  for (int i = 0; i < 3000000; ++i) {
    // operands of every size, quotients around their whole numbers
    const uint32_t d = std::max<uint32_t>(1u, (rng() & 0x7fffffffu) >> (rng() % 31));
    const uint32_t most = 0x7fffffffu / d;
    const uint32_t q = rng() % ((most < (1u << 20) - 1 ? most : (1u << 20) - 2) + 1);
    const int64_t around = static_cast<int64_t>(q) * d + static_cast<int>(rng() % 3) - 1;
    const uint32_t near = around < 0 || around > 0x7fffffff ? q * d : static_cast<uint32_t>(around);
    const uint32_t within = static_cast<uint32_t>(std::min<uint64_t>(uint64_t(q) * d + rng() % d, 0x7fffffffu));
    for (uint32_t x : {near, within}) {
      const uint32_t want = x / d;
      if (want >= (1u << 20)) continue;
      if (gqa::div_small(x, d) != want) ++bad;
      // what a division good to 2 ulp may give instead
      const float f = static_cast<float>(x) / static_cast<float>(d);
      float lo = f, hi = f;
      for (int u = 0; u < 2; ++u) lo = std::nextafterf(lo, 0.f), hi = std::nextafterf(hi, INFINITY);
      if (gqa::div_corrected(lo, x, d) != want || gqa::div_corrected(hi, x, d) != want) ++bad;
    }
    const uint32_t x = rng() & 0x7fffffffu, by = 1u + rng() % (rng() % 2 ? 64u : 4096u);
    if (gqa::div_by(x, gqa::rows_divisor(static_cast<int>(by))) != x / by) ++bad;
  }
  std::printf("%lld bad\n", bad);
  return bad != 0;
}
"""

PLANS = r"""
#include "rows_host.h"
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

using namespace gqa;

#define MUST(c) do { if (!(c)) { std::printf("line %d: %s (B %d nq %d H %d/%d d %d sm %d)\n", __LINE__, #c, d.batch, \
    d.q_tokens, d.q_heads, d.kv_heads, d.head_dim, sm); return false; } } while (0)

bool check(const gqa_desc_t& d, const std::vector<int>& raw, int sm, int (&seen)[5]) {
  const RowsLaunch r = make_launch(&d, nullptr, sm, true);
  MUST(r.status == GQA_OK && r.n == 1);
  const int G = d.q_heads / d.kv_heads, fit = 128 / G;
  const RowsPlanSection& s = r.plan.s[0];
  MUST((r.tiles == 1) == (d.head_dim == 256 || (d.head_dim == 128 && d.q_tokens <= fit && d.batch <= kMaxLoneEntries)));
  MUST(r.plan.dealt || d.batch <= (d.head_dim == 128 && r.tiles == 1 ? kMaxLoneEntries : kMaxRowsEntries));
  const auto& o = r.s[0];
  const int per_group = (o.split_keys ? 1 : r.tiles) * o.tokens;
  MUST(o.groups * per_group >= d.q_tokens && (o.groups - 1) * per_group < d.q_tokens);
  MUST(o.tokens * G <= (o.shift ? 64 : 128) && s.heads == d.kv_heads * o.groups);
  MUST(rows_ws(r).total >= static_cast<size_t>(r.part_rows) * (d.head_dim * 4 + 8) + r.records * 8);
  MUST(r.part_rows == o.pieces * r.tiles * o.tokens * G);
  ++seen[r.every_piece ? 0 : 1];
  if (r.plan.dealt) ++seen[2];
  if (r.tiles == 1 && d.head_dim == 128) ++seen[3];
  if (o.shift) ++seen[4];

  std::vector<int32_t> lens(d.batch);
  std::vector<uint32_t> pre(d.batch + 1, 0);
  for (int b = 0; b < d.batch; ++b) {
    lens[b] = clamp_len(raw[b], s.max_len);
    pre[b + 1] = pre[b] + static_cast<uint32_t>(s.heads) * static_cast<uint32_t>(rows_units(s, lens[b]));
  }
  struct Triple { int blocks = 0, items = 0, pieces = 0, first = -1, last_cta = -1, begin_cta = -1, whole = 0; };
  std::vector<Triple> triples(o.triples);
  std::vector<char> piece_taken(o.pieces, 0);
  long long items = 0;
  for (int c = 0; c < r.plan.num_ctas; ++c) {
    RowsPlanIterT<true> iter;
    iter.init(&r.plan, raw.data(), nullptr, lens.data(), pre.data(), c);
    int begun = 0;
    RowsWork w;
    while (iter.next(w)) {
      MUST(++items < 50000000);
      MUST(w.section == 0 && w.b >= 0 && w.b < d.batch && w.hh >= 0 && w.hh < s.heads && w.L == lens[w.b]);
      MUST(0 <= w.blk_begin && w.blk_begin <= w.blk_end && w.blk_end <= num_blocks(w.L));
      Triple& t = triples[w.b * s.heads + w.hh];
      const int n = w.blk_end - w.blk_begin;
      if (n == 0) {
        MUST(num_blocks(w.L) == 0 && t.items == 0 && w.whole);
        ++t.items;
        if (r.plan.dealt && r.every_piece) MUST(w.b * s.heads + w.hh < o.pieces);
        continue;
      }
      MUST(w.turn >= 0 && w.turn < n && w.blk_begin == t.blocks);  // in order, CTA by CTA
      if (t.items > 0) MUST(t.last_cta == c - 1);
      t.blocks = w.blk_end;
      t.last_cta = c;
      MUST(w.whole == (n == num_blocks(w.L)));
      const bool first = w.blk_begin == 0;
      if (r.every_piece || !w.whole) {
        const int piece = rows_piece(r.every_piece, r.plan.dealt, w.b * s.heads + w.hh, c, first);
        MUST(piece >= 0 && piece < o.pieces && !piece_taken[piece]);
        piece_taken[piece] = 1;
        if (first) {
          t.first = piece;
          t.pieces = w.n_pieces;
          t.begin_cta = c;
          if (!r.every_piece) MUST(++begun == 1);  // a record to a CTA
        } else {
          // where the merges look for it
          MUST(piece == (r.every_piece ? t.first + t.items : 2 * (t.begin_cta + t.items)));
        }
        ++t.items;
      } else {
        ++t.items;
        t.whole = 1;
      }
    }
  }
  for (int b = 0; b < d.batch; ++b)
    for (int h = 0; h < s.heads; ++h) {
      const Triple& t = triples[b * s.heads + h];
      MUST(t.blocks == num_blocks(lens[b]));
      if (t.blocks == 0) {
        MUST(t.items == (r.plan.dealt || !r.every_piece ? 1 : 0));
      } else if (t.whole) {
        MUST(t.items == 1);
      } else {
        MUST(t.pieces == t.items);
        MUST(r.every_piece ? t.first <= o.pieces - t.pieces : 2 * (t.begin_cta + t.pieces) <= o.pieces);
      }
    }
  return true;
}

int main() {
  std::mt19937 rng(7);
  auto upto = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
  auto spread = [&](int lo, int hi) {  // over the logarithm
    return std::min(hi, static_cast<int>(lo * std::exp2(std::log2(static_cast<double>(hi) / lo) * upto(10001) / 10000.0)));
  };
  int seen[5] = {0, 0, 0, 0, 0};
  for (int i = 0; i < 1500; ++i) {
    gqa_desc_t d = {};
    d.head_dim = 64 << upto(3);
    d.kv_heads = spread(1, 16);
    d.q_heads = d.kv_heads * (upto(4) ? 1 << upto(4) : 1 + upto(128));
    d.q_tokens = upto(3) ? spread(1, 256) : 1 + upto(9);
    d.batch = i % 50 == 0 ? 4000 + upto(300) : i % 3 == 0 ? 120 + upto(20) : spread(1, 100);
    const int most = spread(16, i % 50 == 0 ? 600 : 20000);
    d.max_seqlen = upto(5) ? most : std::min(most * 4096ll, 1ll << 30);
    std::vector<int> lens(d.batch);
    const int empty = upto(3);
    for (int& L : lens) L = empty && upto(3) < empty ? 0 : upto(30) ? 1 + upto(most) : upto(2) ? -upto(9) : most + 5;
    if (!check(d, lens, upto(4) ? 152 : 1 + upto(160), seen)) return 1;
  }
  std::printf("all partials %d, whole triples %d, dealt %d, one tile of 128 %d, shifted %d\n", seen[0], seen[1], seen[2],
              seen[3], seen[4]);
  return *std::min_element(seen, seen + 5) < 10;
}
"""


def test_divisions_are_exact(tmp_path):
    """Those of the plan, with whatever error the device's fast division may have."""
    host_program(tmp_path, DIVISIONS)


def test_every_block_of_a_paged_launch_is_in_one_item(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(gbuild._nvcc()))), "include")
    out = host_program(tmp_path, PLANS, "-I", cuda,
                       gbuild.LIB, f"-Wl,-rpath,{gbuild.PKG}")
    print(out)
