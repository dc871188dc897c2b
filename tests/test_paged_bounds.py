"""What the kernels over pages read and write lies inside the caller's buffers.

CPU: the token whose bits a thread fetches, for every place of a row in a tile,
by the function that the kernel calls, compiled for the host.  GPU: the
bounds-checked build, over trees that lie in the middle of a larger tensor."""
import shutil
import subprocess

import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild
from tests.test_paged import (APPEND, BF16, FP16, FP32, STEPS, Case, Step, _branches, _ints, _parents, _randn, _words)
from tests.test_shared_keys import _compare

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.gqa_decode_get_error(clear=True)
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def debug():
    """Calls f with the bounds-checked build in place of the library, which has to stay quiet."""
    gbuild.build_debug()
    release, g._lib = g.lib(), g.load_library(gbuild.DEBUG_LIB)
    checked, g._lib = g._lib, release

    def run(f):
        try:
            g._lib = checked
            assert g.gqa_decode_get_error() == g.GQA_OK
            got = f()
            torch.cuda.synchronize()
            assert g.gqa_decode_get_error() == g.GQA_OK
        finally:
            g._lib = release
        return got

    return run


# Every lane of every tile: rows of `tokens` tokens of G heads, of the second tile from lane `shift` on where both
# hold the same rows.
TOKENS = r"""
#include "paged.h"
#include <cstdio>

int main() {
  long long looked = 0, bad = 0;
  for (int G = 1; G <= 128; ++G)
    for (int nq = 1; nq <= 256; nq = nq < 9 || nq > 253 ? nq + 1 : nq + 7) {
      const int most = 128 / G, tokens = nq < most ? nq : most;
      for (int split = 0; split <= (nq <= most ? 1 : 0); ++split) {
        const int shift = split && tokens * G <= 64 ? 64 : 0, per_group = split ? tokens : 2 * tokens;
        for (int tok0 = 0; tok0 < nq; tok0 += per_group)
          for (int live = 0; live <= nq; live += nq > 8 ? (nq + 3) / 4 : 1)
            for (int t = 0; t < 2; ++t)
              for (int r = 0; r < 128; ++r) {
                const int rr = r - (t == 1 ? shift : 0), tok = tok0 + (split ? 0 : t * tokens) + rr / G;
                const int row = gqa::bits_token(rr, tok, live);
                ++looked;
                if (row < 0 || row >= nq) ++bad;
                if (rr >= 0 && rr < tokens * G && tok < live && row != tok) ++bad;  // a row that is used: its own
              }
      }
    }
  std::printf("%lld lanes, %lld bad\n", looked, bad);
  return bad != 0 || looked < 1000000;
}
"""


def host_program(tmp_path, text, *link):
    """Compiles a program of the kernels' host-side headers and runs it."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "program.cpp", tmp_path / "program"
    source.write_text(text)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", gbuild.CSRC, str(source), *link, "-o", str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout + done.stderr
    return done.stdout


def test_the_bits_fetched_are_those_of_a_token(tmp_path):
    """Lanes in front of a shifted tile's first row fetch no row before the tree's first one."""
    host_program(tmp_path, TOKENS)


def _inside(dev, see):
    """Words of bits in the middle of a tensor of ones, with 64 KB on either side."""
    words = _words(see)
    around = torch.full((words.numel() + (1 << 15),), -1, dtype=torch.int32, device=dev)
    tree = around[1 << 14: (1 << 14) + words.numel()].view(words.shape)
    tree.copy_(words)
    return tree


SPLIT = [  # lens, news, T, H, K, d, page, dtype: split tiles, of at most 64 rows but for the last two
    ([6000] + [3000] * 40, None, 7, 8, 1, 64, 16, BF16),
    ([6000] + [3000] * 9, None, 16, 32, 8, 64, 32, BF16),
    ([5000] + [2000, 900, 17] * 4, None, 9, 12, 12, 64, 16, FP16),        # G = 1
    ([5000] + [2000, 900, 70] * 4, None, 64, 6, 6, 64, 16, BF16),         # G = 1, 64 rows: two words to a token
    ([4000] * 12, [3, 0] * 6, 4, 40, 10, 64, 64, BF16),
    ([2000] + [(i * 97) % 900 for i in range(129)], None, 9, 32, 8, 128, 16, BF16),   # more than one warp stages
    ([2000] + [(i * 97) % 900 for i in range(139)], [i % 4 for i in range(140)], 3, 8, 8, 128, 32, FP16),
    ([4000, 900] * 8, None, 26, 32, 8, 64, 32, BF16),                      # 104 rows
    ([4000, 900] * 8, None, 70, 8, 2, 64, 16, BF16),                       # rows of two tiles and one alone
]


@gpu
@pytest.mark.parametrize("lens,news,T,H,K,d,page,dtype", SPLIT)
def test_trees_inside_a_larger_tensor(dev, debug, lens, news, T, H, K, d, page, dtype):
    """Items of many blocks whose drafts are the second tile's: no row of bits outside the tree is asked for, and the
    results are those of the definition."""
    c = Case(dev, lens, news, T, H, K, d, page, dtype, seed=T)
    branches = [_branches(_parents(T, b)) for b in range(5)]
    tree = _inside(dev, torch.stack([branches[b % 5] for b in range(len(lens))]))
    got = debug(lambda: c.run(tree=tree))
    _compare("inside", *got, c.want(lambda b: branches[b % 5][: c.n[b], : c.n[b]]))
    out, lse = c.run(tree=tree)
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
    assert g.gqa_decode_get_error() == g.GQA_OK


PARTIALS = [  # lens, news, T, H, K, d, page, dtype, out dtype: pieces of each form
    ([4000, 1], None, 1, 32, 8, 128, 16, BF16, None),
    ([900, 65, 300], [64, 64, 10], 64, 64, 8, 128, 128, BF16, None),                # a dead second group
    ([9000, 641, 130], [40, 7, 33], 40, 16, 2, 256, 64, FP16, torch.float32),       # three tiles of one head
    ([3000, 2000, 1, 700], [70, 33, 1, 0], 70, 8, 2, 64, 32, BF16, None),           # a group of two tiles, then one alone
    ([900, 257, 256], [256, 256, 200], 256, 4, 2, 64, 16, BF16, torch.float32),
    ([5000, 0] + [(i * 97) % 300 for i in range(60)], None, 16, 28, 4, 128, 32, FP16, None),   # whole ones and cut ones
    ([4000] + [(i * 331) % 700 for i in range(40)], [9] + [i % 10 for i in range(40)], 9, 24, 8, 256, 64, BF16, None),
    ([700, 650], [3, 2], 3, 100, 1, 128, 1024, FP16, None),                         # G = 100: a token a tile
]


@gpu
@pytest.mark.parametrize("lens,news,T,H,K,d,page,dtype,out_dtype", PARTIALS)
@pytest.mark.parametrize("causal", [False, True])
def test_partials_lie_in_their_tiles(dev, debug, lens, news, T, H, K, d, page, dtype, out_dtype, causal):
    """Each store of a partial row inside its own tile's place in the workspace; the bits of the release build."""
    c = Case(dev, lens, news, T, H, K, d, page, dtype, seed=T)
    got = debug(lambda: c.run(causal=causal, out_dtype=out_dtype))
    out, lse = c.run(causal=causal, out_dtype=out_dtype)
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
    _compare("partials", out, lse, c.want((lambda b: torch.ones(c.n[b], c.n[b]).tril().bool()) if causal else None, out_dtype))


@gpu
@pytest.mark.parametrize("i", range(len(STEPS)))
def test_steps_write_inside_their_buffers(dev, debug, i):
    """Tree, append, attention, merges and keep of a verification step: the bits of the release build."""
    steps = [Step(dev, *STEPS[i], seed=70 + i) for _ in range(2)]
    steps[0].run()
    debug(steps[1].run)
    a, b = ([s.tree, s.positions, s.q_out, s.out, s.lse, s.c.k, s.c.v, s.ends] for s in steps)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    steps[1].check()


@gpu
@pytest.mark.parametrize("lens,news,T,H,K,d,page,dtype,heads_first,dim,interleaved", APPEND)
def test_appends_write_inside_their_buffers(dev, debug, lens, news, T, H, K, d, page, dtype, heads_first, dim, interleaved):
    """Alone in a CTA and in groups, all runs, caches with heads first or last."""
    c = Case(dev, lens, news, T, H, K, d, page, dtype, heads_first, seed=T)
    new = _randn(dev, len(lens), T, H + 2 * K, d, dtype=dtype, seed=5)
    turns = g.rotary_turns(dim, device=dev) if dim else None
    k, v, results = c.k.clone(), c.v.clone(), []

    def append():
        out = torch.zeros_like(c.q)
        c.k.copy_(k)
        c.v.copy_(v)
        g.gqa_paged_append(new[:, :, :H], new[:, :, H: H + K], new[:, :, H + K:], out, c.k, c.v, c.table, c.ln,
                           new_lens=c.new, turns=turns, interleaved=interleaved)
        results.append((out, c.k.clone(), c.v.clone()))

    append()
    debug(append)
    assert all(torch.equal(a, b) for a, b in zip(*results))


@gpu
@pytest.mark.parametrize("T,H,d,dim,interleaved,dtype", [
    (9, 32, 128, 128, False, BF16), (2701, 3, 64, 20, False, FP16), (2703, 9, 64, 64, True, FP32),
    (300, 65, 256, 254, False, BF16), (1, 1, 64, 2, False, FP32), (2709, 2, 64, 2, False, FP32)])
def test_rotations_write_inside_their_buffers(dev, debug, T, H, d, dim, interleaved, dtype):
    """Into part of a larger tensor."""
    x, turns = _randn(dev, T, H, d, dtype=dtype, seed=T), g.rotary_turns(dim, device=dev)
    positions = torch.arange(T, dtype=torch.int32, device=dev)
    want = g.rotary(x, positions, turns, interleaved=interleaved)
    into = torch.full((T, H + 1, d), 7.0, dtype=dtype, device=dev)
    debug(lambda: g.gqa_rotary_apply(x, positions, turns, into[:, 1:], interleaved=interleaved))
    assert torch.equal(into[:, 1:], want) and (into[:, 0] == 7).all()


@gpu
def test_bad_numbers_in_the_checked_build(dev):
    """Pages, parents and branches out of range are flagged as what they are, as by the release build."""
    gbuild.build_debug()
    release, g._lib = g.lib(), g.load_library(gbuild.DEBUG_LIB)
    try:
        c = Case(dev, [300, 200], None, 20, 8, 2, 64, 16, seed=11)
        c.table[1, 12] = -1                                            # positions 192 to 207
        k = _randn(dev, 2, 20, 2, 64, seed=8)
        for call in (lambda: g.gqa_paged_append(None, k, k, None, c.k, c.v, c.table, c.ln), c.run,
                     lambda: g.gqa_paged_keep(c.k, c.v, c.table, c.ln, _ints(dev, [[1], [19]]), _ints(dev, [1, 1]), tokens=20),
                     lambda: g.gqa_paged_keep(c.k, c.v, c.table, c.ln, _ints(dev, [[1], [20]]), _ints(dev, [1, 1]), tokens=20)):
            call()
            assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
        assert g.gqa_decode_get_error() == g.GQA_OK
    finally:
        g._lib = release
