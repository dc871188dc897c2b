"""Calls over pages at the edges of what include/gqa_paged.h allows."""
import math

import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild
from tests.test_paged import BF16, Case, _randn, _words
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


@gpu
@pytest.mark.parametrize("d,T", [(64, 5), (64, 20), (128, 30), (128, 70), (256, 20)])
def test_rows_whose_only_bits_are_of_missing_tokens(dev, d, T):
    """An entry with nothing but T - 2 new tokens, whose rows have set no bits but those of the two that it lacks:
    they see nothing.  Beside it one whose rows see their own token."""
    see = torch.zeros(2, T, T, dtype=torch.bool)
    see[0, :, T - 2:] = True
    see[1] = torch.eye(T)
    c = Case(dev, [T - 2, T], [T - 2, T], T, 8, 2, d, 16, seed=d + T)
    c.poison()
    out, lse = c.run(tree=_words(see).to(dev))
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    _compare("alone", out, lse, c.want(lambda b: see[b, : c.n[b], : c.n[b]]))
    assert g.gqa_decode_get_error() == g.GQA_OK


@pytest.mark.parametrize("t,stride", [
    (torch.empty(2, 0, 8, 64), 512), (torch.empty(2, 0, 12, 64)[:, :, 4:8], 256), (torch.empty(3, 2, 0, 8, 64), 512),
    (torch.empty(0, 3, 8, 64), 512), (torch.empty(0, 8, 64), 512)])
def test_no_tokens_have_a_stride(t, stride):
    """A tensor without tokens has one stride for all of them, wherever its empty dimension is."""
    assert g._paged().stride_of(t) == stride


@gpu
@pytest.mark.parametrize("shape", [(0, 8, 64), (2, 0, 8, 64), (0, 5, 8, 64), (3, 2, 0, 8, 64)])
def test_rotation_of_no_tokens(dev, shape):
    x, turns = torch.empty(shape, dtype=BF16, device=dev), g.rotary_turns(64, device=dev)
    positions = torch.empty(shape[:-2], dtype=torch.int32, device=dev)
    assert g.rotary(x, positions, turns).shape == shape
    g.gqa_rotary_apply(x, positions, turns, x)
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("lens,news,H,K,d,page,m", [
    ([1500, 700, 300, 0], [1000, 513, 256, 0], 8, 2, 128, 16, 256), ([900, 600], [600, 37], 8, 1, 64, 32, 256),
    ([700], [700], 4, 2, 256, 16, 100)])
def test_chunks_longer_than_a_call(dev, lens, news, H, K, d, page, m):
    """A chunk of a prompt appended in one call and seen in several, with the lengths that the header gives: the rows
    of one chain."""
    T, B = max(news), len(lens)
    c = Case(dev, lens, news, T, H, K, d, page, seed=d)
    new = _randn(dev, B, T, H + 2 * K, d, seed=5)
    turns = g.rotary_turns(d, device=dev)
    g.gqa_paged_append(new[:, :, :H], new[:, :, H: H + K], new[:, :, H + K:], c.q, c.k, c.v, c.table, c.ln, new_lens=c.new,
                       turns=turns)
    out, lse = torch.full_like(c.q, math.nan), torch.full((B, T, H), math.nan, device=dev)
    for i in range(0, T, m):
        upto = c.ln - c.new + torch.clamp(c.new, max=i + m)
        here = torch.clamp(c.new - i, 0, m)
        o, l = g.tree_attention(c.q[:, i: i + m].contiguous(), c.k, c.v, c.table, upto, new_lens=here, causal=True)
        out[:, i: i + m], lse[:, i: i + m] = o, l
    _compare("chunk", out, lse, c.want(lambda b: torch.ones(c.n[b], c.n[b]).tril().bool()))
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_an_empty_batch(dev):
    cache, table = _randn(dev, 3, 16, 2, 64), torch.zeros(0, 4, dtype=torch.int32, device=dev)
    q, k = torch.empty(0, 5, 8, 64, dtype=BF16, device=dev), torch.empty(0, 5, 2, 64, dtype=BF16, device=dev)
    none, before = torch.zeros(0, dtype=torch.int32, device=dev), cache.clone()
    tokens = torch.zeros(0, 5, dtype=torch.int32, device=dev)
    tree = torch.zeros(0, 5, 1, dtype=torch.int32, device=dev)
    g.gqa_tree_from_parents(tokens, none, tree, tokens)
    g.gqa_paged_append(q, k, k, q, cache, cache, table, none, positions=tokens, turns=g.rotary_turns(64, device=dev))
    out, lse = g.tree_attention(q, cache, cache, table, none, tree=tree)
    g.gqa_paged_keep(cache, cache, table, none, tokens, none, none, tokens=5)
    assert out.shape == q.shape and lse.shape == (0, 5, 8)
    assert torch.equal(cache, before) and g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("T", [1, 7, 40])
@pytest.mark.parametrize("K,d", [(1, 64), (2, 128), (1, 256)])
def test_a_pool_of_one_page(dev, T, K, d):
    c = Case(dev, [60], None, T, 4 * K, K, d, 64, seed=T, spare=0)
    assert c.k.shape[0] == 1
    out, lse = c.run(causal=True)
    _compare("one page", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool()))
    c.table[0, 0] = 1                                                  # one past the only page: zeros, flagged
    out, lse = c.run(causal=True)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    c.k.zero_(), c.v.zero_()
    c.table[0, 0] = 0
    _compare("no page", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool()))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_caches_inside_larger_tensors(dev, d):
    """Some heads of some pages of a pool, some of each head's elements: strides that are no product of sizes; the rest
    is NaN and stays as it is."""
    T, K, page = 9, 2, 16
    c = Case(dev, [300, 17, 90], None, T, 8, K, d, page, seed=d)
    pools, parts = [], []
    for cache in (c.k, c.v):
        pool = torch.full((cache.shape[0] + 1, 2, page + 3, K + 2, d + 8), math.nan, dtype=BF16, device=dev)
        part = pool[1:, 1, 2: 2 + page, 1: 1 + K, :d]
        part.copy_(cache)
        pools.append(pool)
        parts.append(part)
    c.k, c.v = parts
    new = _randn(dev, 3, T, 8 + 2 * K, d, seed=5)
    turns = g.rotary_turns(d, device=dev)
    g.gqa_paged_append(new[:, :, :8], new[:, :, 8: 8 + K], new[:, :, 8 + K:], c.q, c.k, c.v, c.table, c.ln, turns=turns)
    out, lse = c.run(causal=True)
    _compare("inside", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool()))
    want = [x.clone() for x in parts]
    for x in want:
        for b, L in enumerate(c.lens):
            x[c.places(b, L - T, L - T + 2)] = x[c.places(b, L - T, L)][[1, 5]].clone()
    ends = torch.empty(3, dtype=torch.int32, device=dev)
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, torch.tensor([[1, 5]] * 3, dtype=torch.int32, device=dev),
                     torch.full((3,), 2, dtype=torch.int32, device=dev), ends, tokens=T)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1]) and ends.tolist() == [L - T + 2 for L in c.lens]
    for pool, part in zip(pools, parts):
        part.zero_()
        assert torch.isnan(pool).sum() == pool.numel() - part.numel()
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_sequences_that_share_pages(dev):
    """A prefix in pages that all sequences of a batch name, each with pages of its own behind it."""
    T = 5
    c = Case(dev, [200, 170, 130], None, T, 32, 8, 128, 32, seed=3)
    c.table[1:, :3] = c.table[0, :3]                                   # the first 96 positions
    out, lse = c.run(causal=True)
    _compare("shared", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool()))
    assert g.gqa_decode_get_error() == g.GQA_OK
