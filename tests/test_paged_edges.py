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
