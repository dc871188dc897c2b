"""Paths of the rows kernel (csrc/rows_kernel.cuh) that only calls of certain
shapes take, each with a check, from the plan, that its call takes it.  GPU
results against the definition in fp64, within test_shared_keys.py's bounds.
"""
import math

import numpy as np
import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from tests.test_shared_keys import BF16, _attend, _built, _check_plan, _compare, _desc, _rand, dev, gpu  # noqa: F401


def _items(q, k, lens, prefix=0, room=0):
    """The plan of a call on this device: info [2, 4] and items [n, 9]."""
    B, T, H, d = q.shape
    desc = _desc(batch=B, q_tokens=T, q_heads=H, kv_heads=k.shape[2], head_dim=d, max_seqlen=k.shape[1])
    _, _, info, items = g.gqa_shared_keys_plan(desc, lens, prefix, room)
    return info, items


def _sample(out, lse, q, k, v, b, tokens, L):
    """Rows of some tokens of entry b against all its L keys."""
    at = torch.tensor(tokens, device=q.device)
    sees = torch.ones(len(tokens), L, dtype=torch.bool, device=q.device)
    want = _attend(q[b, at].double(), k[b, :L].double(), v[b, :L].double(), sees, q.shape[3] ** -0.5, q.dtype, out.dtype)
    _compare(f"entry {b}", out[b:b + 1, at], lse[b:b + 1, at], [want])


@gpu
def test_a_tile_without_rows_may_wait_for_long_items(dev, monkeypatch):
    """A last group of rows that fills one tile, over so many keys that its
    part in a CTA outlasts the timeout of a wait (1 ms here), before an item of
    both tiles: the second tile's warps wait for that one all the while."""
    T, K, d, S = 50 * 256 + 44, 3, 64, 512000
    gen = torch.Generator(dev).manual_seed(1)
    q, k, v = _rand(gen, 1, T, K, d), _rand(gen, 1, S, K, d), _rand(gen, 1, S, K, d)
    ln = torch.tensor([S], dtype=torch.int32, device=dev)
    _, items = _items(q, k, [S])
    blocks = items[:, 6] - items[:, 5]
    waits = (items[:-1, 4] == 50) & (items[1:, 4] != 50) & (items[:-1, 0] == items[1:, 0])
    assert blocks[:-1][waits].max() >= 2000   # of ~1 us each
    monkeypatch.setenv("GQA_WAIT_TIMEOUT_MS", "1")
    out, lse = g.cross_attention(q, k, v, ln)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    _sample(out, lse, q, k, v, 0, [0, 127, 128, 255, 256, 6000, 12799, 12800, 12843], S)
