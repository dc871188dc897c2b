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


# ------------------------------------------------------------- the running max
STEP = 9.0   # log2 units between blocks: above the 8 by which a maximum may stand still


def _staircase(q, k, v, keys=128, seed=0):
    """Gives q and k a direction of their own, along which scores climb by STEP
    from block to block for seven blocks and fall back to the first: in a row
    whose sign is positive the maximum moves at every step up, in one whose
    sign is negative hardly ever.  Rows and entries differ in sign."""
    d, dev = q.shape[-1], q.device
    block = torch.arange(k.shape[-3], device=dev) // keys
    step = STEP / (8.0 * d ** -0.5 * math.log2(math.e))
    k[..., -1] = ((block % 8) * step).to(k.dtype)[:, None]
    sign = torch.randint(0, 2, q.shape[:-1], generator=torch.Generator(dev).manual_seed(seed), device=dev) * 2 - 1
    q[..., -1] = (8.0 * sign).to(q.dtype)


CLIMBS = [  # T, H, K, S of one entry; which items the case is for
    ("two tiles", 512, 8, 8, 12000),
    ("a last group of one tile", 300, 8, 8, 12000),
    ("tile groups that begin at different blocks", 700, 4, 4, 20000),
    ("split keys", 30, 8, 4, 70000),
    ("one full tile", 32, 32, 8, 40000),
]


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("name,T,H,K,S", CLIMBS, ids=[c[0] for c in CLIMBS])
def test_maxima_that_climb_within_items(dev, name, T, H, K, S, dtype, d):
    gen = torch.Generator(dev).manual_seed(d)
    q, k, v = _rand(gen, 1, T, H, d, dtype=dtype), _rand(gen, 1, S, K, d, dtype=dtype), _rand(gen, 1, S, K, d, dtype=dtype)
    _staircase(q, k, v)
    ln = torch.tensor([S], dtype=torch.int32, device=dev)
    info, items = _items(q, k, [S])
    blocks = items[:, 6] - items[:, 5]
    assert np.median(blocks) >= (8 if info[0, 2] else 5)   # with split keys, a tile has every other one
    if "groups" in name:
        assert info[0, 1] > 1 and (items[:, 5] > 0).sum() > 100
    out, lse = g.cross_attention(q, k, v, ln)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    tokens = sorted(set(list(range(0, T, 13)) + [min(T - 1, x) for x in (127, 128, 255, 256, 299)] + [T - 1]))
    for at in range(0, len(tokens), 8):
        _sample(out, lse, q, k, v, 0, tokens[at: at + 8], S)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,causal", [(BF16, False), (torch.float16, True)], ids=["bf16", "fp16 causal"])
@pytest.mark.parametrize("B,T,H,K", [(20, 2, 16, 2), (3, 2, 16, 2)], ids=["rows of two tiles", "rows of one"])
def test_maxima_that_climb_behind_a_prefix(dev, B, T, H, K, dtype, causal, d):
    """... within the prefix's items, within those of own keys, and from one section to the other in the merge."""
    P, S = (30000 if B > 3 else 80000), 6000
    lens = [S - 211 * b for b in range(B)]
    gen = torch.Generator(dev).manual_seed(d)
    q = _rand(gen, B, T, H, d, dtype=dtype)
    k, v = _rand(gen, B, S, K, d, dtype=dtype), _rand(gen, B, S, K, d, dtype=dtype)
    kp, vp = _rand(gen, P, K, d, dtype=dtype), _rand(gen, P, K, d, dtype=dtype)
    _staircase(q, kp, vp)
    _staircase(q, k, v)
    _, items = _items(q, k, lens, P, P)
    blocks = items[:, 6] - items[:, 5]
    for section in (0, 1):
        assert np.median(blocks[items[:, 1] == section]) >= 4
    out, lse = g.prefix_decode(q, kp, vp, torch.tensor([P], dtype=torch.int32, device=dev), k, v,
                               torch.tensor(lens, dtype=torch.int32, device=dev), causal=causal)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    for b in range(0, B, 3):
        L = lens[b]
        keys, values = torch.cat([kp, k[b, :L]]).double(), torch.cat([vp, v[b, :L]]).double()
        sees = torch.ones(T, P + L, dtype=torch.bool, device=dev)
        if causal:
            sees[:, P:] = torch.arange(L, device=dev)[None, :] <= (L - T + torch.arange(T, device=dev))[:, None]
        _compare(f"entry {b}", out[b:b + 1], lse[b:b + 1],
                 [_attend(q[b].double(), keys, values, sees, d ** -0.5, dtype, dtype)])
