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
    want = _attend(q[b, at].double(), k[b, :L].double(), v[b, :L].double(), sees, q.shape[3] ** -0.5, q.dtype,
                   out.dtype)
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
    q = _rand(gen, 1, T, H, d, dtype=dtype)
    k, v = _rand(gen, 1, S, K, d, dtype=dtype), _rand(gen, 1, S, K, d, dtype=dtype)
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


# ------------------------------------------------------------------ dealt plans
MANY = 4200   # entries: more than the kernel stages lengths for


def _dealt(items):
    """Every triple whole, triple t of a launch in CTA t mod the grid."""
    order = np.lexsort((items[:, 4], items[:, 3], items[:, 2], items[:, 1]))
    ctas = items[:, 0].max() + 1
    return bool((items[:, 8] <= 1).all() and (items[order, 0] == np.arange(len(items)) % ctas).all())


def _many(dev, T, H, K, d, S, dtype, lens, seed):
    gen = torch.Generator(dev).manual_seed(seed)
    q = _rand(gen, len(lens), T, H, d, dtype=dtype)
    k, v = _rand(gen, len(lens), S, K, d, dtype=dtype), _rand(gen, len(lens), S, K, d, dtype=dtype)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    past = torch.arange(S, device=dev)[None, :] >= ln[:, None]
    k[past], v[past] = math.nan, math.inf
    return q, k, v, ln


@gpu
@pytest.mark.parametrize("d,dtype,T,H,K", [(128, torch.float16, 40, 2, 2), (128, BF16, 129, 2, 1),
                                           (256, BF16, 20, 4, 2), (256, torch.float16, 140, 1, 1)])
def test_dealt_batches(dev, d, dtype, T, H, K):
    lens = [(i * 29) % 301 for i in range(MANY)]
    q, k, v, ln = _many(dev, T, H, K, d, 300, dtype, lens, seed=1)
    assert _dealt(_items(q, k, lens)[1])
    out, lse = g.cross_attention(q, k, v, ln)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    assert torch.isfinite(out).all()
    for b in list(range(0, MANY, 31)) + [MANY - 1]:
        _sample(out, lse, q, k, v, b, range(T), lens[b])


@gpu
@pytest.mark.parametrize("d,dtype,T,H,K,causal", [(128, torch.float16, 3, 4, 2, True), (256, BF16, 2, 4, 1, True),
                                                  (256, torch.float16, 1, 2, 2, False)])
def test_dealt_batches_behind_a_prefix(dev, d, dtype, T, H, K, causal):
    lens, P, room = [(i * 29) % 151 for i in range(MANY)], 333, 400
    q, k, v, ln = _many(dev, T, H, K, d, 150, dtype, lens, seed=2)
    gen = torch.Generator(dev).manual_seed(3)
    kp, vp = _rand(gen, room, K, d, dtype=dtype), _rand(gen, room, K, d, dtype=dtype)
    kp[P:], vp[P:] = math.inf, math.nan
    assert _dealt(_items(q, k, lens, P, room)[1])
    out, lse = g.prefix_decode(q, kp, vp, torch.tensor([P], dtype=torch.int32, device=dev), k, v, ln, causal=causal)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    assert torch.isfinite(out).all()
    for b in list(range(0, MANY, 31)) + [1, 2, MANY - 1]:
        L = lens[b]
        sees = torch.ones(T, P + L, dtype=torch.bool, device=dev)
        if causal:
            sees[:, P:] = torch.arange(L, device=dev)[None, :] <= (L - T + torch.arange(T, device=dev))[:, None]
        _compare(f"entry {b}", out[b:b + 1], lse[b:b + 1],
                 [_attend(q[b].double(), torch.cat([kp[:P], k[b, :L]]).double(), torch.cat([vp[:P], v[b, :L]]).double(),
                          sees, d ** -0.5, dtype, dtype)])


HUGE = dict(batch=2, q_tokens=320000, q_heads=2, kv_heads=2, head_dim=64, max_seqlen=1 << 22)   # 2.3e9 units


def test_units_past_32_bits_are_dealt():
    _check_plan([300, 1000], HUGE["q_tokens"], 2, 2, 64, HUGE["max_seqlen"], 152)
    assert _dealt(g.gqa_shared_keys_plan(_desc(**HUGE), [300, 1000], 0, 0, 152)[3])
    fits = dict(HUGE, q_tokens=290000)
    assert not _dealt(g.gqa_shared_keys_plan(_desc(**fits), [300, 1000], 0, 0, 152)[3])


@gpu
def test_a_call_of_so_many_units(dev):
    lens, T = [300, 1000], HUGE["q_tokens"]
    gen = torch.Generator(dev).manual_seed(4)
    q = _rand(gen, 2, T, 2, 64)
    k, v = (torch.empty(2, HUGE["max_seqlen"], 2, 64, dtype=BF16, device=dev) for _ in range(2))
    for b, L in enumerate(lens):
        k[b, :L], v[b, :L] = _rand(gen, L, 2, 64), _rand(gen, L, 2, 64)
        k[b, L: L + 200], v[b, L: L + 200] = math.nan, math.nan
    out, lse = g.cross_attention(q, k, v, torch.tensor(lens, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    assert torch.isfinite(out).all()
    for b in range(2):
        for at in range(0, T, 40000):
            _sample(out, lse, q, k, v, b, range(at, at + 300), lens[b])
        _sample(out, lse, q, k, v, b, range(T - 300, T), lens[b])


@gpu
def test_debug_build_of_dealt_batches(dev):
    """The bounds-checked build catches no write outside a buffer where triples are dealt whole."""
    import ctypes

    from gqa_decode_blackwell_gb300 import build as gbuild

    gbuild.build_debug()
    L = g.load_library(gbuild.DEBUG_LIB)
    assert L.gqa_decode_get_error(1) == g.GQA_OK
    stream = torch.cuda.current_stream().cuda_stream
    lens = [(i * 29) % 161 for i in range(MANY)]
    kp = torch.ones(130, 2, 128, dtype=BF16, device=dev)
    P = torch.tensor([130], dtype=torch.int32, device=dev)
    for T, prefix in ((40, False), (150, False), (2, True)):
        q, k, v, ln = _many(dev, T, 2, 2, 128, 160, BF16, lens, seed=5)
        want = g.prefix_decode(q, kp, kp, P, k, v, ln) if prefix else g.cross_attention(q, k, v, ln)
        out, lse = torch.full_like(want[0], math.nan), torch.full_like(want[1], math.nan)
        n = g.gqa_prefix_workspace_size(q, kp, k) if prefix else g.gqa_cross_workspace_size(q, k)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
        desc = g.make_desc(q, k)
        end = [ln.data_ptr(), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, stream]
        if prefix:
            rc = L.gqa_prefix_attn(ctypes.byref(desc), q.data_ptr(), kp.data_ptr(), kp.data_ptr(), P.data_ptr(), 130,
                                   k.data_ptr(), v.data_ptr(), *end)
        else:
            rc = L.gqa_cross_attn(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), *end)
        torch.cuda.synchronize()
        assert rc == g.GQA_OK and L.gqa_decode_get_error(1) == g.GQA_OK
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# -------------------------------------------------------- infinities and NaN seen
def _expect(what, out, lse, want):
    """As _compare, with NaN and infinities where the definition has them."""
    o, l, to, tl = want
    got, gl = out.double(), lse.double()
    assert torch.equal(torch.isnan(got), torch.isnan(o)), (what, "NaN of O")
    assert torch.equal(torch.isnan(gl), torch.isnan(l)), (what, "NaN of the LSE")
    for x, w, t in ((got, o, to), (gl, l, tl)):
        far = torch.isinf(w)
        assert torch.equal(x[far], w[far]) and not torch.isinf(x[~far]).any(), (what, "infinities")
        fine = torch.isfinite(w)
        assert ((x - w).abs()[fine] <= t[fine]).all(), (what, (x - w).abs()[fine].max().item())


def _check_seen(dev, T, d, dtype, S, call):
    """One head each: scores of -inf (some, whole blocks, all), a NaN in
    K, in V, in one row of q, infinite V, a score of +inf.  Another head is as it was."""
    K = 9
    gen = torch.Generator(dev).manual_seed(d)
    q = _rand(gen, 1, T, K, d, dtype=dtype)
    k, v = _rand(gen, 1, S, K, d, dtype=dtype), _rand(gen, 1, S, K, d, dtype=dtype)
    ln = torch.tensor([S], dtype=torch.int32, device=dev)
    clean, clean_lse = call(q.abs(), k, v, ln)
    q = q.abs()
    k[0, ::3, 0, 0] = -math.inf           # q is positive: a score of -inf
    k[0, torch.arange(S, device=dev) // 128 % 4 < 2, 1, 5] = -math.inf   # whole blocks, the first ones of many items
    k[0, :, 2, 1] = -math.inf             # nothing left
    k[0, 1234, 3, 2] = math.nan
    v[0, 77, 4, 3] = math.nan
    v[0, S - 1, 5, 4], v[0, 0, 5, 5] = math.inf, -math.inf
    q[0, T // 2, 6, 1] = math.nan
    k[0, 1000, 8, 3] = math.inf
    out, lse = call(q, k, v, ln)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_OK
    assert torch.equal(out[:, :, 7], clean[:, :, 7]) and torch.equal(lse[:, :, 7], clean_lse[:, :, 7])

    sees = torch.ones(T, S, dtype=torch.bool, device=dev)
    for h in range(K):
        qd, kd, vd = q[0, :, h:h + 1].double(), k[0, :, h:h + 1].double(), v[0, :, h:h + 1].double()
        if h < 3:                          # a score of -inf is a key that is not seen
            hidden = torch.isinf(kd).any(-1)[:, 0]
            kd = torch.where(torch.isinf(kd), 0.0, kd)
            o, l, to, tl = _attend(qd, kd, vd, sees & ~hidden[None, :], d ** -0.5, dtype, dtype)
        else:                              # bounds from finite stand-ins, values as they come
            zq, zk, zv = (torch.where(torch.isfinite(x), x, 0.0) for x in (qd, kd, vd))
            o, l, to, tl = _attend(zq, zk, zv, sees, d ** -0.5, dtype, dtype)
            if h in (3, 8):
                o, l = torch.full_like(o, math.nan), torch.full_like(l, math.nan)
            elif h == 4:
                o[..., 3] = math.nan
            elif h == 5:
                o[..., 4], o[..., 5] = math.inf, -math.inf
            elif h == 6:
                o[T // 2], l[T // 2] = math.nan, math.nan
        _expect(f"head {h}", out[0, :, h:h + 1], lse[0, :, h:h + 1], (o, l, to, tl))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [40, 300], ids=["rows of one tile", "rows of two"])
@pytest.mark.parametrize("dtype", [BF16, torch.float16], ids=["bf16", "fp16"])
def test_infinities_and_nan_that_are_seen(dev, T, d, dtype):
    _check_seen(dev, T, d, dtype, 30000, g.cross_attention)


WAYS = {"cross attention": g.cross_attention, "one split": lambda *a: g.decode(*a, num_splits=1),
        "combine": lambda *a: g.decode(*a, num_splits=5, reduction="combine"),
        "many splits": lambda *a: g.decode(*a, num_splits=64, reduction="combine"),
        "cluster": lambda *a: g.decode(*a, num_splits=4, reduction="cluster")}


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 9, 32])
@pytest.mark.parametrize("way", WAYS)
def test_infinities_and_nan_that_few_rows_see(dev, way, T, d):
    """The decode kernel, whose result few rows have, and each of its merges."""
    for dtype, S in ((BF16, 20000), (torch.float16, 1300)):
        _check_seen(dev, T, d, dtype, S, WAYS[way])


@gpu
def test_a_partial_of_nan_is_not_an_empty_one(dev):
    """gqa_decode_combine: an LSE of NaN beside empty splits, and beside full ones, in both of its loops."""
    for n in (3, 64):
        o = torch.randn(n, 4, 64, device=dev)
        lse = torch.zeros(n, 4, device=dev)
        lse[:, 0] = -math.inf
        lse[1, 0] = lse[1, 1] = math.nan
        lse[:, 2] = -math.inf
        out, l = torch.empty(4, 64, device=dev), torch.empty(4, device=dev)
        g.gqa_decode_combine(o, lse, out, l)
        assert torch.isnan(out[:2]).all() and torch.isnan(l[:2]).all()
        assert (out[2] == 0).all() and l[2] == -math.inf
        assert torch.isfinite(out[3]).all() and torch.isfinite(l[3])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_keys_behind_a_prefix_have_one_tile_of_rows(d):
    """The kernel's causal limit is a row's place in its tile: a second tile
    must hold the same rows, whatever the group and the tokens."""
    for G in range(1, 33):
        for nq in {1, 32 // G}:
            desc = _desc(batch=3, q_tokens=nq, q_heads=2 * G, kv_heads=2, head_dim=d, max_seqlen=700, causal=1)
            _, _, info, _ = g.gqa_shared_keys_plan(desc, [700, 0, 3], 500, 600, 152)
            assert info[1, 0] == nq and info[1, 1] == 1 and info[1, 2] == (d != 256)
