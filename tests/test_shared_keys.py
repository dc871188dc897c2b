"""Cross attention and shared-prefix decode (include/gqa_shared_keys.h).

CPU: the refusals, and the tiled kernel's work decomposition.  GPU: every
element against the definition in fp64, within a bound derived per element.

The bound.  With w_j the exact softmax weights, A = sum_j w_j |v_j| and N keys:
- P is rounded once to in_dtype (relative error at most u = eps / 2, the sums
  are of the unrounded p): u A; fp16 also loses up to half its smallest step,
  2^-25, of every p, against a sum that is at least 1 (the running max never
  exceeds the row's): 2^-25 N max|v|;
- a score is an fp32 sum of d exact products, in whatever order and with up to
  a full unit lost at each addition: ds = d 2^-23 scale sum_i |q_i k_i|, and
  the product with the scale and the subtraction of the max, 2^-22 |s| more
  (both in log2 units and back); a weight's relative error is then at most
  2 ds (its own and the sum's) + 2^-20 (exp2 to 2 ulp, and the same of the sum);
- fp32 sums over N keys and the merge of pieces: (N + 64) 2^-23 of A;
- the output's own rounding: half a step of |O|.
For the LSE: ds + 2^-20 + (N + 64) 2^-23, and 2^-22 |lse|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild

gpu = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.gqa_decode_get_error(clear=True)
    return torch.device("cuda:0")


# ------------------------------------------------------------------ refusals
ALIGNED = 1 << 20   # fake, aligned non-null "device" addresses: never dereferenced


def _desc(**kw):
    base = dict(batch=2, q_tokens=100, q_heads=8, kv_heads=2, head_dim=128, max_seqlen=256, scale=0.0, causal=0,
                out_dtype=0, in_dtype=0, reduction=0)
    base.update(kw)
    return g.gqa_desc_t(**base)


def _cross(desc, q=ALIGNED, k=ALIGNED, v=ALIGNED, ln=ALIGNED, out=ALIGNED, lse=None, ws=None, wsb=0):
    return g.lib().gqa_cross_attn(ctypes.byref(desc), q, k, v, ln, out, lse, ws, wsb, None)


def _prefix(desc, q=ALIGNED, kp=ALIGNED, vp=ALIGNED, pl=ALIGNED, room=512, k=ALIGNED, v=ALIGNED, ln=ALIGNED,
            out=ALIGNED, lse=None, ws=None, wsb=0):
    return g.lib().gqa_prefix_attn(ctypes.byref(desc), q, kp, vp, pl, room, k, v, ln, out, lse, ws, wsb, None)


BAD_DESC = [
    (dict(head_dim=96), g.GQA_ERR_UNSUPPORTED),
    (dict(q_heads=6, kv_heads=4), g.GQA_ERR_INVALID_ARG),
    (dict(q_tokens=0), g.GQA_ERR_INVALID_ARG),
    (dict(batch=-1), g.GQA_ERR_INVALID_ARG),
    (dict(max_seqlen=0), g.GQA_ERR_INVALID_ARG),
    (dict(max_seqlen=(1 << 30) + 1), g.GQA_ERR_UNSUPPORTED),
    (dict(out_dtype=7), g.GQA_ERR_INVALID_ARG),
    (dict(in_dtype=1), g.GQA_ERR_INVALID_ARG),
    (dict(out_dtype=2), g.GQA_ERR_UNSUPPORTED),   # fp16 output of bf16 inputs
    (dict(scale=-1.0), g.GQA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), g.GQA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), g.GQA_ERR_INVALID_ARG),
    (dict(reduction=1), g.GQA_ERR_UNSUPPORTED),
    (dict(reduction=2), g.GQA_ERR_UNSUPPORTED),
    (dict(reduction=5), g.GQA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,expect", BAD_DESC + [
    (dict(causal=1), g.GQA_ERR_UNSUPPORTED),
    (dict(q_heads=129, kv_heads=1), g.GQA_ERR_UNSUPPORTED),   # a token's rows exceed a tile
])
def test_cross_refuses(kw, expect):
    assert _cross(_desc(**kw)) == expect
    assert g.lib().gqa_cross_workspace_size(ctypes.byref(_desc(**kw))) == 0


@pytest.mark.parametrize("kw,expect", BAD_DESC + [(dict(q_tokens=9), g.GQA_ERR_UNSUPPORTED)])
def test_prefix_refuses(kw, expect):
    d = _desc(**{"q_tokens": 1, **kw})
    assert _prefix(d) == expect
    assert g.lib().gqa_prefix_workspace_size(ctypes.byref(d), 512) == 0


def test_pointers_and_prefix_capacity():
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(ln=None), dict(out=None), dict(q=ALIGNED + 8),
               dict(k=ALIGNED + 2), dict(v=ALIGNED + 4), dict(out=ALIGNED + 8), dict(ln=ALIGNED + 1),
               dict(lse=ALIGNED + 2)):
        assert _cross(_desc(), **kw) == g.GQA_ERR_INVALID_ARG, kw
        assert _cross(_desc(q_tokens=1), **kw) == g.GQA_ERR_INVALID_ARG, kw   # few rows
        assert _prefix(_desc(q_tokens=1), **kw) == g.GQA_ERR_INVALID_ARG, kw
    for kw in (dict(kp=None), dict(vp=None), dict(pl=None), dict(kp=ALIGNED + 8), dict(vp=ALIGNED + 8),
               dict(pl=ALIGNED + 2), dict(room=0), dict(room=-5)):
        assert _prefix(_desc(q_tokens=1), **kw) == g.GQA_ERR_INVALID_ARG, kw
    assert _prefix(_desc(q_tokens=1), room=(1 << 30) + 1) == g.GQA_ERR_UNSUPPORTED
    assert _cross(_desc(batch=0), q=None, k=None, v=None, ln=None, out=None) == g.GQA_OK
    assert _prefix(_desc(batch=0, q_tokens=1), q=None, kp=None, out=None) == g.GQA_OK
    L = g.lib()
    assert L.gqa_cross_attn(None, *[ALIGNED] * 5, None, None, 0, None) == g.GQA_ERR_INVALID_ARG
    assert L.gqa_cross_workspace_size(None) == 0 and L.gqa_prefix_workspace_size(None, 5) == 0


def test_header_is_plain_c_and_exported(tmp_path):
    import os
    import shutil
    import subprocess

    names = g.header_functions(gbuild.SHARED_KEYS_HEADER)
    assert names == ["gqa_cross_attn", "gqa_cross_workspace_size", "gqa_prefix_attn", "gqa_prefix_workspace_size",
                     "gqa_shared_keys_plan"]
    for n in names:
        assert hasattr(g.lib(), n)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "gqa_shared_keys.h"\nint main(void) {\n  gqa_desc_t d = {0};\n  int64_t n = 0;\n'
                   "  (void)gqa_cross_attn(&d, 0, 0, 0, 0, 0, 0, 0, gqa_cross_workspace_size(&d), 0);\n"
                   "  (void)gqa_prefix_attn(&d, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, gqa_prefix_workspace_size(&d, 1), 0);\n"
                   "  return (int)gqa_shared_keys_plan(&d, 0, 0, 0, 1, 0, 0, 0, 0, 0, &n) == GQA_OK;\n}\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(gbuild.ROOT, "include"), str(src), gbuild.LIB, "-o", str(tmp_path / "use")],
                   check=True)


def test_python_checks_tensors():
    q = torch.zeros(2, 40, 8, 64, dtype=BF16)
    k = torch.zeros(2, 10, 2, 64, dtype=BF16)
    ln = torch.zeros(2, dtype=torch.int32)
    out = torch.empty_like(q)
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=k[:, :5]), dict(kv_lens=ln.long()), dict(kv_lens=ln[:1]),
                dict(q=q.transpose(1, 2)), dict(out=out[:, :1]), dict(out=out.transpose(2, 3)),
                dict(lse=torch.empty(2, 40, 8, dtype=torch.float64)), dict(lse=torch.empty(2, 8, 40)),
                dict()):   # the last: CPU tensors
        with pytest.raises(ValueError):
            g.gqa_cross_attn(**{**dict(q=q, k=k, v=k, kv_lens=ln, out=out), **bad})
    q1, kp = q[:, :1].contiguous(), torch.zeros(7, 2, 64, dtype=BF16)
    good = dict(q=q1, k_prefix=kp, v_prefix=kp, prefix_len=ln[:1], k_cache=k, v_cache=k, seqlens=ln,
                out=torch.empty_like(q1))
    for bad in (dict(k_prefix=kp[None], v_prefix=kp[None]), dict(k_prefix=kp[:, :1], v_prefix=kp[:, :1]),
                dict(v_prefix=kp[:3]), dict(prefix_len=ln), dict(seqlens=ln[:1]), dict()):
        with pytest.raises(ValueError):
            g.gqa_prefix_attn(**{**good, **bad})


# ---------------------------------------------------------------------- plan
def _check_plan(lens, nq, Hq, Hkv, d, s_max, sm, prefix=None):
    """prefix: (length, capacity) of a shared prefix."""
    P, room = prefix or (0, 0)
    desc = _desc(batch=len(lens), q_tokens=nq, q_heads=Hq, kv_heads=Hkv, head_dim=d, max_seqlen=s_max)
    ctas, every, info, items = g.gqa_shared_keys_plan(desc, lens, P, room, sm)
    assert 1 <= ctas <= sm
    G, tiles = Hq // Hkv, 1 if d == 256 else 2
    sections = [([P], nq * len(lens), room), (lens, nq, s_max)] if prefix else [(lens, nq, s_max)]
    assert every == (bool(prefix) or nq <= 128 // G)
    by_triple, used, load = {}, set(), {}
    for cta, sec, b, h, grp, lo, hi, piece, n in items.tolist():
        tokens, groups, split, pieces = info[sec].tolist()
        assert 0 <= cta < ctas and 0 <= h < Hkv and 0 <= grp < groups
        by_triple.setdefault((sec, b, h, grp), []).append((lo, hi, piece, n, cta))
        load[cta] = load.get(cta, 0) + hi - lo
        if piece >= 0 and lo < hi:
            assert piece < pieces and (sec, piece) not in used, "two pieces share a place"
            used.add((sec, piece))
    total = 0
    for sec, (sec_lens, tokens_in, cap) in enumerate(sections):
        tokens, groups, split, _ = info[sec].tolist()
        assert tokens == min(tokens_in, 128 // G) and split == (tiles == 2 and tokens_in <= 128 // G and (d == 64 or tokens_in * G <= 64))
        assert groups == -(-tokens_in // (tokens * (1 if split else tiles)))
        total += len(sec_lens) * Hkv * groups
    assert len(by_triple) == total
    for (sec, b, h, grp), its in by_triple.items():
        sec_lens, _, cap = sections[sec]
        blocks = (min(max(sec_lens[b], 0), cap) + 127) // 128
        if blocks == 0:
            assert len(its) == 1 and its[0][0] == its[0][1] and its[0][3] == 0
            continue
        assert [x[1] for x in its[:-1]] == [x[0] for x in its[1:]] and its[0][0] == 0 and its[-1][1] == blocks
        assert all(lo < hi for lo, hi, _, _, _ in its) and its[0][3] == len(its)
        first, ctas_of = its[0][2], [x[4] for x in its]
        assert ctas_of == list(range(ctas_of[0], ctas_of[0] + len(its)))
        if every:          # consecutive places from the first
            assert [x[2] for x in its] == list(range(first, first + len(its)))
        elif len(its) == 1:
            assert first == -1
        else:              # as the merge finds them
            assert [x[2] for x in its] == [2 * ctas_of[0] + 1] + [2 * c for c in ctas_of[1:]]
    return load


@pytest.mark.parametrize("sm", [1, 7, 152])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,d,s_max", [
    ([4096] * 4, 2048, 32, 8, 128, 4096), ([1, 0, 129, 1000, 128], 77, 12, 12, 64, 1023), ([0, 0], 50, 8, 1, 64, 512),
    ([131072], 64, 64, 8, 128, 131072), ([5001, 4000], 333, 16, 2, 256, 5001), ([700], 33, 3, 1, 128, 700),
    ([-5, 9999, 300], 100, 24, 8, 128, 600), ([1], 1, 128, 1, 64, 1), ([300] * 1100, 40, 4, 4, 64, 300),
    ([300] * 4097, 40, 4, 4, 64, 300), ([300] * 4096, 20, 4, 4, 64, 300),
    ([0, 0, 5, 0, 0, 700, 0], 200, 4, 2, 128, 700), ([100, 90], 129, 2, 2, 64, 128)])
def test_plan_covers_every_block_once(lens, nq, Hq, Hkv, d, s_max, sm):
    load = _check_plan(lens, nq, Hq, Hkv, d, s_max, sm)
    if len(lens) <= 1024 and min(lens) == max(lens) > 0 and sum(load.values()) >= 4 * sm:
        assert max(load.values()) - min(load.values()) <= 6   # equal ranges, but for the items' fixed cost


@pytest.mark.parametrize("lens,nq,prefix", [([0] * 256, 1, (32768, 32768)), ([300] * 128 + [0] * 384, 1, (0, 4096)),
                                            ([0] * 512, 200, None), ([900] * 8 + [0] * 500, 200, None)])
def test_entries_without_keys_are_spread(lens, nq, prefix):
    """A padded batch's empty entries are dealt over the CTAs, not left to one of them."""
    desc = _desc(batch=len(lens), q_tokens=nq, q_heads=32, kv_heads=4, head_dim=128, max_seqlen=1024)
    ctas, _, _, items = g.gqa_shared_keys_plan(desc, lens, *(prefix or (0, 0)), 152)
    empty = items[items[:, 5] == items[:, 6]]
    if prefix:   # records of whole entries, in turn
        most, share = np.bincount(np.unique(empty[:, :3], axis=0)[:, 0]).max(), (len(lens) + 1) / ctas
    else:        # of the plan's line, on which a triple takes 6 units, with keys 16 and 7 a block
        most = np.bincount(empty[:, 0]).max()
        share = (6 * len(empty) + 16 * (len(items) - len(empty)) + 7 * (items[:, 6] - items[:, 5]).sum()) / ctas / 6
    assert most <= math.ceil(share)


@pytest.mark.parametrize("sm", [1, 7, 152])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,d,s_max,prefix", [
    ([5, 700, 0, 128], 1, 8, 2, 128, 700, (1000, 1024)), ([300] * 128, 1, 64, 8, 128, 2048, (32768, 32768)),
    ([0] * 40, 2, 8, 1, 64, 10, (0, 5)), ([40] * 40, 2, 8, 1, 64, 50, (0, 5)), ([7] * 24, 1, 16, 2, 256, 300, (20000, 20480)),
    ([9] * 1100, 4, 32, 4, 64, 9, (130, 130)), ([9] * 4096, 4, 32, 4, 64, 9, (130, 130)),
    ([0] * 900 + [300] * 20, 1, 8, 2, 64, 300, (999, 999)), ([7] * 9 + [0] * 900 + [300] * 20, 1, 8, 2, 64, 300, (0, 9)), ([0, 3], 8, 8, 2, 64, 9, (999, 500))])
def test_plan_with_a_prefix(lens, nq, Hq, Hkv, d, s_max, prefix, sm):
    _check_plan(lens, nq, Hq, Hkv, d, s_max, sm, prefix)


# --------------------------------------------------------- the definition, fp64
def _attend(q, k, v, sees, scale, dtype, out_dtype):
    """q [T, H, d], k / v [N, K, d] (doubles), sees [T, N]: O, lse and the bounds of their errors."""
    T, H, d = q.shape
    N, K = k.shape[:2]
    k, v = k.repeat_interleave(H // K, 1), v.repeat_interleave(H // K, 1)
    s = torch.einsum("thd,jhd->thj", q, k) * scale
    size = torch.einsum("thd,jhd->thj", q.abs(), k.abs()) * scale
    s = s.masked_fill(~sees[:, None, :], -math.inf)
    lse = torch.logsumexp(s, -1) if N else torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    out = torch.einsum("thj,jhd->thd", w, v)
    A = torch.einsum("thj,jhd->thd", w, v.abs())
    if N == 0:
        return out, lse, torch.zeros_like(out), torch.zeros_like(lse)
    s0 = torch.where(s == -math.inf, 0.0, s)
    ds = (d * 2.0 ** -23 * size + 2.0 ** -22 * s0.abs()).masked_fill(~sees[:, None, :], 0.0).amax(-1)
    sums = (N + 64) * 2.0 ** -23
    tol = A * (torch.finfo(dtype).eps / 2 + 2 * ds[..., None] + 2.0 ** -20 + sums)
    if dtype == FP16:
        tol = tol + 2.0 ** -25 * N * v.abs().amax()
    tol = tol + out.abs() * torch.finfo(out_dtype).eps / 2 + 2.0 ** -25   # (fp16 outputs: subnormals)
    tol_lse = ds + 2.0 ** -20 + sums + torch.where(lse == -math.inf, 0.0, lse).abs() * 2.0 ** -22
    return out, lse, tol, tol_lse


def _compare(what, out, lse, want):
    for b, (o, l, to, tl) in enumerate(want):
        got = out[b].double()
        assert torch.isfinite(got).all(), (what, b)
        bad = ((got - o).abs() - to)
        assert bad.max() <= 0, (what, b, "O", bad.max().item(), (got - o).abs().max().item(), to.max().item())
        if lse is None:
            continue
        gl = lse[b].double()
        assert torch.equal(torch.isneginf(gl), torch.isneginf(l)), (what, b, "empty rows")
        e = torch.where(torch.isneginf(l), 0.0, (gl - l).abs())
        assert (e - tl).max() <= 0, (what, b, "lse", e.max().item(), tl.max().item())


def _rand(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _cross_case(dev, B, T, H, K, d, S, lens, dtype=BF16, out_dtype=None, scale=0.0, std=1.0, seed=0, poison=None):
    gen = torch.Generator(dev).manual_seed(seed)
    q, k, v = (_rand(gen, *sh, dtype=dtype, std=std) for sh in ((B, T, H, d), (B, S, K, d), (B, S, K, d)))
    v = v / std
    v = v.to(dtype)
    for b, L in enumerate(lens):
        bad = torch.tensor([math.nan, math.inf, -math.inf], device=dev, dtype=dtype) if poison is None else poison
        n = S - max(min(L, S), 0)
        if n:
            fill = bad[torch.arange(n, device=dev) % len(bad)][:, None, None]
            k[b, S - n:], v[b, S - n:] = fill, fill
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    return q, k, v, ln


def _cross_want(q, k, v, lens, out_dtype, scale=0.0):
    B, T, H, d = q.shape
    S = k.shape[1]
    want = []
    for b, L in enumerate(lens):
        L = max(0, min(L, S))
        sees = torch.ones(T, L, dtype=torch.bool, device=q.device)
        want.append(_attend(q[b].double(), k[b, :L].double(), v[b, :L].double(), sees, scale or d ** -0.5, q.dtype,
                            out_dtype))
    return want


def _run_cross(q, k, v, ln, out_dtype=None, scale=0.0, **kw):
    out, lse = g.cross_attention(q, k, v, ln, out_dtype=out_dtype, scale=scale, **kw)
    torch.cuda.synchronize()
    return out, lse


CROSS = [  # B, T, H, K, d, S, lens, dtype, out dtype
    (1, 33, 1, 1, 64, 1, [1], BF16, None),                       # just past the decode kernel, one key
    (1, 127, 1, 1, 128, 127, [127], FP16, None),
    (1, 128, 1, 1, 256, 128, [128], BF16, FP32),
    (1, 129, 1, 1, 64, 129, [129], BF16, FP32),
    (2, 256, 1, 1, 128, 256, [256, 255], BF16, None),
    (2, 257, 1, 1, 128, 300, [257, 0], FP16, FP32),
    (3, 77, 12, 12, 64, 1023, [1023, 0, 1], FP16, None),
    (3, 43, 24, 8, 128, 513, [513, 384, 385], BF16, None),       # G = 3: 42 tokens of 126 rows a tile
    (2, 52, 10, 2, 256, 641, [641, 130], FP16, None),            # G = 5
    (4, 100, 28, 4, 128, 900, [900, 2, 640, 127], BF16, None),   # G = 7
    (1, 3, 128, 1, 64, 700, [650], BF16, None),                  # G = 128: a token a tile
    (2, 3, 100, 1, 128, 700, [650, 700], FP16, None),            # G = 100
    (2, 333, 16, 2, 256, 5001, [5001, 4000], BF16, None),        # many pieces, one tile and two S slots
    (2, 600, 8, 2, 64, 3000, [3000, 1111], BF16, FP32),
    (1, 64, 8, 1, 128, 40000, [40000], FP16, None),              # one triple over many CTAs
    (5, 40, 4, 4, 128, 260, [0, 0, 0, 0, 0], BF16, None),        # nothing to see at all
    (5, 150, 4, 4, 64, 260, [0, 0, 0, 0, 0], BF16, None),
    (1, 40, 2, 2, 128, 128, [77], BF16, None),                   # one block for the two tiles
    (3, 200, 6, 2, 128, 2000, [2000, 129, 0], BF16, None),       # cut triples of both tiles, and a half-empty last
    (40, 40, 4, 1, 64, 200, [(i * 13) % 201 for i in range(40)], BF16, None),
    (2, 32, 32, 8, 128, 1300, [1300, 257], BF16, None),          # one full tile: its keys are not split
    (3, 16, 32, 8, 128, 1300, [1300, 0, 129], FP16, FP32),       # half a tile: they are
    (300, 40, 4, 1, 64, 300, [0] * 200 + [300] * 100, BF16, None),   # a padded batch: cut triples after empty ones
    (300, 12, 16, 2, 128, 300, [300, 0, 0] * 100, FP16, None),       # and one whose triples all leave partials
]


@gpu
@pytest.mark.parametrize("B,T,H,K,d,S,lens,dtype,out_dtype", CROSS)
def test_cross_matches_the_definition(dev, B, T, H, K, d, S, lens, dtype, out_dtype):
    q, k, v, ln = _cross_case(dev, B, T, H, K, d, S, lens, dtype)
    out, lse = _run_cross(q, k, v, ln, out_dtype)
    _compare("cross", out, lse, _cross_want(q, k, v, lens, out.dtype))
    again = _run_cross(q, k, v, ln, out_dtype)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("order", ["rising", "falling", "huge"])
def test_cross_running_max(dev, d, order):
    """Scores that grow from block to block (every block rescales O), that
    shrink (none does), and that spread over +-60 (few keys take all)."""
    q, k, v, ln = _cross_case(dev, 1, 300, 2, 1, d, 1500, [1500], std=4.0 if order == "huge" else 1.0, seed=d)
    if order != "huge":
        ramp = torch.linspace(0.1, 6.0, 1500, device=dev)
        ramp = ramp if order == "rising" else ramp.flip(0)
        k = (k.float() * ramp[None, :, None, None]).to(BF16)
    out, lse = _run_cross(q, k, v, ln)
    _compare(order, out, lse, _cross_want(q, k, v, [1500], BF16))


@gpu
def test_cross_scale_and_optional_lse(dev):
    q, k, v, ln = _cross_case(dev, 2, 90, 8, 2, 128, 500, [500, 77], seed=3)
    out, lse = _run_cross(q, k, v, ln, FP32, scale=0.3)
    _compare("scale", out, lse, _cross_want(q, k, v, [500, 77], FP32, 0.3))
    ws = torch.empty(g.gqa_cross_workspace_size(q, k, out_dtype=FP32), dtype=torch.uint8, device=dev)
    alone = torch.empty_like(out)
    g.gqa_cross_attn(q, k, v, ln, alone, None, ws, scale=0.3)
    assert torch.equal(alone, out)


@gpu
@pytest.mark.parametrize("T", [1, 8, 100])
def test_cross_writes_its_rows_and_no_others(dev, T):
    """Output 16 bytes into a buffer (so not 32-byte aligned), lse 4 bytes into one: all else stays."""
    q, k, v, ln = _cross_case(dev, 2, T, 8, 2, 64, 300, [300, 200], seed=4)
    want, want_lse = _run_cross(q, k, v, ln)
    n = q.numel()
    buf = torch.full((n + 64,), 7.0, dtype=BF16, device=dev)
    lbuf = torch.full((2 * T * 8 + 8,), 7.0, device=dev)
    out, lse = buf[8: 8 + n].view(q.shape), lbuf[1: 1 + 2 * T * 8].view(2, T, 8)
    ws_n = g.gqa_cross_workspace_size(q, k)
    ws = torch.full((ws_n + 256,), 0xAB, dtype=torch.uint8, device=dev)
    g.gqa_cross_attn(q, k, v, ln, out, lse, ws[:ws_n] if ws_n else None)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all() and lbuf[0] == 7 and (lbuf[1 + 2 * T * 8:] == 7).all()
    assert (ws[ws_n:] == 0xAB).all()


@gpu
def test_cross_refuses_a_small_workspace(dev):
    q, k, v, ln = _cross_case(dev, 2, 100, 8, 2, 64, 300, [300, 200])
    need = g.gqa_cross_workspace_size(q, k)
    out = torch.full_like(q, 7.0)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device=dev),
               torch.empty(need + 256, dtype=torch.uint8, device=dev)[16:]):
        with pytest.raises(g.GQAError) as e:
            g.gqa_cross_attn(q, k, v, ln, out, None, ws)
        assert e.value.status == g.GQA_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert (out == 7).all()


@gpu
def test_few_rows_are_a_decode_call(dev):
    q, k, v, ln = _cross_case(dev, 3, 4, 16, 2, 128, 900, [900, 0, 333], seed=5)
    out, lse = _run_cross(q, k, v, ln)
    want = g.decode(q, k, v, ln)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    _compare("few", out, lse, _cross_want(q, k, v, [900, 0, 333], BF16))


@gpu
def test_bad_lengths_are_clamped_and_flagged(dev):
    for B, T in ((2, 50), (2, 200), (1100, 40)):    # lengths staged, and read per item
        lens = [200] * (B - 2) + [-3, 999]
        q, k, v, ln = _cross_case(dev, B, T, 2, 1, 64, 200, lens, seed=6)
        out, lse = _run_cross(q, k, v, ln)
        assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN
        assert g.gqa_decode_get_error() == g.GQA_OK
        _compare("clamped", out[-2:], lse[-2:], _cross_want(q[-2:], k[-2:], v[-2:], lens[-2:], BF16))


@gpu
def test_more_entries_than_lengths_are_staged(dev):
    for T in (40, 150):
        lens = [(i * 29) % 321 for i in range(1030)]
        q, k, v, ln = _cross_case(dev, 1030, T, 2, 2, 64, 320, lens, seed=7)
        out, lse = _run_cross(q, k, v, ln)
        _compare("batch 1030", out, lse, _cross_want(q, k, v, lens, BF16))
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("T", [40, 150])
def test_a_batch_dealt_whole(dev, T):
    """More entries than the kernel stages: triples go to the CTAs whole, in turn."""
    lens = [(i * 29) % 162 - 1 for i in range(4100)]
    q, k, v, ln = _cross_case(dev, 4100, T, 2, 2, 64, 160, lens, seed=18)
    out, lse = _run_cross(q, k, v, ln)
    _compare("batch 4100", out, lse, _cross_want(q, k, v, lens, BF16))
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN


@gpu
def test_cross_offsets_past_32_bits(dev):
    """K and V of 2.1e9 elements each: only the last batch entry's last head holds anything but zeros."""
    B, S, K, d, T = 2, 8200, 1024, 128, 40
    k = torch.zeros(B, S, K, d, dtype=BF16, device=dev)
    v = torch.zeros(B, S, K, d, dtype=BF16, device=dev)
    gen = torch.Generator(dev).manual_seed(8)
    k[-1, :, -1], v[-1, :, -1] = _rand(gen, S, d), _rand(gen, S, d)
    q = _rand(gen, B, T, K, d)
    ln = torch.tensor([S, S - 5], dtype=torch.int32, device=dev)
    out, lse = _run_cross(q, k, v, ln)
    want = _attend(q[-1, :, -1:].double(), k[-1, : S - 5, -1:].double(), v[-1, : S - 5, -1:].double(),
                   torch.ones(T, S - 5, dtype=torch.bool, device=dev), d ** -0.5, BF16, BF16)
    _compare("far", out[-1:, :, -1:], lse[-1:, :, -1:], [want])
    assert (out[0] == 0).all() and (out[-1, :, :-1] == 0).all()
    assert (lse[0] - math.log(S)).abs().max() < 1e-4


# ------------------------------------------------------------------- prefix
def _prefix_case(dev, B, T, H, K, d, P, room, S, lens, dtype=BF16, seed=0):
    q, k, v, ln = _cross_case(dev, B, T, H, K, d, S, lens, dtype, seed=seed)
    gen = torch.Generator(dev).manual_seed(seed + 1000)
    kp, vp = _rand(gen, room, K, d, dtype=dtype), _rand(gen, room, K, d, dtype=dtype)
    kp[P:], vp[P:] = math.nan, math.inf
    return q, kp, vp, torch.tensor([P], dtype=torch.int32, device=dev), k, v, ln


def _prefix_want(case, P, lens, out_dtype, causal=False, scale=0.0):
    q, kp, vp, _, k, v, _ = case
    T, d = q.shape[1], q.shape[3]
    want = []
    for b, L in enumerate(lens):
        keys, values = torch.cat([kp[:P], k[b, :L]]).double(), torch.cat([vp[:P], v[b, :L]]).double()
        sees = torch.ones(T, P + L, dtype=torch.bool, device=q.device)
        if causal:
            at = torch.arange(L, device=q.device)
            sees[:, P:] = at[None, :] <= (L - T + torch.arange(T, device=q.device))[:, None]
        want.append(_attend(q[b].double(), keys, values, sees, scale or d ** -0.5, q.dtype, out_dtype))
    return want


PREFIX = [  # B, T, H, K, d, P, room, S, lens, dtype, out dtype, causal
    (1, 1, 8, 1, 64, 1, 1, 1, [1], BF16, None, False),
    (4, 1, 8, 1, 64, 500, 512, 64, [1, 64, 0, 33], BF16, None, False),         # few rows: 32
    (5, 1, 8, 1, 64, 500, 512, 64, [1, 64, 0, 33, 5], FP16, FP32, False),      # 40: a tile
    (32, 1, 32, 8, 128, 4000, 4096, 512, [(i * 37) % 513 for i in range(32)], BF16, None, False),
    (16, 4, 16, 2, 64, 1000, 1000, 512, [(i * 37) % 500 + 4 for i in range(16)], FP16, None, True),
    (16, 4, 16, 2, 64, 129, 200, 512, [i % 6 for i in range(16)], BF16, None, True),   # own keys fewer than tokens
    (24, 1, 16, 2, 256, 2000, 2048, 300, [(i * 37) % 300 for i in range(24)], BF16, None, False),
    (9, 2, 10, 2, 256, 700, 700, 130, [130, 0, 2, 129, 128, 1, 7, 99, 64], FP16, FP32, True),
    (24, 1, 16, 2, 128, 0, 2048, 300, [(i * 37) % 300 for i in range(24)], BF16, None, False),  # no prefix
    (24, 1, 16, 2, 128, 0, 64, 300, [0] * 24, BF16, None, False),               # no keys at all
    (24, 1, 16, 2, 64, 777, 800, 300, [0] * 24, BF16, None, False),             # nothing but the prefix
    (3, 1, 8, 1, 128, 0, 64, 300, [0, 5, 300], BF16, None, False),              # few rows, no prefix
    (160, 2, 24, 8, 128, 100, 100, 30, [(i * 37) % 31 for i in range(160)], BF16, None, False),
    (1100, 1, 4, 2, 64, 300, 333, 140, [(i * 7) % 141 for i in range(1100)], BF16, None, False),  # lengths not staged
    (2, 8, 16, 4, 128, 400, 400, 700, [700, 9], BF16, None, True),              # 64 rows, 32 of their own
    (40, 8, 16, 4, 128, 400, 400, 700, [(i * 17) % 701 for i in range(40)], FP16, None, True),
    (3, 1, 128, 4, 64, 260, 260, 40, [40, 1, 0], BF16, None, False),            # G = 32
    (400, 1, 16, 2, 128, 700, 800, 300, [0] * 390 + list(range(10)), FP16, None, False),   # a padded batch
    (400, 1, 8, 4, 256, 0, 800, 300, [300] + [0] * 399, BF16, None, False),
    (4100, 1, 4, 2, 64, 300, 333, 140, [(i * 7) % 141 for i in range(4100)], BF16, None, False),   # lengths not staged
]


@gpu
@pytest.mark.parametrize("B,T,H,K,d,P,room,S,lens,dtype,out_dtype,causal", PREFIX)
def test_prefix_matches_the_definition(dev, B, T, H, K, d, P, room, S, lens, dtype, out_dtype, causal):
    case = _prefix_case(dev, B, T, H, K, d, P, room, S, lens, dtype)
    out, lse = g.prefix_decode(*case, causal=causal, out_dtype=out_dtype)
    torch.cuda.synchronize()
    _compare("prefix", out, lse, _prefix_want(case, P, lens, out.dtype, causal))
    again = g.prefix_decode(*case, causal=causal, out_dtype=out_dtype)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_prefix_equals_decode_over_joined_keys(dev):
    """The two ways a user has of the same step: shared keys held once, or
    copied in front of every sequence's own."""
    lens, P = [40, 1, 300, 129, 7, 64], 1200
    case = _prefix_case(dev, 6, 2, 32, 8, 128, P, 1300, 300, lens, seed=9)
    q, kp, vp, _, k, v, ln = case
    out, lse = g.prefix_decode(*case, causal=True, out_dtype=FP32)
    joined = []
    for own, pre in ((k, kp), (v, vp)):
        j = torch.zeros(6, P + 300, 8, 128, dtype=BF16, device=dev)
        j[:, :P] = pre[:P]
        for b, L in enumerate(lens):
            j[b, P: P + L] = own[b, :L]
        joined.append(j)
    ref, ref_lse = g.decode(q, *joined, (ln + P).contiguous(), causal=True, out_dtype=FP32)
    # both within the bound of the definition, so within twice it of each other
    for b, (_, _, to, tl) in enumerate(_prefix_want(case, P, lens, FP32, True)):
        assert ((out[b] - ref[b]).abs().double() <= 2 * to).all()
        assert ((lse[b] - ref_lse[b]).abs().double() <= 2 * tl).all()


@gpu
def test_prefix_bad_length_and_workspace(dev):
    case = list(_prefix_case(dev, 20, 1, 8, 2, 64, 100, 100, 50, [50] * 20))
    want = _prefix_want(case, 100, [50] * 20, BF16)
    case[3] = torch.tensor([101], dtype=torch.int32, device=dev)
    out, lse = g.prefix_decode(*case)
    torch.cuda.synchronize()
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN
    _compare("clamped prefix", out, lse, want)
    need = g.gqa_prefix_workspace_size(case[0], case[1], case[4])
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device=dev)):
        with pytest.raises(g.GQAError) as e:
            g.gqa_prefix_attn(*case, torch.empty_like(case[0]), None, ws)
        assert e.value.status == g.GQA_ERR_WORKSPACE


# ------------------------------------------------------ together, graphs, streams
@gpu
def test_graph_replay_follows_its_inputs(dev):
    """A prompt's cross attention, a decode step's, and a step behind a
    prefix, captured together and replayed with other inputs and lengths."""
    lens = [700, 33, 500]
    q, k, v, ln = _cross_case(dev, 3, 70, 16, 4, 128, 700, lens, seed=10)
    case = list(_prefix_case(dev, 12, 1, 16, 4, 128, 900, 1024, 200, [200] * 12, seed=11))
    step_q = q[:, -1:].contiguous()
    ws = [torch.empty(n, dtype=torch.uint8, device=dev) for n in (
        g.gqa_cross_workspace_size(q, k), max(1, g.gqa_cross_workspace_size(step_q, k)),
        g.gqa_prefix_workspace_size(case[0], case[1], case[4]))]
    outs = [(torch.empty_like(x), torch.empty(x.shape[:3], device=dev)) for x in (q, step_q, case[0])]

    def all_three(stream=None):
        g.gqa_cross_attn(q, k, v, ln, *outs[0], ws[0], stream=stream)
        g.gqa_cross_attn(step_q, k, v, ln, *outs[1], ws[1], stream=stream)
        g.gqa_prefix_attn(*case, *outs[2], ws[2], stream=stream)

    all_three()
    torch.cuda.synchronize()
    first = [o[0].clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_three()
    new_q, _, _, _ = _cross_case(dev, 3, 70, 16, 4, 128, 700, lens, seed=12)
    q.copy_(new_q)
    step_q.copy_(q[:, -1:])
    new_lens, new_P, new_own = [5, 700, 0], 130, [0, 200, 1] * 4
    good_k, good_v = torch.nan_to_num(k, 0.5, 0.5, 0.5), torch.nan_to_num(v, 0.5, 0.5, 0.5)
    k.copy_(good_k)
    v.copy_(good_v)
    ln.copy_(torch.tensor(new_lens, dtype=torch.int32))
    case[3].fill_(new_P)
    case[6].copy_(torch.tensor(new_own, dtype=torch.int32))
    for _ in range(3):
        for o, l in outs:
            o.fill_(math.nan)
            l.fill_(math.nan)
        graph.replay()
    torch.cuda.synchronize()
    _compare("prompt", *outs[0], _cross_want(q, k, v, new_lens, BF16))
    _compare("step", *outs[1], _cross_want(step_q, k, v, new_lens, BF16))
    _compare("prefix", *outs[2], _prefix_want(case, new_P, new_own, BF16))
    assert not torch.equal(first[0], outs[0][0])
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_two_streams_at_once(dev):
    """Calls on two streams, a workspace each, interleaved: the results of the same calls one by one."""
    a = _cross_case(dev, 2, 400, 8, 2, 128, 3000, [3000, 1700], seed=13)
    b = _prefix_case(dev, 48, 1, 16, 2, 64, 3000, 3000, 400, [(i * 31) % 400 for i in range(48)], seed=14)
    want_a, want_b = _run_cross(*a), g.prefix_decode(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((g.cross_attention(*a, stream=s1), g.prefix_decode(*b, stream=s2.cuda_stream)))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert torch.equal(ga[0], want_a[0]) and torch.equal(ga[1], want_a[1])
        assert torch.equal(gb[0], want_b[0]) and torch.equal(gb[1], want_b[1])
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_calls_in_a_row_share_a_workspace(dev):
    """Different calls back to back on one stream, eagerly and as a graph, in
    one workspace that holds NaNs at first: the results of each alone."""
    a = _cross_case(dev, 2, 400, 8, 2, 128, 3000, [3000, 1700], seed=15)
    b = _prefix_case(dev, 48, 1, 16, 2, 64, 3000, 3000, 400, [(i * 31) % 400 for i in range(48)], seed=16)
    c = _cross_case(dev, 5, 20, 8, 2, 128, 900, [900, 0, 0, 17, 500], seed=17)
    want = [g.cross_attention(*a), g.prefix_decode(*b), g.cross_attention(*c)]
    torch.cuda.synchronize()
    need = max(g.gqa_cross_workspace_size(a[0], a[1]), g.gqa_prefix_workspace_size(b[0], b[1], b[4]),
               g.gqa_cross_workspace_size(c[0], c[1]))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    got = [[torch.empty_like(t) for t in w] for w in want]

    def all_three():
        g.gqa_cross_attn(*a, *got[0], ws)
        g.gqa_prefix_attn(*b, *got[1], ws)
        g.gqa_cross_attn(*c, *got[2], ws)

    def check():
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
            o.fill_(math.nan)
            l.fill_(math.nan)

    for _ in range(5):
        all_three()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(5):
            all_three()
    ws.fill_(255)
    graph.replay()
    check()
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_prompt_then_steps(dev):
    """A decoder's prompt in one call, and its tokens one at a time: the same rows."""
    lens = [450, 90]
    q, k, v, ln = _cross_case(dev, 2, 36, 8, 2, 64, 450, lens, seed=15)
    out, lse = _run_cross(q, k, v, ln, FP32)
    want = _cross_want(q, k, v, lens, FP32)
    for t in range(0, 36, 7):
        o, l = _run_cross(q[:, t: t + 1].contiguous(), k, v, ln, FP32)
        for b in range(2):
            assert ((o[b, 0] - out[b, t]).abs().double() <= 2 * want[b][2][t]).all()
            assert ((l[b, 0] - lse[b, t]).abs().double() <= 2 * want[b][3][t]).all()


@gpu
def test_debug_build_stays_quiet_and_agrees(dev):
    """The bounds-checked build catches no write outside a buffer and gives the same bits."""
    gbuild.build_debug()
    L = g.load_library(gbuild.DEBUG_LIB)
    assert L.gqa_decode_get_error(1) == g.GQA_OK
    stream = torch.cuda.current_stream().cuda_stream
    for B, T, H, K, d, S, lens in ((3, 43, 24, 8, 128, 513, [513, 0, 385]), (2, 90, 16, 2, 256, 1001, [1001, 700]),
                                   (2, 300, 12, 12, 64, 700, [700, 1])):
        q, k, v, ln = _cross_case(dev, B, T, H, K, d, S, lens, seed=16)
        want = _run_cross(q, k, v, ln)
        out, lse = torch.full_like(want[0], math.nan), torch.full_like(want[1], math.nan)
        ws = torch.empty(g.gqa_cross_workspace_size(q, k), dtype=torch.uint8, device=dev)
        desc = g.make_desc(q, k)
        assert L.gqa_cross_attn(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), ln.data_ptr(),
                                out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), stream) == g.GQA_OK
        torch.cuda.synchronize()
        assert L.gqa_decode_get_error(1) == g.GQA_OK
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for B, few in ((20, False), (3, True)):
        case = _prefix_case(dev, B, 1, 16, 2, 128, 700, 800, 90, [(i * 17) % 91 for i in range(B)], seed=17)
        q, kp, vp, pl, k, v, ln = case
        want = g.prefix_decode(*case)
        out, lse = torch.full_like(want[0], math.nan), torch.full_like(want[1], math.nan)
        ws = torch.empty(g.gqa_prefix_workspace_size(q, kp, k), dtype=torch.uint8, device=dev)
        desc = g.make_desc(q, k)
        assert L.gqa_prefix_attn(ctypes.byref(desc), q.data_ptr(), kp.data_ptr(), vp.data_ptr(), pl.data_ptr(), 800,
                                 k.data_ptr(), v.data_ptr(), ln.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                 ws.data_ptr(), ws.numel(), stream) == g.GQA_OK
        torch.cuda.synchronize()
        assert L.gqa_decode_get_error(1) == g.GQA_OK, few
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
