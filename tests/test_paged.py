"""Rotation, paged caches and drafted tokens (include/gqa_paged.h).

CPU: the refusals, the rotation's table and the ABI.  GPU: every element
against the definitions in fp64.

Attention's bound is that of test_shared_keys (_attend), of the same kernel.
The rotation's, for a pair (a, b) turned by an angle of cosine c and sine s and
scaled by m, y = m (a c - b s):
- the angle's fraction of a turn is cut to 2^-32 and, less its nearest quarter,
  rounded to fp32: at most 2^-26 of a half turn, so that c and s are off by
  less than pi (2^-26 + 2^-31) < 2^-24;
- sinpi and cospi are good to an ulp of a number of at most 1, 2^-24;
- m is rounded to fp32 and so is its product with each: 2^-23 together;
- two products and their difference in fp32, 2^-23 of |a| + |b| at most;
in all less than 2^-21 m (|a| + |b|); and half a step of the output's type.
"""
import ctypes
import math
import random

import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild
from tests.test_shared_keys import _attend, _compare

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
    base = dict(batch=2, q_tokens=8, q_heads=8, kv_heads=2, head_dim=128, max_seqlen=256, scale=0.0, causal=0,
                out_dtype=0, in_dtype=0, reduction=0)
    base.update(kw)
    return g.gqa_desc_t(**base)


def _pages(**kw):
    base = dict(num_pages=100, page_size=16, max_pages=16, page_stride=16 * 2 * 128, pos_stride=2 * 128,
                head_stride=128)
    base.update(kw)
    return g.gqa_pages_t(**base)


def _rope(**kw):
    return g.gqa_rotary_t(**{**dict(dim=128, interleaved=0, inverse=0, magnitude=0.0), **kw})


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _tree(desc=None, pages=None, q=ALIGNED, k=ALIGNED, v=ALIGNED, table=ALIGNED, ln=ALIGNED, news=None, tree=None,
          out=ALIGNED, lse=None, ws=None, wsb=0):
    return g.lib().gqa_tree_attn(_ref(desc or _desc()), _ref(pages or _pages()), q, k, v, table, ln, news, tree, out,
                                 lse, ws, wsb, None)


def _append(desc=None, pages=None, rope=None, turns=None, positions=None, q=ALIGNED, qs=1024, k=ALIGNED, ks=256,
            v=ALIGNED, vs=256, q_out=ALIGNED, kc=ALIGNED, vc=ALIGNED, table=ALIGNED, ln=ALIGNED, news=None):
    return g.lib().gqa_paged_append(_ref(desc or _desc()), _ref(pages or _pages()), _ref(rope), turns, positions, q,
                                    qs, k, ks, v, vs, q_out, kc, vc, table, ln, news, None)


def _keep(desc=None, pages=None, kc=ALIGNED, vc=ALIGNED, table=ALIGNED, ln=ALIGNED, news=None, path=ALIGNED, n=4,
          keep=ALIGNED, out=None):
    return g.lib().gqa_paged_keep(_ref(desc or _desc()), _ref(pages or _pages()), kc, vc, table, ln, news, path, n,
                                  keep, out, None)


def _apply(rope=None, turns=ALIGNED, positions=ALIGNED, tokens=5, heads=3, d=128, dtype=0, x=ALIGNED, xs=384,
           out=ALIGNED, outs=384):
    return g.lib().gqa_rotary_apply(_ref(rope or _rope()), turns, positions, tokens, heads, d, dtype, x, xs, out,
                                    outs, None)


INVALID, UNSUPPORTED = g.GQA_ERR_INVALID_ARG, g.GQA_ERR_UNSUPPORTED
PAGED_DESC = [(dict(batch=-1), INVALID), (dict(q_tokens=0), INVALID), (dict(kv_heads=0), INVALID),
              (dict(max_seqlen=0), INVALID), (dict(max_seqlen=257), INVALID), (dict(in_dtype=1), INVALID),
              (dict(head_dim=96), UNSUPPORTED), (dict(batch=1 << 20, q_tokens=1 << 12), UNSUPPORTED)]
PAGED_PAGES = [(dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=0), INVALID),
               (dict(page_size=8, max_pages=99), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
               (dict(page_size=1 << 17), UNSUPPORTED), (dict(page_stride=0), INVALID), (dict(pos_stride=-256), INVALID),
               (dict(head_stride=132), INVALID), (dict(head_stride=64), INVALID), (dict(pos_stride=260), INVALID),
               (dict(page_stride=1 << 39), UNSUPPORTED)]


@pytest.mark.parametrize("kw,expect", PAGED_DESC)
def test_descriptions_are_checked(kw, expect):
    assert _append(_desc(**kw)) == expect
    assert _keep(_desc(**kw)) == expect
    assert _tree(_desc(**kw)) == expect
    assert g.lib().gqa_tree_workspace_size(_ref(_desc(**kw)), _ref(_pages())) == 0


@pytest.mark.parametrize("kw,expect", PAGED_PAGES)
def test_geometries_are_checked(kw, expect):
    assert _append(pages=_pages(**kw)) == expect
    assert _keep(pages=_pages(**kw)) == expect
    assert _tree(pages=_pages(**kw)) == expect
    assert g.lib().gqa_tree_workspace_size(_ref(_desc()), _ref(_pages(**kw))) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(q_heads=7), INVALID), (dict(q_heads=258), UNSUPPORTED), (dict(q_tokens=257), UNSUPPORTED),
    (dict(out_dtype=2), UNSUPPORTED), (dict(out_dtype=9), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(reduction=1), UNSUPPORTED), (dict(reduction=9), INVALID),
    (dict(batch=1 << 22, q_tokens=256, q_heads=256), UNSUPPORTED)])
def test_tree_refuses(kw, expect):
    assert _tree(_desc(**kw)) == expect
    assert g.lib().gqa_tree_workspace_size(_ref(_desc(**kw)), _ref(_pages())) == 0


def test_pointers():
    off = dict(kc=ALIGNED + 8, vc=ALIGNED + 8, table=ALIGNED + 2, ln=ALIGNED + 1, news=ALIGNED + 2)
    none = dict(kc=None, vc=None, table=None, ln=None)
    for name, at in [*off.items(), *none.items()]:
        t = {"kc": "k", "vc": "v"}.get(name, name)
        assert _tree(**{t: at}) == INVALID, name
        assert _append(**{name: at}) == INVALID, name
        assert _keep(**{name: at}) == INVALID, name
    for kw in (dict(q=None), dict(out=None), dict(q=ALIGNED + 8), dict(out=ALIGNED + 8), dict(lse=ALIGNED + 2),
               dict(tree=ALIGNED + 2)):
        assert _tree(**kw) == INVALID, kw
    assert _tree(_desc(causal=1), tree=ALIGNED) == INVALID            # a tree, or a chain
    for kw in (dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(q=ALIGNED + 8), dict(k=ALIGNED + 2),
               dict(q_out=ALIGNED + 4), dict(positions=ALIGNED + 2), dict(rope=_rope()), dict(turns=ALIGNED),
               dict(rope=_rope(), turns=ALIGNED + 4), dict(rope=_rope(inverse=1), turns=ALIGNED),
               dict(rope=_rope(dim=130), turns=ALIGNED), dict(rope=_rope(dim=7), turns=ALIGNED),
               dict(rope=_rope(magnitude=-1.0), turns=ALIGNED), dict(qs=1016), dict(ks=248), dict(vs=260),
               dict(qs=2048)):                                         # q_out is q, which is not dense
        assert _append(**kw) == INVALID, kw
    assert _append(ks=1 << 61) == UNSUPPORTED
    for kw in (dict(path=None), dict(keep=None), dict(path=ALIGNED + 2), dict(keep=ALIGNED + 2), dict(n=0),
               dict(out=ALIGNED + 2)):
        assert _keep(**kw) == INVALID, kw
    L, empty = g.lib(), _desc(batch=0)
    assert _tree(empty, q=None, k=None, v=None, table=None, ln=None, out=None) == g.GQA_OK
    assert _append(empty, q=None, q_out=None, k=None, v=None, kc=None, vc=None, table=None, ln=None) == g.GQA_OK
    assert _keep(empty, kc=None, vc=None, table=None, ln=None, path=None, keep=None) == g.GQA_OK
    assert L.gqa_tree_attn(None, _ref(_pages()), *[ALIGNED] * 5, None, None, ALIGNED, None, None, 0, None) == INVALID
    assert L.gqa_tree_workspace_size(None, None) == 0


def test_rotary_apply_refuses():
    for kw in (dict(rope=_rope(dim=0)), dict(rope=_rope(dim=3)), dict(rope=_rope(dim=130)), dict(tokens=-1),
               dict(rope=_rope(magnitude=float("nan"))), dict(rope=_rope(magnitude=float("inf"))), dict(heads=0),
               dict(dtype=5), dict(xs=380), dict(outs=376), dict(x=None), dict(out=None), dict(turns=None),
               dict(positions=None), dict(x=ALIGNED + 8), dict(out=ALIGNED + 4), dict(turns=ALIGNED + 4),
               dict(positions=ALIGNED + 2), dict(xs=392)):              # in place with two strides
        assert _apply(**kw) == INVALID, kw
    assert _apply(d=96) == UNSUPPORTED and _apply(tokens=1 << 31) == UNSUPPORTED
    assert _apply(xs=1 << 61, outs=1 << 61) == UNSUPPORTED
    assert _apply(tokens=0, x=None, out=None, turns=None, positions=None) == g.GQA_OK


def test_tree_from_parents_refuses():
    f, A = g.lib().gqa_tree_from_parents, ALIGNED
    for args in ((-1, 8, 9, A, A, None, A, A), (2, 0, 9, A, A, None, A, A), (2, 8, 0, A, A, None, A, A),
                 (2, 8, 9, None, A, None, A, A), (2, 8, 9, A, None, None, A, A), (2, 8, 9, A, A, None, None, A),
                 (2, 8, 9, A, A, A + 2, A, A), (2, 8, 9, A, A, None, A + 2, A), (2, 8, 9, A, A, None, A, A + 1)):
        assert f(*args, None) == INVALID, args
    assert f(2, 257, 9, A, A, None, A, A, None) == UNSUPPORTED
    assert f(0, 8, 9, None, None, None, None, None, None) == g.GQA_OK


def test_header_is_plain_c_and_exported(tmp_path):
    import os
    import shutil
    import subprocess

    names = g.header_functions(gbuild.PAGED_HEADER)
    assert names == ["gqa_paged_append", "gqa_paged_keep", "gqa_rotary_apply", "gqa_rotary_turns",
                     "gqa_tree_attn", "gqa_tree_from_parents", "gqa_tree_workspace_size"]
    for n in names:
        assert hasattr(g.lib(), n)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "gqa_paged.h"\nint main(void) {\n  gqa_desc_t d = {0};\n  gqa_pages_t p = {0};\n'
                   "  gqa_rotary_t r = {0};\n  uint64_t t[2];\n"
                   "  (void)gqa_rotary_turns(4, 10000.0, GQA_ROTARY_NONE, 1.0, 0, 1.0, 32.0, t);\n"
                   "  (void)gqa_rotary_apply(&r, 0, 0, 0, 1, 64, 0, 0, 64, 0, 64, 0);\n"
                   "  (void)gqa_paged_append(&d, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0);\n"
                   "  (void)gqa_tree_from_parents(0, 1, 1, 0, 0, 0, 0, 0, 0);\n"
                   "  (void)gqa_tree_attn(&d, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, gqa_tree_workspace_size(&d, &p), 0);\n"
                   "  return (int)gqa_paged_keep(&d, &p, 0, 0, 0, 0, 0, 0, 1, 0, 0, 0) == GQA_OK;\n}\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(gbuild.ROOT, "include"), str(src), gbuild.LIB, "-o", str(tmp_path / "use")],
                   check=True)


def test_status_of_an_index_out_of_range():
    assert g.GQA_ERR_BAD_INDEX == 8
    assert "out of range" in g.gqa_status_string(g.GQA_ERR_BAD_INDEX)
    assert g.gqa_status_string(g.GQA_ERR_BAD_INDEX) != g.gqa_status_string(g.GQA_ERR_BAD_SEQLEN)


def test_python_checks_tensors():
    """Refused before anything reaches the library (these are CPU tensors, the last of whose faults that is)."""
    k = torch.zeros(2, 5, 2, 64, dtype=BF16)
    q, cache = torch.zeros(2, 5, 8, 64, dtype=BF16), torch.zeros(9, 16, 2, 64, dtype=BF16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.gqa_paged_append(q, k, k, torch.empty_like(q), cache, cache, torch.zeros(2, 4, dtype=torch.int32), ints)
    with pytest.raises(ValueError):
        g.gqa_tree_attn(q, cache, cache, torch.zeros(2, 4, dtype=torch.int32), ints, torch.empty_like(q))
    with pytest.raises(ValueError):
        g.gqa_paged_keep(cache, cache, torch.zeros(2, 4, dtype=torch.int32), ints, torch.zeros(2, 5, dtype=torch.int32),
                         ints, tokens=5)
    with pytest.raises(ValueError):
        g.gqa_tree_from_parents(torch.zeros(2, 5, dtype=torch.int32), ints, torch.zeros(2, 5, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.gqa_rotary_apply(q, torch.zeros(2, 5, dtype=torch.int32), torch.zeros(32, dtype=torch.int64), q)
    with pytest.raises(ValueError):
        g.rotary_turns(64, scaling="other")


@pytest.mark.parametrize("t,stride", [
    (torch.empty(3, 5, 4, 64), 256), (torch.empty(3, 5, 12, 64)[:, :, 4:8], 768), (torch.empty(7, 4, 64), 256),
    (torch.empty(3, 5, 12, 64)[:, :1, :4], 3840), (torch.empty(1, 1, 4, 64), 256), (torch.empty(0, 5, 4, 64), 256),
    (torch.empty(3, 5, 4, 64).transpose(1, 2), None), (torch.empty(5, 3, 4, 64).transpose(0, 1), None),
    (torch.empty(3, 5, 4, 128)[..., :64], None), (torch.empty(3, 9, 4, 64)[:, :5], None)])
def test_one_stride_for_all_tokens(t, stride):
    if stride is None:
        with pytest.raises(ValueError):
            g._paged().stride_of(t)
    else:
        assert g._paged().stride_of(t) == stride


# ------------------------------------------------------- the rotation's table
def _frequencies(dim, base, scaling="none", factor=1.0, original=0, slow=1.0, fast=32.0):
    out = []
    for i in range(dim // 2):
        b = base * factor ** (dim / (dim - 2)) if scaling == "base" and dim > 2 else base
        f = b ** (-2 * i / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            w = min(1.0, max(0.0, (original * f / (2 * math.pi) - slow) / (fast - slow)))
            f = f * w + f / factor * (1 - w)
        out.append(f)
    return out


@pytest.mark.parametrize("dim,base,kw", [
    (2, 10000.0, {}), (128, 10000.0, {}), (256, 500000.0, {}), (20, 10000.0, dict(scaling="linear", factor=4.0)),
    (64, 10000.0, dict(scaling="base", factor=8.0)), (2, 10000.0, dict(scaling="base", factor=8.0)),
    (128, 500000.0, dict(scaling="parts", factor=8.0, original_length=8192)),
    (128, 10000.0, dict(scaling="parts", factor=2.0, original_length=1, slow=0.0, fast=0.5))])
def test_turns_are_the_frequencies(dim, base, kw):
    turns = g.rotary_turns(dim, base, **kw)
    kw = {"original" if k == "original_length" else k: v for k, v in kw.items()}
    want = _frequencies(dim, base, **kw)
    assert turns.dtype == torch.int64 and turns.shape == (dim // 2,)
    for t, f in zip(turns.tolist(), want):
        assert 0 < t < 2 ** 64 / 6
        # a few roundings of fp64, pow's among them, and half a step of the table, 2^-64 of a turn (which is more
        # than all of those for a slow pair: 2^-65 = 2.7e-20 against 4.8e-5 * 2^-52 = 1.1e-20)
        assert abs(t / 2 ** 64 - f / (2 * math.pi)) <= f * 2.0 ** -50 + 2.0 ** -65


@pytest.mark.parametrize("args", [
    (3, 1e4, 0, 1.0, 0, 1.0, 32.0), (0, 1e4, 0, 1.0, 0, 1.0, 32.0), (258, 1e4, 0, 1.0, 0, 1.0, 32.0),
    (64, 1.0, 0, 1.0, 0, 1.0, 32.0), (64, float("inf"), 0, 1.0, 0, 1.0, 32.0), (64, float("nan"), 0, 1.0, 0, 1.0, 2.0),
    (64, 1e4, 4, 1.0, 0, 1.0, 32.0), (64, 1e4, -1, 1.0, 0, 1.0, 32.0), (64, 1e4, 0, 2.0, 0, 1.0, 32.0),
    (64, 1e4, 1, 0.5, 0, 1.0, 32.0), (64, 1e4, 3, 2.0, 0, 1.0, 32.0), (64, 1e4, 3, 2.0, 100, 2.0, 2.0),
    (64, 1e4, 3, 2.0, 100, -1.0, 2.0), (64, 1e4, 3, 2.0, 100, 1.0, float("inf")), (4, 1e300, 2, 1e100, 0, 1.0, 2.0)])
def test_turns_refuse(args):
    assert g.lib().gqa_rotary_turns(*args, ALIGNED) == INVALID


# ----------------------------------------------------------------- rotation
def _turned(x, positions, turns, interleaved=False, inverse=False, magnitude=1.0):
    """x [..., heads, d] in fp64, rotated to positions [...], and the bound of the
    kernel's error.  The angles' whole turns are taken off in integers."""
    table, dim = turns.tolist(), 2 * turns.numel()
    angle = torch.tensor([[(p * t + 2 ** 63) % 2 ** 64 - 2 ** 63 for t in table] for p in positions.flatten().tolist()],
                         dtype=torch.int64).view(*positions.shape, 1, dim // 2).to(x.device)
    angle = angle.double() * (2 * math.pi / 2 ** 64) * (-1 if inverse else 1)
    c, s = angle.cos(), angle.sin()
    i = torch.arange(dim // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    a, b = x.double()[..., lo], x.double()[..., hi]
    y[..., lo], y[..., hi] = magnitude * (a * c - b * s), magnitude * (a * s + b * c)
    tol[..., lo] = tol[..., hi] = magnitude * (a.abs() + b.abs()) * 2.0 ** -21
    # half a step, of fp16 at least its smallest one's
    tol[..., :dim] += y[..., :dim].abs() * torch.finfo(x.dtype).eps / 2 + (2.0 ** -25 if x.dtype == FP16 else 0)
    return y, tol


def _randn(dev, *shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator(dev).manual_seed(seed), device=dev).to(dtype)


def _ints(dev, values):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _check_turned(got, want):
    y, tol = want
    err = (got.double() - y).abs() - tol
    assert err.max() <= 0, (err.max().item(), tol.max().item())


ROTARY = [  # tokens, heads, d, dim, interleaved, dtype, scaling
    (1, 1, 64, 64, False, BF16, {}), (1, 1, 64, 2, True, BF16, {}), (8, 32, 128, 128, False, BF16, {}),
    (5, 3, 256, 256, True, FP16, {}), (7, 12, 64, 20, False, FP16, dict(scaling="linear", factor=4.0)),
    (7, 12, 64, 20, True, FP32, dict(scaling="linear", factor=4.0)), (3, 5, 128, 2, False, FP32, {}),
    (300, 7, 128, 64, False, FP32, dict(scaling="parts", factor=8.0, original_length=4096)),
    (300, 7, 128, 64, True, BF16, dict(scaling="base", factor=4.0)), (2, 65, 256, 254, False, BF16, {}),
    (2, 65, 256, 254, True, BF16, {}), (6000, 2, 64, 48, False, FP16, {})]


@gpu
@pytest.mark.parametrize("T,H,d,dim,interleaved,dtype,kw", ROTARY)
@pytest.mark.parametrize("far", [0, 10 ** 6, 2 ** 31 - 7000, -10 ** 6])
def test_rotary_matches_the_definition(dev, T, H, d, dim, interleaved, dtype, kw, far):
    x = _randn(dev, T, H, d, dtype=dtype, seed=T)
    positions = (torch.arange(T, device=dev) + far).to(torch.int32)
    turns = g.rotary_turns(dim, 10000.0, device=dev, **kw)
    for inverse in (False, True):
        got = g.rotary(x, positions, turns, interleaved=interleaved, inverse=inverse, magnitude=1.25)
        _check_turned(got, _turned(x, positions, turns, interleaved, inverse, 1.25))
        assert torch.equal(got[..., dim:], x[..., dim:])
    same = x.clone()
    g.gqa_rotary_apply(same, positions, turns, same, interleaved=interleaved, inverse=True, magnitude=1.25)
    assert torch.equal(same, got)                                     # in place


@gpu
@pytest.mark.parametrize("T,H,d,dim,interleaved,dtype", [
    (2700, 1, 64, 64, False, BF16), (2701, 3, 64, 20, False, FP16), (2702, 8, 64, 18, True, BF16), (2703, 9, 64, 64, True, FP32),
    (2704, 5, 128, 24, False, FP32), (2705, 8, 128, 128, False, BF16), (2706, 3, 256, 256, False, BF16),
    (2707, 4, 256, 250, True, FP16), (2708, 1, 64, 18, False, BF16), (2709, 2, 64, 2, False, FP32)])
def test_rotary_of_many_tokens_of_few_heads(dev, T, H, d, dim, interleaved, dtype):
    """Tokens that share a CTA, the last one's not full; out of a view and into one."""
    wide = _randn(dev, T, H + 2, d, dtype=dtype, seed=T)
    into = torch.full((T, H + 1, d), 7.0, dtype=dtype, device=dev)
    x, out = wide[:, 1: H + 1], into[:, 1:]
    positions = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), device=dev, generator=torch.Generator(dev).manual_seed(T)).to(torch.int32)
    turns = g.rotary_turns(dim, 10000.0, device=dev)
    for inverse in (False, True):
        g.gqa_rotary_apply(x, positions, turns, out, interleaved=interleaved, inverse=inverse, magnitude=0.5)
        _check_turned(out, _turned(x, positions, turns, interleaved, inverse, 0.5))
        assert torch.equal(out[..., dim:], x[..., dim:]) and (into[:, 0] == 7).all()
    before = wide.clone()
    g.gqa_rotary_apply(x, positions, turns, x, interleaved=interleaved, inverse=True, magnitude=0.5)
    assert torch.equal(x, out)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, H + 1:], before[:, H + 1:])


@gpu
@pytest.mark.parametrize("dim,interleaved", [(64, False), (20, False), (20, True)])
def test_rotary_of_views_keeps_what_is_around(dev, dim, interleaved):
    """Heads out of one projection's output, into part of another tensor; elements that are not rotated pass
    through whatever they are."""
    qkv = _randn(dev, 3, 9, 10, 64, seed=1)
    qkv[1, 2, 4:7, dim:] = math.nan
    into = torch.full((3, 9, 7, 64), 7.0, dtype=BF16, device=dev)
    positions, turns = _ints(dev, [[i * 100 + j for j in range(9)] for i in range(3)]), g.rotary_turns(dim, device=dev)
    x, out = qkv[:, :, 4:7], into[:, :, 2:5]
    before = qkv.clone()
    g.gqa_rotary_apply(x, positions, turns, out, interleaved=interleaved)
    want, tol = _turned(x, positions, turns, interleaved)
    assert torch.equal(torch.isnan(out), torch.isnan(x))
    _check_turned(torch.nan_to_num(out), (torch.nan_to_num(want), torch.nan_to_num(tol)))
    assert (into[:, :, :2] == 7).all() and (into[:, :, 5:] == 7).all()
    assert torch.equal(qkv.view(torch.int16), before.view(torch.int16))
    g.gqa_rotary_apply(x, positions, turns, x, interleaved=interleaved)   # in place, in a view
    assert torch.equal(x.contiguous().view(torch.int16), out.contiguous().view(torch.int16))
    qkv[:, :, 4:7] = before[:, :, 4:7]
    assert torch.equal(qkv.view(torch.int16), before.view(torch.int16))


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_gradient(dev, interleaved):
    """Of L(x) = sum w R(x), against the formula and against differences: R is linear, so a
    difference of any size is the derivative, up to the rounding of its two sides."""
    T, H, d, dim = 5, 2, 64, 48
    x, w = _randn(dev, T, H, d, dtype=FP32, seed=2), _randn(dev, T, H, d, dtype=FP32, seed=3)
    positions, turns = _ints(dev, [0, 1, 77, 1000, 123456]), g.rotary_turns(dim, device=dev)
    kw = dict(interleaved=interleaved, magnitude=0.75)
    grad = g.rotary(w, positions, turns, inverse=True, **kw)
    _check_turned(grad, _turned(w, positions, turns, interleaved, True, 0.75))
    y = g.rotary(x, positions, turns, **kw).double()
    for e in (0, 1, 24, 25, 46, 47, 48, 63):
        moved = x.clone()
        moved[..., e] += 1.0
        step = (moved.double() - x.double())[..., e]
        slope = ((g.rotary(moved, positions, turns, **kw).double() - y) * w.double()).sum(-1) / step
        # each side of the two elements that move is off by 2^-21 (|a| + |b|) and a rounding
        size = (x.abs().amax() + 1).double() * 2 * w.abs().amax().double() * 4
        assert ((slope - grad[..., e].double()).abs() <= size * 2.0 ** -20).all(), e


# ------------------------------------------------------------- paged caches
class Case:
    """Sequences of lengths lens (with news[b] of T new tokens) in pages dealt in no order."""

    def __init__(self, dev, lens, news, T, H, K, d, page, dtype=BF16, heads_first=False, seed=0, spare=3, room=0,
                 pool=False):
        self.dev, self.lens, self.news, self.T, self.H, self.K, self.d, self.page = dev, lens, news, T, H, K, d, page
        self.dtype, B = dtype, len(lens)
        gen = torch.Generator().manual_seed(seed)
        cols = max(1, -(-max(max(lens), room) // page))
        pages = B * cols + spare
        order = torch.randperm(pages, generator=gen)[: B * cols].view(B, cols)
        used = torch.arange(cols)[None] * page < torch.tensor(lens)[:, None]
        self.table = torch.where(used, order, torch.tensor(-7)).to(torch.int32).to(dev)
        shape = (pages, 2, page, K, d) if pool else (pages, K, page, d) if heads_first else (pages, page, K, d)
        k = _randn(dev, *shape, dtype=dtype, seed=seed + 1)
        v = k if pool else _randn(dev, *shape, dtype=dtype, seed=seed + 2)
        self.k, self.v = (k[:, 0], v[:, 1]) if pool else (k.transpose(1, 2), v.transpose(1, 2)) if heads_first else (k, v)
        self.ln = _ints(dev, lens)
        self.new = None if news is None else _ints(dev, news)
        self.n = [min(T, L) for L in lens] if news is None else [min(n, L) for n, L in zip(news, lens)]
        self.q = _randn(dev, B, T, H, d, dtype=dtype, seed=seed + 3)

    def places(self, b, first, last):
        j = torch.arange(first, last, device=self.dev)
        return self.table[b].long()[j // self.page], j % self.page

    def poison(self):
        """NaN and infinities everywhere but in the sequences' positions."""
        keep = torch.zeros(self.k.shape[:2], dtype=torch.bool, device=self.dev)
        for b, L in enumerate(self.lens):
            keep[self.places(b, 0, L)] = True
        for cache in (self.k, self.v):
            cache[~keep] = torch.tensor([math.nan, math.inf], device=self.dev, dtype=self.dtype).repeat(self.d // 2)

    def want(self, sees=None, out_dtype=None, scale=0.0):
        """sees(b) -> [n_b, n_b] truth values of new tokens (None: all)."""
        result = []
        for b, L in enumerate(self.lens):
            n, at = self.n[b], self.places(b, 0, L)
            see = torch.ones(n, L, dtype=torch.bool, device=self.dev)
            if sees is not None:
                see[:, L - n:] = sees(b).to(self.dev)
            o, l, to, tl = (torch.zeros(self.T, self.H, self.d, dtype=torch.float64, device=self.dev),
                            torch.full((self.T, self.H), -math.inf, dtype=torch.float64, device=self.dev),
                            torch.zeros(self.T, self.H, self.d, dtype=torch.float64, device=self.dev),
                            torch.zeros(self.T, self.H, dtype=torch.float64, device=self.dev))
            if n:
                got = _attend(self.q[b, :n].double(), self.k[at].double(), self.v[at].double(), see,
                              scale or self.d ** -0.5, self.dtype, out_dtype or self.dtype)
                o[:n], l[:n], to[:n], tl[:n] = got
            result.append((o, l, to, tl))
        return result

    def run(self, **kw):
        out, lse = g.tree_attention(self.q, self.k, self.v, self.table, self.ln, new_lens=self.new, **kw)
        torch.cuda.synchronize()
        return out, lse


def _parents(T, seed, kind="random"):
    gen = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return [t - 1 for t in range(T)]
    if kind == "roots":
        return [-1] * T
    return [int(torch.randint(-1, t, (1,), generator=gen)) for t in range(T)]


def _branches(parents):
    T = len(parents)
    see = torch.zeros(T, T, dtype=torch.bool)
    for t, p in enumerate(parents):
        if p >= 0:
            see[t] = see[p]
        see[t, t] = True
    return see


def _words(see):
    """[..., n] truth values as int32 words."""
    n = see.shape[-1]
    see = torch.nn.functional.pad(see, (0, -n % 32)).view(*see.shape[:-1], -1, 32).long()
    return (see << torch.arange(32)).sum(-1).to(torch.int32)


@gpu
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 100, 255, 256])
@pytest.mark.parametrize("kind", ["random", "chain", "roots"])
def test_trees_from_parents(dev, T, kind):
    news = [T, max(1, T // 2), 0, T, 1]
    lens = [T + 5, 4000, 9, T, 0]                       # the last has a token, but no position for it
    parents = [_parents(T, 10 * T + b, kind) for b in range(5)]
    n = [min(a, b) for a, b in zip(news, lens)]
    W = (T + 31) // 32
    tree = torch.full((5, T, W), -1, dtype=torch.int32, device=dev)
    positions = torch.full((5, T), -1, dtype=torch.int32, device=dev)
    args = (_ints(dev, parents), _ints(dev, lens))
    g.gqa_tree_from_parents(*args, tree, positions, new_lens=_ints(dev, news))
    for b in range(5):
        see = _branches(parents[b])
        see[n[b]:] = False
        assert torch.equal(tree[b].cpu(), _words(see)), b
        depth = torch.tensor([lens[b] - n[b] + int(r.sum()) - 1 if t < n[b] else 0 for t, r in enumerate(see)])
        assert torch.equal(positions[b].cpu(), depth.to(torch.int32)), b
    again = torch.empty_like(tree)
    g.gqa_tree_from_parents(*args, again, None, new_lens=_ints(dev, news))
    assert torch.equal(again, tree)
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_bad_parents_are_roots_and_flagged(dev):
    tree, positions = torch.empty(1, 6, 1, dtype=torch.int32, device=dev), torch.empty(1, 6, dtype=torch.int32, device=dev)
    for bad in (3, 9, -2, 2 ** 31 - 1, -2 ** 31):
        g.gqa_tree_from_parents(_ints(dev, [[-1, 0, 0, bad, 3, 1]]), _ints(dev, [10]), tree, positions)
        assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
        assert tree.flatten().tolist() == [1, 3, 5, 8, 24, 35] and positions.flatten().tolist() == [4, 5, 5, 4, 5, 6]
    g.gqa_tree_from_parents(_ints(dev, [[-1, 0, 0, 9, 3, 1]]), _ints(dev, [10]), tree, positions, new_lens=_ints(dev, [3]))
    assert g.gqa_decode_get_error() == g.GQA_OK          # behind the last token nothing is read
    g.gqa_tree_from_parents(_ints(dev, [[-1, 0, 0, 1, 3, 1]]), _ints(dev, [10]), tree, positions, new_lens=_ints(dev, [7]))
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX and positions[0, 0] == 4
    g.gqa_tree_from_parents(_ints(dev, [[-1, 0, 0, 1, 3, 1]]), _ints(dev, [11]), tree, positions, max_seqlen=10)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN and positions[0, 0] == 4


APPEND = [  # lens, news, T, H, K, d, page, dtype, heads first, dim, interleaved
    ([1], None, 1, 8, 1, 64, 16, BF16, False, 64, False),
    ([17, 4000, 16, 1], None, 1, 32, 8, 128, 16, BF16, False, 128, False),
    ([200, 1023, 77], [5, 77, 77], 77, 12, 12, 64, 16, FP16, False, 20, True),
    ([200, 1023, 77], [5, 0, 77], 77, 12, 12, 64, 32, FP16, True, 20, False),
    ([3000, 500, 0, 129], [1000, 500, 0, 1], 1000, 24, 8, 128, 64, BF16, True, 64, False),
    ([700, 300], None, 40, 10, 2, 256, 256, FP16, False, 256, True),
    ([9, 3], None, 12, 4, 4, 64, 16, BF16, False, 0, False),          # more tokens than positions, nothing rotated
    ([70000], [4], 4, 3, 3, 128, 65536, BF16, False, 96, False),
    ([2000, 0, 900, 1300], [900, 0, 1, 877], 900, 8, 1, 64, 16, BF16, False, 64, False),   # many tokens of few heads, some dead
    ([1500, 1300], None, 1300, 2, 1, 128, 32, FP16, True, 50, True),
    ([1299, 1300, 5], None, 1300, 1, 1, 64, 16, BF16, False, 0, False),
    ([1299, 1300, 5], None, 1300, 2, 2, 64, 16, BF16, True, 20, False),
]


@gpu
@pytest.mark.parametrize("lens,news,T,H,K,d,page,dtype,heads_first,dim,interleaved", APPEND)
@pytest.mark.parametrize("with_q,explicit", [(True, False), (True, True), (False, False)])
def test_append_matches_the_definition(dev, lens, news, T, H, K, d, page, dtype, heads_first, dim, interleaved,
                                       with_q, explicit):
    c = Case(dev, lens, news, T, H, K, d, page, dtype, heads_first, seed=T)
    B = len(lens)
    qkv = _randn(dev, B, T, H + 2 * K, d, dtype=dtype, seed=5)
    q, k, v = qkv[:, :, :H], qkv[:, :, H: H + K], qkv[:, :, H + K:]
    turns = g.rotary_turns(dim, 10000.0, device=dev) if dim else None
    positions = _ints(dev, [[(b * 7919 + t * 31) % 100000 for t in range(T)] for b in range(B)]) if explicit else None
    q_out = torch.full((B, T, H, d), 7.0, dtype=dtype, device=dev)
    old_k, old_v = c.k.clone(), c.v.clone()
    for n in range(B):
        for t in range(c.n[n], T):
            qkv[n, t] = math.nan                                     # behind the last token
    g.gqa_paged_append(q if with_q else None, k, v, q_out if with_q else None, c.k, c.v, c.table, c.ln,
                       new_lens=c.new, positions=positions, turns=turns, interleaved=interleaved,
                       magnitude=1.5 if dim else 0.0)
    assert g.gqa_decode_get_error() == g.GQA_OK
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool, device=dev)
    for b, L in enumerate(lens):
        n = c.n[b]
        if n == 0:
            continue
        at = c.places(b, L - n, L)
        touched[at] = True
        where = positions[b, :n] if explicit else torch.arange(L - n, L, device=dev)
        assert torch.equal(c.v[at], v[b, :n])
        if dim:
            _check_turned(c.k[at], _turned(k[b, :n], where, turns, interleaved, False, 1.5))
            if with_q:
                _check_turned(q_out[b, :n], _turned(q[b, :n], where, turns, interleaved, False, 1.5))
        else:
            assert torch.equal(c.k[at], k[b, :n]) and (not with_q or torch.equal(q_out[b, :n], q[b, :n]))
        assert (q_out[b, n:] == 7).all()
    assert torch.equal(c.k[~touched], old_k[~touched]) and torch.equal(c.v[~touched], old_v[~touched])
    assert with_q or (q_out == 7).all()


@gpu
def test_append_in_place_and_into_one_pool(dev):
    """q rotated where it is; K and V pages side by side in one pool."""
    c = Case(dev, [100, 40], None, 6, 8, 2, 64, 16, pool=True, seed=3)
    pool = c.k._base
    q, k, v = c.q.clone(), _randn(dev, 2, 6, 2, 64, seed=8), _randn(dev, 2, 6, 2, 64, seed=9)
    turns, out, before = g.rotary_turns(64, device=dev), torch.empty_like(q), pool.clone()
    g.gqa_paged_append(q, k, v, out, c.k, c.v, c.table, c.ln, turns=turns)
    once = pool.clone()
    pool.copy_(before)
    g.gqa_paged_append(q, k, v, q, c.k, c.v, c.table, c.ln, turns=turns)
    assert torch.equal(q, out) and torch.equal(pool, once) and not torch.equal(before, once)
    for b, L in enumerate(c.lens):
        at = c.places(b, L - 6, L)
        assert torch.equal(c.v[at], v[b])
        _check_turned(c.k[at], _turned(k[b], torch.arange(L - 6, L, device=dev), turns))


@gpu
def test_append_to_bad_pages_and_lengths(dev):
    """A page out of range takes nothing, and is flagged; lengths are clamped."""
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Case(dev, [40, 40], None, 20, 4, 2, 64, 16, seed=4)
        good = c.table.clone()
        k = _randn(dev, 2, 20, 2, 64, seed=8)
        c.table[1, 1] = bad                                          # positions 16 to 31, of which 20 on are new
        want_k, want_v = c.k.clone(), c.v.clone()
        for b in range(2):
            for j in range(20, 40):
                if b == 0 or j >= 32:
                    want_k[good[b, j // 16].long(), j % 16] = want_v[good[b, j // 16].long(), j % 16] = k[b, j - 20]
        g.gqa_paged_append(None, k, k, None, c.k, c.v, c.table, c.ln)
        assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
        assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    # many tokens of few heads, of which those of one page are lost
    c = Case(dev, [2000, 1500], None, 1400, 4, 2, 64, 16, seed=4)
    many = _randn(dev, 2, 1400, 2, 64, seed=8)
    lost = int(c.table[0, 60])
    c.table[0, 60] = -5                                              # positions 960 to 975
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, L in enumerate(c.lens):
        there = [j for j in range(L - 1400, L) if b == 1 or not 960 <= j < 976]
        at, off = c.table[b].long()[torch.tensor(there, device=dev) // 16], torch.tensor(there, device=dev) % 16
        new = torch.tensor(there, device=dev) - (L - 1400)
        want_k[at, off] = want_v[at, off] = many[b, new]
    g.gqa_paged_append(None, many, many, None, c.k, c.v, c.table, c.ln)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v) and lost >= 0
    c = Case(dev, [48, 0], None, 20, 4, 2, 64, 16, seed=4)
    before = c.k.clone()
    g.gqa_paged_append(None, k, k, None, c.k, c.v, c.table, _ints(dev, [999, -5]))
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN
    at = c.places(0, 28, 48)
    assert torch.equal(c.k[at], k[0])
    before[at] = k[0]
    assert torch.equal(c.k, before)


TREE = [  # lens, news, T, H, K, d, page, dtype, out dtype, heads first
    ([1], None, 1, 1, 1, 64, 16, BF16, None, False),
    ([512], None, 1, 8, 1, 64, 16, BF16, None, False),
    ([4000, 0, 1, 127, 128, 129, 1000, 17], None, 1, 32, 8, 128, 16, BF16, None, False),
    ([300, 5, 64, 1023], [7, 5, 0, 3], 7, 8, 1, 64, 16, FP16, FP32, False),
    ([3000, 26, 27, 155, 700], [26, 26, 3, 27, 1], 27, 32, 8, 128, 32, BF16, None, False),    # 108 rows: one tile
    ([3000, 26, 0, 155], [16, 16, 16, 2], 16, 32, 8, 128, 64, FP16, None, True),             # 64: keys in turn
    ([2500, 400, 641], [40, 7, 33], 40, 16, 2, 256, 64, FP16, None, True),
    ([641, 130], None, 12, 10, 2, 256, 128, BF16, FP32, False),                              # G = 5
    ([4000, 65, 300], [64, 64, 10], 64, 64, 8, 128, 128, BF16, None, False),                 # two groups, one of them dead
    ([1500, 200], [100, 1], 100, 24, 8, 128, 256, BF16, None, False),                        # G = 3, pages of two blocks
    ([900, 257, 256], [256, 256, 200], 256, 4, 2, 64, 16, BF16, FP32, False),                # the most tokens
    ([700, 650], [3, 2], 3, 100, 1, 128, 1024, FP16, None, False),                           # G = 100: a token a tile
    ([300] * 40 + [0] * 60, [9] * 40 + [0] * 60, 9, 12, 12, 64, 16, BF16, None, False),      # a padded batch
    ([(i * 29) % 300 for i in range(300)], None, 30, 8, 2, 64, 16, BF16, None, False),       # fewer positions than tokens
    ([3000, 2000, 1, 700], [70, 33, 1, 0], 70, 8, 2, 64, 32, BF16, None, False),             # a group of two tiles, then one alone
    ([5000, 130], None, 50, 16, 2, 64, 16, FP16, None, False),                               # the same, cut many times
    ([(i * 97) % 700 for i in range(200)], [i % 10 for i in range(200)], 9, 32, 8, 128, 16, BF16, None, False),  # more
    ([(i * 97) % 300 for i in range(140)], None, 40, 8, 2, 128, 32, FP16, None, False),      # entries than one warp stages
    ([(i * 97) % 400 for i in range(150)], [i % 20 for i in range(150)], 19, 8, 1, 256, 16, BF16, None, False),
    ([(i * 29) % 150 for i in range(4100)], None, 20, 2, 2, 64, 16, BF16, None, False),      # more entries than are staged
    ([(i * 29) % 150 for i in range(4100)], [(i * 7) % 70 for i in range(4100)], 70, 4, 1, 64, 32, FP16, None, False),
    # enough rows of one tile for whole triples to write their own: some cut, some without keys
    ([(i * 331) % 900 for i in range(60)], [i % 13 for i in range(60)], 12, 32, 8, 128, 16, BF16, None, False),
    ([5000, 0] + [(i * 97) % 300 for i in range(60)], None, 16, 28, 4, 128, 32, FP16, FP32, True),
    ([4000] + [(i * 331) % 700 for i in range(40)], [9] + [i % 10 for i in range(40)], 9, 24, 8, 256, 64, BF16, None, False),
    ([(i * 53) % 400 for i in range(140)], [i % 21 for i in range(140)], 20, 8, 2, 128, 32, BF16, None, False),
    ([(i * 29) % 40 for i in range(4100)], None, 2, 2, 1, 256, 16, FP16, None, False),
]


@gpu
@pytest.mark.parametrize("lens,news,T,H,K,d,page,dtype,out_dtype,heads_first", TREE)
@pytest.mark.parametrize("kind", ["tree", "chain", "all"])
def test_tree_attention_matches_the_definition(dev, lens, news, T, H, K, d, page, dtype, out_dtype, heads_first, kind):
    c = Case(dev, lens, news, T, H, K, d, page, dtype, heads_first, seed=T)
    c.poison()
    branches = [_branches(_parents(T, b)) for b in range(min(len(lens), 7))]
    sees, kw = None, {}
    if kind == "tree":
        def sees(b):
            return branches[b % 7][: c.n[b], : c.n[b]]
        kw = dict(tree=_words(torch.stack([branches[b % 7] for b in range(len(lens))])).to(dev))
    elif kind == "chain":
        def sees(b):
            return torch.ones(c.n[b], c.n[b]).tril().bool()
        kw = dict(causal=True)
    for b, n in enumerate(c.n):
        c.q[b, n:] = math.nan                                        # behind the last token
    out, lse = c.run(out_dtype=out_dtype, **kw)
    _compare(kind, out, lse, c.want(sees, out_dtype))
    again = c.run(out_dtype=out_dtype, **kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("d,T", [(64, 5), (128, 30), (256, 20)])
def test_any_bits_hide_new_tokens(dev, d, T):
    """Bits that are no tree's: none set, only others', those of tokens a sequence lacks; without a position
    before the new ones such rows see nothing."""
    gen = torch.Generator().manual_seed(d)
    lens, news = [T, T, 700, 200], [T, T - 2, T, T - 1]
    see = torch.rand(4, T, T, generator=gen) < 0.3
    see[0, ::3] = False
    see[1, :, : T - 2] = False                                       # only tokens that it lacks
    see[2] = False
    c = Case(dev, lens, news, T, 8, 2, d, 16, seed=6)
    c.poison()
    out, lse = c.run(tree=_words(see).to(dev))
    _compare("bits", out, lse, c.want(lambda b: see[b, : c.n[b], : c.n[b]]))
    assert (out[0, ::3] == 0).all() and torch.isneginf(lse[0, ::3]).all()
    assert (out[1, :3] == 0).all() or c.lens[1] > c.n[1]
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 40])
def test_hidden_keys_may_be_anything(dev, d, T):
    """K of positions that a row does not see: NaN, infinities and the type's extremes."""
    c = Case(dev, [600, 170], None, T, 8, 2, d, 16, seed=7)
    see = torch.eye(T).bool()
    out, lse = c.run(tree=_words(see[None].expand(2, T, T)).to(dev))
    for b, L in enumerate(c.lens):
        want = c.want(lambda b: see)[b]
        _compare("alone", out[b: b + 1], lse[b: b + 1], [want])
    # token 0 alone sees its own key: made NaN, only its rows are
    for b, L in enumerate(c.lens):
        page, at = c.places(b, L - T, L - T + 1)
        c.k[page, at] = math.nan
    got, got_lse = c.run(tree=_words(see[None].expand(2, T, T)).to(dev))
    assert torch.isnan(got[:, 0]).all() and torch.isnan(got_lse[:, 0]).all()
    assert torch.equal(got[:, 1:], out[:, 1:]) and torch.equal(got_lse[:, 1:], lse[:, 1:])
    for value in (math.inf, -math.inf, torch.finfo(BF16).max, torch.finfo(BF16).min):
        for b, L in enumerate(c.lens):
            page, at = c.places(b, L - T, L - T + 1)
            c.k[page, at] = value
        got, got_lse = c.run(tree=_words(see[None].expand(2, T, T)).to(dev))
        assert torch.equal(got[:, 1:], out[:, 1:]) and torch.equal(got_lse[:, 1:], lse[:, 1:])


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_maxima_that_climb(dev, d):
    """Scores that grow from page to page, so that O is rescaled again and again."""
    for T in (3, 30):
        c = Case(dev, [1500, 40], None, T, 8, 2, d, 16, seed=8)
        for b, L in enumerate(c.lens):
            at = c.places(b, 0, L)
            ramp = torch.linspace(0.1, 6.0, L, device=dev)[:, None, None]
            c.k[at] = (c.k[at].float() * ramp).to(BF16)
        out, lse = c.run(causal=True, scale=0.2)
        _compare("climb", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool(), scale=0.2))


@gpu
def test_paged_equals_dense(dev):
    """A chain over pages, and the decode call over the same keys side by side: within twice the bound."""
    c = Case(dev, [700, 4, 129, 300], None, 4, 32, 8, 128, 16, seed=9)
    out, lse = c.run(causal=True, out_dtype=FP32)
    k, v = torch.zeros(4, 704, 8, 128, dtype=BF16, device=dev), torch.zeros(4, 704, 8, 128, dtype=BF16, device=dev)
    for b, L in enumerate(c.lens):
        k[b, :L], v[b, :L] = c.k[c.places(b, 0, L)], c.v[c.places(b, 0, L)]
    ref, ref_lse = g.decode(c.q, k, v, c.ln, causal=True, out_dtype=FP32)
    for b, (_, _, to, tl) in enumerate(c.want(lambda b: torch.ones(4, 4).tril().bool(), FP32)):
        assert ((out[b] - ref[b]).abs().double() <= 2 * to).all() and ((lse[b] - ref_lse[b]).abs().double() <= 2 * tl).all()


@gpu
@pytest.mark.parametrize("T", [1, 6, 40])
def test_tree_writes_its_rows_and_no_others(dev, T):
    """Output 16 bytes into a buffer, lse 4 bytes into one, a workspace of the size asked for: all else stays."""
    c = Case(dev, [300, 200, 90], None, T, 8, 2, 64, 16, seed=10)
    want, want_lse = c.run(causal=True)
    n, ws_n = c.q.numel(), g.gqa_tree_workspace_size(c.q, c.k, c.table)
    buf, lbuf = torch.full((n + 64,), 7.0, dtype=BF16, device=dev), torch.full((3 * T * 8 + 8,), 7.0, device=dev)
    out, lse = buf[8: 8 + n].view(c.q.shape), lbuf[1: 1 + 3 * T * 8].view(3, T, 8)
    ws = torch.full((ws_n + 256,), 0xAB, dtype=torch.uint8, device=dev)
    k, v, table = c.k.clone(), c.v.clone(), c.table.clone()
    g.gqa_tree_attn(c.q, c.k, c.v, c.table, c.ln, out, lse, ws[:ws_n] if ws_n else None, causal=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all() and lbuf[0] == 7 and (lbuf[1 + 3 * T * 8:] == 7).all()
    assert (ws[ws_n:] == 0xAB).all()
    assert torch.equal(k, c.k) and torch.equal(v, c.v) and torch.equal(table, c.table)
    alone = torch.empty_like(out)
    g.gqa_tree_attn(c.q, c.k, c.v, c.table, c.ln, alone, None, ws[:ws_n] if ws_n else None, causal=True)
    assert torch.equal(alone, want)
    if ws_n:
        for small in (None, ws[: ws_n - 1], ws[16:]):
            with pytest.raises(g.GQAError) as e:
                g.gqa_tree_attn(c.q, c.k, c.v, c.table, c.ln, alone, None, small, causal=True)
            assert e.value.status == g.GQA_ERR_WORKSPACE


@gpu
@pytest.mark.parametrize("T", [1, 40])
def test_bad_pages_read_as_zeros(dev, T):
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Case(dev, [300, 200], None, T, 8, 2, 64, 32, seed=11)
        page = int(c.table[1, 2])
        c.table[1, 2] = bad
        out, lse = c.run()
        assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
        c.table[1, 2] = page
        c.k[page] = c.v[page] = 0
        _compare("bad page", out, lse, c.want())


@gpu
@pytest.mark.parametrize("T", [1, 40])
def test_bad_lengths_are_clamped_and_flagged(dev, T):
    c = Case(dev, [304, 0, 90], [T] * 3, T, 8, 2, 64, 16, seed=12)
    want = c.want()
    c.ln = _ints(dev, [305, -3, 90])
    out, lse = c.run()
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_SEQLEN
    _compare("lengths", out, lse, want)
    c.ln, c.new = _ints(dev, [304, 0, 90]), _ints(dev, [T + 1, 0, -1])
    out, lse = c.run()
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    c.n = [T, 0, 0]
    _compare("tokens", out, lse, c.want())


@gpu
def test_offsets_past_32_bits(dev):
    """A pool of 2.4e9 elements: the sequence's pages are its first and its last ones."""
    pages, K, d, P = 1200, 8, 128, 2048
    k = torch.zeros(pages, P, K, d, dtype=BF16, device=dev)
    v = torch.zeros(pages, P, K, d, dtype=BF16, device=dev)
    rows = [0, pages - 1, 1, pages - 2]
    L = 4 * P - 77
    table = _ints(dev, [rows + [-1]])
    for T in (1, 30):
        c = Case(dev, [L], None, T, 32, K, d, P, seed=13)
        turns = g.rotary_turns(d, device=dev)
        new = _randn(dev, 1, T, 48, d, seed=14)
        for i, p in enumerate(rows):
            k[p], v[p] = _randn(dev, P, K, d, seed=20 + i), _randn(dev, P, K, d, seed=30 + i)
        c.k, c.v, c.table, c.ln = k, v, table, _ints(dev, [L])
        g.gqa_paged_append(new[:, :, :32], new[:, :, 32:40], new[:, :, 40:], c.q, k, v, table, c.ln, turns=turns)
        _check_turned(k[pages - 2, P - 77 - T: P - 77], _turned(new[0, :, 32:40], torch.arange(L - T, L), turns))
        out, lse = c.run(causal=True)
        _compare("far", out, lse, c.want(lambda b: torch.ones(T, T).tril().bool()))
    path, keep = _ints(dev, [[3, 7, 29]]), _ints(dev, [3])
    moved = k[pages - 2, P - 77 - 30 + torch.tensor([3, 7, 29])].clone()
    g.gqa_paged_keep(k, v, table, c.ln, path, keep, tokens=30)
    assert torch.equal(k[pages - 2, P - 77 - 30: P - 77 - 27], moved)
    assert g.gqa_decode_get_error() == g.GQA_OK


# ------------------------------------------------------------ accepted branch
@gpu
@pytest.mark.parametrize("K,d,page,dtype,heads_first", [(1, 64, 16, BF16, False), (8, 128, 16, FP16, True),
                                                        (2, 256, 64, BF16, False), (40, 128, 32, BF16, False)])
def test_keep_moves_the_branch(dev, K, d, page, dtype, heads_first):
    T = 40
    lens, news = [1000, 40, 63, 100, 17, 0, 300], [40, 40, 31, 1, 17, 5, 0]
    c = Case(dev, lens, news, T, K, K, d, page, dtype, heads_first, seed=15)
    paths = [[0, 1, 2, 5, 9, 17, 18, 19, 20, 38, 39], list(range(40)), [30], [0], [4, 5, 16], [], []]
    path = torch.full((7, T), -9, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    keep, ends = _ints(dev, [len(p) for p in paths]), torch.full((7,), -1, dtype=torch.int32, device=dev)
    want = [c.k.clone(), c.v.clone()]
    for cache in want:
        for b, p in enumerate(paths):
            if p:
                first = lens[b] - c.n[b]
                rows = cache[c.places(b, first, lens[b])][p].clone()
                cache[c.places(b, first, first + len(p))] = rows
    before = [c.k.clone(), c.v.clone()]
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, path.to(dev), keep, ends, tokens=T, new_lens=c.new)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert ends.tolist() == [L - n + len(p) for L, n, p in zip(lens, c.n, paths)]
    c.k.copy_(before[0])
    c.v.copy_(before[1])
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, path.to(dev), keep, c.ln, tokens=T, new_lens=c.new)   # lengths in place
    assert torch.equal(c.k, want[0]) and torch.equal(c.ln, ends)
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_keep_moves_long_branches(dev):
    """More tokens than a CTA has threads; one branch ends at a bad token far along, of one a page is lost."""
    T, lens = 900, [2000, 900, 1500]
    c = Case(dev, lens, None, T, 2, 2, 64, 16, seed=17)
    paths = [sorted(random.Random(b).sample(range(T), n)) for b, n in enumerate((700, 257, 513))]
    path = torch.zeros(3, 700, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    path[0, 600] = path[0, 599]                                      # not past the one before it
    paths[0] = paths[0][:600]
    c.table[2, 1400 // 16] = -3                                      # positions 1392 to 1407
    want = [c.k.clone(), c.v.clone()]
    for cache in want:
        old = cache.clone()
        for b, p in enumerate(paths):
            first = lens[b] - T
            for i, at in enumerate(p):
                if b != 2 or not (1392 <= first + at < 1408 or 1392 <= first + i < 1408):
                    cache[c.places(b, first + i, first + i + 1)] = old[c.places(b, first + at, first + at + 1)]
    ends = torch.empty(3, dtype=torch.int32, device=dev)
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, path.to(dev), _ints(dev, [700, 257, 513]), ends, tokens=T)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert ends.tolist() == [L - T + len(p) for L, p in zip(lens, paths)]


@gpu
def test_keep_ends_at_a_bad_token(dev):
    c = Case(dev, [50, 50, 50, 50, 50], [9] * 5, 9, 2, 2, 64, 16, seed=16)
    want_k = c.k.clone()
    good = [[1, 4], [], [2], [0, 1, 2], [8]]
    path = _ints(dev, [[1, 4, 4, 5], [-1, 2, 3, 4], [2, 1, 3, 4], [0, 1, 2, 9], [8, 2 ** 31 - 1, 0, 0]])
    for b, p in enumerate(good):
        rows = want_k[c.places(b, 41, 50)][p].clone()
        want_k[c.places(b, 41, 41 + len(p))] = rows
    ends = torch.empty(5, dtype=torch.int32, device=dev)
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, path, _ints(dev, [4] * 5), ends, tokens=9, new_lens=c.new)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    assert torch.equal(c.k, want_k) and ends.tolist() == [41 + len(p) for p in good]
    before = c.k.clone()
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, path, _ints(dev, [-1, 5, 0, 0, 0]), ends, tokens=9, new_lens=c.new)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    assert ends.tolist() == [41, 41, 41, 41, 41] and torch.equal(c.k, before)
    c.table[0, 3] = -1                                               # positions 48 and 49
    g.gqa_paged_keep(c.k, c.v, c.table, c.ln, _ints(dev, [[2, 8]] + [[0, 1]] * 4), _ints(dev, [2] * 5), ends, tokens=9,
                     new_lens=c.new)
    assert g.gqa_decode_get_error() == g.GQA_ERR_BAD_INDEX
    at = c.places(0, 41, 44)
    before[at[0][0], at[1][0]] = before[at[0][2], at[1][2]].clone()  # token 2 moves, token 8 has no page
    assert torch.equal(c.k, before) and ends[0] == 43


# ----------------------------------------------------- together, graphs, streams
class Step:
    """A verification step of drafts for a batch, as a serving loop makes it, and what it should leave behind."""

    def __init__(self, dev, lens, news, T, H, K, d, page, seed):
        self.c = c = Case(dev, lens, news, T, H, K, d, page, seed=seed, room=max(lens) + 2 * T)
        B = len(lens)
        free = [p for p in range(c.k.shape[0]) if p not in set(c.table.flatten().tolist())]
        for b in range(B):                                           # pages for the next step too
            for i in range(c.table.shape[1]):
                if c.table[b, i] < 0 and free:
                    c.table[b, i] = free.pop()
        self.turns = g.rotary_turns(d, 500000.0, device=dev)
        self.qkv = _randn(dev, B, T, H + 2 * K, d, seed=seed + 7)
        self.parents = [_parents(T, seed + b) for b in range(B)]
        self.par = _ints(dev, self.parents)
        self.tree = torch.empty(B, T, (T + 31) // 32, dtype=torch.int32, device=dev)
        self.positions = torch.empty(B, T, dtype=torch.int32, device=dev)
        self.q_out = torch.zeros(B, T, H, d, dtype=BF16, device=dev)
        self.out, self.lse = torch.empty_like(self.q_out), torch.empty(B, T, H, device=dev)
        n = g.gqa_tree_workspace_size(self.q_out, c.k, c.table)
        self.ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev) if n else None
        self.path, self.keep = torch.zeros(B, T, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
        for b in range(B):
            if c.n[b]:
                kept = _branches(self.parents[b])[(b * 5 + seed) % c.n[b]].nonzero().flatten()
                self.path[b, : len(kept)], self.keep[b] = kept.to(torch.int32).to(dev), len(kept)
        self.ends = torch.empty(B, dtype=torch.int32, device=dev)

    def run(self, stream=None):
        c, H, K = self.c, self.c.H, self.c.K
        g.gqa_tree_from_parents(self.par, c.ln, self.tree, self.positions, new_lens=c.new, stream=stream)
        g.gqa_paged_append(self.qkv[:, :, :H], self.qkv[:, :, H: H + K], self.qkv[:, :, H + K:], self.q_out, c.k, c.v,
                           c.table, c.ln, new_lens=c.new, positions=self.positions, turns=self.turns, stream=stream)
        g.gqa_tree_attn(self.q_out, c.k, c.v, c.table, c.ln, self.out, self.lse, self.ws, new_lens=c.new,
                        tree=self.tree, stream=stream)
        g.gqa_paged_keep(c.k, c.v, c.table, c.ln, self.path, self.keep, self.ends, tokens=c.T, new_lens=c.new,
                         stream=stream)

    def check(self):
        """Attention against the definition over the keys as they were before the branch moved: the new ones are
        found by rotating again."""
        c, H, K = self.c, self.c.H, self.c.K
        whole_k, whole_v = c.k.clone(), c.v.clone()
        for b, L in enumerate(c.lens):
            n = c.n[b]
            if n == 0:
                continue
            depth = torch.tensor([int(r.sum()) - 1 for r in _branches(self.parents[b])[:n]])
            want = _turned(self.qkv[b, :n, H: H + K], L - n + depth, self.turns)
            m = int(self.keep[b])
            kept = self.path[b, :m].long()
            _check_turned(c.k[c.places(b, L - n, L - n + m)], (want[0][kept], want[1][kept]))
            _check_turned(self.q_out[b, :n], _turned(self.qkv[b, :n, :H], L - n + depth, self.turns))
            assert torch.equal(c.v[c.places(b, L - n, L - n + m)], self.qkv[b, kept, H + K:])
            assert int(self.ends[b]) == L - n + m
            # (rounded as the kernel does wherever the definition does not say how)
            again = g.rotary(self.qkv[b, :n, H: H + K].contiguous(), _ints(c.dev, (L - n + depth).tolist()), self.turns)
            at = c.places(b, L - n, L)
            c.k[at], c.v[at] = again, self.qkv[b, :n, H + K:]
        c.q = self.q_out
        want = c.want(lambda b: _branches(self.parents[b])[: c.n[b], : c.n[b]])
        c.k.copy_(whole_k)
        c.v.copy_(whole_v)
        _compare("step", self.out, self.lse, want)


STEPS = [([100, 33, 600, 7], [7, 1, 5, 7], 7, 8, 1, 64, 16), ([700, 300, 0, 129, 64], [16, 3, 0, 16, 9], 16, 32, 8, 128, 32),
         ([900, 50], None, 40, 16, 2, 256, 64)]


@gpu
@pytest.mark.parametrize("i", range(len(STEPS)))
def test_verification_steps_in_a_row(dev, i):
    lens, news, T, H, K, d, page = STEPS[i]
    s = Step(dev, lens, news, T, H, K, d, page, seed=40 + i)
    s.run()
    s.check()
    # the next step begins where the accepted branch ended
    ends = s.ends.tolist()
    again = Step(dev, [e + n for e, n in zip(ends, s.c.n)], s.c.n, T, H, K, d, page, seed=50 + i)
    again.c.k, again.c.v, again.c.table = s.c.k, s.c.v, s.c.table
    if s.c.table.shape[1] * page >= max(again.c.lens):
        again.run()
        again.check()
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_graph_of_a_step_follows_its_inputs(dev):
    """Captured once, replayed with other tokens, trees, lengths and pages."""
    lens, news, T, H, K, d, page = STEPS[1]
    s = Step(dev, lens, news, T, H, K, d, page, seed=60)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    other = Step(dev, [701, 0, 90, 16, 640], [16, 0, 16, 16, 2], T, H, K, d, page, seed=70)
    assert other.c.table.shape[1] <= s.c.table.shape[1] and other.c.k.shape[0] <= s.c.k.shape[0]
    for a, b in ((s.qkv, other.qkv), (s.par, other.par), (s.path, other.path), (s.keep, other.keep),
                 (s.c.ln, other.c.ln), (s.c.new, other.c.new)):
        a.copy_(b)
    s.c.table.fill_(-1)
    s.c.table[:, : other.c.table.shape[1]] = other.c.table
    s.c.k[: other.c.k.shape[0]], s.c.v[: other.c.k.shape[0]] = other.c.k, other.c.v
    s.c.lens, s.c.n, s.parents = other.c.lens, other.c.n, other.parents
    s.out.fill_(math.nan)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    s.check()
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
@pytest.mark.parametrize("B,T,H,K,d,page", [(60, 16, 32, 8, 128, 32), (40, 9, 24, 8, 256, 16), (30, 5, 16, 2, 64, 16),
                                            (3, 70, 16, 2, 64, 16)])
def test_graph_over_a_workspace_of_anything(dev, B, T, H, K, d, page):
    """Captured with one set of lengths, replayed with others, over a workspace that held NaNs before each."""
    lens = [(i * 331) % 800 for i in range(B)]
    c = Case(dev, lens, [i % (T + 1) for i in range(B)], T, H, K, d, page, seed=B)
    ws = torch.empty(g.gqa_tree_workspace_size(c.q, c.k, c.table), dtype=torch.uint8, device=dev)
    out, lse = torch.empty_like(c.q), torch.empty(B, T, H, device=dev)

    def run():
        g.gqa_tree_attn(c.q, c.k, c.v, c.table, c.ln, out, lse, ws, new_lens=c.new, causal=True)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for shift in (0, 1, 7):
        now, news = [lens[i] if i % 7 < shift else lens[i] // (1 + shift) for i in range(B)], [(i * 5 + shift) % (T + 1) for i in range(B)]
        c.lens, c.n = now, [min(n, L) for n, L in zip(news, now)]
        c.ln.copy_(_ints(dev, now))
        c.new.copy_(_ints(dev, news))
        ws.fill_(255)
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        _compare("graph", out, lse, c.want(lambda b: torch.ones(c.n[b], c.n[b]).tril().bool()))
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_tensors_that_do_not_fit_are_refused(dev):
    """Types, shapes, strides and devices, each wrong by itself; nothing is launched, and nothing changes."""
    c = Case(dev, [40, 90], None, 6, 8, 2, 64, 16, seed=98)
    k = _randn(dev, 2, 6, 2, 64, seed=99)
    parents, tree, at = _ints(dev, [[-1] * 6] * 2), torch.zeros(2, 6, 1, dtype=torch.int32, device=dev), _ints(dev, [[0] * 6] * 2)
    turns, path = g.rotary_turns(64, device=dev), _ints(dev, [[0, 2]] * 2)
    keep, news = _ints(dev, [2, 2]), _ints(dev, [6, 5])
    out, lse = torch.zeros_like(c.q), torch.zeros(2, 6, 8, device=dev)
    ws = torch.zeros(max(g.gqa_tree_workspace_size(c.q, c.k, c.table), 1), dtype=torch.uint8, device=dev)
    calls = {
        "apply": (g.gqa_rotary_apply, dict(x=c.q, positions=at, turns=turns, out=c.q.clone())),
        "append": (g.gqa_paged_append, dict(q=c.q, k=k, v=k, q_out=out, k_cache=c.k, v_cache=c.v, page_table=c.table,
                                            seqlens=c.ln, new_lens=news, positions=at, turns=turns)),
        "parents": (g.gqa_tree_from_parents, dict(parents=parents, seqlens=c.ln, tree=tree, positions=at, new_lens=news)),
        "attn": (g.gqa_tree_attn, dict(q=c.q, k_cache=c.k, v_cache=c.v, page_table=c.table, seqlens=c.ln, out=out, lse=lse,
                                       workspace=ws, new_lens=news, tree=tree)),
        "keep": (g.gqa_paged_keep, dict(k_cache=c.k, v_cache=c.v, page_table=c.table, seqlens=c.ln, path=path,
                                        keep_lens=keep, seqlens_out=c.ln.clone(), new_lens=news, tokens=6)),
    }
    for name, (fn, args) in calls.items():
        fn(**args)                                                     # as they are, they do fit
        torch.cuda.synchronize()
        held = {n: t.clone() for n, t in args.items() if isinstance(t, torch.Tensor)}
        for n, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            wrong = [t.cpu(), t.to(torch.float64), t[:1] if n != "turns" else t[None], t[..., None]]
            if n == "workspace":
                wrong = [t.cpu(), torch.cat([t, t])[::2]]
            elif n != "turns":
                wrong.append(torch.cat([t, t], dim=-1)[..., ::2])
            for w in wrong:
                with pytest.raises(ValueError):
                    fn(**{**args, n: w})
            with pytest.raises(TypeError):
                fn(**{**args, n: "a tensor"})
            if n not in ("q", "q_out", "lse", "workspace", "new_lens", "turns", "tree", "positions", "seqlens_out"):
                with pytest.raises(ValueError):
                    fn(**{**args, n: None})
        torch.cuda.synchronize()
        for n, t in held.items():
            assert torch.equal(args[n], t), (name, n)
    with pytest.raises(ValueError):
        g.gqa_paged_append(c.q, k, k, None, c.k, c.v, c.table, c.ln)   # q without a place for it
    with pytest.raises(TypeError):
        g.gqa_tree_attn(**{**calls["attn"][1], "scale": "a number"})
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_capacity_far_beyond_the_lengths(dev):
    """A table for 2^24 positions of each sequence, of which they have a few thousand."""
    for T in (1, 20):
        c = Case(dev, [3000, 40, 0, 777], None, T, 16, 4, 128, 16, seed=96)
        wide = torch.full((4, 1 << 20), -1, dtype=torch.int32, device=dev)
        wide[:, : c.table.shape[1]] = c.table
        c.table = wide
        out, lse = c.run(causal=True)
        _compare("capacity", out, lse, c.want(lambda b: torch.ones(c.n[b], c.n[b]).tril().bool()))
    assert g.gqa_decode_get_error() == g.GQA_OK


@gpu
def test_steps_back_to_back_without_waiting(dev):
    """Twenty steps in a row on one cache, each reading what the one before has just written: the results of the
    same steps with the GPU waited for after every call."""
    def many(wait):
        s = Step(dev, *STEPS[1], seed=97)
        outs = []
        for i in range(20):
            s.qkv.copy_(_randn(dev, *s.qkv.shape, seed=200 + i))
            s.run()
            if wait:
                torch.cuda.synchronize()
            outs.append((s.out.clone(), s.lse.clone(), s.c.k.clone()))
        torch.cuda.synchronize()
        return outs

    for a, b in zip(many(True), many(False)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_two_streams_at_once(dev):
    """Steps of two batches on two streams, a workspace and a cache each: the results of each alone."""
    steps = [Step(dev, *STEPS[i], seed=80 + i) for i in (0, 2)]
    wants = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        wants.append([t.clone() for t in (s.out, s.lse, s.c.k, s.c.v, s.ends)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        steps[0].run(stream=streams[0])
        steps[1].run(stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    for s, want in zip(steps, wants):
        for got, w in zip((s.out, s.lse, s.c.k, s.c.v, s.ends), want):
            assert torch.equal(got, w)


@gpu
def test_calls_share_a_workspace_with_other_operators(dev):
    """Tree attention, cross attention and a decode step back to back in one workspace that holds NaNs at first."""
    a, b = Case(dev, [900, 30, 400], None, 30, 32, 8, 128, 16, seed=90), Case(dev, [700, 90], None, 2, 8, 2, 64, 16, seed=91)
    q, k = _randn(dev, 2, 60, 8, 64, seed=92), _randn(dev, 2, 500, 2, 64, seed=93)
    ln = _ints(dev, [500, 77])
    want = [a.run(causal=True), b.run(causal=True), g.cross_attention(q, k, k, ln)]
    sizes = [g.gqa_tree_workspace_size(a.q, a.k, a.table), g.gqa_tree_workspace_size(b.q, b.k, b.table),
             g.gqa_cross_workspace_size(q, k)]
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device=dev)
    got = [[torch.empty_like(t) for t in w] for w in want]
    for _ in range(5):
        g.gqa_tree_attn(a.q, a.k, a.v, a.table, a.ln, *got[0], ws, causal=True)
        g.gqa_cross_attn(q, k, k, ln, *got[2], ws)
        g.gqa_tree_attn(b.q, b.k, b.v, b.table, b.ln, *got[1], ws, causal=True)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])


@gpu
def test_debug_build_stays_quiet_and_agrees(dev):
    """The bounds-checked build catches no write outside a buffer and gives the same bits."""
    gbuild.build_debug()
    release, g._lib = g.lib(), g.load_library(gbuild.DEBUG_LIB)
    debug, g._lib = g._lib, release
    for args in (([300, 5, 64, 1023], [7, 5, 0, 3], 7, 8, 1, 64, 16, BF16), ([900, 65, 300], [64, 64, 10], 64, 64, 8, 128, 128, BF16),
                 ([641, 130], None, 40, 10, 2, 256, 32, FP16), ([4000, 1], None, 1, 32, 8, 128, 16, BF16)):
        c = Case(dev, *args, seed=95)
        want = c.run(causal=True)
        try:
            g._lib = debug
            assert g.gqa_decode_get_error() == g.GQA_OK
            got = c.run(causal=True)
            assert g.gqa_decode_get_error() == g.GQA_OK
        finally:
            g._lib = release
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
