"""The rotation's table, and what it turns at far positions, against frequencies of 40 digits.

The table is computed in fp64 and is within 2^-54 of a turn of f / (2 pi): the
bound that include/gqa_paged.h gives.  (f <= 1, so that f / (2 pi) < 2^-2.6, and
half a step of it is 2^-56: the constant 2 pi and the division are off by as much
each, pow by little more, and its argument and a stretched base by less than
2^-56 together, as x exp(-x) <= 1 / e.)  A position's angle is then off by
|position| 2^-54 turns, beside what the kernel adds, which test_paged.py derives:
less than 2^-21 m (|a| + |b|) of a pair (a, b), and half a step of the output."""
import math
import random
from decimal import Decimal, getcontext

import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild

gpu = pytest.mark.gpu
getcontext().prec = 40
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
STEP = Decimal(2) ** -54


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def turns_of(dim, base, scaling="none", factor=1.0, original_length=0, slow=1.0, fast=32.0):
    """f_i / (2 pi) by the header's definitions."""
    base, factor, slow, fast = (Decimal(x) for x in (base, factor, slow, fast))
    log_base = base.ln() + (factor.ln() * dim / (dim - 2) if scaling == "base" and dim > 2 else 0)
    out = []
    for i in range(dim // 2):
        f = (-log_base * 2 * i / dim).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            w = min(Decimal(1), max(Decimal(0), (original_length * f / TWO_PI - slow) / (fast - slow)))
            f *= (1 - w) / factor + w
        out.append(f / TWO_PI)
    return out


def _draw(seed):
    rng = random.Random(seed)
    dim, base, scaling = 2 * rng.randint(1, 128), 10 ** rng.uniform(0.01, 7), rng.choice(["none", "linear", "base", "parts"])
    if scaling == "none":
        return dim, base, {}
    kw = dict(scaling=scaling, factor=10 ** rng.uniform(0, 2))
    if scaling == "parts":
        slow = rng.uniform(0, 4)
        fast = slow + 10 ** rng.uniform(-1, 1.6)
        least = math.ceil(16 * fast * fast / (fast - slow))              # the header's condition
        kw.update(slow=slow, fast=fast, original_length=least + rng.randint(0, 10 ** 5))
    return dim, base, kw


TABLES = [(128, 10000.0, {}), (256, 500000.0, {}), (64, 1.0000001, {}), (2, 10000.0, {}),
          (64, 10000.0, dict(scaling="base", factor=8.0)), (20, 10000.0, dict(scaling="linear", factor=4.0)),
          (128, 500000.0, dict(scaling="parts", factor=8.0, original_length=8192))] + [_draw(i) for i in range(8)]


@pytest.mark.parametrize("dim,base,kw", TABLES)
def test_the_table_is_within_its_bound(dim, base, kw):
    table = g.rotary_turns(dim, base, **kw).tolist()
    for i, (t, want) in enumerate(zip(table, turns_of(dim, base, **kw))):
        assert abs(Decimal(t) / 2 ** 64 - want) <= STEP, i


@gpu
@pytest.mark.parametrize("dim,base,kw", [TABLES[0], TABLES[1], TABLES[4], TABLES[6]])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_turn_by_the_frequencies(dim, base, kw, interleaved):
    """Angles from the frequencies, not from the table; fp32, whose rounding hides least."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    positions = [0, 1, 4095, 131071, 10 ** 6, 10 ** 9, 2 ** 31 - 1, -10 ** 9]
    head = dim if dim in (64, 128, 256) else 256
    x = torch.randn(len(positions), 2, head, generator=torch.Generator(dev).manual_seed(dim), device=dev)
    y = g.rotary(x, torch.tensor(positions, dtype=torch.int32, device=dev), g.rotary_turns(dim, base, device=dev, **kw),
                 interleaved=interleaved)
    f = turns_of(dim, base, **kw)
    angle = torch.tensor([[float(p * t % 1 * TWO_PI) for t in f] for p in positions], dtype=torch.float64)[:, None]
    c, s = angle.cos(), angle.sin()
    i = torch.arange(dim // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
    x, y = x.cpu().double(), y.cpu().double()
    a, b = x[..., lo], x[..., hi]
    far = torch.tensor([abs(p) * 2.0 ** -54 * 2 * math.pi for p in positions], dtype=torch.float64)[:, None, None]
    for got, want in ((y[..., lo], a * c - b * s), (y[..., hi], a * s + b * c)):
        tol = (a.abs() + b.abs()) * (2.0 ** -21 + far) + want.abs() * 2.0 ** -24
        assert ((got - want).abs() <= tol).all()
    assert torch.equal(y[..., dim:], x[..., dim:])
