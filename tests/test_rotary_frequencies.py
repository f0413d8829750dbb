"""rotary_frequencies against the published formulas of the stretched kinds, at every
pair, with the defaults that each kind is published with; and against the
frequencies that perf/more_operators.py measures with."""
import math

import pytest

from moe_expert_layer_warp_gb300 import batch
from perf import more_operators

SIZES = [(128, 10000.0, 4096, 8.0), (128, 500000.0, 8192, 8.0), (64, 1000000.0, 32768, 4.0),
         (96, 10000.0, 2048, 16.0), (16, 150000.0, 4096, 32.0)]


def bands(n, base, original, factor):
    """By wavelengths: those shorter than original / 4 stay, those longer than
    original / 1 are stretched by the factor, and between them the share that stays is
    linear in original / wavelength."""
    out = []
    for i in range(n // 2):
        f = 1.0 / base ** (2 * i / n)
        wave = 2 * math.pi / f
        if wave < original / 4.0:
            out.append(f)
        elif wave > original / 1.0:
            out.append(f / factor)
        else:
            smooth = (original / wave - 1.0) / (4.0 - 1.0)
            out.append((1 - smooth) * f / factor + smooth * f)
    return out


def ramp(n, base, original, factor):
    """By the pairs' index: the pair that turns 32 times within the original positions,
    rounded down, begins the ramp, and the one that turns once, rounded up, ends it."""
    def pair(turns):
        return n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), n - 1)
    out = []
    for i in range(n // 2):
        f = base ** -(2 * i / n)
        stretched = min(max((i - low) / (high - low), 0.0), 1.0)
        out.append(f / factor * stretched + f * (1 - stretched))
    return out


@pytest.mark.parametrize("n, base, original, factor", SIZES)
@pytest.mark.parametrize("kind, published", [("bands", bands), ("ramp", ramp)])
def test_published_values(kind, published, n, base, original, factor):
    got = batch.rotary_frequencies(n, base, scaling=kind, factor=factor, original=original)
    want = published(n, base, original, factor)
    assert len(got) == len(want) == n // 2
    # powers, logarithms and quotients in 64 bits, a few roundings each
    assert all(abs(a - b) <= 2.0 ** -48 * b for a, b in zip(got, want))
    # each kind has pairs that stay, that are stretched and that are between
    ratio = [a * base ** (2 * i / n) for i, a in enumerate(got)]
    assert max(ratio) > 1 - 1e-9 and min(ratio) < 1 / factor + 1e-9


def test_given_ends_are_kept():
    for kind in ("bands", "ramp"):
        default = {"bands": 4.0, "ramp": 32.0}[kind]
        args = dict(scaling=kind, factor=8.0, original=8192)
        assert batch.rotary_frequencies(128, fast=default, slow=1.0, **args) == (
            batch.rotary_frequencies(128, **args))
        assert batch.rotary_frequencies(128, fast=9.0, **args) != batch.rotary_frequencies(128, **args)
        with pytest.raises(ValueError):
            batch.rotary_frequencies(128, slow=default, **args)


@pytest.mark.parametrize("kind", ["none", "linear", "base", "ramp", "bands"])
@pytest.mark.parametrize("n", [16, 64, 80, 192])
def test_measured_cases_use_the_same(kind, n):
    case = {"rotated": n, "factor": 1.0 if kind == "none" else 8.0, "scaling": kind}
    got = batch.rotary_frequencies(n, scaling=kind, factor=case["factor"])
    want = more_operators._frequencies(case)
    assert all(abs(a - b) <= 2.0 ** -48 * b for a, b in zip(got, want))
