"""The rotation tables' frequencies for stretched contexts, on the CPU, against
hand-worked values and each ramp's definition written out for itself."""
import math

import pytest
import torch

from linear_exl3_input_amd import attention as at


def frequencies(dim, base, linear=1.0, ntk=1.0, yarn=None, turns=(1.0, 32.0), gain=None, ramp="pairs"):
    return at._frequencies(dim, base, linear, ntk, yarn, turns, gain, ramp)


def by_pairs(dim, base, factor, trained, lo, hi):
    """The ramp over indexes: 0 (kept) up to `first`, 1 (slowed) from `last` on."""
    where = [dim * math.log(trained / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (hi, lo)]
    first, last = max(math.floor(where[0]), 0), min(math.ceil(where[1]), dim - 1)
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        r = min(max((i - first) / ((last - first) or 0.001), 0.0), 1.0)
        out.append(f / factor * r + f * (1 - r))
    return torch.tensor(out, dtype=torch.float64)


def by_turns(dim, base, factor, trained, lo, hi):
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        s = min(max((trained * f / (2 * math.pi) - lo) / (hi - lo), 0.0), 1.0)
        out.append((1 - s) * f / factor + s * f)
    return torch.tensor(out, dtype=torch.float64)


SHAPES = [(128, 1e6, 4.0, 32768, 1.0, 32.0), (64, 1e4, 40.0, 4096, 1.0, 32.0), (128, 5e5, 8.0, 8192, 1.0, 4.0),
          (64, 1e4, 4.0, 100, 1.0, 32.0), (256, 1e4, 16.0, 2048, 2.0, 20.0), (16, 1e4, 2.0, 7, 0.5, 30.0)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("ramp,want", [("pairs", by_pairs), ("turns", by_turns)])
def test_ramps(shape, ramp, want):
    dim, base, factor, trained, lo, hi = shape
    inv, gain = frequencies(dim, base, yarn=(factor, trained), turns=(lo, hi), ramp=ramp)
    assert ((inv / want(*shape)) - 1).abs().max() < 1e-12
    assert gain == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-15)


def test_the_ramp_over_pairs_by_hand():
    """64 dims, base 10^4, 4096 positions: 32 turns at pair 10.47, one at 22.51, so the ramp runs from 10 to 23; pair
    16 (frequency 1/100) is 6/13 of the way."""
    inv, _ = frequencies(64, 1e4, yarn=(40.0, 4096))
    assert inv[16].item() == pytest.approx(0.01 * (7 / 13 + 6 / 13 / 40), rel=1e-14)
    assert inv[10].item() == pytest.approx(1e4 ** (-10 / 32), rel=1e-14)
    assert inv[23].item() == pytest.approx(1e4 ** (-23 / 32) / 40, rel=1e-14)
    assert inv[11] < 1e4 ** (-11 / 32) and inv[22] > 1e4 ** (-22 / 32) / 40


def test_the_two_ramps_differ():
    for shape, count, worst in ((SHAPES[0], 16, 0.42), (SHAPES[1], 12, 0.77)):
        ratio = by_turns(*shape) / by_pairs(*shape)
        off = torch.maximum(1 - ratio, 1 - 1 / ratio)  # the smaller below the larger
        assert int((off > 1e-9).sum()) == count and off.max().item() == pytest.approx(worst, abs=0.005)


def test_the_default_ramp_is_the_one_over_pairs():
    shape = SHAPES[0]
    inv, _ = at._frequencies(128, 1e6, 1.0, 1.0, (4.0, 32768), (1.0, 32.0), None, "pairs")
    import inspect

    import linear_exl3_input_amd as ex
    assert inspect.signature(ex.Rope.make).parameters["yarn_ramp"].default == "pairs"
    assert ((inv / by_pairs(*shape)) - 1).abs().max() < 1e-12


def test_without_a_ramp():
    inv, gain = frequencies(64, 1e4, linear=2.0)
    assert gain == 1.0 and inv[0].item() == 0.5 and inv[16].item() == pytest.approx(0.005, rel=1e-15)
    inv, _ = frequencies(64, 1e4, ntk=4.0)
    assert inv[0].item() == 1.0 and inv[31].item() == pytest.approx(1e4 ** (-31 / 32) / 4, rel=1e-12)


@pytest.mark.parametrize("kw,what", [
    (dict(turns=(2.0, 2.0)), "yarn_turns"), (dict(turns=(32.0, 1.0)), "yarn_turns"), (dict(turns=(0.0, 32.0)), "yarn_turns"),
    (dict(turns=(math.nan, 32.0)), "yarn_turns"), (dict(ramp="index"), "yarn_ramp"), (dict(base=1.0), "base"),
    (dict(base=math.nan), "base"), (dict(base=-5.0), "base"), (dict(linear=math.nan), "linear"), (dict(ntk=0.0), "ntk"),
    (dict(yarn=(math.nan, 100)), "yarn"), (dict(yarn=(4.0, 0)), "yarn"), (dict(dim=24), "rotary_dim"),
])
def test_refusals(kw, what):
    with pytest.raises(ValueError, match=what):
        frequencies(**{**dict(dim=64, base=1e4, yarn=(4.0, 4096)), **kw})


def test_a_table_needs_a_position():
    import linear_exl3_input_amd as ex
    with pytest.raises(ValueError, match="positions=0"):
        ex.Rope.make(64, 1e4, 0, device="cpu")
