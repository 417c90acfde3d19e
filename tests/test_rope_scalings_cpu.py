"""The two blends of YaRN's frequencies, without a GPU: by the number of turns, and by the pair's index."""
import math

import numpy as np
import pytest

import speculative_decoding_block_dflash_gb300 as dfl

TWO_PI = 2 * math.pi


def frequencies(rope):
    """The f_i of a table, below one turn a position."""
    return np.array([t % 2 ** 64 for t in rope.turns.tolist()], dtype=np.float64) / 2.0 ** 64 * TWO_PI


# (rotary dims, base, factor, original length, turns that keep a pair, turns below which it is divided) and the blend's ends, by
# hand: pair i makes L base^(-2i/r) / 2 pi turns, so that n turns are made at i = r ln(L / 2 pi n) / (2 ln base)
CASES = [
    ((128, 1e4, 4.0, 32768, 32.0, 1.0), (35, 60)),    # 35.4 and 59.5
    ((64, 5e5, 8.0, 8192, 32.0, 1.0), (9, 18)),       # 9.04 and 17.5
    ((64, 1e4, 40.0, 4096, 32.0, 1.0), (10, 23)),     # 10.5 and 22.5
    ((128, 1e6, 2.0, 4, 2.0, 0.1), (0, 9)),           # -5.3 and 8.6: the faster end lies before the first pair
]


@pytest.mark.parametrize("args,ends", CASES)
def test_blend_by_the_pairs_index(args, ends):
    r, base, factor, old, fast, slow = args
    rope = dfl.make_rope(r, base=base, scaling="yarn_index", factor=factor, original_len=old, beta_fast=fast, beta_slow=slow,
                         device="cpu")
    f, got = base ** (-np.arange(0, r, 2) / r), frequencies(rope)
    first, last = ends
    for i in range(r // 2):
        share = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)  # of the divided frequency
        want = f[i] * (share / factor + 1 - share)
        assert abs(got[i] / want - 1) < 1e-12, i
    assert abs(rope.gain - (0.1 * math.log(factor) + 1)) < 1e-15


def test_the_two_blends_differ_as_stated():
    kw = dict(base=1e4, factor=4.0, original_len=32768, device="cpu")
    by_turns, by_index = (frequencies(dfl.make_rope(128, scaling=s, **kw)) for s in ("yarn", "yarn_index"))
    f = 1e4 ** (-np.arange(0, 128, 2) / 128)
    keep = np.clip((32768 * f / TWO_PI - 1) / 31, 0, 1)
    assert np.allclose(by_turns, f / 4 * (1 - keep) + f * keep, rtol=1e-12, atol=0)
    apart = np.abs(by_turns / by_index - 1)
    assert (apart > 1e-9).sum() == 24 and 0.42 < apart.max() < 0.43
    assert np.allclose(by_turns[:36], f[:36], rtol=1e-12) and np.allclose(by_index[60:], f[60:] / 4, rtol=1e-12)


def test_a_blend_without_a_pair_between():
    # both ends at the same pair: a step
    rope = dfl.make_rope(8, base=1e4, scaling="yarn_index", factor=2.0, original_len=10 ** 9, beta_fast=2.0, beta_slow=1.0,
                         device="cpu")
    f = 1e4 ** (-np.arange(0, 8, 2) / 8)
    assert np.allclose(frequencies(rope), f, rtol=1e-12)  # every pair turns more than twice


def test_refusals():
    for bad in (dict(), dict(original_len=9, beta_fast=1.0), dict(original_len=9, base=1.0), dict(original_len=9, base=0.5),
                dict(original_len=9, beta_slow=0.0), dict(original_len=9, inv_freq=[1.0, 0.5])):
        with pytest.raises(ValueError):
            dfl.make_rope(4, scaling="yarn_index", device="cpu", **bad)
