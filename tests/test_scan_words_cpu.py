"""The words through which the recurrence's workgroups hand their states on, on the host: what a state is formed
from, words that are missing, and the range of a group's product of decays."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from gated_deltaproduct_recurrence_amd import build

MISSING = (1 << 64) - 1
NOTHING = 0x3F800000 << 32
f32 = ctypes.c_float


@pytest.fixture(scope="module")
def words(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not installed")
    out = str(tmp_path_factory.mktemp("words") / "words.so")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    subprocess.run([build.HIPCC, "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{build.CSRC}",
                    os.path.join(os.path.dirname(__file__), "scan_words_host.cpp"), "-o", out], check=True, env=env)
    lib = ctypes.CDLL(out)
    u64, p = ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64)
    for name, res, args in (("tile_word", u64, [f32, f32]), ("group_word", u64, [p, ctypes.c_int]),
                            ("span_word", u64, [p]), ("span_applied", f32, [p, f32]),
                            ("group_word_applied", f32, [u64, f32]), ("drops", ctypes.c_int, [u64]),
                            ("fold_tiles", f32, [p]), ("fold_groups", f32, [p])):
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def array(values):
    return (ctypes.c_uint64 * len(values))(*values)


def group(words, *tiles):
    """The word of tiles (A, B), in the order of the rows."""
    return words.group_word(array([words.tile_word(a, b) for a, b in reversed(tiles)]), len(tiles))


@pytest.mark.parametrize("kind", ["fold_tiles", "fold_groups"])
def test_a_missing_word_makes_the_state_unknown(words, kind):
    """Nearest word first: one missing, and the next one knows its state."""
    word = words.tile_word if kind == "fold_tiles" else lambda a, b: group(words, (a, b))
    fold = getattr(words, kind)
    known, pair = word(0.0, 3.0), word(0.5, 1.0)
    assert fold(array([pair, pair, known] + [MISSING] * 5)) == 2.25
    assert fold(array([known] + [MISSING] * 7)) == 3.0
    assert math.isnan(fold(array([MISSING, known] + [pair] * 6)))
    assert math.isnan(fold(array([pair, MISSING, known] + [pair] * 5)))
    assert math.isnan(fold(array([pair] * 8)))  # none knows its state
    assert fold(array([pair, known, MISSING, known] + [pair] * 4)) == 2.5
    assert fold(array([pair, 0] + [0] * 6)) == 1.0  # nothing before the first tile


def test_a_missing_word_makes_a_group_unknown(words):
    known, pair = words.tile_word(0.0, 3.0), words.tile_word(0.5, 1.0)
    assert words.span_applied(array([pair, pair] + [NOTHING] * 13), 4.0) == 2.5
    assert words.span_applied(array([NOTHING] * 15), 4.0) == 4.0
    assert math.isnan(words.span_applied(array([pair, MISSING, pair] + [NOTHING] * 12), 4.0))
    assert math.isnan(words.span_applied(array([MISSING, known] + [NOTHING] * 13), 4.0))
    assert words.span_applied(array([pair, known, MISSING] + [NOTHING] * 12), 4.0) == 2.5
    assert words.span_applied(array([pair, known, MISSING] + [NOTHING] * 12), math.nan) == 2.5


def test_no_word_reads_as_missing(words):
    for a in (math.nan, math.inf, 3.4e38, 1e-45, 0.0):
        for b in (math.nan, math.inf, -math.inf, -0.0):
            assert words.tile_word(a, b) != MISSING
            assert group(words, (a, b), (a, b)) != MISSING and group(words, *[(a, b)] * 16) != MISSING


def test_the_range_of_a_group(words):
    """Products of 16 decays between 2^-255 and 2^255 on states between 2^-126 and 2^127."""
    rng = random.Random(5)
    for _ in range(3000):
        log2 = rng.uniform(-250, 250) / 16
        tiles = [(f32(2.0 ** (log2 + rng.uniform(-1, 1))).value, 0.0) for _ in range(16)]
        product = math.prod(a for a, _ in tiles)
        h = f32(rng.choice([-1, 1]) * 2.0 ** rng.uniform(-126, 127)).value
        got = words.group_word_applied(group(words, *tiles), h)
        want = product * h
        if abs(want) >= 2.0 ** 128:
            assert got == math.copysign(math.inf, want)
        elif abs(want) > 2.0 ** 128 * (1 - 2.0 ** -19):
            continue  # infinity or not by the roundings
        else:  # 15 products and the last one, half a step each; below 2^-126 nothing need be left
            assert abs(got - want) <= abs(want) * 17 * 2.0 ** -24 + 2.0 ** -126, (product, h, got, want)


def test_growth_of_zero_is_zero(words):
    for a in (1e10, 1e38):
        assert words.group_word_applied(group(words, *[(a, 0.0)] * 16), 0.0) == 0.0
        assert words.span_applied(array([words.tile_word(a, 0.0)] * 15), 0.0) == 0.0


def test_what_a_group_drops(words):
    """Below 2^-126 a state is dropped where no state of float32 could move B by half a step, or where less than
    2^-126 of the largest would be left; not elsewhere."""
    quarter = (2.0 ** -10, 0.0)
    assert words.drops(group(words, *[quarter] * 15, (2.0 ** -10, 1.0)))
    assert not words.drops(group(words, *[quarter] * 15, (2.0 ** -10, 2.0 ** -40)))
    assert not words.drops(group(words, *[quarter] * 12, (1.0, 1.0)))  # 2^-120
    assert not words.drops(group(words, *[quarter] * 16))  # 2^-160 and B = 0
    assert words.drops(group(words, *[(2.0 ** -17, 0.0)] * 16))  # 2^-272
    assert words.drops(group(words, (1e30, 0.0), (0.0, 2.0), (1e30, 0.0), (1e30, 0.0)))


def test_a_product_that_is_no_number(words):
    for bad in (math.nan, math.inf):
        word = group(words, (bad, math.nan), (0.5, 1.0))
        assert math.isnan(words.group_word_applied(word, 0.0))
        word = group(words, (bad, math.nan), (0.0, 7.0), (0.5, 1.0))
        assert words.group_word_applied(word, math.nan) == 4.5
