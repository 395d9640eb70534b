"""How sequences are cut into chunks and where what belongs to a chunk lies, on the host: every row once, every place its
own, and with boundaries that do not rise every place within what is allocated."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

from gated_deltaproduct_recurrence_amd import build

i64, int32 = ctypes.c_int64, ctypes.c_int


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not installed")
    out = str(tmp_path_factory.mktemp("chunks") / "chunks.so")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    subprocess.run([build.HIPCC, "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{build.CSRC}",
                    os.path.join(os.path.dirname(__file__), "chunks_host.cpp"), "-o", out], check=True, env=env)
    lib = ctypes.CDLL(out)
    for name, args in (("numbers", [i64, i64, int32]), ("slots", [i64, int32]), ("followed", [i64, int32]),
                       ("checkpoint", [int32, int32, int32, int32])):
        getattr(lib, name).restype, getattr(lib, name).argtypes = i64, args
    lib.chunks.restype, lib.chunks.argtypes = None, [ctypes.POINTER(i64), int32, int32, int32, ctypes.c_void_p]
    return lib


def chunks(lib, cu, T, shift):
    N = len(cu) - 1
    out = (i64 * 8 * lib.numbers(T, N, shift))()
    lib.chunks((i64 * (N + 1))(*cu), T, N, shift, out)
    return [tuple(row) for row in out]


def check(lib, cu, T, shift, rising):
    """Bounds of everything a chunk names; where the boundaries rise, also that it is all there and its own."""
    N, places = len(cu) - 1, lib.slots(T, shift)
    rows, behind, points, starts = [0] * T, set(), set(), []
    for begin, end, first, last, seq, index, after, before in chunks(lib, cu, T, shift):
        if begin < 0:
            continue
        assert 0 <= first <= begin <= end <= last <= T and 0 <= seq < N and end - begin <= 1 << shift
        for t in range(begin, end):
            rows[t] += 1
        starts += [seq] * (index == 0)
        if end < last:
            assert end - begin == 1 << shift and 0 <= after < places and after == (first >> shift) + index
            assert not rising or after not in behind
            behind.add(after)
        if index > 0:
            assert 0 <= before < places and before == (first >> shift) + index - 1
        fine = min(shift, 2)  # checkpoints of up to 4 rows
        for t in range(begin, end, 1 << fine):
            row = lib.checkpoint(first, seq, t, fine)
            assert 0 <= row < lib.numbers(T, N, fine)
            assert not rising or row not in points
            points.add(row)
    for i in range(N):  # the walk over a sequence's hand-overs
        first = max(0, min(cu[i], T))
        full = lib.followed(max(0, min(cu[i + 1], T)) - first, shift)
        assert full <= 0 or (first >> shift) + full <= places
        if rising:
            assert {(first >> shift) + c for c in range(full)} <= behind
    if rising:
        inside = [cu[0] <= t < cu[-1] for t in range(T)]
        assert rows == [int(x) for x in inside] and starts == list(range(N))


@pytest.mark.parametrize("T,N", [(0, 2), (1, 2), (3, 3), (5, 2), (8, 2), (4, 3)])
def test_all_boundaries_of_few_rows(lib, T, N):
    for cu in itertools.product(range(-1, T + 2), repeat=N + 1):
        rising = all(a <= b for a, b in zip(cu, cu[1:])) and cu[0] >= 0 and cu[-1] <= T
        for shift in (0, 1, 2):
            check(lib, cu, T, shift, rising)


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 130, 4097])
def test_rising_boundaries(lib, N):
    rng = random.Random(N)
    for T in (1, 50, 700, 3000):
        for _ in range(4):
            cu = sorted(rng.randint(0, T) for _ in range(N + 1))
            for shift in (1, 3, 4, 7):
                check(lib, cu, T, shift, True)


@pytest.mark.parametrize("N", [1, 3, 64, 65, 300])
def test_boundaries_that_do_not_rise(lib, N):
    rng = random.Random(N)
    for T in (1, 50, 700):
        for _ in range(20):
            cu = [rng.choice([rng.randint(-9, T + 9), 0, T, 1 << 40, -1 << 40]) for _ in range(N + 1)]
            for shift in (1, 3, 4, 7):
                check(lib, cu, T, shift, False)


def test_the_largest_numbers(lib):
    """The last rows of what a row's number holds."""
    T = 1 << 30
    for shift in (3, 4, 11):
        for cu in ([0, T], [T - 1, T], [0, 1, T - 5, T - 5, T]):
            N, places = len(cu) - 1, lib.slots(T, shift)
            assert lib.numbers(T, N, shift) == (T >> shift) + N and places == (T - 1) >> shift
            for i in range(N):
                full = lib.followed(cu[i + 1] - cu[i], shift)
                assert full <= 0 or (cu[i] >> shift) + full <= places
            assert lib.checkpoint(cu[-2], N - 1, cu[-1] - 1 & ~15 if cu[-2] == 0 else cu[-2], 4) < lib.numbers(T, N, 4)
