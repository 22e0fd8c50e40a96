"""The workgroups of a packed linear-attention batch, on the host: whatever the
offsets, each sequence's segments are each taken by one workgroup of those that
are launched, and by no thread against another."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++ in this image")
    lib = str(tmp_path_factory.mktemp("places") / "places.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "gated_deltanet_recurrence_delta_amd", "csrc"),
                    os.path.join(HERE, "linear_places_host.cpp"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).linear_places
    fn.restype = None

    def call(which, cu, T, rows, threads):
        """(place, sequence, segment, uncut) of every workgroup of a launch that has work."""
        B = len(cu) - 1
        places = T // rows + (B if which == 0 else 0)
        found = (ctypes.c_int * max(1, 4 * places))()
        fn(which, (ctypes.c_int32 * len(cu))(*cu), B, T, rows, threads, places, found)
        got = []
        for at in range(places):
            n, seg, uncut, taken = found[4 * at:4 * at + 4]
            assert taken == (n >= 0), (at, taken)  # one thread, or none
            if n >= 0:
                got.append((at, n, seg, bool(uncut)))
        return got

    return call


def check(walk, cu, T, rows, threads):
    B = len(cu) - 1
    at = [min(max(x, 0), T) for x in cu]
    lens = [max(0, e - b) for b, e in zip(at, at[1:])]
    falls = any(e < b for b, e in zip(at, at[1:]))
    outputs = [x[1:] for x in walk(0, cu, T, rows, threads)]
    states = walk(1, cu, T, rows, threads)
    assert len(outputs) == len(set(outputs)), "a segment is taken twice"
    if falls:
        assert sorted(outputs) == [(n, 0, True) for n in range(B)] and not states
        return
    assert sorted(outputs) == [(n, s, False) for n in range(B) for s in range(max(1, -(-lens[n] // rows)))]
    # a segment that others follow leaves its state in a slot of its own
    assert sorted(x[1:3] for x in states) == [(n, s) for n in range(B) for s in range(-(-lens[n] // rows) - 1)]
    assert all(place == at[n] // rows + seg and place < T // rows for place, n, seg, _ in states)


@pytest.mark.parametrize("cu,T", [
    ([0], 0), ([0, 0], 0), ([0, 1000], 1000), ([9, 3, 30], 90), ([9, 3, 300], 1300),
    ([0, 32768, 0, 32768], 32768),                                       # the same rows twice
    ([256, 0] + list(range(10, 10 * 64 + 1, 10)), 1000),                 # no row twice, 65 sequences
    ([1000] + [0] * 64 + [1000], 1000),
    (list(range(1300, -1, -20)), 1300),                                  # 65 sequences, all empty
    ([-5, 40, 1400], 1300), ([0, 128, 128, 256, 256, 256, 1024], 1024),
])
@pytest.mark.parametrize("threads", [128, 512])
def test_given_offsets(walk, cu, T, threads):
    for rows in (64, 256, T + 1):
        check(walk, cu, T, rows, threads)


@pytest.mark.parametrize("kind", ["ascending", "gaps", "any", "one falls"])
@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 200])
def test_random_offsets(walk, kind, B):
    rnd = random.Random(B * 10 + len(kind))
    for _ in range(30):
        T, rows = rnd.choice([0, 7, 300, 2000]), 64 * rnd.randint(1, 6)
        cu = [rnd.randint(-3, T + 3) for _ in range(B + 1)]
        if kind != "any":
            cu.sort()
        if kind == "ascending":
            cu[0], cu[-1] = 0, T
        if kind == "one falls":
            i = rnd.randint(1, B)
            cu[i] = rnd.randint(0, T)
        check(walk, cu, T, rows, rnd.choice([128, 256, 512]))
