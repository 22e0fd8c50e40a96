"""The order in which a pool's slots are moved, on the host against plain
indexing: lists within their bounds, groups that do not meet, each slot read
before it is written."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gated_deltanet_recurrence_delta_amd", "csrc")
LIMIT = 320  # steps of one launch


@pytest.fixture(scope="module")
def move(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++ in this image")
    lib = str(tmp_path_factory.mktemp("move") / "move.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-Werror", "-D_GLIBCXX_ASSERTIONS", "-I",
                    CSRC, os.path.join(HERE, "move_plan_host.cpp"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).move_plan

    def call(src, dst, slots):
        """Carries the pairs out; the number of launches."""
        ints = lambda x: (ctypes.c_int * max(1, len(x)))(*x)  # noqa: E731
        pool, count = ints(range(1, slots + 1)), ctypes.c_int()
        want = list(pool)
        for s, d in zip(src, dst):
            want[d] = s + 1 if s >= 0 else 0
        assert fn(slots, ints(src), ints(dst), len(src), pool, len(src), ctypes.byref(count)) == 0
        assert list(pool)[:slots] == want[:slots]
        return count.value

    return call


def singles(n, at):
    """n pairs of slots of their own."""
    return [at + 2 * i for i in range(n)], [at + 2 * i + 1 for i in range(n)], at + 2 * n


def chain(n, at):
    """n pairs, each taking what the next one overwrites."""
    return list(range(at + 1, at + n + 1)), list(range(at, at + n)), at + n + 1


def cycle(n, at):
    return list(range(at + 1, at + n)) + [at], list(range(at, at + n)), at + n


def tree(n, at):
    """A chain that ends in a cycle: n pairs of each."""
    s, d, end = cycle(n, at)
    return s + [at] + list(range(end, end + n - 1)), d + list(range(end, end + n)), end + n


@pytest.mark.parametrize("first", [0, 1, 318, 319, 320, 321, 639, 640, 641])
@pytest.mark.parametrize("kind", [chain, cycle, tree])
@pytest.mark.parametrize("n", [2, 317, 318, 319, 320, 321, 330, 700])
def test_a_long_list_behind_full_launches(move, first, kind, n):
    s, d, at = singles(first, 0)
    s2, d2, at = kind(n, at)
    launches = move(s + s2, d + d2, at)
    steps = len(s) + len(s2)
    assert launches <= 2 + 2 * (steps // LIMIT + 1)
    # and one more list of each kind behind that
    s3, d3, at = cycle(n, at)
    s4, d4, at = chain(3, at)
    move(s + s2 + s3 + s4, d + d2 + d3 + d4, at)


@pytest.mark.parametrize("kind", ["random", "clear", "permutation", "few sources", "shift"])
@pytest.mark.parametrize("slots", [1, 2, 9, 64, 350, 1500])
def test_random_maps(move, kind, slots):
    rnd = random.Random(slots * 7 + len(kind))
    for _ in range(20):
        dst = rnd.sample(range(slots), rnd.randint(0, slots))
        src = {"random": [rnd.randrange(slots) for _ in dst], "clear": [rnd.choice([-1, rnd.randrange(slots)]) for _ in dst],
               "permutation": rnd.sample(dst, len(dst)), "few sources": [rnd.randrange(min(3, slots)) for _ in dst],
               "shift": [(d + 1) % slots for d in dst]}[kind]
        move(src, dst, slots)


def test_one_launch_for_usual_lists(move):
    assert move(*singles(300, 0)) == 1 and move(*cycle(300, 0)) == 1 and move(*chain(320, 0)) == 1
    assert move([0] * 300, list(range(1, 301)), 301) == 1
