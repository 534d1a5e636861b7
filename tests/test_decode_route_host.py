"""Which kernels a decode call takes, and how they share its items: the host's own rules, run on
the CPU."""
import random

import pytest

from decode_route import CASES, DENSE, constants, groups, routes


def test_no_item_is_described_by_two_blocks():
    """decode_walks_kernel gives block b the items from b * group on and describes whole rounds of
    them: a group of a part of a round would reach into the next block's items."""
    c = constants()
    most = c["kPlanBlocks"] * c["kPlanThreads"]
    rng = random.Random(0)
    items = [1, most - 1, most, most + 1, 2 ** 31 - 1] + [int(2 ** rng.uniform(0, 31)) for _ in range(500)]
    pairs = [(n, 1 << k) for n in items for k in range(5)]
    for (n, lanes), group in zip(pairs, groups(pairs)):
        assert -(-n // group) <= most
        assert group == 1 if n <= most else group % (c["kWalkThreads"] // lanes) == 0


def test_the_calls_of_the_gpu_tests_take_the_routes_that_they_are_for():
    names = list(CASES)
    for name, got in zip(names, routes([CASES[n] for n in names])):
        want = CASES[name]["want"]
        assert {k: got[k] for k in want} == want, name


@pytest.mark.parametrize("d", [64, 128])
def test_routes_fit_what_the_kernels_hold(d):
    """Over random calls: a team's blocks run at once and have partials for every warp, and warps
    and groups stay within the workspace."""
    rng, c = random.Random(d), constants()
    calls = []
    for _ in range(3000):
        Hkv, G = int(2 ** rng.uniform(0, 6)), int(2 ** rng.uniform(0, 6))
        pats = [(int(2 ** rng.uniform(0, 21)), int(2 ** rng.uniform(0, 8))) for _ in range(rng.randint(1, 16))]
        T = int(2 ** rng.uniform(0, 12))
        calls.append(dict(T=T, B=rng.choice((T, T, max(1, T // 2), max(1, T // 5))), H=Hkv * G, Hkv=Hkv, d=d,
                          pats=rng.choice((pats, DENSE)), longest=16 * int(2 ** rng.uniform(0, 17)), of_seq=True))
    for call, a in zip(calls, routes(calls)):
        G = call["H"] // call["Hkv"]
        tiles = sum(-(-(-(-min(w, call["longest"]) // r)) // 32) for w, r in call["pats"])
        assert a["heads"] in (1, 2, 4, 8, 16) and a["walks"] <= a["lanes"] <= 16 and a["items"] >= 1
        assert a["nsub"] * a["heads"] >= G and a["tokens"] * G <= max(a["heads"], G)
        if a["team"] > 0:
            assert a["items"] * a["team"] <= 256 and tiles <= 8 * c["kTeamWarps"] * a["team"] and not a["grouped"]
        elif a["team"] == 0:
            assert tiles <= 16 and not a["grouped"]
        assert a["warps"] % c["kDecWarps"] == 0 and a["warps"] >= c["kDecWarps"]
        assert a["warps"] <= 148 * 4 * c["kDecWarps"]
        assert not a["grouped"] or (a["dense"] and a["tokens"] > 0 and call["T"] > call["B"])
        assert not a["plan_alone"] or a["items"] * a["lanes"] <= c["kPlanAlone"]
