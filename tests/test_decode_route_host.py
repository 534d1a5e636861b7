"""Which kernels a decode call takes, and how they share its items: the host's own rules, run on
the CPU."""
import random

from decode_route import ask, constants


def test_no_item_is_described_by_two_blocks():
    """decode_walks_kernel gives block b the items from b * group on and describes whole rounds of
    them: a group of a part of a round would reach into the next block's items."""
    c = constants()
    most = c["kPlanBlocks"] * c["kPlanThreads"]
    rng = random.Random(0)
    items = [1, most - 1, most, most + 1, 2 ** 31 - 1] + [int(2 ** rng.uniform(0, 31)) for _ in range(500)]
    lines = [(n, 1 << k) for n in items for k in range(5)]
    for (n, lanes), (group,) in zip(lines, ask(lines)):
        assert -(-n // group) <= most
        assert group == 1 if n <= most else group % (c["kWalkThreads"] // lanes) == 0
