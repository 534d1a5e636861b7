"""Decoding where the tiles of all items are cut into ranges (plan, main kernel, join) and not
done in one launch: long tables, many items."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_util import Pair, bf16, check_decode, f64, filled, i32, normal, tables
from sparse_long_sequence_dilated_b200 import dilattn

pytestmark = pytest.mark.gpu

DENSE = [(1 << 20, 1)]
SPREAD = [(1 << 20, 2), (1 << 20, 3), (8192, 1)]  # r that do not divide one another


def widened(table, rows, columns=1200):
    """The table with unused rows and columns: contexts that no team of blocks would be given."""
    wide = np.full((rows, columns), -1)
    wide[:len(table), :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("pats", [DENSE, SPREAD], ids=["dense", "spread"])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_empty_slots_may_hold_anything(d, G, pats):
    """NaN and infinities in the queries of empty slots, of tokens without a page and of sequences
    that there are not: zeros and -infinity come out, and other tokens have their results."""
    rng = np.random.default_rng(G + d)
    pair, table = filled(rng, [300, 40], 1, 16, d, "int8")
    bad = np.array([np.nan, np.inf, -np.inf, np.nan])
    for T, B, of_seq in ((6, 6, False), (300, 300, False), (12, 2, True), (6, 6, True)):
        wide = widened(table, B)
        q = normal(rng, T, G, d)
        seq = np.arange(T) % B
        pos = np.full(T, -1)
        pos[:2] = 299, 39
        q[2:] = bad[rng.integers(0, 4, (T - 2, G, d))]
        q[3, :, 1:] = 1.0  # one number of a head is enough
        want = ref.decode(q[:2], pair.ref, table, pos[:2], seq[:2], pats)
        out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(wide), i32(pos), pats, seq=i32(seq) if of_seq else None)
        torch.cuda.synchronize()
        assert dilattn.device_error() == 0
        check_decode((out[:2], lse[:2]), want, q[:2], pair)
        assert (f64(out[2:]) == 0).all() and torch.isneginf(lse[2:]).all()
    # pages that there are not: no row is left
    wide = widened(table, 6)
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(wide), i32([299, 39, 5, 350, -1, 19199]), pats)
    torch.cuda.synchronize()
    assert dilattn.device_error() == 4
    check_decode((out[:2], lse[:2]), want, q[:2], pair)
    assert (f64(out[2:]) == 0).all() and torch.isneginf(lse[2:]).all()
