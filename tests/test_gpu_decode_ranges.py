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


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("wide", [False, True])
def test_tiny_queries_over_large_keys(wide, fmt):
    """Queries down to bf16's smallest numbers over keys up to its largest: scores near one, which
    fp32 holds as well as those of ordinary sizes."""
    rng = np.random.default_rng(41)
    e = 120 if fmt == "e4m3" else 124
    table, pages = tables(rng, [300], 16)
    pair = Pair(pages, 1, 16, 64, fmt)
    k = f64(bf16(normal(rng, 300, 1, 64) * 2.0 ** e))
    pair.write(k, normal(rng, 300, 1, 64), table, [0], [0, 300])
    # the smallest step of bf16 is 2^-133: as few as six bits are left of these
    q = f64(bf16(normal(rng, 6, 2, 64) * 2.0 ** -np.array([96, 100, 110, 118, 122, 127])[:, None, None]))
    pos, seq = [299, 298, 200, 17, 15, 3], [0] * 6
    dev_table = widened(table, 6) if wide else table
    for pats in (DENSE, SPREAD):
        out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(dev_table), i32(pos), pats, seq=i32(seq))
        torch.cuda.synchronize()
        assert dilattn.device_error() == 0
        check_decode((out, lse), ref.decode(q, pair.ref, table, pos, seq, pats), q, pair)
