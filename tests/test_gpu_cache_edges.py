"""Writes whose positions lie partly outside the table, against the float64 model."""
import numpy as np
import pytest

from cache_util import bf16, f64, filled, i32, normal
from sparse_long_sequence_dilated_b200 import dilattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,P", [(64, 16), (128, 32), (128, 128)])
@pytest.mark.parametrize("few", [True, False])
def test_a_stretch_that_reaches_out_of_the_table(few, d, P, fmt):
    """Positions below zero and past the table are skipped and reported, one by one: those of the
    same sequence that the table holds are written, as they are read."""
    rng = np.random.default_rng(P + few)
    held = 2 * P
    pair, table = filled(rng, [held] * 5, 2, P, d, fmt)
    if few:  # eight tokens a sequence at most, on average
        start, n = [-1, held - 1, -3, 2 ** 31 - 1, -2 ** 31], [3, 2, 9, 4, 2]
    else:
        start, n = [-2, held - 2, -P - 4, 2 ** 31 - 3, -2 ** 31], [P + 5, P + 9, P + 14, 70, 60]
    offsets = np.concatenate([[0], np.cumsum(n)])
    k, v = normal(rng, offsets[-1], 2, d) * 9, normal(rng, offsets[-1], 2, d)
    assert (offsets[-1] <= 8 * len(n)) == few
    dilattn.cache_write(pair.dev, bf16(k).cuda(), bf16(v).cuda(), i32(table), i32(start), i32(offsets))
    assert dilattn.device_error() == 4
    k, v = f64(bf16(k)), f64(bf16(v))
    for b in range(len(n)):
        lo, hi = max(start[b], 0), min(start[b] + n[b], held)
        if lo < hi:
            t = offsets[b] + lo - start[b]
            pair.ref.write(k[t:t + hi - lo], v[t:t + hi - lo], table[b:b + 1], [lo], [0, hi - lo])
    pair.check()
    kk, vv = dilattn.cache_read(pair.dev, i32(table), i32(start), i32(offsets), int(offsets[-1]))
    assert dilattn.device_error() == 4
    for z, got in enumerate((f64(kk), f64(vv))):
        for b in range(len(n)):
            x = np.arange(n[b]) + start[b]
            ok = (x >= 0) & (x < held)
            part = got[offsets[b]:offsets[b + 1]]
            assert (part[~ok] == 0).all()
            assert np.array_equal(part[ok], pair.ref.rows(z, table[b], x[ok]))
