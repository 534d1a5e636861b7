"""The cache tests' float64 model against independent statements of the same things, on the CPU."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import oracle
from sparse_long_sequence_dilated_b200.workloads import e4m3_values


def test_rounding_matches_the_format_tables():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000)])
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_to_format(y.astype(np.float32).astype(np.float64), "e4m3"), want)
    vals = np.unique(e4m3_values()[np.isfinite(e4m3_values())])
    assert np.array_equal(ref.round_to_format(vals, "e4m3"), vals)
    mid = (vals[1:] + vals[:-1]) / 2  # ties go to one of the neighbours whose code is even
    got = ref.round_to_format(mid, "e4m3")
    assert np.array_equal(got, torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_least_that_holds(fmt):
    for a in (0.0, 1e-40, 1e-6, 0.99, 1.0, ref.TOP[fmt], ref.TOP[fmt] * 1.01, 3e38):
        s = ref.block_scale(a, fmt)
        assert a <= ref.TOP[fmt] * s and (s == 2.0 ** -126 or a > ref.TOP[fmt] * s / 2)


@pytest.mark.parametrize("pats", [((100, 1),), ((16, 1), (32, 2), (100, 4)), ((30, 4), (50, 7))])
def test_decode_is_a_row_of_the_whole_sequence_forward(pats):
    rng = np.random.default_rng(1)
    N, H, Hkv, d, P = 70, 4, 2, 64, 16
    c = ref.Cache(5, Hkv, P, d, "int8")
    k, v = rng.standard_normal((N, Hkv, d)), rng.standard_normal((N, Hkv, d))
    table = [[3, 1, 4, 0, 2]]
    c.write(k, v, table, [0], [0, N])
    kk, vv = c.read(table, [0], [0, N])
    q = rng.standard_normal((N, H, d))
    got, lse, _ = ref.decode(q, c, table, np.arange(N), np.zeros(N, int), pats)
    rep = lambda a: np.repeat(a, H // Hkv, axis=1)[None]
    want, wl = oracle.fwd(q[None], rep(kk), rep(vv), list(pats), True)
    assert np.allclose(got, want[0], atol=1e-12)
    fin = np.isfinite(wl[0].T)
    assert np.array_equal(np.isfinite(lse), fin) and np.allclose(lse[fin], wl[0].T[fin], atol=1e-12)


def test_appends_equal_one_write_where_the_scale_does_not_grow():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((40, 2, 64))
    x[0, :, 0] = x[16, :, 0] = x[32, :, 0] = 7.0  # each page's largest comes first
    a, b = ref.Cache(3, 2, 16, 64, "e4m3"), ref.Cache(3, 2, 16, 64, "e4m3")
    table = [[2, 0, 1]]
    a.write(x, x, table, [0], [0, 40])
    for t in range(40):
        b.write(x[t:t + 1], x[t:t + 1], table, [t])
    assert np.array_equal(a.codes, b.codes) and np.array_equal(a.scale, b.scale)
