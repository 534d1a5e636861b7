"""Writing the 8-bit cache and reading it back, against the float64 model: codes and scales
are whole-number facts of the definition, so every comparison is exact."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_util import Pair, bf16, f64, filled, i32, normal, tables
from sparse_long_sequence_dilated_b200 import dilattn

pytestmark = pytest.mark.gpu

FMTS = ["e4m3", "int8"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_ragged_prompts_in_two_calls(fmt, d, P, Hkv):
    """Lengths from zero to several pages, then a second call that goes on mid-page with larger
    numbers, so that scales grow and codes are rounded again."""
    rng = np.random.default_rng(P + d)
    first, more = [0, 1, P - 1, P, P + 1, 3 * P + 5], [5, 0, 1, 2 * P, P - 1, 1]
    table, pages = tables(rng, [a + b for a, b in zip(first, more)], P)
    pair = Pair(pages, Hkv, P, d, fmt)
    for lens, start, size in ((first, [0] * 6, 1.0), (more, first, 100.0)):
        T = sum(lens)
        k = f64(bf16(normal(rng, T, Hkv, d) * size ** rng.uniform(-1, 1, (T, Hkv, 1))))
        v = f64(bf16(normal(rng, T, Hkv, d) * size ** rng.uniform(-1, 1, (T, Hkv, 1))))
        pair.write(k, v, table, start, np.concatenate([[0], np.cumsum(lens)]))
        pair.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(fmt, d):
    """One token a call for each of several sequences, growing and shrinking in size."""
    rng = np.random.default_rng(3)
    B, P, Hkv = 5, 16, 2
    table, pages = tables(rng, [40] * B, P)
    pair = Pair(pages, Hkv, P, d, fmt)
    start = np.array([0, 3, 7, 15, 16])
    pair.write(normal(rng, B * 8, Hkv, d), normal(rng, B * 8, Hkv, d), table, start, np.arange(B + 1) * 8)
    for t in range(12):
        size = 2.0 ** rng.integers(-6, 7, (B, Hkv, 1))
        pair.write(normal(rng, B, Hkv, d) * size, normal(rng, B, Hkv, d) / size, table, start + 8 + t)
        pair.check()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_call_that_goes_back(fmt):
    """Rewriting rows in the middle keeps the page's other rows, and row 0 starts a page afresh."""
    rng = np.random.default_rng(4)
    pair, table = filled(rng, [40, 30], 2, 16, 64, fmt)
    pair.write(normal(rng, 9, 2, 64) * 50, normal(rng, 9, 2, 64) * 0.01, table, [5, 20], [0, 6, 9])
    pair.check()
    pair.write(normal(rng, 3, 2, 64) * 0.01, normal(rng, 3, 2, 64) * 0.01, table, [16, 0], [0, 2, 3])
    pair.check()


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_numbers(fmt):
    """Zeros, the smallest and the largest bf16 numbers, and the formats' own edges."""
    Hkv, d, P = 1, 64, 16
    big = float(torch.finfo(torch.bfloat16).max)
    rows = [0.0, 2.0 ** -133, 2.0 ** -126, 1e-30, 1.0, ref.TOP[fmt], big]
    x = np.zeros((len(rows) * P, Hkv, d))
    for i, a in enumerate(rows):
        a = f64(bf16(np.array([a])))[0]
        x[i * P:(i + 1) * P] = a * np.linspace(-1, 1, 64)
        x[i * P, 0, 0] = a
    x = f64(bf16(x))
    table, pages = tables(np.random.default_rng(0), [len(x)], P)
    pair = Pair(pages, Hkv, P, d, fmt)
    pair.write(x, x[::-1].copy(), table, [0], [0, len(x)])
    pair.check()
    # a page of zeros grows from the smallest scale to the largest
    pair.write(x[-1:], x[:1], table, [3])
    pair.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_numbers_that_no_code_holds(fmt, bad):
    rng = np.random.default_rng(5)
    pair, table = filled(rng, [40], 2, 16, 64, fmt)
    k, v = normal(rng, 2, 2, 64), normal(rng, 2, 2, 64)
    k[1, 1, 63] = bad
    pair.write(k, v, table, [20], [0, 2])
    assert np.isnan(pair.ref.scale[0]).sum() == 1 and not np.isnan(pair.ref.scale[1]).any()
    pair.check()
    pair.write(normal(rng, 1, 2, 64), v[:1], table, [22])  # a NaN stays ...
    assert np.isnan(pair.ref.scale[0]).sum() == 1
    pair.check()
    got = dilattn.cache_read(pair.dev, i32(table), i32([0]), i32([0, 40]), 40)
    want = pair.ref.read(table, [0], [0, 40])
    for g, w in zip(got, want):
        assert np.array_equal(f64(g), w, equal_nan=True)
    pair.write(normal(rng, 1, 2, 64), v[:1], table, [16])  # ... until row 0 is written
    assert not np.isnan(pair.ref.scale[0]).any()
    pair.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 128])
def test_read_back(fmt, d, P):
    rng = np.random.default_rng(6)
    lens = [200, 1, 77, 300]
    pair, table = filled(rng, lens, 3, P, d, fmt, spread=4)
    start, n = [17, 0, 76, 0], [150, 1, 0, 300]
    offsets = np.concatenate([[0], np.cumsum(n)])
    total = int(offsets[-1]) + 7  # rows behind the last sequence stay as they are
    k = torch.full((total, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    dilattn.cache_read(pair.dev, i32(table), i32(start), i32(offsets), total, k=k, v=v)
    want = pair.ref.read(table, start, offsets)
    for got, w in zip((k, v), want):
        assert np.array_equal(f64(got)[:-7], w)
        assert (f64(got)[-7:] == 7).all()
    # one token of each sequence
    k, v = dilattn.cache_read(pair.dev, i32(table), i32([5, 0, 76, 299]))
    want = pair.ref.read(table, [5, 0, 76, 299], [0, 1, 2, 3, 4])
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    assert dilattn.device_error() == 0


def test_strided_rows_and_rows_behind_the_last_sequence():
    """k and v as slices of a fused projection, with unused rows at the end (NaN: never read);
    reading back into the slices leaves what is between them."""
    rng = np.random.default_rng(7)
    table, pages = tables(rng, [20, 30], 16)
    pair = Pair(pages, 2, 16, 64, "e4m3")
    fused = torch.full((53, 6, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = normal(rng, 50, 2, 64), normal(rng, 50, 2, 64)
    fused[:50, 2:4], fused[:50, 4:6] = bf16(k).cuda(), bf16(v).cuda()
    dilattn.cache_write(pair.dev, fused[:, 2:4], fused[:, 4:6], i32(table), i32([0, 0]), i32([0, 20, 50]))
    pair.ref.write(k, v, table, [0, 0], [0, 20, 50])
    pair.check()
    fused.fill_(3.0)
    dilattn.cache_read(pair.dev, i32(table), i32([0, 0]), i32([0, 20, 50]), 53, k=fused[:, :2], v=fused[:, 4:])
    want = pair.ref.read(table, [0, 0], [0, 20, 50])
    assert np.array_equal(f64(fused[:50, :2]), want[0]) and np.array_equal(f64(fused[:50, 4:]), want[1])
    assert (f64(fused[50:]) == 3).all() and (f64(fused[:, 2:4]) == 3).all()


def test_positions_and_pages_out_of_range_are_skipped_and_reported():
    """Every bad index is one that the kernels check: nothing else is touched, and the error
    word says so."""
    rng = np.random.default_rng(8)
    pair, table = filled(rng, [32, 32], 1, 16, 64, "int8")
    before = [t.view(torch.uint8).clone() for t in (pair.dev.k, pair.dev.v)]
    x = bf16(normal(rng, 2, 1, 64)).cuda()
    pages = pair.ref.codes.shape[1]
    for bad, start in ((table, [-1, 32]), (table, [32, 2 ** 31 - 1]),
                       (np.array([[0, pages], [-1, 2 ** 31 - 1]]), [16, 0]),
                       (np.array([[0, -2 ** 31], [pages + 5, 0]]), [31, 15])):
        dilattn.cache_write(pair.dev, x, x, i32(bad), i32(start))
        assert dilattn.device_error() == 4
        k, v = dilattn.cache_read(pair.dev, i32(bad), i32(start))
        assert dilattn.device_error() == 4
        assert (f64(k) == 0).all() and (f64(v) == 0).all()
        for t, b in zip((pair.dev.k, pair.dev.v), before):
            assert torch.equal(t.view(torch.uint8), b)
    pair.check()


def test_on_another_stream_and_in_a_graph():
    """Write and read captured once, replayed with other positions and numbers."""
    rng = np.random.default_rng(9)
    pair, table = filled(rng, [20, 40], 2, 32, 128, "e4m3")
    dev_table, start = i32(table), i32([20, 10])
    k, v = (torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dilattn.cache_write(pair.dev, k, v, dev_table, start)
        pair.ref.write(f64(k), f64(v), table, [20, 10])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            dilattn.cache_write(pair.dev, k, v, dev_table, start)
            rk, rv = dilattn.cache_read(pair.dev, dev_table, start)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(3):
        a, b = normal(rng, 2, 2, 128) * 4 ** t, normal(rng, 2, 2, 128)
        k.copy_(bf16(a)), v.copy_(bf16(b)), start.copy_(i32([20 + t, 31 + t]))
        g.replay()
        pair.ref.write(a, b, table, [20 + t, 31 + t])
        pair.check()
        want = pair.ref.read(table, [20 + t, 31 + t], [0, 1, 2])
        assert np.array_equal(f64(rk), want[0]) and np.array_equal(f64(rv), want[1])


def test_a_cache_past_32_bits():
    """Pages whose bytes lie past 2^32, the last of them among them."""
    P, Hkv, d = 128, 32, 128
    pages = (1 << 32) // (P * Hkv * d) + 5
    dev = dilattn.new_cache(pages, Hkv, P, d, "int8")
    rng = np.random.default_rng(10)
    small = ref.Cache(2, Hkv, P, d, "int8")
    x, y = normal(rng, 2, Hkv, d), normal(rng, 2, Hkv, d)
    table = np.array([[pages - 1], [pages - 3]])
    dilattn.cache_write(dev, bf16(x).cuda(), bf16(y).cuda(), i32(table), i32([0, 127]))
    small.scale[:] = 1
    small.write(x, y, [[0], [1]], [0, 127])
    ids = [pages - 1, pages - 3]
    for z, (c, s) in enumerate(((dev.k, dev.k_scale), (dev.v, dev.v_scale))):
        assert np.array_equal(f64(c[ids]), small.codes[z]) and np.array_equal(f64(s[ids]), small.scale[z])
    k, v = dilattn.cache_read(dev, i32(table), i32([0, 127]))
    want = small.read([[0], [1]], [0, 127], [0, 1, 2])
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    assert dilattn.device_error() == 0
