"""Dilated attention of single tokens over the 8-bit cache, against the float64 model and
against the full-sequence forward."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_util import Pair, bf16, check_decode, f64, filled, i32, normal, tables
from sparse_long_sequence_dilated_b200 import dilattn

pytestmark = pytest.mark.gpu

PATS = {
    "dense": [(1 << 20, 1)],
    "nested": [(64, 1), (128, 2), (256, 4), (512, 8)],
    "uneven": [(50, 1), (128, 3), (200, 6), (333, 4)],    # w not a multiple of r, r of no other
    "no_r1": [(60, 2), (100, 3), (400, 12)],              # some tokens are kept by no pattern
    "twice": [(96, 2), (300, 1), (96, 1), (300, 1)],      # repeated and unsorted
    "far": [(40, 64), (7, 9)],                            # offsets past a segment's end
}


def run(pair, table, q, pos, pats, seq=None, **kw):
    seq = np.arange(len(pos)) if seq is None else np.asarray(seq)
    got = dilattn.decode(bf16(q).cuda(), pair.dev, i32(table), i32(pos), pats, seq=i32(seq), **kw)
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    return got, ref.decode(q, pair.ref, table, pos, seq, pats)


@pytest.mark.parametrize("copies", [1, 7])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2), (4, 1), (7, 1), (13, 1)])
@pytest.mark.parametrize("pats", sorted(PATS))
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_few_tokens_and_many(copies, H, Hkv, pats, fmt, d):
    """The same tokens few at a time (a cluster for each token and KV head) and seven times over
    (ranges of the whole call's tiles): every copy has the token's result."""
    rng = np.random.default_rng(d + H)
    lens = [1, 40, 333, 1900]
    pair, table = filled(rng, lens, Hkv, 16, d, fmt, spread=3)
    pos, seq = [0, 39, 332, 1899, 1030, -1], [0, 1, 2, 3, 3, 0]
    q = normal(rng, len(pos), H, d)
    want = ref.decode(q, pair.ref, table, pos, seq, PATS[pats])
    out, lse = dilattn.decode(bf16(np.tile(q, (copies, 1, 1))).cuda(), pair.dev, i32(table), i32(pos * copies),
                              PATS[pats], seq=i32(seq * copies))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    n = len(pos)
    for k in range(copies):
        check_decode((out[k * n:(k + 1) * n], lse[k * n:(k + 1) * n]), want, q, pair)


@pytest.mark.parametrize("pats", sorted(PATS))
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_patterns(pats, fmt, d):
    rng = np.random.default_rng(d)
    lens = [1, 2, 17, 333, 700]
    pair, table = filled(rng, lens, 2, 32, d, fmt, spread=3)
    pos = [0, 1, 16, 332, 699, 50, 511, 128, -1]
    seq = [0, 1, 2, 3, 4, 4, 4, 3, 0]
    q = normal(rng, len(pos), 4, d)
    got, want = run(pair, table, q, pos, PATS[pats], seq)
    check_decode(got, want, q, pair)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 5), (6, 2), (8, 1), (14, 2), (9, 1), (16, 1), (20, 1), (40, 1), (33, 3)])
@pytest.mark.parametrize("pats", ["dense", "nested"])
def test_head_layouts(H, Hkv, pats):
    rng = np.random.default_rng(H)
    pair, table = filled(rng, [130, 301], Hkv, 16, 64, "int8")
    q = normal(rng, 4, H, 64)
    got, want = run(pair, table, q, [129, 300, 100, 16], PATS[pats], [0, 1, 1, 0])
    check_decode(got, want, q, pair)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_drafted_tokens(G, d, fmt):
    """More tokens than sequences under dense attention: drafts in order, and tokens of any sequence
    and position in any order, the same one twice, with empty slots between."""
    rng = np.random.default_rng(G + d)
    lens, Hkv = [900, 40, 3, 1, 66], 2
    pair, table = filled(rng, lens, Hkv, 16, d, fmt, spread=3)
    wide = np.full((len(lens), 1200), -1)  # a table for contexts that no team of blocks would be given
    wide[:, :table.shape[1]] = table
    drafts = [(b, n - 1 - k) for b, n in enumerate(lens) for k in range(min(n, 5) - 1, -1, -1)]
    mixed = [(int(b), int(rng.integers(0, lens[b]))) for b in rng.integers(0, len(lens), 21)]
    for tokens in (drafts, drafts + [(0, -1)] * 3, mixed + [(1, -1)] + mixed[:2] + [(4, -1), (0, 899)]):
        seq, pos = [t[0] for t in tokens], [t[1] for t in tokens]
        q = normal(rng, len(tokens), G * Hkv, d)
        got, want = run(pair, wide, q, pos, PATS["dense"], seq)
        check_decode(got, want, q, pair)
    # segments end inside the sequences: tokens of one need not share rows
    seq, pos = [t[0] for t in drafts] * 8, [t[1] for t in drafts] * 8
    q = normal(rng, len(seq), G * Hkv, d)
    for w in (600, 64, 3):
        got, want = run(pair, wide, q, pos, [(w, 1)], seq)
        check_decode(got, want, q, pair)
    # a sequence that there is not, and a position past the table, among drafts
    seq, pos = [0, 9, 0, 0, 1, 1], [5, 5, 2 ** 31 - 1, 7, 2, 39]
    q = normal(rng, 6, G * Hkv, d)
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(wide), i32(pos), PATS["dense"], seq=i32(seq))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 4
    ok = [0, 3, 4, 5]
    want = ref.decode(q[ok], pair.ref, table, [pos[i] for i in ok], [seq[i] for i in ok], PATS["dense"])
    check_decode((out[ok], lse[ok]), want, q[ok], pair)
    assert (f64(out[1:3]) == 0).all() and torch.isneginf(lse[1:3]).all()


def test_the_largest_patterns():
    """Segment lengths and dilations up to the largest int: each keeps one row of one head at most."""
    rng = np.random.default_rng(24)
    top = 2 ** 31 - 1
    pair, table = filled(rng, [40], 1, 16, 64, "int8")
    q = normal(rng, 4, 5, 64)
    for pats in ([(top, top)], [(top, top), (top, 1)], [(1, top), (3, top - 1), (8, 2)]):
        got, want = run(pair, table, q, [0, 1, 3, 39], pats, [0] * 4)
        check_decode(got, want, q, pair)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_every_short_length(P, d):
    """Positions around tile and page ends, each token in its own sequence."""
    rng = np.random.default_rng(P)
    lens = [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257]
    pair, table = filled(rng, lens, 1, P, d, "e4m3")
    q = normal(rng, len(lens), 2, d)
    for pats in (PATS["dense"], [(1 << 20, 3), (1 << 20, 2)]):
        got, want = run(pair, table, q, [n - 1 for n in lens], pats)
        check_decode(got, want, q, pair)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_long_rows_are_split(fmt):
    rng = np.random.default_rng(11)
    pair, table = filled(rng, [20000, 3], 1, 64, 64, fmt)
    q = normal(rng, 2, 8, 64)
    for pats in (PATS["dense"], [(2048, 1), (4096, 2), (8192, 4), (16384, 8), (32768, 16)]):
        got, want = run(pair, table, q, [19999, 2], pats)
        check_decode(got, want, q, pair)


def test_many_short_tokens():
    """More items than any launch has blocks, most of them short."""
    rng = np.random.default_rng(12)
    lens = list(rng.integers(1, 60, 150)) + [900]
    pair, table = filled(rng, lens, 4, 16, 64, "int8")
    T = 600
    seq = rng.integers(0, len(lens), T)
    pos = np.array([rng.integers(-1, lens[s]) for s in seq])
    q = normal(rng, T, 8, 64)
    for pats in (PATS["dense"], [(32, 1), (64, 2)]):
        got, want = run(pair, table, q, pos, pats, seq)
        check_decode(got, want, q, pair)


@pytest.mark.parametrize("T,H,Hkv,pats", [
    (1400, 8, 4, "dense"),                        # a token of each of 1400 sequences
    (1100, 8, 4, [(1000, 1), (1000, 2)]),
    (4200, 8, 8, "dense"),                        # tokens of some of them together
])
def test_more_items_than_the_plan_describes_at_once(T, H, Hkv, pats):
    rng = np.random.default_rng(25)
    lens = list(rng.integers(1, 30, 1399)) + [700]  # the long one keeps the table wide
    pair, table = filled(rng, lens, Hkv, 16, 64, "int8")
    seq = np.arange(T) if T <= len(lens) else np.sort(rng.integers(0, len(lens), T))
    pos = np.array([rng.integers(-1, lens[s]) for s in seq])
    pos[-1] = lens[seq[-1]] - 1
    q = normal(rng, T, H, 64)
    pats = PATS["dense"] if pats == "dense" else pats
    got, want = run(pair, table, q, pos, pats, seq)
    check_decode(got, want, q, pair)


def test_sharp_and_flat_softmax():
    """Queries whose scores differ by hundreds, and zero queries (the mean of the rows)."""
    rng = np.random.default_rng(13)
    pair, table = filled(rng, [3000], 1, 64, 128, "e4m3")
    q = normal(rng, 3, 4, 128)
    q[0] *= 16
    q[1] = 0
    q[2] *= 2.0 ** -130
    got, want = run(pair, table, q, [2999] * 3, PATS["dense"], [0] * 3)
    check_decode(got, want, q, pair)


def test_pages_of_very_different_sizes():
    """V pages 2^60 apart: the rows that matter are those whose weight times size is largest."""
    rng = np.random.default_rng(14)
    table, pages = tables(rng, [48], 16)
    pair = Pair(pages, 1, 16, 64, "e4m3")
    k, v = normal(rng, 48, 1, 64), normal(rng, 48, 1, 64)
    v[:16] *= 2.0 ** -30
    v[16:32] *= 2.0 ** 30
    pair.write(k, v, table, [0], [0, 48])
    q = normal(rng, 3, 2, 64)
    got, want = run(pair, table, q, [47, 31, 15], PATS["dense"], [0] * 3)
    check_decode(got, want, q, pair)


def test_nan_reaches_only_the_heads_that_attend_it():
    rng = np.random.default_rng(15)
    pair, table = filled(rng, [64, 64], 1, 16, 64, "e4m3")
    k, v = normal(rng, 1, 1, 64), normal(rng, 1, 1, 64)
    pair.write(np.full_like(k, np.nan), v, table, [3, 999], [0, 1, 1])    # K of page 0, sequence 0
    pair.write(k, np.full_like(v, np.inf), table, [999, 20], [0, 0, 1])   # V of page 1, sequence 1
    q = normal(rng, 4, 2, 64)
    # pattern (64, 2): position 62 and head 0, or 63 and head 1; (16, 1) sees the last page alone
    pats = [(16, 1), (64, 2)]
    pos, seq = [62, 63, 62, 63], [0, 0, 1, 1]
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(table), i32(pos), pats, seq=i32(seq))
    out, lse = f64(out), f64(lse)
    for i in range(4):
        hit = i % 2
        assert np.isnan(out[i, hit]).all() and np.isfinite(out[i, 1 - hit]).all()
        assert np.isnan(lse[i, hit]) == (i < 2) and np.isfinite(lse[i, 1 - hit])
    with np.errstate(invalid="ignore"):
        wo, wl, sp = ref.decode(q, pair.ref, table, pos, seq, pats)
    ok = np.array([[False, True], [True, False]] * 2)
    assert (np.abs(out[ok] - wo[ok]) <= 2.0 ** -8 * np.abs(wo[ok]) + 2.0 ** -10 * sp[ok]).all()


def test_nan_queries():
    rng = np.random.default_rng(16)
    pair, table = filled(rng, [64], 1, 16, 64, "int8")
    q = normal(rng, 2, 3, 64)
    q[0, 1, 5], q[1, 0, 0] = np.nan, np.inf
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(table), i32([63, 10]), PATS["dense"], seq=i32([0, 0]))
    bad = np.zeros((2, 3), bool)
    bad[0, 1] = bad[1, 0] = True
    assert np.array_equal(np.isnan(f64(lse)), bad) and np.array_equal(np.isnan(f64(out)).all(-1), bad)
    assert np.array_equal(np.isnan(f64(out)).any(-1), bad)


def test_codes_behind_the_last_token_are_not_read():
    """Garbage (NaN codes, NaN scales) in rows and pages past the token changes nothing."""
    rng = np.random.default_rng(17)
    pair, table = filled(rng, [37], 2, 16, 64, "e4m3")
    q = normal(rng, 1, 4, 64)
    args = bf16(q).cuda(), pair.dev, i32(table), i32([36]), PATS["nested"]
    want = [t.clone() for t in dilattn.decode(*args)]
    used = table[0, :3]
    for c, s in ((pair.dev.k, pair.dev.k_scale), (pair.dev.v, pair.dev.v_scale)):
        raw = c.view(torch.uint8)
        keep = raw[used.tolist()].clone()
        raw.fill_(0x7f)
        raw[used.tolist()] = keep
        raw[used[2], :, 5:] = 0xff
        for p in range(len(s)):
            if p not in used:
                s[p] = float("nan")
    for a, b in zip(dilattn.decode(*args), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,pats,wide", [(3, "dense", False), (300, "dense", False), (3, "nested", False), (300, "dense", True),
                                         (3, "dense", True), (300, "nested", True), (300, "uneven", True)])
@pytest.mark.parametrize("H", [2, 8, 16, 32])
def test_empty_slots_over_a_cache_that_holds_nothing(T, pats, wide, H):
    """Codes and scales that nothing has written (NaN all of them) do not reach slots without rows,
    nor a token whose pages are elsewhere."""
    cache = dilattn.new_cache(40, 2, 16, 64, "e4m3")
    for t in cache:
        t.view(torch.uint8).fill_(0xff)
    table = np.full((2, 1200 if wide else 4), -1)
    q = bf16(np.random.default_rng(26).standard_normal((T, H, 64))).cuda()
    pats = [(30000, 1), (30000, 2)] if pats == "nested" and wide else PATS[pats]
    out, lse = dilattn.decode(q, cache, i32(table), i32([-1] * T), pats, seq=i32([0] * T))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    assert (f64(out) == 0).all() and torch.isneginf(lse).all()
    # a token with one page of finite numbers, its other page missing
    one = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    table[1, 0] = 7
    dilattn.cache_write(cache, one, one, i32(table[1:]), i32([0]))
    out, lse = dilattn.decode(q, cache, i32(table), i32([0] + [-1] * (T - 1)), [(1 << 20, 1)], seq=i32([1] + [0] * (T - 1)))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    assert (f64(out[0]) == 1).all() and torch.isfinite(lse[0]).all()
    assert (f64(out[1:]) == 0).all() and torch.isneginf(lse[1:]).all()
    out, lse = dilattn.decode(q, cache, i32(table), i32([20] * T), [(4, 1)], seq=i32([1] * T))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 4
    assert (f64(out) == 0).all() and torch.isneginf(lse).all()


def test_pages_and_positions_out_of_range_are_skipped_and_reported():
    rng = np.random.default_rng(18)
    pair, table = filled(rng, [48, 48], 1, 16, 64, "int8")
    q = normal(rng, 2, 2, 64)
    dq = bf16(q).cuda()
    pages = pair.ref.codes.shape[1]
    # a position past the table, a sequence that there is not: empty slots
    for pos, seq in (([48, 10], [0, 1]), ([2 ** 31 - 1, 10], [0, 1]), ([5, 10], [2, 1]), ([5, 10], [-1, 1])):
        out, lse = dilattn.decode(dq, pair.dev, i32(table), i32(pos), PATS["dense"], seq=i32(seq))
        assert dilattn.device_error() == 4
        assert (f64(out[0]) == 0).all() and torch.isneginf(lse[0]).all()
        wo, wl, sp = ref.decode(q[1:], pair.ref, table, [10], [1], PATS["dense"])
        check_decode((out[1:], lse[1:]), (wo, wl, sp), q[1:], pair)
    # a page that there is not: its rows are left out
    for page in (pages, -1, 2 ** 31 - 1, -2 ** 31):
        bad = table.copy()
        bad[0, 1] = page
        out, lse = dilattn.decode(dq, pair.dev, i32(bad), i32([47, 47]), PATS["dense"])
        assert dilattn.device_error() == 4
        short = np.delete(table[:1], 1, axis=1)  # the sequence without that page
        wo, wl, sp = ref.decode(q[:1], pair.ref, short, [31], [0], PATS["dense"])
        check_decode((out[:1], lse[:1]), (wo, wl, sp), q[:1], pair)


def test_strided_queries_and_given_outputs():
    rng = np.random.default_rng(19)
    pair, table = filled(rng, [100, 90], 2, 16, 64, "int8")
    fused = bf16(normal(rng, 2, 8, 64)).cuda()
    q = fused[:, 2:6]
    out = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 4), device="cuda")
    ws = dilattn.decode_workspace(2, 4, 2, 64)
    ws.fill_(255)
    got = dilattn.decode(q, pair.dev, i32(table), i32([99, 89]), PATS["nested"], out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    check_decode(got, ref.decode(f64(q), pair.ref, table, [99, 89], [0, 1], PATS["nested"]), f64(q), pair)


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(20)
    pair, table = filled(rng, [5000, 700, 60], 2, 64, 128, "e4m3")
    args = bf16(normal(rng, 3, 8, 128)).cuda(), pair.dev, i32(table), i32([4999, 699, 59]), PATS["dense"]
    first = [t.clone() for t in dilattn.decode(*args)]
    for _ in range(10):
        for a, b in zip(dilattn.decode(*args), first):
            assert torch.equal(a, b)


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(21)
    pair, table = filled(rng, [9000, 8000], 2, 64, 64, "int8")
    dev_table = i32(table)
    calls, want = [], []
    for b, n in enumerate((8999, 7999)):
        q = bf16(normal(rng, 1, 8, 64)).cuda()
        calls.append((q, pair.dev, dev_table, i32([n]), PATS["dense"], i32([b])))
        want.append([t.clone() for t in dilattn.decode(*calls[-1])])
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[dilattn.decode(*c, stream=s) for c, s in zip(calls, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pairs in got:
        for g, w in zip(pairs, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_a_captured_step_of_a_padded_batch():
    """One decoding step (write, then attend) captured once and replayed along the sequences."""
    rng = np.random.default_rng(22)
    lens, H, Hkv, d = [100, 31, 0], 4, 2, 64
    pats = [(64, 1), (128, 2)]
    table, pages = tables(rng, [n + 10 for n in lens], 16)
    pair = Pair(pages, Hkv, 16, d, "e4m3")
    pair.write(normal(rng, 131, Hkv, d), normal(rng, 131, Hkv, d), table, [0, 0, 0], [0, 100, 131, 131])
    dev_table = i32(table)
    # four query slots; the batch fills three
    start, seq, pos = i32(lens), i32([0, 1, 2, 0]), i32(lens + [-1])
    k, v = (torch.zeros((3, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((4, H, d), dtype=torch.bfloat16, device="cuda")
    ws = dilattn.decode_workspace(4, H, Hkv, d)

    def step():
        dilattn.cache_write(pair.dev, k, v, dev_table, start)
        return dilattn.decode(q, pair.dev, dev_table, pos, pats, seq=seq, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = step()
    torch.cuda.current_stream().wait_stream(side)
    pair.ref.write(f64(k), f64(v), table, lens)
    for t in range(8):
        a, b, c = normal(rng, 3, Hkv, d), normal(rng, 3, Hkv, d), normal(rng, 4, H, d)
        at = [n + t for n in lens]
        k.copy_(bf16(a)), v.copy_(bf16(b)), q.copy_(bf16(c)), start.copy_(i32(at)), pos.copy_(i32(at + [-1]))
        g.replay()
        pair.ref.write(a, b, table, at)
        pair.check()
        check_decode(got, ref.decode(c, pair.ref, table, at + [-1], [0, 1, 2, 0], pats), c, pair)


@pytest.mark.parametrize("tokens", [2, 90])
def test_calls_on_forked_streams_in_one_graph(tokens):
    """K and V rows made on one stream, queries on another, joined before the write and the decode;
    two decodes side by side afterwards, with a workspace each; memory set and copied in between."""
    rng = np.random.default_rng(27)
    lens, H, Hkv, d = [70, 900], 4, 2, 64
    pair, table = filled(rng, lens, Hkv, 16, d, "int8")
    dev_table, start = i32(table), i32([69, 899])
    seq = i32(np.arange(tokens) % 2)
    pos = i32(np.where(np.arange(tokens) % 2, 899, 69))
    rows, q0 = normal(rng, 2, Hkv, d), normal(rng, tokens, H, d)
    src_rows, src_q = bf16(rows).cuda(), bf16(q0).cuda()
    rows_in, q_in = torch.empty_like(src_rows), torch.empty_like(src_q)
    ws = [dilattn.decode_workspace(tokens, H, Hkv, d) for _ in range(2)]
    main, other = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        cur = torch.cuda.current_stream()
        rows_in.zero_()
        other.wait_stream(cur)
        with torch.cuda.stream(other):
            q_in.copy_(src_q)
        rows_in.copy_(src_rows)
        cur.wait_stream(other)
        dilattn.cache_write(pair.dev, rows_in, rows_in, dev_table, start)
        other.wait_stream(cur)
        with torch.cuda.stream(other):
            b = dilattn.decode(q_in, pair.dev, dev_table, pos, PATS["nested"], seq=seq, workspace=ws[1])
        a = dilattn.decode(q_in, pair.dev, dev_table, pos, PATS["dense"], seq=seq, workspace=ws[0])
        cur.wait_stream(other)
        return a, b

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            got = step()
    torch.cuda.current_stream().wait_stream(main)
    for t in range(3):
        rows, q0 = normal(rng, 2, Hkv, d), normal(rng, tokens, H, d)
        src_rows.copy_(bf16(rows))
        src_q.copy_(bf16(q0))
        if t == 0:  # what the pass before the capture wrote
            first = f64(rows_in)
            pair.ref.write(first, first, table, [69, 899])
        g.replay()
        pair.ref.write(rows, rows, table, [69, 899])
        pair.check()
        for (out, lse), pats in zip(got, ("dense", "nested")):
            want = ref.decode(q0, pair.ref, table, f64(pos).astype(int), f64(seq).astype(int), PATS[pats])
            check_decode((out, lse), want, q0, pair)


@pytest.mark.parametrize("d", [64, 128])
def test_the_set_together_with_the_forward(d):
    """A prompt through the full-sequence forward and into the cache; the cache read back and run
    through the forward gives, row by row, what decoding gives at those positions."""
    rng = np.random.default_rng(23)
    N, H = 640, 4
    pats = [(128, 1), (256, 2), (640, 4)]
    table, pages = tables(rng, [N], 64)
    q, k, v = (bf16(normal(rng, 1, N, H, d)).cuda() for _ in range(3))
    cache = dilattn.new_cache(pages, H, 64, d, "int8")
    t, zero, offsets = i32(table), i32([0]), i32([0, N])
    dilattn.cache_write(cache, k[0], v[0], t, zero, offsets)
    kk, vv = dilattn.cache_read(cache, t, zero, offsets, N)
    out, lse = dilattn.fwd(q, kk[None], vv[None], pats)
    got, gl = dilattn.decode(q[0], cache, t, i32(np.arange(N)), pats, seq=i32(np.zeros(N)))
    # both round to bf16 (2^-8 of the value each); the forward also rounds its probabilities to bf16
    diff = np.abs(f64(got) - f64(out[0]))
    assert (diff <= 2.0 ** -7 * np.abs(f64(out[0])) + 2.0 ** -7).all(), diff.max()
    assert np.abs(f64(gl) - f64(lse[0].t())).max() <= 1e-3
