"""Decoding where the tiles of all items are cut into ranges (plan, main kernel, join) and not
done in one launch: long tables, many items. That the calls of CASES go this way is tested on the
CPU (test_decode_route_host.py)."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_util import Pair, bf16, check_decode, f64, filled, i32, normal, tables
from decode_route import CASES, DENSE, PATS, case
from sparse_long_sequence_dilated_b200 import dilattn

pytestmark = pytest.mark.gpu

SPREAD = PATS["spread"]


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


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", case("few") + case("many") + case("team"))
def test_walks_cut_into_ranges(name, fmt):
    """Tokens few at a time, their items cut into some thirty ranges each, and so often that no team
    takes them: every copy has the token's result."""
    c = CASES[name]
    rng = np.random.default_rng(c["d"] + c["H"])
    pair, table = filled(rng, [1, 40, 333, 1900], c["Hkv"], 16, c["d"], fmt, spread=3)
    pos, seq = [0, 39, 332, 1899, 1030, -1, 777], [0, 1, 2, 3, 3, 0, 3]
    q = normal(rng, 7, c["H"], c["d"])
    n = c["T"] // 7
    out, lse = dilattn.decode(bf16(np.tile(q, (n, 1, 1))).cuda(), pair.dev, i32(widened(table, c["B"])), i32(pos * n),
                              c["pats"], seq=i32(seq * n))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    want = ref.decode(q, pair.ref, table, pos, seq, c["pats"])
    check_decode((out, lse), [np.tile(x, (n,) + (1,) * (x.ndim - 1)) for x in want], np.tile(q, (n, 1, 1)), pair)


@pytest.mark.parametrize("name", case("long"))
def test_items_of_many_partials(name):
    """One token's walks over more than a thousand ranges, alone and among hundreds of short ones,
    where another has some three hundred."""
    c = CASES[name]
    rng = np.random.default_rng(43)
    fmt = "e4m3" if c["d"] == 64 else "int8"
    lens = [70000, 3]
    if name.startswith("long_among"):
        lens = list(rng.integers(1, 60, 320))
        lens[200], lens[7] = 40000, 20000
    pair, table = filled(rng, lens, 1, 64, c["d"], fmt)
    assert table.shape == (c["B"], c["longest"] // 64)
    pos = np.array(lens) - 1
    q = normal(rng, len(lens), c["H"], c["d"])
    args = bf16(q).cuda(), pair.dev, i32(table), i32(pos), c["pats"]
    out, lse = dilattn.decode(*args)
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    check_decode((out, lse), ref.decode(q, pair.ref, table, pos, np.arange(len(lens)), c["pats"]), q, pair)
    for a, b in zip(dilattn.decode(*args), (out, lse)):
        assert torch.equal(a, b)


LENS, H, HKV = [1900, 333, 40], 8, 2


class Again:
    """The calls of the "again" cases over one cache."""

    def __init__(self, d, fmt, seed=44):
        self.rng, self.d = np.random.default_rng(seed), d
        self.pair, self.table = filled(self.rng, LENS, HKV, 16, d, fmt, spread=2)
        self.wide = i32(widened(self.table, 3))

    def workspace(self):
        return dilattn.decode_workspace(200, H, HKV, self.d)

    def tokens(self, T):
        seq = np.sort(self.rng.integers(0, 3, T))
        pos = np.array([self.rng.integers(-1 if T > 3 else 0, LENS[b]) for b in seq])
        return normal(self.rng, T, H, self.d), seq, pos

    def inputs(self, name):
        q, seq, pos = self.tokens(CASES[name]["T"])
        return dict(q=bf16(q).cuda(), seq=i32(seq), pos=i32(pos), pats=CASES[name]["pats"])

    def call(self, x, ws=None, **kw):
        return dilattn.decode(x["q"], self.pair.dev, self.wide, x["pos"], x["pats"], seq=x["seq"], workspace=ws, **kw)

    def check(self, x, got):
        q, seq, pos = f64(x["q"]), f64(x["seq"]).astype(int), f64(x["pos"]).astype(int)
        check_decode(got, ref.decode(q, self.pair.ref, self.table, pos, seq, x["pats"]), q, self.pair)


def names_again(d):
    return [n for n in case("again") if CASES[n]["d"] == d]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", case("again"))
def test_the_same_bits_whatever_the_workspace_holds(name, fmt):
    a = Again(CASES[name]["d"], fmt)
    x, ws = a.inputs(name), a.workspace()
    ws.fill_(255)
    first = [t.clone() for t in a.call(x, ws)]
    a.check(x, first)
    for fill in (lambda: ws.zero_(), lambda: ws.random_(0, 256), lambda: ws, lambda: ws.fill_(0x7f), lambda: ws):
        fill()
        for t, f in zip(a.call(x, ws), first):
            assert torch.equal(t, f)
    assert dilattn.device_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_one_workspace_from_call_to_call_in_a_graph(d, fmt):
    """Calls of every kind one behind the other on one workspace, captured once and replayed over
    other tokens: each launch begins while the one before it still runs."""
    a = Again(d, fmt)
    names = names_again(d)
    names = names + names[::-1]
    xs, ws = [a.inputs(n) for n in names], a.workspace()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for x in xs:
            a.call(x, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = [a.call(x, ws) for x in xs]
    torch.cuda.current_stream().wait_stream(stream)
    for t in range(3):
        for n, x in zip(names, xs):
            for k, v in a.inputs(n).items():
                if k != "pats":
                    x[k].copy_(v)
        torch.cuda.synchronize()
        for _ in range(4):
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, got):
            for p, r in zip(y, a.call(x)):
                assert torch.equal(p, r)
        if t == 0:
            for x, y in zip(xs[:len(xs) // 2], got):
                a.check(x, y)
    assert dilattn.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_two_streams_with_a_workspace_each_in_ranges(d):
    """Calls that run at the same time, each chain of launches on a stream and workspace of its own."""
    a = Again(d, "int8")
    names = names_again(d)
    xs = [a.inputs(n) for n in names]
    want = [[t.clone() for t in a.call(x)] for x in xs]
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [a.workspace() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(8):
        for i in range(len(xs)):
            for s in range(2):  # the second stream takes the calls the other way round
                j = i if s == 0 else len(xs) - 1 - i
                got.append((j, a.call(xs[j], ws[s], stream=streams[s])))
    torch.cuda.synchronize()
    for j, y in got:
        for p, r in zip(y, want[j]):
            assert torch.equal(p, r)
    for x, y in zip(xs, want):
        a.check(x, y)
    assert dilattn.device_error() == 0


@pytest.mark.parametrize("pats", [DENSE, SPREAD], ids=["dense", "spread"])
def test_a_captured_step_in_ranges(pats):
    """Write, then attend, captured once and replayed along the sequences, with a padded slot."""
    rng, d = np.random.default_rng(45), 64
    lens = [1000, 331, 0]
    table, pages = tables(rng, [n + 10 for n in lens], 16)
    pair = Pair(pages, HKV, 16, d, "e4m3")
    n = sum(lens)
    pair.write(normal(rng, n, HKV, d), normal(rng, n, HKV, d), table, [0, 0, 0], np.concatenate([[0], np.cumsum(lens)]))
    wide = i32(widened(table, 3))
    start, seq, pos = i32(lens), i32([0, 1, 2, 0]), i32(lens + [-1])
    k, v = (torch.zeros((3, HKV, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((4, H, d), dtype=torch.bfloat16, device="cuda")
    ws = dilattn.decode_workspace(4, H, HKV, d)

    def step():
        dilattn.cache_write(pair.dev, k, v, wide, start)
        return dilattn.decode(q, pair.dev, wide, pos, pats, seq=seq, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = step()
    torch.cuda.current_stream().wait_stream(side)
    pair.ref.write(f64(k), f64(v), table, lens)
    for t in range(6):
        a, b, c = normal(rng, 3, HKV, d), normal(rng, 3, HKV, d), normal(rng, 4, H, d)
        at = [m + t for m in lens]
        k.copy_(bf16(a)), v.copy_(bf16(b)), q.copy_(bf16(c)), start.copy_(i32(at)), pos.copy_(i32(at + [-1]))
        ws.fill_(0xff - t)
        g.replay()
        pair.ref.write(a, b, table, at)
        pair.check()
        check_decode(got, ref.decode(c, pair.ref, table, at + [-1], [0, 1, 2, 0], pats), c, pair)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", case("padded"))
def test_padded_batches_and_drafts(name, fmt):
    """A token of each of 32 sequences with padded slots, more than one of some, and four of each;
    among them a sequence that there is not and positions past the table."""
    c = CASES[name]
    rng = np.random.default_rng(c["T"])
    lens = [700] + list(rng.integers(1, 90, 31))
    pair, table = filled(rng, lens, c["Hkv"], 16, c["d"], fmt)
    T = c["T"]
    seq = np.sort(np.arange(T) % 32)
    left = np.array([np.sum(seq[i:] == seq[i]) for i in range(T)])  # drafts end at their sequence's last token
    pos = np.array([lens[b] for b in seq]) - left
    seq[-3:], pos[-3:], pos[5] = [31, 32, -1], [-1, 5, 5], c["longest"]
    q = normal(rng, T, c["H"], c["d"])
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(widened(table, 32)), i32(pos), c["pats"], seq=i32(seq))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 4
    pos[[5, -2, -1]], seq[-2:] = -1, 0
    check_decode((out, lse), ref.decode(q, pair.ref, table, pos, seq, c["pats"]), q, pair)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [0, 12, 20, 24, 33, 60])
def test_channels_that_only_small_pages_fill(e, d, fmt, wide):
    """Each page of V fills a channel of its own, pages 2^e apart. A row's probability times its V
    scale, z, is rounded to 11 bits, or, below 2^-21 of the largest z, by up to 2^-32 of that: a
    channel is off by 2^-32 max z sum |code| / sum p beside the usual bound."""
    rng = np.random.default_rng(46)
    table, pages = tables(rng, [64], 16)
    pair = Pair(pages, 1, 16, d, fmt)
    k, v = f64(bf16(normal(rng, 64, 1, d) / 8)), np.zeros((64, 1, d))
    for page in range(4):
        v[16 * page:16 * page + 16, 0, 9 * page] = rng.integers(1, 8, 16) * 2.0 ** (e * (page % 2) - page)
    pair.write(k, v, table, [0], [0, 64])
    q = normal(rng, 2, 2, d)
    pos, seq = [63, 40], [0, 0]
    out, lse = dilattn.decode(bf16(q).cuda(), pair.dev, i32(widened(table, 2) if wide else table), i32(pos), DENSE,
                              seq=i32(seq))
    torch.cuda.synchronize()
    assert dilattn.device_error() == 0
    want = ref.decode(q, pair.ref, table, pos, seq, DENSE)
    if e <= 20:
        check_decode((out, lse), want, q, pair)
    wo, wl, spread = want
    assert np.abs(f64(lse) - wl).max() <= 1e-4
    for i in range(2):
        x = np.arange(pos[i] + 1)
        codes = np.abs(pair.ref.codes[1, table[0][x // 16], 0, x % 16])           # [rows, d]
        scale = pair.ref.scale[1, table[0][x // 16], 0]
        for h in range(2):
            p = np.exp(pair.ref.rows(0, table[0], x)[:, 0] @ q[i, h] / np.sqrt(d) - wl[i, h])  # sums to one
            tol = 2.0 ** -8 * np.abs(wo[i, h]) + 2.0 ** -10 * spread[i, h] + 2.0 ** -32 * (p * scale).max() * codes.sum(0)
            assert (np.abs(f64(out[i, h]) - wo[i, h]) <= tol).all()
