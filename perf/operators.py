"""Cases for the 8-bit key/value cache and the attention over it: writing, reading back, decoding.

The cache is paged: codes [pages, Hkv, P, d] in e4m3 or int8, and one float32 scale for each
(page, KV head), for K and V apart. Three operators:

* write: new K and V rows (bf16) are quantised into the pages of their sequences. A page's scale
  is the least power of two that holds every magnitude written to it; rows already there are
  re-rounded when it grows; writing a page's row 0 starts the page afresh.
* read: tokens of the cache come back as bf16.
* decode: merged dilated attention of single query tokens over the cache. Pattern (w, r) gives a
  token at position t, for the heads h with h mod r = (t - s) mod r, the rows t, t - r, ... down to
  its segment's start s = floor(t / w) w; the softmax runs over the multiset union of all patterns'
  rows. Dense attention is the pattern (w >= length, 1).

Outputs that are held in 8 bits are returned as the float8 (or int8) numbers beside their scales,
which are powers of two; the value is their product.
"""
import math
import random

import torch

own = False

BASE = "2048/1 4096/2 8192/4 16384/6 32768/12"
WIDE = "2048/1 4096/2 8192/4 16384/8 32768/16 65536/32 131072/64"
SWEEP = "2048/1 4096/2 8192/4 16384/8 32768/16"


def listed():
    return [
        # one new token of one sequence, LongNet-base heads: the per-step append of a single stream
        _write("append_1_base", 1, 1, 1, 32000, 12, 64, 64, "e4m3"),
        # one new token for each of 64 sequences of a wide layer: the per-step append of a server
        _write("append_64_wide", 64, 1, 1, 4096, 32, 128, 64, "int8"),
        # ragged prompts, some of them continuing sequences in the middle of a page
        _write("prompts_16_base", 16, 1, 8191, 1000, 12, 64, 32, "int8"),
        # a whole 128K prompt of a wide layer
        _write("prompt_128k_wide", 1, 131072, 131072, 0, 32, 128, 128, "e4m3"),
        # a few ragged stretches read back, pages smaller than a tile
        _read("read_5_base", 5, 1, 700, 5000, 12, 64, 16, "int8"),
        # a whole 128K sequence read back, to run the full-sequence forward on it
        _read("read_128k_wide", 1, 131072, 131072, 0, 32, 128, 128, "e4m3"),
        # one stream of LongNet-base at 32K: latency
        _decode("decode_1_base", 1, 1, 0, 32768, 32768, 12, 12, 64, 64, "e4m3", BASE),
        # a padded serving batch of LongNet-base, ragged lengths
        _decode("decode_64_base", 64, 1, 4, 100, 32768, 12, 12, 64, 64, "e4m3", BASE),
        # a wide layer's batch at up to 128K
        _decode("decode_16_wide", 16, 1, 0, 40000, 131072, 32, 32, 128, 64, "e4m3", WIDE),
        # four drafted tokens for each of eight sequences, small pages
        _decode("drafts_8x4_sweep", 8, 4, 0, 3000, 32768, 12, 12, 64, 16, "int8", SWEEP),
        # dense attention with four query heads to a KV head, a ragged batch
        _decode("dense_32_shared", 32, 1, 0, 500, 32768, 32, 8, 128, 64, "int8", "32768/1"),
        # one very long context, dense: the long axis has to be split
        _decode("dense_1_million", 1, 1, 0, 1048576, 1048576, 32, 8, 128, 128, "e4m3", "1048576/1"),
    ]


def _write(name, B, least, most, ctx, heads, d, page, fmt, mix=1):
    return dict(name=name, op="write", B=B, least=least, most=most, ctx=ctx, heads=heads, d=d,
                page=page, fmt=fmt, mix=mix)


def _read(name, B, least, most, ctx, heads, d, page, fmt, mix=1):
    return dict(_write(name, B, least, most, ctx, heads, d, page, fmt, mix), op="read")


def _decode(name, B, per, pad, least, most, H, heads, d, page, fmt, patterns, mix=1):
    return dict(name=name, op="decode", B=B, per=per, pad=pad, least=least, most=most, H=H,
                heads=heads, d=d, page=page, fmt=fmt, patterns=patterns, mix=mix)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode"))
    d = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    fmt = rng.choice(("e4m3", "int8"))
    mix = rng.randrange(1 << 20)
    if op != "decode":
        heads = rng.choice((1, 2, 4, 8, 12, 20, 32))
        B = _log_int(rng, 1, 64)
        # at most the rows of the 128K prompt of the wide layer
        most = _log_int(rng, 1, max(1, min(131072, 131072 * 32 * 128 // (B * heads * d))))
        make = _write if op == "write" else _read
        c = make("", B, 1, most, _log_int(rng, 1, 8192), heads, d, page, fmt, mix)
        del c["name"]
        return c
    heads = rng.choice((1, 2, 4, 8, 12, 20, 32))
    G = rng.choice((1, 1, 2, 4, 7, 8, 16)) if heads <= 8 else 1
    per = rng.choice((1, 1, 1, 2, 5))
    dense = rng.random() < 0.4
    B = _log_int(rng, 1, 64)
    # the cache holds at most what the wide layer's batch holds, and the rows that a pass attends
    # are at most those of the longest dense case
    room = (1 << 30) // (heads * d * per * B) if dense else (1 << 33) // (heads * d * B)
    most = _log_int(rng, 1, max(1, min(1 << 20 if dense else 1 << 17, room)))
    least = _log_int(rng, 1, most)
    if dense:
        patterns = "%d/1" % (1 << 20)
    else:
        patterns = rng.choice((BASE, WIDE, SWEEP, "1000/1 3001/3 10000/7", "512/2 4096/4", "256/1 9000/5"))
    c = _decode("", B, per, rng.choice((0, 0, 1, 3)), max(per, least), max(per, most), heads * G,
                heads, d, page, fmt, patterns, mix)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that follow from a case
def _lengths(case):
    """Tokens of each sequence (write and read: new or read ones; decode: held ones)."""
    rng = random.Random(case["mix"])
    n = [_log_int(rng, case["least"], case["most"]) for _ in range(case["B"])]
    n[rng.randrange(case["B"])] = case["most"]
    return n


def _starts(case):
    """Position of each sequence's first written or read token."""
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(0, case["ctx"]) if case["ctx"] else 0 for _ in range(case["B"])]


def _queries(case):
    """(sequence, position) of every query token; padded slots have position -1."""
    got = [(b, n - case["per"] + k) for b, n in enumerate(_lengths(case)) for k in range(case["per"])]
    return got + [(0, -1)] * case["pad"]


def _patterns(case):
    return [tuple(int(x) for x in p.split("/")) for p in case["patterns"].split()]


def _rows(case, t, heads):
    """The sets of positions that a token at t gives any of these query heads, each as (start, step)
    of an arithmetic progression that ends at t."""
    got = []
    for w, r in _patterns(case):
        s = t // w * w
        o = (t - s) % r
        if any(h % r == o for h in heads):
            got.append((s + o, r))
    return got


def _distinct(progressions, t):
    """How many different positions progressions that end at t hold together."""
    if not progressions:
        return 0
    lowest = min(s for s, _ in progressions)
    held = torch.zeros(t - lowest + 1, dtype=torch.bool)
    for s, r in progressions:
        held[s - lowest::r] = True
    return int(held.sum())


def work(case):
    d = case["d"]
    if case["op"] != "decode":
        n = sum(_lengths(case)) * case["heads"] * d * 2  # K and V
        return {"bytes": 3 * n, "flops": 0}
    G = case["H"] // case["heads"]
    bytes_, flops, seen = 0, 0, {}
    for b, t in _queries(case):
        if t < 0:
            continue
        by_set = {}
        for g in range(case["heads"]):
            p = tuple(_rows(case, t, range(g * G, (g + 1) * G)))
            seen.setdefault((b, g), []).append((p, t))
            for h in range(g * G, (g + 1) * G):
                p = tuple(_rows(case, t, (h,)))
                if p not in by_set:
                    by_set[p] = _distinct(p, t)
                flops += 4 * d * by_set[p]
    unions = {}
    for tokens in seen.values():
        key = tuple(tokens)
        if key not in unions:
            top = max(t for _, t in tokens)
            held = torch.zeros(top + 1, dtype=torch.bool)
            for p, t in tokens:
                for s, r in p:
                    held[s:t + 1:r] = True
            unions[key] = int(held.sum())
        bytes_ += 2 * d * unions[key]
    T = case["B"] * case["per"] + case["pad"]
    return {"bytes": bytes_ + T * case["H"] * (4 * d + 4), "flops": flops}


# ------------------------------------------------------------------ inputs
_DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _codes(shape, fmt, gen):
    """Codes of normally distributed values whose largest sits near the format's top."""
    out = torch.empty(shape, dtype=_DTYPE[fmt], device="cuda")
    rows = max(1, (1 << 28) // max(1, out[0].numel()))
    for i in range(0, shape[0], rows):
        x = torch.randn(out[i:i + rows].shape, device="cuda", generator=gen)
        if fmt == "e4m3":
            out[i:i + rows] = x.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        else:
            out[i:i + rows] = x.mul_(28).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _scales(pages, case, gen):
    """Powers of two that bring the codes' values to a standard deviation near one."""
    low = -7 if case["fmt"] == "e4m3" else -5
    e = torch.randint(low, low + 2, (pages, case["heads"]), device="cuda", generator=gen)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    P, d, heads = case["page"], case["d"], case["heads"]
    n = _lengths(case)
    start = _starts(case) if case["op"] != "decode" else [0] * len(n)
    held = [-(-(s + k) // P) for s, k in zip(start, n)]
    pages = sum(held) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(n), max(held)), -1, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for b, k in enumerate(held):
        table[b, :k] = order[at:at + k]
        at += k
    shape = (pages, heads, P, d)
    s = dict(case=case, table=table.cuda(), kc=_codes(shape, case["fmt"], gen),
             vc=_codes(shape, case["fmt"], gen), ks=_scales(pages, case, gen),
             vs=_scales(pages, case, gen))
    if case["op"] == "decode":
        q = _queries(case)
        s["seq"] = torch.tensor([b for b, _ in q], dtype=torch.int32, device="cuda")
        s["pos"] = torch.tensor([t for _, t in q], dtype=torch.int32, device="cuda")
        s["q"] = torch.randn((len(q), case["H"], d), device="cuda", generator=gen).bfloat16()
        s["patterns"] = _patterns(case)
        s["w"] = torch.tensor([w for w, _ in s["patterns"]], device="cuda")
        s["r"] = torch.tensor([r for _, r in s["patterns"]], device="cuda")
        # the rows that one pattern can give one token, at most
        s["most"] = max(-(-min(w, case["most"]) // r) for w, r in s["patterns"])
    else:
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        offsets = [0]
        for k in n:
            offsets.append(offsets[-1] + k)
        s["total"] = offsets[-1]
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        if case["op"] == "write":
            s["k"] = _tokens(s["total"], heads, d, gen)
            s["v"] = _tokens(s["total"], heads, d, gen)
    if own:
        from sparse_long_sequence_dilated_b200 import dilattn
        s["cache"] = dilattn.Cache(s["kc"], s["vc"], s["ks"], s["vs"])
        if case["op"] == "decode":
            s["workspace"] = dilattn.decode_workspace(len(q), case["H"], heads, d, device="cuda")
    return s


def _tokens(n, heads, d, gen):
    out = torch.empty((n, heads, d), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // (heads * d))
    for i in range(0, n, step):
        out[i:i + step] = torch.randn(out[i:i + step].shape, device="cuda", generator=gen)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from sparse_long_sequence_dilated_b200 import dilattn
        if op == "write":
            dilattn.cache_write(s["cache"], s["k"], s["v"], s["table"], s["start"], s["offsets"])
            return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
        if op == "read":
            return dilattn.cache_read(s["cache"], s["table"], s["start"], s["offsets"], s["total"])
        return dilattn.decode(s["q"], s["cache"], s["table"], s["pos"], s["patterns"],
                              seq=s["seq"], workspace=s["workspace"])
    if op == "write":
        seq, at, page, row = _places(s)
        _plain_write(s["kc"], s["ks"], s["k"], s, page, row)
        _plain_write(s["vc"], s["vs"], s["v"], s, page, row)
        return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "read":
        seq, at, page, row = _places(s)
        return (_fetch(s["kc"], s["ks"], page, row).bfloat16(),
                _fetch(s["vc"], s["vs"], page, row).bfloat16())
    return _plain_decode(s)


def _places(s):
    """Sequence, position, page and row of every token that is written or read."""
    tok = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["offsets"][1:].long(), tok, right=True)
    at = s["start"].long()[seq] + tok - s["offsets"].long()[seq]
    P = s["case"]["page"]
    return seq, at, s["table"][seq, at // P].long(), at % P


def _power_scale(amax, fmt):
    """The least power of two (from 2^-126) whose product with the format's largest number holds amax."""
    m, e = torch.frexp(amax)
    top, bits = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)
    e = torch.where(amax == 0, -126, e - bits + (m > top)).clamp(min=-126)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _encode(x, fmt):
    """The codes of values in units of their scale, as bytes."""
    if fmt == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _plain_write(codes, scale, x, s, page, row):
    fmt, P = s["case"]["fmt"], s["case"]["page"]
    x = x.float()
    held = torch.full_like(scale, -1.0)
    held.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    fresh = torch.zeros(scale.shape[0], device="cuda")
    fresh.scatter_reduce_(0, page, (row == 0).float(), "amax")
    need = _power_scale(held.clamp(min=0), fmt)
    new = torch.where(held < 0, scale, torch.where(fresh[:, None] > 0, need, torch.maximum(need, scale)))
    # a sequence's first page alone can hold rows already: they are re-rounded to the new scale
    first = s["table"].gather(1, (s["start"].long() // P)[:, None])[:, 0].long()
    old = codes.view(torch.uint8)[first].view(codes.dtype).float()
    ratio = torch.where(fresh[first][:, None] > 0, 1.0, scale[first] / new[first])
    raw = codes.view(torch.uint8)
    raw[first] = _encode(old * ratio[:, :, None, None], fmt)
    raw[page, :, row] = _encode(x / new[page][:, :, None], fmt)
    scale.copy_(new)


def _fetch(codes, scale, page, row):
    """Rows [..., Hkv, d] of the cache in 32 bits."""
    x = codes.view(torch.uint8)[page, :, row].view(codes.dtype).float()
    return x.mul_(scale[page][..., None])


def _plain_decode(s):
    case = s["case"]
    H, heads, d, P = case["H"], case["heads"], case["d"], case["page"]
    t, w, r = s["pos"].long()[:, None], s["w"][None], s["r"][None]
    T = t.shape[0]
    low = t.clamp(min=0) // w * w                                       # [T, npat]
    takes = torch.arange(H, device="cuda")[None, :, None] % r[:, None] == ((t - low) % r)[:, None]
    x = t[..., None] - r[..., None] * torch.arange(s["most"], device="cuda")  # [T, npat, most]
    valid = (x >= low[..., None]) & (t[..., None] >= 0)
    keep = (takes[..., None] & valid[:, None]).flatten(2)               # [T, H, rows]
    x = x.clamp(min=0).flatten(1)
    page = s["table"].long()[s["seq"].long()[:, None], (x // P).clamp(max=s["table"].shape[1] - 1)]
    page, row = page.clamp(min=0), x % P
    q = s["q"].float().view(T, heads, H // heads, d)
    k = _fetch(s["kc"], s["ks"], page, row).permute(0, 2, 3, 1)         # [T, Hkv, d, rows]
    scores = (q @ k).view(T, H, -1).mul_(1 / math.sqrt(d))
    scores = scores.masked_fill_(~keep, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = scores.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    v = _fetch(s["vc"], s["vs"], page, row).permute(0, 2, 1, 3)         # [T, Hkv, rows, d]
    out = (p.view(T, heads, H // heads, -1) @ v).view(T, H, d)
    out = torch.where(z > 0, out / z, 0.0)
    return out.bfloat16(), (top + z.log())[..., 0]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"] == "read":
        return _exact_read(case, s)
    return _exact_write(case, s)


def _values(codes, scale, pages, P, lo, hi):
    """Positions lo to hi - 1 of a sequence with these pages: [hi - lo, Hkv, d] in 64 bits."""
    ids = pages[lo // P:(hi - 1) // P + 1].long()
    x = codes.view(torch.uint8)[ids].view(codes.dtype).double() * scale[ids].double()[:, :, None, None]
    x = x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])
    return x[lo % P:lo % P + hi - lo]


def _exact_read(case, s):
    ks, vs = [], []
    for b, (lo, n) in enumerate(zip(_starts(case), _lengths(case))):
        ks.append(_values(s["kc"], s["ks"], s["table"][b], case["page"], lo, lo + n))
        vs.append(_values(s["vc"], s["vs"], s["table"][b], case["page"], lo, lo + n))
    return torch.cat(ks), torch.cat(vs)


def _round_to_format(y, fmt):
    """The format's nearest number, ties to the even code, from the spacing of its numbers."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    _, e = torch.frexp(y)
    # e4m3: three fraction bits from 2^-6 on, a spacing of 2^-9 below
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_write(case, s):
    P, top = case["page"], 448.0 if case["fmt"] == "e4m3" else 127.0
    starts, lengths = _starts(case), _lengths(case)
    out = {}
    for name, codes, scale, x in (("k", s["kc"], s["ks"], s["k"]), ("v", s["vc"], s["vs"], s["v"])):
        codes, scale = codes.double(), scale.double()
        at = 0
        for b, (lo, n) in enumerate(zip(starts, lengths)):
            new = x[at:at + n].double().permute(1, 0, 2)  # [Hkv, n, d]
            at += n
            # stretches that lie in one page, and the whole pages between them at once
            ends = [lo] + ([e for e in (-(-(lo + 1) // P) * P, (lo + n) // P * P) if lo < e < lo + n]) + [lo + n]
            for a, e in zip(ends, ends[1:]):
                if e <= a:
                    continue
                ids = s["table"][b, a // P:(e - 1) // P + 1].long()
                y = new[:, a - lo:e - lo]
                y = y.reshape(y.shape[0], len(ids), -1, y.shape[2]).transpose(0, 1)  # [pages, Hkv, rows, d]
                big = y.abs().amax((2, 3))
                p = torch.ceil(torch.log2(big / top))
                p = torch.where(torch.exp2(p - 1) * top >= big, p - 1, p)  # log2's own rounding
                p = torch.where(torch.exp2(p) * top < big, p + 1, p).clamp(min=-126)
                need = torch.exp2(p)
                if a % P:
                    was = scale[ids]
                    need = torch.maximum(need, was)
                    codes[ids] = _round_to_format(codes[ids] * (was / need)[:, :, None, None], case["fmt"])
                scale[ids] = need
                r0 = a % P
                codes[ids, :, r0:r0 + y.shape[2]] = _round_to_format(y / need[:, :, None, None], case["fmt"])
        out[name], out[name + "_scale"] = codes, scale
    if case["fmt"] == "int8":
        out["k"], out["v"] = out["k"].to(torch.int8), out["v"].to(torch.int8)
    return out


def _exact_decode(case, s):
    H, heads, d, P = case["H"], case["heads"], case["d"], case["page"]
    G = H // heads
    queries = _queries(case)
    out = torch.zeros((len(queries), H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((len(queries), H), -math.inf, dtype=torch.float64, device="cuda")
    h = torch.arange(H, device="cuda")[:, None]
    for i, (b, t) in enumerate(queries):
        if t < 0:
            continue
        x = torch.arange(t + 1, device="cuda")[None]
        count = torch.zeros((H, t + 1), dtype=torch.int8, device="cuda")
        for w, r in s["patterns"]:
            low = t // w * w
            kept = (x >= low) & ((x - low) % r == h % r)  # rows of the token's segment that the head keeps
            count += kept & kept[:, t:]
        used = count.any(0).nonzero()[:, 0]
        if not len(used):
            continue
        ids, row = s["table"][b].long()[used // P], used % P

        def rows(codes, scale):
            got = codes.view(torch.uint8)[ids, :, row].view(codes.dtype).double()
            return (got * scale[ids].double()[:, :, None]).transpose(0, 1)  # [Hkv, rows, d]

        c = count[:, used].double()
        scores = (s["q"][i].double().view(heads, G, d) @ rows(s["kc"], s["ks"]).transpose(1, 2)).view(H, -1)
        scores = torch.where(c > 0, scores / math.sqrt(d), -math.inf)
        some = c.sum(1) > 0
        top = torch.where(some, scores.amax(1), 0.0)
        p = c * torch.exp(scores - top[:, None])
        z = p.sum(1)
        o = (p.view(heads, G, -1) @ rows(s["vc"], s["vs"])).view(H, d)
        out[i] = torch.where(some[:, None], o / z[:, None], 0.0)
        lse[i] = torch.where(some, top + torch.log(z), -math.inf)
    return out, lse
