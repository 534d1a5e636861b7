"""Shared by the cache tests: a device cache beside its float64 model, and the tolerances."""
import numpy as np
import torch

import cache_reference as ref
from sparse_long_sequence_dilated_b200 import dilattn


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()


def f64(t):
    if t.dtype in (torch.float8_e4m3fn, torch.int8, torch.bfloat16):
        t = t.float()
    return t.detach().cpu().double().numpy()


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def tables(rng, lengths, P, spare=3):
    """Shuffled page tables for sequences of these lengths (unused entries -1) and the page count."""
    need = [max(1, -(-n // P)) for n in lengths]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lengths), max(need)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(need) + spare


class Pair:
    """A device cache and its model, written and compared together."""

    def __init__(self, pages, Hkv, P, d, fmt):
        self.dev = dilattn.new_cache(pages, Hkv, P, d, fmt)
        self.ref = ref.Cache(pages, Hkv, P, d, fmt)
        self.Hkv, self.d = Hkv, d

    def write(self, k, v, table, start, offsets=None):
        """k, v: float64 arrays; both sides get their bf16 values."""
        k, v = bf16(k), bf16(v)
        dilattn.cache_write(self.dev, k.cuda(), v.cuda(), i32(table), i32(start),
                            None if offsets is None else i32(offsets))
        self.ref.write(f64(k), f64(v), table, start, offsets)

    def check(self):
        torch.cuda.synchronize()
        assert dilattn.device_error() == 0
        for z, (codes, scale) in enumerate(((self.dev.k, self.dev.k_scale), (self.dev.v, self.dev.v_scale))):
            assert np.array_equal(f64(scale), self.ref.scale[z], equal_nan=True)
            assert np.array_equal(f64(codes), self.ref.codes[z])


def normal(rng, *shape):
    """Normal numbers that bf16 holds exactly, as float64."""
    return f64(bf16(rng.standard_normal(shape)))


def filled(rng, lengths, Hkv, P, d, fmt, spread=0.0):
    """A pair whose sequences hold these lengths, and its table; spread: log2 of the range of
    sizes that single tokens have."""
    table, pages = tables(rng, lengths, P)
    pair = Pair(pages, Hkv, P, d, fmt)
    T = int(sum(lengths))
    k, v = normal(rng, T, Hkv, d), normal(rng, T, Hkv, d)
    if spread:
        k = f64(bf16(k * 2.0 ** rng.uniform(-spread, 0, (T, 1, 1))))
        v = f64(bf16(v * 2.0 ** rng.uniform(-spread, spread, (T, 1, 1))))
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    pair.write(k, v, table, [0] * len(lengths), offsets)
    return pair, table


def check_decode(got, want, q, cache):
    """out: half a bf16 step of the value (2^-8), and the roundings of the probabilities to 11
    bits (2^-11 of each term, so 2^-11 of the weighted mean of |v|) and of fp32 scores: a score
    is a sum of d products and a scale factor, off by at most (d / 8 + 8) 2^-23 of the largest
    sum of |q k| it stands for. lse: that score error and 2^-20 for exp2, log2 and the sums."""
    (out, lse), (wo, wl, spread) = got, want
    out, lse = f64(out), f64(lse)
    d = q.shape[-1]
    kmax = np.nanmax(np.abs(cache.ref.codes[0]) * cache.ref.scale[0][:, :, None, None])
    size = np.abs(q).sum(-1) * kmax / np.sqrt(d)  # [T, H]: at least any sum of |q k|
    es = (d / 8 + 8) * 2.0 ** -23 * size
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    f = ~empty
    tol_l = es[f] + 2.0 ** -20 * (1 + np.abs(wl[f]))
    assert (np.abs(lse[f] - wl[f]) <= tol_l).all(), np.max(np.abs(lse[f] - wl[f]) / tol_l)
    tol = 2.0 ** -8 * np.abs(wo[f]) + (2.0 ** -11 + 2 * es[f][:, None] + 2.0 ** -18) * spread[f]
    err = np.abs(out[f] - wo[f])
    assert (err <= tol).all(), np.max(err / np.maximum(tol, 1e-300))
