"""Plain float64 model of the 8-bit cache and of single-token dilated attention over it.

Written from the definitions alone, with numpy; nothing of the package is imported."""
import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def round_to_format(y, fmt):
    """Nearest number of the format to y (|y| within its range), ties to the even code."""
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)  # spacing: 3 fraction bits from 2^-6 on
    return np.clip(np.rint(y / step) * step, -448, 448)


def block_scale(amax, fmt):
    """The least power of two 2^e, e >= -126, with amax <= top * 2^e."""
    e = -126
    while TOP[fmt] * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


class Cache:
    """Codes (as numbers) and scales, K and V in one array of two."""

    def __init__(self, pages, Hkv, P, d, fmt):
        self.fmt, self.P = fmt, P
        self.codes = np.zeros((2, pages, Hkv, P, d))
        self.scale = np.ones((2, pages, Hkv))

    def write(self, k, v, table, start, offsets=None):
        B, P = len(table), self.P
        offsets = list(range(B + 1)) if offsets is None else list(offsets)
        for b in range(B):
            n = offsets[b + 1] - offsets[b]
            for pg in range(start[b] // P, (start[b] + n - 1) // P + 1 if n else 0):
                lo, hi = max(start[b], pg * P), min(start[b] + n, (pg + 1) * P)
                page, r0, r1 = table[b][pg], lo - pg * P, hi - pg * P
                t0 = offsets[b] + lo - start[b]
                for z, x in enumerate((k, v)):
                    for h in range(self.codes.shape[2]):
                        self._block(z, page, h, r0, r1, x[t0:t0 + hi - lo, h])

    def _block(self, z, page, h, r0, r1, x):
        codes, was = self.codes[z, page, h], self.scale[z, page, h]
        old = [i for i in range(self.P) if not r0 <= i < r1]
        if not np.isfinite(x).all() or (r0 > 0 and np.isnan(was)):
            self.scale[z, page, h] = np.nan
            codes[r0:r1] = 0
            return
        now = block_scale(np.abs(x).max(), self.fmt)
        if r0 > 0:
            now = max(now, was)
            if now > was:
                codes[old] = round_to_format(codes[old] * (was / now), self.fmt)
        codes[r0:r1] = round_to_format(x / now, self.fmt)
        self.scale[z, page, h] = now

    def rows(self, z, pages, positions):
        """Values of positions of a sequence with these pages: [n, Hkv, d]."""
        ids, row = np.asarray(pages)[positions // self.P], positions % self.P
        return self.codes[z, ids, :, row] * self.scale[z, ids][:, :, None]

    def read(self, table, start, offsets):
        out = []
        for z in range(2):
            got = [self.rows(z, table[b], np.arange(start[b], start[b] + offsets[b + 1] - offsets[b]))
                   for b in range(len(table)) if offsets[b + 1] > offsets[b]]
            out.append(np.concatenate(got))
        return out


def multiplicity(t, h, patterns):
    """How many patterns give position x to head h of the token at t, for x = 0 .. t."""
    x = np.arange(t + 1)
    count = np.zeros(t + 1)
    for w, r in patterns:
        s = t // w * w
        kept = (x >= s) & ((x - s) % r == h % r)
        if kept[t]:
            count += kept
    return count


def decode(q, cache, table, pos, seq, patterns):
    """(out [T, H, d], lse [T, H], spread [T, H, d]): spread is the softmax-weighted mean of |v|."""
    T, H, d = q.shape
    Hkv = cache.codes.shape[2]
    out, spread = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse = np.full((T, H), -np.inf)
    for i in range(T):
        if pos[i] < 0:
            continue
        for h in range(H):
            c = multiplicity(pos[i], h, patterns)
            x = np.nonzero(c)[0]
            if len(x) == 0:
                continue
            k = cache.rows(0, table[seq[i]], x)[:, h // (H // Hkv)]
            v = cache.rows(1, table[seq[i]], x)[:, h // (H // Hkv)]
            s = k @ q[i, h] / np.sqrt(d)
            m = s.max()
            p = c[x] * np.exp(s - m)
            out[i, h], spread[i, h] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
            lse[i, h] = m + np.log(p.sum())
    return out, lse, spread
