"""Plain 64-bit (and, for the codes, exact 32-bit) forms of the 8-bit paged
cache for the tests: numpy only, one sequence and token at a time."""
import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}
TINY = np.float32(np.finfo(np.float32).tiny)


def e4m3_table():
    """The 256 values of e4m3 (NaN at 0x7f and 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_table()


def value(codes, kind):
    """Codes (uint8) as float64."""
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else E4M3[codes]


def round_code(y, kind):
    """float32 scaled values to codes (uint8), half to even."""
    y = np.asarray(y, np.float32)
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    a = np.rint(a / step) * step
    i = np.searchsorted(E4M3[:127], a)
    assert np.array_equal(E4M3[i], a)
    return (i + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


class Ref:
    """One layer: codes [pages, heads, P, d] of keys and values, scales."""

    def __init__(self, kind, pages, heads, page, d):
        self.kind, self.P = kind, page
        self.c = [np.zeros((pages, heads, page, d), np.uint8) for _ in range(2)]
        self.s = [np.zeros((pages, heads), np.float32) for _ in range(2)]

    def load(self, k, v, ks, vs):
        n, h, p, d = self.c[0].shape
        self.c = [k.copy(), v.transpose(0, 1, 2, 4, 3).reshape(n, h, p, d).copy()]
        self.s = [ks.copy(), vs.copy()]

    def append(self, table, length, x):
        """x = (k, v), float32 [n, heads, d]: the last n of `length` tokens."""
        n = x[0].shape[0]
        for w in range(2):
            t = length - n
            while t < length:
                page, lo = t // self.P, t % self.P
                hi = min(self.P, lo + length - t)
                i = table[page]
                rows = x[w][t - (length - n):t - (length - n) + hi - lo]
                for h in range(rows.shape[1]):
                    a = np.max(np.abs(rows[:, h]))        # NaN stays
                    old = self.s[w][i, h] if lo else np.float32(0)
                    s = np.float32(a / np.float32(TOP[self.kind])) if np.isfinite(a) else np.float32(np.nan)
                    if s < TINY:
                        s = np.float32(0)
                    s = np.float32(np.nan) if np.isnan(s) or np.isnan(old) else max(s, old)
                    c = self.c[w][i, h]
                    if not s > 0:
                        c[:hi] = 0
                    else:
                        if lo and s != old:
                            c[:lo] = round_code(value(c[:lo], self.kind).astype(np.float32) * np.float32(old / s), self.kind)
                        c[lo:hi] = round_code(rows[:, h] * np.float32(np.float32(1) / s), self.kind)
                    self.s[w][i, h] = s
                t += hi - lo

    def tokens(self, w, table, n):
        """float64 [n, heads, d] of a sequence's first n tokens."""
        out = np.zeros((n, self.c[w].shape[1], self.c[w].shape[3]))
        for t in range(n):
            i = table[t // self.P]
            out[t] = value(self.c[w][i, :, t % self.P], self.kind) * self.s[w][i, :, None].astype(np.float64)
        return out


def attention(q, k, v, limits, scale):
    """q [n, H, d], k and v [T, heads, d] in float64; row i sees limits[i]
    tokens.  Returns out, lse and two sizes for error bounds: the weighted
    magnitudes sum w |v| [n, H, d] and the largest sum |q||k| * |scale| [n, H]."""
    n, H, d = q.shape
    G = H // k.shape[1]
    out, lse = np.zeros((n, H, d)), np.full((n, H), -np.inf)
    mag, dot = np.zeros((n, H, d)), np.zeros((n, H))
    for i in range(n):
        L = max(0, min(limits[i], k.shape[0]))
        if L == 0:
            continue
        for h in range(H):
            kk, vv = k[:L, h // G], v[:L, h // G]
            x = kk @ q[i, h] * scale
            m = x.max()
            w = np.exp(x - m)
            lse[i, h] = m + np.log(w.sum())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            dot[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h])) * abs(scale)
    return out, lse, mag, dot


class Pool:
    """Pages of rows, one operation after the other."""

    def __init__(self, rows, max_pages, pages, page):
        self.t = np.full((rows, max_pages), -1, np.int32)
        self.lens, self.ref = np.zeros(rows, np.int32), np.zeros(pages, np.int32)
        self.P, self.moves = page, []

    def count(self, n):
        return -(-int(n) // self.P)

    def extend(self, add):
        """Error bits."""
        free, at, bits, short = list(np.nonzero(self.ref == 0)[0]), 0, 0, False
        for r, a in enumerate(add):
            have, want = self.count(self.lens[r]), self.count(self.lens[r] + a)
            if a < 0 or self.lens[r] + a > self.t.shape[1] * self.P:
                bits |= 16
                continue
            if want > have:
                short |= at + want - have > len(free)
                if short:
                    bits |= 32
                    continue
                self.t[r, have:want] = free[at:at + want - have]
                self.ref[free[at:at + want - have]] = 1
                at += want - have
            self.lens[r] += a
        return bits

    def fork(self, src, dst):
        """(done, pages copied [(from, to)], error bits)."""
        free, at, short = list(np.nonzero(self.ref == 0)[0]), 0, False
        before, lens = self.t.copy(), self.lens.copy()
        done, copies, seen = [], [], set()
        R = len(lens)
        for a, z in zip(src, dst):
            ok = 0 <= a < R and 0 <= z < R and lens[z] == 0 and z not in seen
            if ok:
                seen.add(z)
                n = int(lens[a])
                part = n % self.P != 0
                if part and (short or at >= len(free)):
                    short, ok = True, False
            if ok:
                full = n // self.P
                self.t[z, :full] = before[a, :full]
                self.ref[before[a, :full]] += 1
                if part:
                    self.t[z, full] = free[at]
                    self.ref[free[at]] = 1
                    copies.append((before[a, full], free[at]))
                    at += 1
                self.lens[z] = n
            done.append(int(ok))
        return np.array(done, np.int32), copies, 0 if all(done) else 32

    def free(self, rows):
        bits = 0
        for r in rows:
            if not 0 <= r < len(self.lens):
                bits |= 32
                continue
            n = self.count(self.lens[r])
            np.subtract.at(self.ref, self.t[r, :n], 1)
            self.t[r, :n] = -1
            self.lens[r] = 0
        return bits

    def compact(self):
        """(pages in use, pages copied [(from, to)])."""
        live = int((self.ref > 0).sum())
        holes, movers = np.nonzero(self.ref[:live] == 0)[0], np.nonzero(self.ref[live:] > 0)[0] + live
        to = dict(zip(movers, holes))
        for r in range(len(self.lens)):
            for j in range(self.count(self.lens[r])):
                self.t[r, j] = to.get(self.t[r, j], self.t[r, j])
        self.ref[holes] = self.ref[movers]
        self.ref[movers] = 0
        return live, list(to.items())
