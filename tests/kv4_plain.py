"""Plain 64-bit implementation of the 4-bit K/V cache for the tests: the page format, the
rounding, attention and the page bookkeeping, written from their definitions with numpy."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(bits):
    bits = np.asarray(bits).astype(np.int64)
    e, f = bits >> 3 & 15, bits & 7
    v = np.where(e > 0, (1.0 + f / 8.0) * np.exp2(e - 7.0), f * 2.0 ** -9)
    v = np.where((bits & 127) == 127, np.nan, v)
    return np.where(bits & 128, -v, v)


E4M3 = e4m3_value(np.arange(127))  # the non-negative finite values, ascending


def nearest_even(x, grid):
    """Index of the value of the ascending `grid` nearest to x >= 0; ties to the even index."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(x, ts):
    """Codes and scale bits of x [..., D] (float64 holding the input values)."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    b = x.reshape(*x.shape[:-1], -1, 16)
    sb = nearest_even(np.abs(b).max(-1) / (6.0 * ts), E4M3)
    d = (E4M3[sb] * ts)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(d > 0, b / np.where(d > 0, d, 1.0), 0.0)
    code = nearest_even(np.abs(y), E2M1) | np.where(y < 0, 8, 0)
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def values(code, sb, ts):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, 16) * (e4m3_value(sb) * ts)[..., None]).reshape(v.shape)


def tile_fields(tile, D):
    """K and V codes [16, D] and scale bits [16, D / 16] of one tile (18 D bytes)."""
    tile = np.asarray(tile)
    k = tile[:8 * D].reshape(D // 32, 16, 16).transpose(1, 0, 2).reshape(16, D // 2)
    v = tile[8 * D:16 * D].reshape(16, D // 2)
    both = []
    for c in (k, v):
        o = np.empty((16, D), dtype=np.uint8)
        o[:, 0::2], o[:, 1::2] = c & 15, c >> 4
        both.append(o)
    return both[0], both[1], tile[16 * D:17 * D].reshape(16, D // 16), tile[17 * D:].reshape(16, D // 16)


def make_tile(kc, vc, ks, vs):
    """The inverse of tile_fields."""
    D = kc.shape[1]
    pack = [c[:, 0::2] | (c[:, 1::2] << 4) for c in (kc, vc)]
    return np.concatenate([pack[0].reshape(16, D // 32, 16).transpose(1, 0, 2).reshape(-1), pack[1].reshape(-1),
                           ks.reshape(-1), vs.reshape(-1)]).astype(np.uint8)


def tile_at(pool, table, s, pos, h, heads, D, page):
    """The 18 D bytes (a view) that hold token `pos` of sequence s and head h; pool [pages, bytes]."""
    p = int(table[s, pos // page])
    at = (h * (page // 16) + pos % page // 16) * 18 * D
    return pool[p, at:at + 18 * D]


def kv_of(pool, table, s, n, h, heads, D, page, k_ts, v_ts):
    """K and V [n, D] in 64 bits of the first n tokens of a sequence and head."""
    k, v = np.zeros((n, D)), np.zeros((n, D))
    for t in range(0, n, 16):
        kc, vc, ks, vs = tile_fields(tile_at(pool, table, s, t, h, heads, D, page), D)
        m = min(16, n - t)
        k[t:t + m] = values(kc, ks, k_ts)[:m]
        v[t:t + m] = values(vc, vs, v_ts)[:m]
    return k, v


def visible(n_tokens, first, row, window, tree):
    """Which of the sequence's tokens the step's row sees; first: the position of the step's row 0."""
    t = np.arange(n_tokens)
    if tree is not None:
        j = t - first
        bits = np.array([(int(tree) >> int(x)) & 1 if 0 <= x < 64 else 0 for x in j], dtype=bool)
        return (j < 0) | bits
    see = t <= first + row
    return see & (t > first + row - window) if window else see


def attend_row(q, k, v, see, scale):
    """One head's output and log-sum-exp in 64 bits, with the quantities that bound a kernel's error:
    sum p|v| / sum p, the largest sum |q k| * scale, and the largest |v|."""
    if not see.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0, 0.0
    k, v = k[see], v[see]
    z = k @ q * scale
    m = z.max()
    p = np.exp(z - m)
    l = p.sum()
    return p @ v / l, m + np.log(l), p @ np.abs(v) / l, float((np.abs(k) @ np.abs(q)).max() * abs(scale)), float(np.abs(v).max())


class PlainPages:
    """The page bookkeeping, one sequence after the other; pool [layers, pages, bytes] is changed in place."""

    def __init__(self, pool, table, lens, refs, heads, D, page):
        self.pool, self.table, self.lens, self.refs = pool, table, lens, refs
        self.heads, self.D, self.page = heads, D, page
        self.no_page = False

    def pages_of(self, n):
        return -(-int(n) // self.page)

    def drop(self, s, keep_pages):
        for j in range(keep_pages, self.table.shape[1]):
            if self.table[s, j] >= 0:
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1

    def trim(self, to):
        for s in range(len(self.lens)):
            n = min(max(int(to[s]), 0), int(self.lens[s]))
            self.drop(s, self.pages_of(n))
            self.lens[s] = n

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.drop(d, 0)
            self.table[d] = self.table[s]
            self.lens[d] = self.lens[s]
            for p in self.table[d]:
                if p >= 0:
                    self.refs[p] += 1

    def reserve(self, new):
        before = self.refs.copy()
        free = [p for p in range(len(before)) if before[p] == 0]
        full = False
        for s in range(len(self.lens)):
            n = max(int(new[s]), 0)
            if n == 0:
                continue
            have, want = self.pages_of(self.lens[s]), self.pages_of(self.lens[s] + n)
            if want > self.table.shape[1]:
                self.no_page = True
                continue
            copy = self.lens[s] % self.page != 0 and before[self.table[s, have - 1]] > 1
            need = want - have + int(copy)
            if need and (full or need > len(free)):
                full = self.no_page = True
                continue
            if copy:
                p, old = free.pop(0), self.table[s, have - 1]
                self.pool[:, p] = self.pool[:, old]
                self.refs[old] -= 1
                self.refs[p] += 1
                self.table[s, have - 1] = p
            for j in range(have, want):
                p = free.pop(0)
                self.refs[p] += 1
                self.table[s, j] = p
            self.lens[s] += n

    def row_parts(self, layer, s, pos, h):
        """The four byte ranges of one token and head, as views."""
        D = self.D
        tile = tile_at(self.pool[layer], self.table, s, pos, h, self.heads, D, self.page)
        i = pos % 16
        return (tile[:8 * D].reshape(D // 32, 16, 16)[:, i], tile[8 * D:16 * D].reshape(16, D // 2)[i],
                tile[16 * D:17 * D].reshape(16, D // 16)[i], tile[17 * D:].reshape(16, D // 16)[i])

    def compact(self, keep, cu):
        for s in range(len(self.lens)):
            n = int(cu[s + 1] - cu[s])
            if n == 0:
                continue
            first = int(self.lens[s]) - n
            kept = [i for i in range(min(n, 64)) if keep[cu[s] + i]]
            for rank, i in enumerate(kept):
                if rank == i:
                    continue
                for layer in range(self.pool.shape[0]):
                    for h in range(self.heads):
                        for a, b in zip(self.row_parts(layer, s, first + rank, h), self.row_parts(layer, s, first + i, h)):
                            a[...] = b
            self.lens[s] = first + len(kept)
            self.drop(s, self.pages_of(self.lens[s]))
