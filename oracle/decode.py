"""fp64 / integer reference of the 8-bit tree cache and its single-token attention.

Written from the definitions only: e4m3 codes through a table of the format's 256
values, page scales by trial over powers of two, attention query by query over the
tokens of the query's own root path.
"""
from __future__ import annotations

import numpy as np

PAGE = 64
MIN_EXP = -100


def e4m3_values() -> np.ndarray:
    """The value of every byte: sign, 4 exponent bits (bias 7), 3 mantissa bits, no
    infinities; 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


VALUES = e4m3_values()


def encode(x) -> np.ndarray:
    """Bytes of the nearest e4m3 values (ties to the even mantissa); beyond 448
    saturates, NaN is NaN, the sign of zero is kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    table = VALUES[:127]
    hi = np.minimum(np.searchsorted(table, np.where(np.isnan(a), 0, a)), 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - table[lo], table[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def page_exp(x) -> int:
    """Exponent of the scale of a page's values: the smallest e >= -100 with the
    largest finite magnitude at most 448 * 2^e."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    amax = np.max(x[np.isfinite(x)], initial=0.0)
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """The pages as numpy arrays, with the writes of the definition."""

    def __init__(self, k8, v8, ks, vs):
        self.k8, self.v8 = k8.copy(), v8.copy()      # uint8 [P, hkv, 64, d], [P, hkv, d, 64]
        self.ks, self.vs = ks.copy(), vs.copy()      # float [P, hkv]

    def write_page(self, page, k, v):
        """k, v [n <= 64, hkv, d]: the page's first n tokens."""
        n = k.shape[0]
        for h in range(k.shape[1]):
            for x, s in ((k, self.ks), (v, self.vs)):
                s[page, h] = 2.0 ** page_exp(x[:, h])
            self.k8[page, h, :n] = encode(k[:, h] / float(self.ks[page, h]))
            self.v8[page, h, :, :n] = encode(v[:, h] / float(self.vs[page, h])).T

    def append(self, page, slot, k, v):
        """k, v [hkv, d]: token `slot` of the page, after `slot` older ones."""
        for h in range(k.shape[0]):
            for x, s, codes in ((k[h], self.ks, self.k8[page, h]), (v[h], self.vs, self.v8[page, h].T)):
                new = 2.0 ** page_exp(x)
                if slot and float(s[page, h]) > new:
                    new = float(s[page, h])
                if slot and new > float(s[page, h]):
                    codes[:slot] = encode(VALUES[codes[:slot]] * (float(s[page, h]) / new))
                codes[slot] = encode(x / new)
                s[page, h] = new

    def tokens(self, page, h, n):
        """(k, v) [n, d] in fp64."""
        k = VALUES[self.k8[page, h, :n]] * float(self.ks[page, h])
        v = VALUES[self.v8[page, h, :, :n].T] * float(self.vs[page, h])
        return k, v


def node_pages(capacity, pages):
    """Page numbers of every node from the list by node id."""
    out, at = [], 0
    for c in capacity:
        n = -(-int(c) // PAGE)
        out.append([int(p) for p in pages[at:at + n]])
        at += n
    return out


def decode(cache: Cache, parent, lens, capacity, pages, query_nodes, q, scale):
    """o [R, hq, d], lse [hq, R] in fp64, with what their error bounds need:
    mass [R, hq, d] = sum_j p_j |v_j|, reach [hq, R] = max_j scale * sum_f |q_f k_jf| and
    coarse [R, hq, d] = max_j(p_j s_j) * sum_j |v_j / s_j|, s_j the scale of j's page.
    Rows of padding queries (-1) are NaN."""
    R, hq, d = q.shape
    hkv = cache.k8.shape[1]
    q = np.asarray(q, dtype=np.float64)
    at = node_pages(capacity, pages)
    o, lse = np.full((R, hq, d), np.nan), np.full((hq, R), np.nan)
    mass, coarse, reach = np.zeros((R, hq, d)), np.zeros((R, hq, d)), np.zeros((hq, R))
    for r in range(R):
        path, u = [], int(query_nodes[r])
        if u < 0:
            continue
        while u >= 0:
            path.append(u)
            u = int(parent[u])
        for h in range(hkv):
            ks, vs, sc = [np.zeros((0, d))], [np.zeros((0, d))], [np.zeros(0)]
            for u in path:
                left = max(0, min(int(lens[u]), int(capacity[u])))
                for p in at[u]:
                    n = min(PAGE, left)
                    if n > 0:
                        k, v = cache.tokens(p, h, n)
                        ks.append(k)
                        vs.append(v)
                        sc.append(np.full(n, float(cache.vs[p, h])))
                        left -= n
            k, v, sc = np.concatenate(ks), np.concatenate(vs), np.concatenate(sc)
            for a in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                if not len(k):
                    o[r, a], lse[a, r] = 0, -np.inf
                    continue
                s = scale * (k @ q[r, a])
                top = s.max()
                w = np.exp(s - top)
                lse[a, r] = top + np.log(w.sum())
                w = w / w.sum()
                o[r, a], mass[r, a] = w @ v, w @ np.abs(v)
                coarse[r, a] = (w * sc).max() * np.abs(v / sc[:, None]).sum(0)
                reach[a, r] = scale * (np.abs(k) @ np.abs(q[r, a])).max()
    return o, lse, mass, coarse, reach
