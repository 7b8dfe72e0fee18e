"""CPU oracle of the 8-bit paged key/value cache (np_kv_*), numpy in 64 bits.

Restates the operations that include/np.h defines for the cache, page by page
and token by token: reserve, fork, release, compact, append, attend.  Test
infrastructure only.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even), saturating at +-448; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def scale_for(amax: float) -> float:
    """Smallest 2^e, -40 <= e <= 40, with amax <= 448 * 2^e."""
    for e in range(-40, 41):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 40


class KvError(Exception):
    pass


class KvOracle:
    """One cache.  Codes are held as the values they stand for (code units):
    k [L][pages][H][64][D], v [L][pages][H][D][64] float64."""

    def __init__(self, n_layers, n_pages, n_kv_heads, head_dim, max_seqs, max_pages):
        self.L, self.P, self.H, self.D = n_layers, n_pages, n_kv_heads, head_dim
        self.k = np.zeros((n_layers, n_pages, n_kv_heads, PAGE, head_dim))
        self.v = np.zeros((n_layers, n_pages, n_kv_heads, head_dim, PAGE))
        self.ks = np.zeros((n_layers, n_pages, n_kv_heads))
        self.vs = np.zeros((n_layers, n_pages, n_kv_heads))
        self.table = np.full((max_seqs, max_pages), -1, dtype=np.int64)
        self.len = np.zeros(max_seqs, dtype=np.int64)
        self.refs = np.zeros(n_pages, dtype=np.int64)

    # -- pages ---------------------------------------------------------------
    def reserve(self, n_new, seqs=None):
        seqs = range(len(n_new)) if seqs is None else seqs
        table, refs, length = self.table.copy(), self.refs.copy(), self.len.copy()
        free = [p for p in range(self.P) if refs[p] == 0]
        copies, fresh = [], []
        for row, m in zip(seqs, n_new):
            if length[row] + m > table.shape[1] * PAGE:
                raise KvError("row too short")
            slot, off = divmod(int(length[row]), PAGE)
            first = slot + (off > 0)
            if m and off and refs[table[row, slot]] > 1:
                if not free:
                    raise KvError("no page")
                new = free.pop(0)
                copies.append((table[row, slot], new))
                refs[table[row, slot]] -= 1
                refs[new] = 1
                table[row, slot] = new
            for s in range(first, -(-int(length[row] + m) // PAGE)):
                if not free:
                    raise KvError("no page")
                table[row, s] = free.pop(0)
                refs[table[row, s]] = 1
                fresh.append(table[row, s])
            length[row] += m
        self.table, self.refs, self.len = table, refs, length
        for a, b in copies:
            self._copy(a, b)

    def _copy(self, a, b):
        for t in (self.k, self.v, self.ks, self.vs):
            t[:, b] = t[:, a]

    def fork(self, src, dst):
        if len(set(dst)) != len(dst):
            raise KvError("repeated dst")
        rows, lens = self.table[list(src)].copy(), self.len[list(src)].copy()
        for r in rows:
            for p in r[r >= 0]:
                self.refs[p] += 1
        for d in dst:
            for p in self.table[d][self.table[d] >= 0]:
                self.refs[p] -= 1
        self.table[list(dst)], self.len[list(dst)] = rows, lens

    def release(self, seqs, window=0, sinks=0):
        for row in seqs:
            for s in range(self.table.shape[1]):
                p = self.table[row, s]
                if p < 0:
                    continue
                if window:
                    # a later query, at position >= len, sees j > len - window and j < sinks
                    if any(j > self.len[row] - window or j < sinks for j in range(s * PAGE, s * PAGE + PAGE)):
                        continue
                self.refs[p] -= 1
                self.table[row, s] = -1
            if not window:
                self.len[row] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        ends = [p for p in range(live, self.P) if self.refs[p] > 0]
        for a, b in zip(ends, holes):
            self._copy(a, b)
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0

    # -- tokens ----------------------------------------------------------------
    def append(self, layer, k, v, counts, seqs=None):
        """k, v float64 [tokens][H][D]."""
        seqs = range(len(counts)) if seqs is None else seqs
        at = 0
        for row, n in zip(seqs, counts):
            pos = int(self.len[row]) - n
            while pos < self.len[row]:
                slot, off = divmod(pos, PAGE)
                m = min(PAGE - off, int(self.len[row]) - pos)
                p = self.table[row, slot]
                for h in range(self.H):
                    kk, vv = k[at:at + m, h].copy(), v[at:at + m, h].copy()
                    kk[np.isnan(vv).any(1), 0] = np.nan
                    top_k = _nanmax(k[at:at + m, h])
                    top_v = _nanmax(vv)
                    vv[np.isnan(vv)] = 0.0
                    self.ks[layer, p, h] = _write(self.k[layer, p, h], self.ks[layer, p, h], kk, off, top_k)
                    self.vs[layer, p, h] = _write(self.v[layer, p, h].T, self.vs[layer, p, h], vv, off, top_v)
                pos += m
                at += m

    def keys_values(self, layer, row, h):
        """(k, v, present) of a row's tokens, in real units."""
        n = int(self.len[row])
        k, v = np.zeros((n, self.D)), np.zeros((n, self.D))
        present = np.zeros(n, dtype=bool)
        for s in range(-(-n // PAGE)):
            p = self.table[row, s]
            if p < 0:
                continue
            m = min(PAGE, n - s * PAGE)
            with np.errstate(invalid="ignore"):
                k[s * PAGE:s * PAGE + m] = self.k[layer, p, h, :m] * self.ks[layer, p, h]
                v[s * PAGE:s * PAGE + m] = self.v[layer, p, h, :, :m].T * self.vs[layer, p, h]
            present[s * PAGE:s * PAGE + m] = True
        return k, v, present

    def attend(self, layer, q, counts, scale, window=0, sinks=0, seqs=None):
        """q float64 [tokens][heads][D] -> (out, magnitude, reach), where
        magnitude = sum_j p_j |v_j| (what rounding of the weights scales with)
        and reach = (visible keys, max_j scale sum_d |q_d k_jd|, max |v|)."""
        seqs = range(len(counts)) if seqs is None else seqs
        heads = q.shape[1]
        out, mag = np.zeros_like(q), np.zeros_like(q)
        reach = np.zeros(q.shape[:2] + (3,))
        at = 0
        for row, n in zip(seqs, counts):
            length = int(self.len[row])
            for h in range(heads):
                k, v, present = self.keys_values(layer, row, h // (heads // self.H))
                for i in range(n):
                    p = length - n + i
                    j = np.arange(length)
                    see = (j <= p) & present
                    if window:
                        see &= (j > p - window) | (j < sinks)
                    if not see.any():
                        continue
                    qi = q[at + i, h]
                    with np.errstate(invalid="ignore"):
                        z = k[see] @ qi * scale
                        w = np.exp(z - z.max())
                        w /= w.sum()
                        out[at + i, h] = w @ v[see]
                        mag[at + i, h] = w @ np.abs(v[see])
                        reach[at + i, h] = (see.sum(), (np.abs(k[see]) @ np.abs(qi)).max() * scale,
                                            np.abs(v[see]).max())
            at += n
        return out, mag, reach


def _nanmax(x):
    a = np.abs(x)
    a = a[~np.isnan(a)]
    return float(a.max()) if a.size else 0.0


def _write(codes, scale, x, off, top):
    """Tokens x [m][D] into codes [64][D] from row `off`; the new scale."""
    now = scale_for(top)
    if off:
        now = max(now, scale)
        if now != scale:
            codes[:off] = e4m3_round(codes[:off] * (scale / now))
    codes[off:off + len(x)] = e4m3_round(x / now)
    return now
