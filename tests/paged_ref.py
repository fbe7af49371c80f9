"""Plain implementations of the paged-cache operators for the tests: page accounting as
Python loops over numpy arrays, norm, rotation and attention in float64."""
import math

import numpy as np


def pages_of(n, ps):
    return -(-n // ps)


class Pages:
    """Page accounting with the rules of mk_pages_resize / fork / compact. `slot[p]` stands for
    a page's contents: one number per slot."""

    def __init__(self, n_pages, n_seqs, max_pages, ps):
        self.ps = ps
        self.table = np.full((n_seqs, max_pages), -1, np.int32)
        self.len = np.zeros(n_seqs, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.slot = np.zeros((n_pages, ps), np.int64)

    def copy(self):
        o = Pages(len(self.ref), len(self.len), self.table.shape[1], self.ps)
        o.table, o.len, o.ref, o.slot = self.table.copy(), self.len.copy(), self.ref.copy(), self.slot.copy()
        return o

    def _free(self):
        return [p for p in range(len(self.ref)) if self.ref[p] == 0]

    def resize(self, seqs, lens):
        """False (and nothing changed) with too few free pages."""
        o, ps = self.copy(), self.ps
        for s, n in zip(seqs, lens):
            for j in range(pages_of(n, ps), pages_of(int(o.len[s]), ps)):
                o.ref[o.table[s, j]] -= 1
                o.table[s, j] = -1
        own = [min(int(o.len[s]), n) % ps > 0 and o.ref[o.table[s, min(int(o.len[s]), n) // ps]] > 1 for s, n in zip(seqs, lens)]
        free = o._free()
        for s, n, mine in zip(seqs, lens, own):
            low = min(int(o.len[s]), n)
            new = ([low // ps] if mine else []) + list(range(pages_of(low, ps), pages_of(n, ps)))
            if len(free) < len(new):
                return False
            for j in new:
                p = free.pop(0)
                if mine and j == low // ps:
                    o.slot[p, :low % ps] = o.slot[o.table[s, j], :low % ps]
                    o.ref[o.table[s, j]] -= 1
                o.ref[p], o.table[s, j] = 1, p
            o.len[s] = n
        self.__dict__.update(o.__dict__)
        return True

    def fork(self, src, dst):
        o, ps = self.copy(), self.ps
        for b in dst:
            for j in range(pages_of(int(o.len[b]), ps)):
                o.ref[o.table[b, j]] -= 1
            o.table[b] = -1
        free = o._free()
        for a, b in zip(src, dst):
            n = int(o.len[a])
            for j in range(pages_of(n, ps)):
                p = o.table[a, j]
                if (j + 1) * ps <= n:
                    o.ref[p] += 1
                else:
                    if not free:
                        return False
                    to = free.pop(0)
                    o.slot[to, :n % ps] = o.slot[p, :n % ps]
                    o.ref[to], p = 1, to
                o.table[b, j] = p
            o.len[b] = n
        self.__dict__.update(o.__dict__)
        return True

    def compact(self):
        live = [p for p in range(len(self.ref)) if self.ref[p] > 0]
        to = dict(zip([p for p in live if p >= len(live)], [p for p in range(len(live)) if self.ref[p] == 0]))
        for a, b in to.items():
            self.slot[b] = self.slot[a]
            self.ref[b], self.ref[a] = self.ref[a], 0
        for s in range(len(self.len)):
            for j in range(pages_of(int(self.len[s]), self.ps)):
                self.table[s, j] = to.get(int(self.table[s, j]), self.table[s, j])


def rope(x, gain, pos, rot, eps, theta):
    """x float64 [rows][heads][d] -> (result, |normed a| + |normed b| per entry: the scale of its rounding errors)."""
    d = x.shape[-1]
    if gain is not None:
        x = x * gain / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, mag = x.copy(), np.abs(x)
    h = rot // 2
    if h:
        ang = pos[:, None].astype(np.float64) * np.array([math.pow(theta, -2.0 * i / rot) for i in range(h)])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * c - b * s, b * c + a * s
        mag[..., :h] = mag[..., h:rot] = np.abs(a) + np.abs(b)
    assert d >= rot
    return y, mag


def attention(q, k, v, pos, scale):
    """q [rows][hq][d], k, v [positions][hkv][d] (float64), pos [rows] -> (o, sum of w |v|, largest sum |q||k|)."""
    rows, hq, d = q.shape
    g = hq // k.shape[1] if k.shape[1] else 1
    o, mag, big = np.zeros_like(q), np.zeros_like(q), 0.0
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        z = q[:, h] @ kk.T * scale
        z = np.where(np.arange(len(kk))[None, :] <= pos[:, None], z, -np.inf)
        seen = pos >= 0
        if not seen.any() or not len(kk):
            continue
        zz = z[seen]
        w = np.exp(zz - zz.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        o[seen, h], mag[seen, h] = w @ vv, w @ np.abs(vv)
        big = max(big, float((np.abs(q[:, h]) @ np.abs(kk).T).max()))
    return o, mag, big


def attention_bound(o, mag, big, scale, d):
    """How far a bf16 result may be from o. Inputs are exact in bf16; each score is an fp32 sum of d
    products, so it is off by at most e = (d + 2) 2^-24 scale sum|q||k|, and a weight by the
    factor exp(2 e) together with its sum; exp and the fp32 sums add 2^-18; a weight enters
    the value product as bf16, off by 2^-8 of itself, while the sum of weights does not; the result is rounded once, 2^-8 of itself."""
    e = (d + 2) * 2.0 ** -24 * abs(scale) * big
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + math.expm1(2 * e) + 2.0 ** -18) * mag * (1 + 2.0 ** -8) + 1e-30
