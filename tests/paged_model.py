"""A plain numpy model of the paged FP4 cache and of the operators around it,
in 64 bits, one page and one row at a time (what include/csa2.h says, nothing
shared with the library)."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """Values of the codes 0 .. 126."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def nearest_even(x, table):
    """Index of the nearest value of an ascending table (ties: the even index)."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    d = (x - table[lo]) - (table[hi] - x)
    return np.where((d < 0) | ((d == 0) & (lo % 2 == 0)), lo, hi)


def quantise(x):
    """float64 [..., D] -> (rows uint8 [..., D/2 + D/16], their values float64)."""
    D = x.shape[-1]
    g = x.reshape(x.shape[:-1] + (D // 16, 16))
    scale = nearest_even(np.abs(g).max(-1, keepdims=True) / 6.0, e4m3_values())
    s = e4m3_values()[scale]
    mag = nearest_even(np.abs(g) / np.where(s == 0, 1.0, s), E2M1)
    mag = np.where(s == 0, 0, mag)
    code = (mag + 8 * (np.signbit(g) & (s != 0))).reshape(x.shape)
    rows = np.concatenate([code[..., 0::2] | code[..., 1::2] << 4, scale[..., 0]], -1)
    return rows.astype(np.uint8), (E2M1[mag] * np.where(np.signbit(g), -1.0, 1.0) * s).reshape(x.shape)


def values(rows, D):
    """uint8 rows -> float64 values."""
    code = np.stack([rows[..., : D // 2] & 15, rows[..., : D // 2] >> 4], -1).reshape(
        rows.shape[:-1] + (D,))
    s = e4m3_values()[np.minimum(rows[..., D // 2:], 126)]
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(s, 16, axis=-1)


def turns(R, base=10000.0, scaling="plain", factor=1.0, context=0.0, fast=32.0, slow=1.0):
    """theta_i / (2 pi), as float64."""
    if R == 0:
        return np.zeros(0)
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2.0))
    theta = base ** (-2.0 * np.arange(R // 2) / R)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "yarn":
        g = np.clip((context * theta / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        theta = (1 - g) * theta / factor + g * theta
    return theta / (2 * math.pi)


def norm_rope(x, pos, fixed, begin, interleaved, inverse=False, rot_scale=1.0, eps=1e-6,
              norm=True, weight=None):
    """x float64 [n, ..., D], pos [n], fixed: the turns as integers times 2^64."""
    y = np.array(x, np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight
    out = y.copy()
    R = 2 * len(fixed)
    for n in range(len(pos)):
        for i, t in enumerate(fixed):
            frac = (int(pos[n]) * int(t)) % (1 << 64)
            phi = 2 * math.pi * (frac / 2.0 ** 64) * (-1.0 if inverse else 1.0)
            u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            a, b = y[n, ..., begin + u], y[n, ..., begin + v]
            out[n, ..., begin + u] = rot_scale * (a * math.cos(phi) - b * math.sin(phi))
            out[n, ..., begin + v] = rot_scale * (b * math.cos(phi) + a * math.sin(phi))
    return out


def attention(q, v, scale):
    """q float64 [H][D], v float64 [n][D] (keys and values) -> (out [H][D], lse [H])."""
    if len(v) == 0:
        return np.zeros(q.shape), np.full(q.shape[0], -np.inf)
    x = q @ v.T * scale
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    return p @ v / p.sum(-1, keepdims=True), (m + np.log(p.sum(-1, keepdims=True)))[:, 0]


class Cache:
    """rows [P][page][row bytes], table [S][M], length [S], refs [P]; one thing at a time."""

    def __init__(self, rows, S, M):
        self.rows = rows
        self.P, self.page = rows.shape[:2]
        self.table = np.full((S, M), -1, np.int32)
        self.length = np.zeros(S, np.int32)
        self.refs = np.zeros(self.P, np.int32)
        self.no_pages = self.bad = False

    def pages_for(self, n):
        return -(-n // self.page)

    def _sound(self, slots):
        S = len(self.length)
        slots = [int(s) for s in slots]
        ok = [0 <= s < S and slots.count(s) == 1 for s in slots]
        if not all(ok):
            self.bad = True
        return ok

    def resize(self, seq, new_len):
        ok = self._sound(seq)
        before, refs = [p for p in range(self.P) if self.refs[p] == 0], self.refs.copy()
        wanted = 0                                   # pages asked for so far, carried out or not
        for i, s in enumerate(seq):
            if not ok[i]:
                continue
            new, cur = int(new_len[i]), int(self.length[s])
            if not 0 <= new <= self.table.shape[1] * self.page:
                self.bad = True
                continue
            have, want = self.pages_for(cur), self.pages_for(new)
            tail = self.table[s, have - 1] if new > cur and cur % self.page else -1
            copy = tail >= 0 and refs[tail] > 1
            need = max(0, want - have) + copy
            first, wanted = wanted, wanted + need
            if need and wanted > len(before):
                self.no_pages = True
                continue
            take = before[first:wanted]
            if copy:
                p, take = take[0], take[1:]
                self.rows[p, : cur % self.page] = self.rows[tail, : cur % self.page]
                self.table[s, have - 1] = p
                self.refs[p] = 1
                self.refs[tail] -= 1
            for j, p in enumerate(take):
                self.table[s, have + j] = p
                self.refs[p] = 1
            for j in range(want, have):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.length[s] = new

    def fork(self, src, dst):
        S = len(self.length)
        ok = [o and 0 <= int(a) < S for o, a in zip(self._sound(dst), src)]
        if not all(ok):
            self.bad = True
        table, length = self.table.copy(), self.length.copy()
        for i, (a, b) in enumerate(zip(src, dst)):
            if ok[i]:
                for p in table[a][table[a] >= 0]:
                    self.refs[p] += 1
                for p in table[b][table[b] >= 0]:
                    self.refs[p] -= 1
                self.table[b], self.length[b] = table[a], length[a]

    def compact(self):
        used = int((self.refs > 0).sum())
        holes = [p for p in range(used) if self.refs[p] == 0]
        moved = [p for p in range(used, self.P) if self.refs[p] > 0]
        for a, b in zip(moved, holes):
            self.rows[b] = self.rows[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return used

    def entries(self, s, n=None):
        n = int(self.length[s]) if n is None else n
        at = np.arange(n)
        return self.rows[self.table[s, at // self.page], at % self.page]
