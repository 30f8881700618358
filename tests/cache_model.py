"""A plain model of the 4-bit key/value cache in NumPy, for the tests: the
documented layout, written byte by byte from the oracle's codes, and attention
in 64 bits from the definition, with the bound its outputs are held to."""
import numpy as np

import oracle


def blocks(D):
    return next(c for c in (2, 3, 4, 6, 8) if 32 * c >= D)


class Model:
    """Host arrays of one cache in the layout of include/int4dq_cache.h."""

    def __init__(self, pages, page_size, heads, D, group, affine, fill=0):
        self.P, self.S, self.H, self.D, self.affine = pages, page_size, heads, D, affine
        self.group = min(group, D)
        self.C, self.G = blocks(D), -(-D // self.group)
        DB, u = 16 * self.C, (pages, heads, page_size // 16)
        self.packed = {"k": np.full((pages, heads, page_size, DB), fill, np.uint8),
                       "v": np.full((*u, DB, 16), fill, np.uint8)}
        self.scales = {s: np.full((*u, self.G, 16), fill, np.uint16).view(np.float16) for s in "kv"}
        self.zeros = {s: np.full((*u, self.G, 16), fill, np.uint8) if affine else None for s in "kv"}

    # ---------------------------------------------------------------- rows
    def place(self, table, lengths, starts, t):
        """(sequence, position, page or -1) of row t, or None."""
        B = len(lengths)
        if starts is None:
            b, end = t, t + 1
        else:
            own = [b for b in range(B) if starts[b] <= t < starts[b + 1]]
            if not own:
                return None
            b, end = own[0], int(starts[own[0] + 1])
        pos = int(lengths[b]) - (end - t)
        return b, pos, self.page(table, b, pos)

    def page(self, table, b, pos):
        if pos < 0 or pos // self.S >= table.shape[1]:
            return -1
        p = int(table[b, pos // self.S])
        return p if 0 <= p < self.P else -1

    # ---------------------------------------------------------------- write
    def write(self, k, v, table, lengths, starts):
        for t in range(k.shape[0]):
            at = self.place(table, lengths, starts, t)
            if at is None or at[2] < 0:
                continue
            self.put("k", k[t], at[2], at[1] % self.S)
            self.put("v", v[t], at[2], at[1] % self.S)

    def put(self, side, x, page, slot):
        """x [H, D] float32 at one slot."""
        if self.affine:
            packed, scales, zeros, _ = oracle.quantize_int4_affine(np.ascontiguousarray(x), self.group)
            self.zeros[side][page, :, slot // 16, :, slot % 16] = zeros
        else:
            packed, scales, _ = oracle.quantize_int4(np.ascontiguousarray(x), self.group)
        row = np.zeros((self.H, 16 * self.C), np.uint8)
        row[:, :packed.shape[1]] = packed                # byte j: channels 2j, 2j + 1
        self.scales[side][page, :, slot // 16, :, slot % 16] = scales
        if side == "v":
            self.packed["v"][page, :, slot // 16, :, slot % 16] = row
        else:
            self.packed["k"][page, :, slot] = row[:, self.key_order()]

    def key_order(self):
        """Natural byte of each byte of a key row."""
        p = np.arange(16 * self.C)
        a, i, e = p // (4 * self.C), p % (4 * self.C) // 4, p % 4
        return 16 * i + 4 * a + e

    # ---------------------------------------------------------------- values
    def values(self, side, page, slot):
        """float32 [H, D] that one slot stands for, and the scale of each channel."""
        if side == "v":
            row = self.packed["v"][page, :, slot // 16, :, slot % 16]
        else:
            row = np.empty((self.H, 16 * self.C), np.uint8)
            row[:, self.key_order()] = self.packed["k"][page, :, slot]
        u = np.stack([row & 15, row >> 4], -1).reshape(self.H, -1)[:, :self.D].astype(np.int32)
        g = np.arange(self.D) // self.group
        s = self.scales[side][page, :, slot // 16, :, slot % 16].astype(np.float32)[:, g]
        if self.affine:
            c = u - self.zeros[side][page, :, slot // 16, :, slot % 16].astype(np.int32)[:, g]
        else:
            c = np.where(u > 7, u - 16, u)
        return c.astype(np.float32) * s, s

    def read(self, rows, table, lengths, starts):
        k = np.zeros((rows, self.H, self.D), np.float32)
        v = np.zeros_like(k)
        owned = np.zeros(rows, bool)
        for t in range(rows):
            at = self.place(table, lengths, starts, t)
            if at is None:
                continue
            owned[t] = True
            if at[2] >= 0:
                k[t], v[t] = self.values("k", at[2], at[1] % self.S)[0], self.values("v", at[2], at[1] % self.S)[0]
        return k, v, owned

    # ---------------------------------------------------------------- attention
    def attend(self, q, table, lengths, starts, scale, causal=True, window=0):
        """q [rows, Hq, D] in 64 bits: out, lse, which rows a sequence owns, and the
        bounds of out (without the rounding of its type) and lse:

        scores: a sum of D products of queries with offset codes up to 15, in
          binary32: delta = scale 2^-24 (D + 16) sum_d |q_d| 16 s_jd, and 2^-22 of
          the score itself for the scaling and the exponential's argument;
        weights: one rounding to binary16, 2^-11, the exponential's and the sum's
          few binary32 roundings, 2^-20; values whose scale is far below another's
          of the same head are held to 2^-24 of the largest;
        values: offset codes up to 15 summed in binary32, one rounding for each 32
          tokens."""
        rows, Hq, D = q.shape
        R = Hq // self.H
        q = q.astype(np.float64)
        out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
        tol, ltol = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
        owned = np.zeros(rows, bool)
        held = {}
        for t in range(rows):
            at = self.place(table, lengths, starts, t)
            if at is None:
                continue
            owned[t] = True
            b, pos, _ = at
            if b not in held:
                js = [j for j in range(int(lengths[b])) if self.page(table, b, j) >= 0]
                got = [(self.values("k", self.page(table, b, j), j % self.S),
                        self.values("v", self.page(table, b, j), j % self.S)) for j in js]
                held[b] = (np.array(js, np.int64),
                           *(np.array([g[i][n] for g in got], np.float64).reshape(-1, self.H, D)
                             for i in (0, 1) for n in (0, 1)))
            js, k, ks, v, vs = held[b]
            see = np.ones(len(js), bool) if not causal else (js <= pos)
            if window:
                see &= js > pos - window
            if not see.any():
                continue
            n = int(see.sum())
            for h in range(Hq):
                kk, kss, vv, vss = (x[see, h // R] for x in (k, ks, v, vs))
                a = kk @ q[t, h] * scale
                m = a.max()
                p = np.exp(a - m)
                w = p / p.sum()
                out[t, h], lse[t, h] = w @ vv, m + np.log(p.sum())
                delta = (scale * 2.0 ** -24 * (D + 16) * (16 * kss @ np.abs(q[t, h])) + 2.0 ** -22 * np.abs(a)).max()
                tol[t, h] = ((2.0 ** -11 + 2 * delta + 2.0 ** -20) * (w @ np.abs(vv))
                             + (n / 32 + 64) * 2.0 ** -24 * 15 * (w @ vss) + 2.0 ** -24 * vss.max())
                ltol[t, h] = delta + 2.0 ** -20 + 2.0 ** -22 * abs(lse[t, h])
        return out, lse, owned, tol, ltol


def plan(rng, lengths, new, page_size, spare=3):
    """Page table of random distinct pages (unused entries -1), and the page count."""
    need = [-(-int(n) // page_size) for n in lengths]
    total = sum(need) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(lengths), max(need + [1])), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return table, total, starts
