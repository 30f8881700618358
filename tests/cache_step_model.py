"""A plain model of a serving step around the 4-bit cache, for the tests: the page
table of a batch in Python lists, and norms and rotation in NumPy, both in the
documented order of roundings and in 64 bits."""
import numpy as np

INT32_MAX = 2 ** 31 - 1


def _count(said, pages):
    return min(max(int(said), 0), pages)


def _entries(length, S, most):
    return min(-(-max(int(length), 0) // S), most)


def release(table, lengths, free, count, S, done, shared=None):
    """(lengths, free, count) afterwards; arrays as the call takes them."""
    pages, free = len(free), free.copy()
    left = _count(count[0], pages)
    skip = max(int(shared), 0) // S if shared is not None else 0
    new = lengths.copy()
    for b in range(len(lengths)):
        if not done[b]:
            continue
        new[b] = 0
        for i in range(skip, _entries(lengths[b], S, table.shape[1])):
            if 0 <= table[b, i] < pages and left < pages:
                free[left] = table[b, i]
                left += 1
    return new, free, np.array([left, 0], np.int32)


def extend(table, lengths, free, count, S, added, rows):
    """(table, lengths, starts, slots, count) afterwards."""
    table, most, pages = table.copy(), table.shape[1], len(free)
    left, lacking = _count(count[0], pages), 0
    new, starts, slots = [], [0], np.full(rows, -1, np.int64)
    for b in range(len(lengths)):
        n, m = max(int(lengths[b]), 0), max(int(added[b]), 0)
        for i in range(_entries(n, S, most), _entries(n + m, S, most)):
            if left > 0:
                left -= 1
                table[b, i] = free[left]
            else:
                lacking += 1
                table[b, i] = -1
        for i in range(m):
            t, p = starts[-1] + i, n + i
            if t < rows and p // S < most and 0 <= table[b, p // S] < pages:
                slots[t] = int(table[b, p // S]) * S + p % S
        new.append(min(n + m, INT32_MAX))
        starts.append(min(starts[-1] + m, INT32_MAX))
    return (table, np.array(new, np.int32), np.array(starts, np.int32), slots, np.array([left, lacking], np.int32))


def rope_table(positions, rotary, base=10000.0):
    angle = np.outer(np.arange(positions), base ** (-np.arange(rotary // 2) / (rotary // 2)))
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def pairs(rotary, interleaved):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def transform(x, weight, eps, rope, interleaved):
    """x float32 [rows, heads, D], rope the rows' float32 [rows, rotary] or None, in the
    documented roundings: float32 [rows, heads, D]."""
    x = x.astype(np.float32)
    if weight is not None:
        mean = (x.astype(np.float64) ** 2).sum(-1, keepdims=True) / x.shape[-1]
        with np.errstate(divide="ignore", invalid="ignore"):
            r = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
            x = (x * r) * weight.astype(np.float32)
    if rope is None:
        return x
    half = rope.shape[1] // 2
    a, b = pairs(2 * half, interleaved)
    c, s = rope[:, None, :half], rope[:, None, half:]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def transform64(x, weight, eps, rope, interleaved):
    """The same in 64 bits, and a bound of the roundings' difference from it: r, its
    product and the weight's are 3 roundings of a normalised value, each product with a
    cosine or sine and the sum one more: 5 x 2^-24 of |y_a cos| + |y_b sin|."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / x.shape[-1] + eps) * weight.astype(np.float64)
    size = np.abs(x)
    if rope is not None:
        half = rope.shape[1] // 2
        a, b = pairs(2 * half, interleaved)
        c, s = rope[:, None, :half].astype(np.float64), rope[:, None, half:].astype(np.float64)
        y, z = x.copy(), size.copy()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        z[..., a] = size[..., a] * np.abs(c) + size[..., b] * np.abs(s)
        z[..., b] = size[..., b] * np.abs(c) + size[..., a] * np.abs(s)
        x, size = y, z
    return x, 5.0 * 2.0 ** -24 * size * (1 + 2.0 ** -20) + 2.0 ** -148


class Sinks:
    """Makes a cache model's attention (tests/cache_model.py) one with first tokens that
    stay visible, from its own bounds: those tokens and the window's are all that a row's
    part of the cache holds."""

    def __init__(self, model, sinks):
        self.model, self.sinks = model, sinks

    def __getattr__(self, name):
        return getattr(self.model, name)

    def attend(self, q, table, lengths, starts, scale, causal=True, window=0):
        m, rows = self.model, q.shape[0]
        if not window:
            return m.attend(q, table, lengths, starts, scale, causal, window)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        lse, ltol = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
        owned = np.zeros(rows, bool)
        for t in range(rows):
            at = m.place(table, lengths, starts, t)
            if at is None:
                continue
            owned[t] = True
            b, pos, _ = at
            top = min(pos + 1, int(lengths[b]))
            # one row that sees all keys of a cache whose pages between the first tokens and
            # the window are gone; tokens of the pages at the two borders one by one
            gone = _Hidden(m, lambda j: self.sinks <= j <= pos - window)
            o, l, _, tl, ll = gone.attend(q[t:t + 1], table[b:b + 1], [max(top, 0)], None, scale, False)
            out[t], lse[t], tol[t], ltol[t] = o[0], l[0], tl[0], ll[0]
        return out, lse, owned, tol, ltol


class _Hidden:
    """A model in which some positions have no page."""

    def __init__(self, model, hides):
        self.m, self.hides = model, hides
        self.H, self.S = model.H, model.S
        self.values, self.place = model.values, model.place

    def page(self, table, b, pos):
        return -1 if self.hides(pos) else self.m.page(table, b, pos)

    def attend(self, *a):
        return type(self.m).attend(self, *a)
