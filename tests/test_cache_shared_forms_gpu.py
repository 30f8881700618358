"""Attention over the 4-bit cache for a batch that shares its first tokens, on MI355X, in every
pair of tile heights that the two parts can have, and where the library itself decides that
sharing pays: against the model's attention over whole sequences, within its bounds. Which
heights each case has is checked on the host too (tests/test_sanitize_parts_cpu.py)."""
import numpy as np
import pytest
import torch

from tests.cache_step_model import Sinks
from tests.test_cache_gpu import BF16, F16, check_attention, cache_of, dq, rounded, say  # noqa: F401
from tests.test_cache_shared_gpu import DEV, batch

pytestmark = pytest.mark.gpu


class Batch(Sinks):
    """The model's attention with a sequence's rows and one head at a time; the bounds of
    cache_model.Model.attend, of the worst visible key likewise."""

    def held(self):
        if not hasattr(self, "_held"):
            m = self.model
            got = [[m.values(s, p, j) for p in range(m.P) for j in range(m.S)] for s in "kv"]
            self._held = [np.array([x[i] for x in g], np.float64).reshape(m.P, m.S, m.H, m.D) for g in got for i in (0, 1)]
        return self._held

    def attend(self, q, table, lengths, starts, scale, causal=True, window=0):
        m, D = self.model, q.shape[2]
        q = q.astype(np.float64)
        starts = np.arange(len(lengths) + 1) if starts is None else starts
        out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
        tol, ltol, owned = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(len(q), bool)
        for b, n in enumerate(lengths):
            rows = np.arange(starts[b], starts[b + 1])
            owned[rows] = True
            js = np.arange(min(max(int(n), 0), table.shape[1] * m.S))
            page = table[b, js // m.S]
            js = js[(page >= 0) & (page < m.P)]
            if len(js) == 0 or len(rows) == 0:
                continue
            k, ks, v, vs = (x[table[b, js // m.S], js % m.S] for x in self.held())
            pos = (int(n) - len(rows) + rows - rows[0])[:, None]
            see = (js <= pos) if causal else np.ones((len(rows), len(js)), bool)
            if window:
                see = see & ((js > pos - window) | (js < self.sinks))
            some = see.any(1)
            rows, see = rows[some], see[some]
            if len(rows) == 0:
                continue
            js, k, ks, v, vs = (x[see.any(0)] for x in (js, k, ks, v, vs))
            see = see[:, see.any(0)]
            count = see.sum(1)[:, None]
            for h in range(q.shape[1]):
                kh, x = h // (q.shape[1] // m.H), q[rows, h]
                a = np.where(see, x @ k[:, kh].T * scale, -np.inf)
                top = a.max(1, keepdims=True)
                p = np.exp(a - top)
                w = p / p.sum(1, keepdims=True)
                out[rows, h], lse[rows, h] = w @ v[:, kh], top[:, 0] + np.log(p.sum(1))
                delta = np.where(see, scale * 2.0 ** -24 * (D + 16) * 16 * (np.abs(x) @ ks[:, kh].T)
                                 + 2.0 ** -22 * np.abs(np.where(see, a, 0)), 0).max(1, keepdims=True)
                tol[rows, h] = ((2.0 ** -11 + 2 * delta + 2.0 ** -20) * (w @ np.abs(v[:, kh]))
                                + (count / 32 + 64) * 2.0 ** -24 * 15 * (w @ vs[:, kh])
                                + 2.0 ** -24 * np.where(see, vs[:, kh].max(1), 0).max(1, keepdims=True))
                ltol[rows, h] = delta[:, 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[rows, h])
        return out, lse, owned, tol, ltol


# D, group, affine, heads, ratio, page, dtype, shared pages, table entries (0: what it needs), own tokens, new rows,
# then the tile heights of the sequences' own part and of the shared one
FORMS = [
    (64, 64, False, 1, 4, 64, F16, 11, 0, [150, 93, 300, 91, 120, 200, 95, 97], [90, 93, 120, 91, 88, 130, 95, 97], 128, 128),
    (128, 64, True, 1, 8, 32, BF16, 30, 0, [70, 52, 90, 48, 61], [60, 52, 61, 48, 61], 128, 128),
    (192, 64, False, 1, 4, 64, BF16, 10, 0, [100, 70, 99, 130, 140, 90, 120], [77, 70, 71, 75, 80, 81, 76], 128, 128),
    (64, 32, True, 1, 16, 16, BF16, 40, 0, [1 + n % 37 for n in range(130)], [1] * 130, 16, 128),
    (64, 64, False, 1, 4, 64, BF16, 12, 0, [13 + n for n in range(40)], [13] * 40, 32, 128),
    (96, 96, False, 2, 6, 32, F16, 20, 0, [20 + 3 * n for n in range(60)], [6] * 60, 32, 128),
    (64, 64, False, 1, 3, 256, F16, 3, 70, [100 + 11 * n for n in range(3)], [100, 99, 101], 128, 32),
    (128, 128, False, 1, 4, 64, BF16, 11, 0, [90, 150, 95], [85, 85, 86], 128, 16),
    (128, 128, False, 1, 4, 64, BF16, 11, 0, [90, 150, 95, 70], [55, 60, 56, 59], 32, 16),
    (128, 128, False, 2, 4, 128, BF16, 5, 130, [75 + n for n in range(22)], [3] * 22, 16, 32),
    (64, 64, False, 1, 3, 256, F16, 3, 66, [31 + n for n in range(10)], [10] * 10, 32, 32),
    (80, 128, False, 1, 5, 256, BF16, 2, 64, [31 + n for n in range(60)], [1, 7] * 30, 32, 128),
    (256, 128, True, 1, 8, 64, F16, 9, 0, [40 + n for n in range(65)], [4] * 65, 16, 128),
    (256, 32, True, 1, 8, 64, BF16, 9, 0, [30 + n for n in range(65)], [4] * 65, 16, 16),
]


def table_of(table, entries):
    more = max(0, entries - table.shape[1])
    return np.concatenate([table, np.full((len(table), more), -1, np.int32)], 1)


def call(dq, m, cache, table, lengths, starts, q, dtype, shared, window=0, sinks=0, share_from=1, **kw):
    m.sinks = sinks
    n = torch.tensor([shared], dtype=torch.int32, device=DEV)
    return check_attention(dq, m, table, lengths, starts, q, dtype, window=window, sinks=sinks, shared=n, cache=cache,
                           share_from=share_from, **kw)


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,pages,entries,own,new,own_rows,shared_rows", FORMS)
def test_forms(dq, D, group, affine, heads, ratio, page, dtype, pages, entries, own, new, own_rows, shared_rows):
    rng = np.random.default_rng(D + len(own))
    lengths = [pages * page + n for n in own]
    plain, table, starts = batch(rng, heads, D, group, affine, page, pages, lengths, new)
    table = table_of(table, entries)
    m, cache = Batch(plain, 0), cache_of(dq, plain)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    whole = pages * page
    say("case: forms", D, group, affine, heads, ratio, page, len(own), own_rows, shared_rows)
    for shared in (whole, whole - 37, 5):              # the last two end inside a step
        call(dq, m, cache, table, lengths, starts, q, dtype, shared)
    for window, sinks in ((200, 0), (300, 70), (30, 2 ** 31), (whole // 2, 3)):
        say("case: forms, window", window, sinks)
        call(dq, m, cache, table, lengths, starts, q, dtype, whole - 11, window=window, sinks=sinks)
    call(dq, m, cache, table, lengths, starts, q, dtype, whole - 3, causal=False)
    # sequences that end within the shared tokens, rows whose positions lie among them, an empty one
    short = list(lengths)
    short[0], short[1], short[-1] = whole - 50, whole + 1, 0
    call(dq, m, cache, table, short, starts, q, dtype, whole)
    call(dq, m, cache, table, short, starts, q, dtype, whole, window=90, sinks=20)
    # the keys that no row sees may hold anything: NaN in what is behind and between
    gone = table.copy()
    gone[:, 4:5] = -1
    call(dq, m, cache, gone, lengths, starts, q, dtype, whole)


# the same without heights: cases in which the library shares by itself
PAYS = [
    (64, 64, False, 1, 4, 64, F16, 24, 0, [5 + 7 * n for n in range(16)], [1] * 16),
    (64, 32, True, 1, 2, 256, BF16, 24, 0, [9, 70, 300, 1], [1] * 4),
    (64, 64, False, 1, 5, 256, F16, 64, 0, [20 + 5 * n for n in range(9)], [14 + n for n in range(9)]),
]


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,pages,entries,own,new", PAYS)
def test_where_it_pays(dq, D, group, affine, heads, ratio, page, dtype, pages, entries, own, new):
    """The library's own choice: the same bits as with sharing asked for, below its length those of a call
    without; a workspace made for it."""
    rng = np.random.default_rng(len(own))
    lengths = [pages * page + n for n in own]
    plain, table, starts = batch(rng, heads, D, group, affine, page, pages, lengths, new)
    m, cache = Batch(plain, 0), cache_of(dq, plain)
    T = int(starts[-1])
    q = rounded(rng.normal(size=(T, heads * ratio, D)).astype(np.float32), dtype)
    whole = pages * page
    say("case: pays", D, heads, ratio, len(own), T)
    kw = dict(window=0, sinks=0)
    asked = call(dq, m, cache, table, lengths, starts, q, dtype, whole, share_from=1, **kw)
    chosen = call(dq, m, cache, table, lengths, starts, q, dtype, whole, share_from=None, **kw)
    assert torch.equal(asked[0], chosen[0]) and torch.equal(asked[1], chosen[1])
    n = dq.cache_attention_workspace_bytes(cache, len(own), T, heads * ratio, shared=True)
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    kept = call(dq, m, cache, table, lengths, starts, q, dtype, whole, share_from=None, workspace=ws[:n], **kw)
    assert torch.equal(asked[0], kept[0]) and torch.equal(asked[1], kept[1]) and (ws[n:] == 0xFF).all()
    # few shared tokens: the choice leaves them to the sequences
    few = call(dq, m, cache, table, lengths, starts, q, dtype, 100, share_from=None, **kw)
    alone = check_attention(dq, m, table, lengths, starts, q, dtype, cache=cache)
    assert few[0].shape == alone[0].shape
    call(dq, m, cache, table, lengths, starts, q, dtype, whole, share_from=None, window=whole // 2, sinks=9)
