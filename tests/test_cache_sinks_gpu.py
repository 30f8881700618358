"""Attention over the 4-bit cache with a window and first tokens that stay visible
(int4_cache_attention, sinks=) on MI355X, against the plain model and its bounds."""
import numpy as np
import pytest
import torch

from tests.cache_model import plan
from tests.cache_step_model import Sinks
from tests.test_cache_gpu import BF16, DEV, F16, cache_of, check_attention, dev, dq, filled, rounded, say, values  # noqa: F401
from tests.test_cache_plans_gpu import with_holes

pytestmark = pytest.mark.gpu


def check(dq, m, table, lengths, starts, q, dtype, window, sinks, cache=None, **kw):
    cache = cache or cache_of(dq, m)
    return check_attention(dq, Sinks(m, sinks), table, lengths, starts, q, dtype, window=window, sinks=sinks, cache=cache, **kw)


CASES = [  # D, group, affine, heads, ratio, page, dtype, lengths, new rows
    (128, 128, False, 1, 4, 16, BF16, [1, 300, 77], [1, 1, 1]),
    (128, 64, True, 2, 3, 64, F16, [700, 64, 1], [1, 1, 1]),
    (64, 32, False, 2, 1, 16, F16, [500, 3], [9, 3]),
    (96, 96, True, 1, 6, 32, BF16, [400, 200], [33, 5]),
    (192, 64, False, 1, 2, 16, BF16, [210, 130], [7, 2]),
    (256, 128, True, 1, 8, 32, F16, [333], [4]),
    # the form for prompts
    (128, 128, False, 1, 4, 64, BF16, [500, 140], [200, 140]),
    (64, 64, True, 1, 2, 16, F16, [600], [400]),
    (128, 32, True, 1, 2, 32, BF16, [400], [300]),
]
WINDOWS = [(1, 1), (1, 200), (50, 4), (64, 64), (64, 65), (130, 63), (100, 1000), (5000, 7), (33, 2 ** 40)]


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,lengths,new", CASES)
def test_sinks(dq, D, group, affine, heads, ratio, page, dtype, lengths, new):
    rng = np.random.default_rng(300 + D + sum(new))
    m, table, starts = filled(rng, heads, D, group, affine, page, lengths, new)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    for window, sinks in WINDOWS if sum(new) < 50 else WINDOWS[2:6]:
        say("case: sinks", D, group, affine, heads, ratio, page, lengths, new, window, sinks)
        check(dq, m, table, lengths, starts, q, dtype, window, sinks, cache=cache)
    if set(new) == {1}:
        check(dq, m, table, lengths, None, q, dtype, 40, 5, cache=cache)


def test_without_a_window_sinks_do_nothing(dq):
    rng = np.random.default_rng(31)
    m, table, starts = filled(rng, 1, 64, 64, False, 16, [200, 30], [3, 30])
    q = rounded(rng.normal(size=(33, 2, 64)).astype(np.float32), BF16)
    check(dq, m, table, [200, 30], starts, q, BF16, 0, 9)
    check(dq, m, table, [200, 30], starts, q, BF16, 0, 9, causal=False)


@pytest.mark.parametrize("lengths,new", [([4000, 900, 2500], [1, 1, 1]), ([3000, 1500], [3, 9]), ([2300, 400], [150, 90])])
def test_shared_out_over_blocks(dq, lengths, new):
    """Long windows, whose steps are cut into blocks, the first tokens' steps among them."""
    rng = np.random.default_rng(sum(lengths))
    m, table, starts = filled(rng, 1, 64, 64, False, 64, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), 4, 64)).astype(np.float32), F16)
    cache = cache_of(dq, m)
    for window, sinks in ((2000, 4), (1300, 700), (100, 1500), (64, 64)):
        say("case: shared out", lengths, new, window, sinks)
        check(dq, m, table, lengths, starts, q, F16, window, sinks, cache=cache)


class Prompts(Sinks):
    """The model with all rows of a sequence and head at once, for prompts that it would take minutes
    for row by row; its bounds (cache_model.Model.attend) are those of the worst visible key likewise."""

    def attend(self, q, table, lengths, starts, scale, causal=True, window=0):
        m, D = self.model, q.shape[2]
        q = q.astype(np.float64)
        out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
        tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:2])
        for b, n in enumerate(lengths):
            got = [[m.values(s, table[b, j // m.S], j % m.S) for j in range(n)] for s in "kv"]
            k, v = (np.array([x[0] for x in g], np.float64) for g in got)
            ks, vs = (np.array([x[1] for x in g], np.float64).reshape(n, m.H, D) for g in got)
            rows = np.arange(starts[b], starts[b + 1])
            pos, js = (n - len(rows) + rows - rows[0])[:, None], np.arange(n)
            see = (js <= pos) & ((js > pos - window) | (js < self.sinks))
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
        return out, lse, np.ones(len(q), bool), tol, ltol


@pytest.mark.parametrize("lengths,new", [([1800, 1500], [600, 520]), ([1300, 1400, 1250], [500, 900, 700])])
def test_last_round(dq, lengths, new):
    """Prompts of a few more tiles than the GPU has places: 35 and 66 on 32 of 16 heads. Those of the
    last round are cut, unless the workspace has no room for it or the window is short."""
    rng = np.random.default_rng(sum(lengths))
    m, table, starts = filled(rng, 16, 64, 64, False, 64, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), 64, 64)).astype(np.float32), F16)
    cache = cache_of(dq, m)
    for window, sinks, kw in ((1100, 70, {}), (1100, 70, dict(workspace=torch.empty(0, dtype=torch.uint8, device=DEV))),
                              (300, 10, {})):
        say("case: last round", lengths, new, window, sinks, list(kw))
        check_attention(dq, Prompts(m, sinks), table, lengths, starts, q, F16, window=window, sinks=sinks, cache=cache, **kw)


def test_large_batch(dq):
    """More sequences than a wavefront looks through at once."""
    rng = np.random.default_rng(33)
    lengths = rng.integers(1, 60, size=90)
    lengths[[3, 50, 88]] = [1500, 1100, 1700]
    m, table, starts = filled(rng, 1, 64, 64, True, 16, lengths, np.ones(90, np.int64))
    q = rounded(rng.normal(size=(90, 2, 64)).astype(np.float32), BF16)
    check(dq, m, table, lengths, None, q, BF16, 1100, 20)
    check(dq, m, table, lengths, starts, q, BF16, 16, 130)


BAD = [
    (1, 64, 64, False, 4, 16, F16, [2600, -5, 1900, 0, 40, 1300], [2, 1, 7, 3, 4, 2]),
    (1, 128, 128, True, 3, 32, BF16, [400, 90, 300], [200, 95, 150]),
]


@pytest.mark.parametrize("heads,D,group,affine,ratio,page,dtype,lengths,new", BAD)
def test_bad_plans(dq, heads, D, group, affine, ratio, page, dtype, lengths, new):
    """Pages that are missing, among the first tokens' too, lengths past the table (a window that
    sees nothing while the first tokens are there), rows that no sequence owns."""
    rng = np.random.default_rng(400 + D)
    m, table, claimed, starts, T = with_holes(rng, (heads, D, group, affine), lengths, new, page)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(T, heads * ratio, D)).astype(np.float32), dtype)
    for window, sinks in ((150, 20), (10, 100), (60, 64)):
        say("case: bad plan", heads, D, lengths, new, window, sinks)
        check(dq, m, table, claimed, starts, q, dtype, window, sinks, cache=cache)
    if claimed[-1] > 0:                                # far past the table: only the first tokens are seen
        far = claimed.copy()
        far[-1] = table.shape[1] * page + 5000
        check(dq, m, table, far, starts, q, dtype, 30, 70, cache=cache)


def test_pages_between_are_gone(dq):
    """What lies between the first tokens and the window may be on no page any more, and hold anything."""
    rng = np.random.default_rng(35)
    m, table, starts = filled(rng, 2, 128, 64, False, 16, [800], [1])
    q = rounded(rng.normal(size=(1, 4, 128)).astype(np.float32), BF16)
    whole = check(dq, m, table, [800], None, q, BF16, 100, 10)
    less = table.copy()
    less[0, 1:43] = -1
    gone = check(dq, m, less, [800], None, q, BF16, 100, 10)
    assert torch.equal(whole[0], gone[0]) and torch.equal(whole[1], gone[1])
    for p in table[0, 1:43]:
        for s in "kv":
            m.scales[s][p] = np.float16("nan")
    poisoned = check(dq, m, table, [800], None, q, BF16, 100, 10)
    assert torch.equal(whole[0], poisoned[0]) and torch.equal(whole[1], poisoned[1])


def test_in_a_graph(dq):
    """A captured step replays with the lengths of that time."""
    rng = np.random.default_rng(36)
    m, table, starts = filled(rng, 1, 64, 64, False, 16, [900, 300], [1, 1])
    cache, t, n = cache_of(dq, m), dev(table), dev(np.array([500, 20], np.int32))
    q = rounded(rng.normal(size=(2, 2, 64)).astype(np.float32), F16)
    qd = dev(q).to(F16)
    ws = dq.cache_attention_workspace(cache, 2, 2, 2)
    dq.int4_cache_attention(qd, cache, t, n, window=60, sinks=5, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n += 70
        out = dq.int4_cache_attention(qd, cache, t, n, window=60, sinks=5, workspace=ws)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        now = [500 + 70 * (i + 1), 20 + 70 * (i + 1)]
        want, _ = check(dq, m, table, now, None, q, F16, 60, 5, cache=cache)
        assert torch.equal(out, want), i


def test_refusals(dq):
    rng = np.random.default_rng(37)
    m, table, _ = filled(rng, 1, 64, 64, False, 16, [40], [1])
    cache, t, n = cache_of(dq, m), dev(table), dev(np.array([40], np.int32))
    q = torch.zeros(1, 1, 64, dtype=F16, device=DEV)
    for kw in (dict(sinks=-1, window=5), dict(sinks=4, window=-1), dict(sinks=4, window=3, causal=False),
               dict(shared=torch.zeros(1, dtype=torch.int32)), dict(shared=torch.zeros(2, dtype=torch.int32, device=DEV)),
               dict(shared=torch.zeros(1, dtype=torch.int64, device=DEV)), dict(shared=5)):
        with pytest.raises(ValueError):
            dq.int4_cache_attention(q, cache, t, n, **kw)
