"""Attention over the 4-bit cache for a batch whose sequences begin with the same tokens
(int4_cache_attention, shared=) on MI355X: the model's attention over whole sequences,
within its bounds, whichever way the call takes them."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model
from tests.cache_step_model import Sinks
from tests.test_cache_gpu import BF16, DEV, F16, cache_of, check_attention, dev, dq, rounded, say, values  # noqa: F401

pytestmark = pytest.mark.gpu


def batch(rng, heads, D, group, affine, page, shared_pages, lengths, new, spare=3):
    """A model whose sequences have their first pages in common; lengths count them."""
    own = [max(0, -(-int(n) // page) - shared_pages) for n in lengths]
    total = shared_pages + sum(own) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(lengths), shared_pages + max(own + [1])), -1, np.int32)
    table[:, :shared_pages] = order[:shared_pages]
    at = shared_pages
    for b, n in enumerate(own):
        table[b, shared_pages:shared_pages + n] = order[at:at + n]
        at += n
    m = Model(total, page, heads, D, group, affine, fill=0x7E)
    for p in order[:at]:
        for slot in range(page):
            m.put("k", values(rng, heads, D), int(p), slot)
            m.put("v", values(rng, heads, D), int(p), slot)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return m, table, starts


def check(dq, m, table, lengths, starts, q, dtype, shared, window=0, sinks=0, cache=None, share_from=1, **kw):
    """share_from: 1, whatever it costs; None: where it pays."""
    cache = cache or cache_of(dq, m)
    n = torch.tensor([shared], dtype=torch.int32, device=DEV)
    return check_attention(dq, Sinks(m, sinks), table, lengths, starts, q, dtype, window=window, sinks=sinks, shared=n,
                           cache=cache, share_from=share_from, **kw)


CASES = [  # D, group, affine, heads, ratio, page, dtype, shared pages, own tokens, new rows
    (128, 128, False, 1, 4, 64, BF16, 18, [1, 30, 200, 65], [1, 1, 1, 1]),
    (128, 64, True, 2, 2, 16, F16, 80, [3, 300, 17], [1, 1, 1]),
    (64, 64, False, 2, 1, 16, F16, 70, [1] * 40, [1] * 40),
    (64, 32, True, 1, 5, 32, BF16, 36, [9, 70, 40, 100, 3], [9, 2, 1, 30, 3]),
    (96, 96, False, 1, 6, 32, F16, 40, [40, 200], [13, 5]),
    (80, 128, True, 1, 3, 16, BF16, 66, [20, 1, 7], [3, 1, 4]),
    (192, 64, False, 1, 2, 32, BF16, 34, [21, 40], [7, 2]),
    (256, 128, True, 1, 8, 64, F16, 17, [33, 5], [4, 1]),
    # as many rows as fill the form for prompts with the shared tokens
    (64, 64, False, 1, 8, 64, F16, 17, [3] * 45, [1] * 45),
    (128, 128, True, 1, 4, 128, BF16, 9, [50] * 12, [6] * 12),
]


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,pages,own,new", CASES)
def test_shared(dq, D, group, affine, heads, ratio, page, dtype, pages, own, new):
    rng = np.random.default_rng(500 + D + sum(own))
    lengths = [pages * page + n for n in own]
    m, table, starts = batch(rng, heads, D, group, affine, page, pages, lengths, new)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    # all shared pages, a number of tokens that ends inside a step, or inside a unit, few, none
    for shared in (pages * page, pages * page - 37, 64 * (pages * page // 64) // 2 + 5, 3, 0, -8):
        say("case: shared", D, group, affine, heads, ratio, page, own, new, shared)
        check(dq, m, table, lengths, starts, q, dtype, shared, cache=cache)
        check(dq, m, table, lengths, starts, q, dtype, shared, cache=cache, share_from=None)
    if set(new) == {1}:
        check(dq, m, table, lengths, None, q, dtype, pages * page, cache=cache)
    check(dq, m, table, lengths, starts, q, dtype, pages * page, cache=cache, share_from=pages * page)
    check(dq, m, table, lengths, starts, q, dtype, pages * page, cache=cache, share_from=pages * page + 1)
    shared = pages * page - 11
    for window, sinks in ((20, 0), (500, 0), (20, 7), (700, 90), (pages * page // 2, 30), (60, 2 ** 31)):
        say("case: shared, window", window, sinks)
        check(dq, m, table, lengths, starts, q, dtype, shared, window=window, sinks=sinks, cache=cache)
    check(dq, m, table, lengths, starts, q, dtype, shared, causal=False, cache=cache)


def test_shared_past_some_sequences(dq):
    """Sequences that end within the shared tokens, rows whose positions lie among them, empty ones."""
    rng = np.random.default_rng(41)
    page, pages = 32, 40
    lengths, new = [1280, 500, 1300, 0, 1, 1281, 33], [3, 9, 40, 0, 1, 2, 33]
    m, table, starts = batch(rng, 1, 64, 64, False, page, pages, lengths, new)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(int(starts[-1]), 3, 64)).astype(np.float32), BF16)
    for shared in (1280, 1277, 600, 40):
        say("case: past some", shared)
        check(dq, m, table, lengths, starts, q, BF16, shared, cache=cache)
        check(dq, m, table, lengths, starts, q, BF16, shared, window=50, sinks=4, cache=cache)
        check(dq, m, table, lengths, starts, q, BF16, shared, causal=False, cache=cache)
    # rows that no sequence owns, before and behind
    q = rounded(rng.normal(size=(int(starts[-1]) + 9, 3, 64)).astype(np.float32), BF16)
    check(dq, m, table, lengths, starts + 4, q, BF16, 1280, cache=cache)
    # lengths below 0 and past the table, pages that are none, shared past everything
    lengths = [1280, -5, 1300, 0, 1, 2000, 33]
    table[:, 7] = -1
    table[2, 40] = m.P
    check(dq, m, table, lengths, starts + 4, q, BF16, 1280, cache=cache)
    # one conversation in all of them: shared past everything
    table[:] = table[:1]
    check(dq, m, table, [1280, 700, 1312, 1290, 1, 1281, 33], starts + 4, q, BF16, 2 ** 31 - 1, cache=cache)


def test_large_batch(dq):
    rng = np.random.default_rng(42)
    for n, new in ((130, [1] * 130), (70, [1, 3, 0, 2, 1] * 14)):
        lengths = (1152 + rng.integers(3, 60, size=n)).tolist()
        m, table, starts = batch(rng, 1, 64, 64, False, 64, 18, lengths, new)
        q = rounded(rng.normal(size=(int(starts[-1]), 2, 64)).astype(np.float32), F16)
        say("case: large batch", n)
        check(dq, m, table, lengths, starts, q, F16, 1152)
        check(dq, m, table, lengths, starts, q, F16, 1100, window=200, sinks=9)


def test_workspaces(dq):
    """Of the size asked for, larger, too small for the parts, none: the same within bounds; its
    contents do not matter, and what lies behind it is left as it was."""
    rng = np.random.default_rng(43)
    lengths, new = [1216 + n for n in (5, 90, 41)], [1, 1, 1]
    m, table, starts = batch(rng, 2, 64, 64, False, 64, 19, lengths, new)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(3, 4, 64)).astype(np.float32), BF16)
    n = dq.cache_attention_workspace_bytes(cache, 3, 3, 4, shared=True, share_from=1)
    assert n >= dq.cache_attention_workspace_bytes(cache, 3, 3, 4) > 0
    outs = []
    for size in (n, n + 4096, n // 2, 0):
        ws = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        outs.append(check(dq, m, table, lengths, None, q, BF16, 1216, cache=cache, workspace=ws[:size]))
        assert (ws[size:] == 0xFF).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_in_a_graph(dq):
    """A captured step replays with the lengths and the number of shared tokens of that time."""
    rng = np.random.default_rng(44)
    m, table, starts = batch(rng, 1, 64, 64, False, 16, 72, [1152 + 500] * 5, [1] * 5)
    cache, t = cache_of(dq, m), dev(table)
    lengths = np.array([1160, 1153, 1300, 1200, 1190], np.int32)
    n, s = dev(lengths), torch.tensor([1152], dtype=torch.int32, device=DEV)
    q = rounded(rng.normal(size=(5, 2, 64)).astype(np.float32), F16)
    qd = dev(q).to(F16)
    ws = dq.cache_attention_workspace(cache, 5, 5, 2, shared=True, share_from=400)
    dq.int4_cache_attention(qd, cache, t, n, shared=s, workspace=ws, share_from=400)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n += 7
        out = dq.int4_cache_attention(qd, cache, t, n, shared=s, workspace=ws, share_from=400)
    for i, shared in enumerate((1152, 0, 700, 1100, 1152)):
        s.fill_(shared)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = check(dq, m, table, lengths + 7 * (i + 1), None, q, F16, shared, cache=cache, workspace=ws, share_from=400)
        assert torch.equal(out, want), i


def test_on_another_stream(dq):
    rng = np.random.default_rng(45)
    lengths = [1216 + n for n in (5, 90, 41)]
    m, table, starts = batch(rng, 2, 64, 64, False, 64, 19, lengths, [1] * 3)
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(3, 4, 64)).astype(np.float32), BF16)
    here = check(dq, m, table, lengths, None, q, BF16, 1216, cache=cache)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            there = check(dq, m, table, lengths, None, q, BF16, 1216, cache=cache)
            assert torch.equal(here[0], there[0]) and torch.equal(here[1], there[1])
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
