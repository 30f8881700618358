"""Pages of a serving batch on MI355X (int4_cache_release, int4_cache_extend) against
the list model of tests/cache_step_model.py: every entry, length, slot and count."""
import numpy as np
import pytest
import torch

from tests.cache_step_model import extend, release

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def dq():
    import dequantizing_gemm_amd as dq
    return dq


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def say(*a):
    print(*a, flush=True)


def state(rng, lengths, S, most, spare):
    """Table, free pages and count of a batch that holds its pages."""
    held = [min(-(-max(int(n), 0) // S), most) for n in lengths]
    order = rng.permutation(sum(held) + spare).astype(np.int32)
    table = np.full((len(lengths), most), -7, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    free = np.full(len(order), -9, np.int32)
    free[:spare] = order[at:]
    return table, free, np.array([spare, 5], np.int32)


def check_extend(dq, table, lengths, free, count, S, added, rows, **kw):
    t, n, f, c = dev(table), dev(lengths), dev(free), dev(count)
    got = dq.int4_cache_extend(t, n, f, c, S, None if added is None else dev(added), rows=rows, **kw)
    torch.cuda.synchronize()
    want = extend(table, lengths, free, count, S, np.ones(len(lengths), np.int32) if added is None else added, rows)
    for name, x, y in zip(("table", "lengths", "starts", "slots", "count"), (t, *got), want):
        if x is not None:
            assert x.dtype == (torch.int64 if name == "slots" else torch.int32)
            assert np.array_equal(x.cpu().numpy(), y), name
    assert np.array_equal(f.cpu().numpy(), free) and np.array_equal(n.cpu().numpy(), lengths)
    return got


EXTEND = [  # batch, page, longest, most new (None: one each), pages to spare, entries of the table, extra rows
    (1, 16, 700, None, 3, 60, 0),
    (1, 64, 0, None, 1, 1, 0),
    (128, 64, 4000, None, 40, 70, 0),
    (128, 64, 4000, None, 2, 70, 0),               # too few pages
    (5, 16, 100, 300, 200, 40, 7),                 # rows behind the last sequence
    (5, 16, 100, 300, 200, 12, 0),                 # past the table
    (7, 256, 1000, 5000, 400, 80, 0),              # slots by their own kernel
    (48, 16, 900, 400, 3000, 120, 100),
    (1025, 32, 300, None, 500, 20, 0),             # past a thread each
    (1500, 16, 50, 9, 4000, 20, 3),
    (3000, 16, 100, 3, 10, 8, 0),
    (2, 1 << 20, 5, 70, 2, 3, 0),
]


@pytest.mark.parametrize("batch,S,longest,most_new,spare,most,extra", EXTEND)
def test_extend(dq, batch, S, longest, most_new, spare, most, extra):
    rng = np.random.default_rng(batch + S + longest)
    lengths = rng.integers(0, longest + 1, size=batch).astype(np.int32)
    added = None if most_new is None else rng.integers(0, most_new + 1, size=batch).astype(np.int32)
    table, free, count = state(rng, lengths, S, most, spare)
    rows = (batch if added is None else int(added.sum())) + extra
    say("case: extend", batch, S, longest, most_new, spare, most, rows)
    check_extend(dq, table, lengths, free, count, S, added, rows)
    check_extend(dq, table, lengths, free, count, S, added, max(rows - 3, 0))        # fewer rows than starts has
    check_extend(dq, table, lengths, free, count, S, added, rows, slots=False)


def test_extend_edges_of_contents(dq):
    """Lengths and counts below 0 and past their range, a table that holds what is no page."""
    rng = np.random.default_rng(3)
    lengths = np.array([-5, 3, 1000, -2 ** 31, 2 ** 31 - 1, 0, 17, 2 ** 31 - 3], np.int32)
    added = np.array([4, -9, 2, 40, 3, 0, -2 ** 31, 2], np.int32)
    for said in (0, -1, -2 ** 31, 9, 2 ** 31 - 1):
        table = rng.integers(-3, 60, size=(8, 6)).astype(np.int32)
        free = rng.integers(-2, 60, size=9).astype(np.int32)
        say("case: contents", said)
        check_extend(dq, table, lengths, free, np.array([said, 1], np.int32), 16, added, 60)


def test_extend_nothing(dq):
    empty, one = np.zeros(0, np.int32), np.array([4, 4], np.int32)
    check_extend(dq, np.zeros((0, 3), np.int32), empty, np.arange(4, dtype=np.int32), one, 16, empty, 0)
    check_extend(dq, np.zeros((0, 3), np.int32), empty, np.arange(4, dtype=np.int32), one, 16, None, 0)
    check_extend(dq, np.zeros((3, 0), np.int32), np.zeros(3, np.int32), np.arange(4, dtype=np.int32), one, 16, None, 3)
    check_extend(dq, np.zeros((3, 2), np.int32), np.zeros(3, np.int32), empty, one, 16, np.ones(3, np.int32), 3)
    check_extend(dq, np.zeros((3, 2), np.int32), np.zeros(3, np.int32), empty, one, 16, np.zeros(3, np.int32), 0)


def check_release(dq, table, lengths, free, count, S, done, shared=None):
    t, n, f, c = dev(table), dev(lengths), dev(free), dev(count)
    got = dq.int4_cache_release(t, n, f, c, S, dev(done), shared=None if shared is None else dev(np.array([shared], np.int32)))
    torch.cuda.synchronize()
    want = release(table, lengths, free, count, S, done, shared)
    for name, x, y in zip(("lengths", "free", "count"), (got[0], f, got[1]), want):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lengths)


@pytest.mark.parametrize("batch,S,longest,share", [(1, 16, 50, 1.0), (128, 64, 4000, 0.1), (40, 16, 3000, 0.5),
                                                    (2100, 16, 90, 0.7), (3, 32, 100000, 1.0), (6, 16, 200, 0.0)])
def test_release(dq, batch, S, longest, share):
    rng = np.random.default_rng(batch + longest)
    lengths = rng.integers(0, longest + 1, size=batch).astype(np.int32)
    table, free, count = state(rng, lengths, S, -(-longest // S) + 1, 13)
    done = rng.random(batch) < share
    say("case: release", batch, S, longest, share)
    check_release(dq, table, lengths, free, count, S, done)
    check_release(dq, table, lengths, free, count, S, done.astype(np.uint8) * 200)
    for shared in (0, 1, S, 3 * S - 1, longest, 2 ** 31 - 1, -4):
        check_release(dq, table, lengths, free, count, S, done, shared)
    table[rng.random(table.shape) < 0.3] = -1      # pages that were lacking
    table[rng.random(table.shape) < 0.1] = len(free)
    check_release(dq, table, lengths, free, count, S, done)
    check_release(dq, table, lengths, free, np.array([len(free) - 2, 0], np.int32), S, done)     # no room for all
    check_release(dq, table, -lengths, free, count, S, done)


def test_in_place_and_strides(dq):
    """Lengths and count of a step are those of the next; a table that is part of another."""
    rng = np.random.default_rng(11)
    S, batch = 16, 37
    lengths = rng.integers(0, 60, size=batch).astype(np.int32)
    table, free, count = state(rng, lengths, S, 9, 400)
    big = torch.full((batch, 31), 77, dtype=torch.int32, device=DEV)
    t = big[:, 5:14]
    t.copy_(dev(table))
    n, f, c = dev(lengths), dev(free), dev(count)
    starts, slots = torch.empty(batch + 1, dtype=torch.int32, device=DEV), torch.empty(200, dtype=torch.int64, device=DEV)
    for step in range(12):
        done = rng.random(batch) < 0.2
        added = rng.integers(0, 6, size=batch).astype(np.int32)
        dq.int4_cache_release(t, n, f, c, S, dev(done), out=(n, c))
        lengths, free, count = release(table, lengths, free, count, S, done)
        assert np.array_equal(f.cpu().numpy(), free)
        dq.int4_cache_extend(t, n, f, c, S, dev(added), rows=200, out=(n, starts, slots, c))
        table, lengths, want_starts, want_slots, count = extend(table, lengths, free, count, S, added, 200)
        for x, y in ((t, table), (n, lengths), (starts, want_starts), (slots, want_slots), (c, count)):
            assert np.array_equal(x.cpu().numpy(), y), step
    assert (big[:, :5] == 77).all() and (big[:, 14:] == 77).all()
    # no sequence shares a page with another, and none of theirs is free
    held = [p for b in range(batch) for p in table[b, :min(-(-lengths[b] // S), 9)] if p >= 0]
    assert sorted(held + list(free[:count[0]])) == sorted(set(held) | set(free[:count[0]]))


def test_pages_in_a_graph(dq):
    """A captured step replays with what the tensors hold at that time."""
    rng = np.random.default_rng(12)
    S, batch = 16, 20
    lengths = np.zeros(batch, np.int32)
    table, free, count = state(rng, lengths, S, 300, 5000)
    t, n, f, c = dev(table), dev(lengths), dev(free), dev(count)
    d, a = torch.zeros(batch, dtype=torch.bool, device=DEV), torch.zeros(batch, dtype=torch.int32, device=DEV)
    starts, slots = torch.empty(batch + 1, dtype=torch.int32, device=DEV), torch.empty(4000, dtype=torch.int64, device=DEV)

    def step():
        dq.int4_cache_release(t, n, f, c, S, d, out=(n, c))
        dq.int4_cache_extend(t, n, f, c, S, a, rows=4000, out=(n, starts, slots, c))

    step()                                         # nothing new, nothing done
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    for i in range(6):
        done, added = rng.random(batch) < 0.3, rng.integers(0, 190, size=batch).astype(np.int32)
        d.copy_(dev(done))
        a.copy_(dev(added))
        graph.replay()
        torch.cuda.synchronize()
        lengths, free, count = release(table, lengths, free, count, S, done)
        table, lengths, want_starts, want_slots, count = extend(table, lengths, free, count, S, added, 4000)
        for x, y in ((t, table), (n, lengths), (f, free), (starts, want_starts), (slots, want_slots), (c, count)):
            assert np.array_equal(x.cpu().numpy(), y), i


def test_pages_on_another_stream(dq):
    rng = np.random.default_rng(13)
    lengths = rng.integers(0, 900, size=300).astype(np.int32)
    added = rng.integers(0, 30, size=300).astype(np.int32)
    table, free, count = state(rng, lengths, 32, 60, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check_extend(dq, table, lengths, free, count, 32, added, int(added.sum()))
    torch.cuda.current_stream().wait_stream(side)
