"""Pages of a serving batch on MI355X where sequences end at 2^31 - 1 tokens, the most that a
length can say: the same slots whether one block or the whole GPU writes them, those of the
positions that the other calls derive from lengths and starts, and no page taken that the
lengths do not cover."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MOST = 2 ** 31 - 1
S = 1 << 20


@pytest.fixture(scope="module")
def dq():
    import dequantizing_gemm_amd as dq
    return dq


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("lengths,added", [
    ([MOST - 10, 7], [3000, 5]),               # past the end
    ([MOST, 5, 1500 * S], [2900, 200, 1]),     # at the end before
    ([MOST - 3000, 7], [3000, 5]),             # up to it
    ([40, 9], [100, MOST - 49]),               # more tokens than rows: starts end at 2^31 - 1 too
    ([3 * S - 7, 2 ** 30], [2500, 2500]),      # nowhere near
])
def test_ends_of_sequences(dq, lengths, added):
    batch, most, pages = len(lengths), 2049, 7000
    rng = np.random.default_rng(batch)
    order = rng.permutation(pages).astype(np.int32)
    table, at = np.full((batch, most), -1, np.int32), 0
    for b, n in enumerate(lengths):
        held = -(-n // S)
        table[b, :held] = order[at:at + held]
        at += held
    free = np.concatenate([order[at:], np.full(at, -1, np.int32)])
    new = [min(n + m, MOST) for n, m in zip(lengths, added)]
    need = [-(-n // S) - -(-o // S) for n, o in zip(new, lengths)]
    left = pages - at
    for b in range(batch):
        held = -(-lengths[b] // S)
        for i in range(need[b]):
            left -= 1
            table[b, held + i] = free[left]
    starts = np.minimum(np.concatenate([[0], np.cumsum(np.array(added, np.int64))]), MOST)
    rows = int(min(sum(added), 3100)) + 9
    slots = np.full(rows, -1, np.int64)
    first = 0
    for b in range(batch):
        t = np.arange(first, min(first + added[b], rows))
        pos = new[b] - added[b] + t - first
        slots[t] = table[b, pos // S].astype(np.int64) * S + pos % S
        first += added[b]
    print("case: ends", lengths, added, rows, flush=True)
    got = None
    for n in (rows, 2048, 1000):               # on the whole GPU, by one block, the fewest
        t, f = i32(table.tolist()), i32(free.tolist())
        for b in range(batch):
            t[b, -(-lengths[b] // S):] = -5
        got = dq.int4_cache_extend(t, i32(lengths), f, i32([pages - at, 0]), S, i32(added), rows=n)
        for x, want in zip(got, (new, starts, slots[:n], [left, 0])):
            assert np.array_equal(x.cpu().numpy(), np.asarray(want)), n
        for b in range(batch):
            held = -(-new[b] // S)
            assert np.array_equal(t[b, :held].cpu().numpy(), table[b, :held])
    # in place: the lengths that the slots go by are the new ones then
    n, c, s0, sl = i32(lengths), i32([pages - at, 0]), i32([0] * (batch + 1)), torch.zeros(rows, dtype=torch.int64, device=DEV)
    t = i32(table.tolist())
    dq.int4_cache_extend(t, n, f, c, S, i32(added), rows=rows, out=(n, s0, sl, c))
    assert np.array_equal(sl.cpu().numpy(), slots) and n.tolist() == new
    # all pages come back
    done = torch.ones(batch, dtype=torch.bool, device=DEV)
    _, count = dq.int4_cache_release(t, n, f, c, S, done)
    assert count.tolist() == [pages, 0]
    assert sorted(f.tolist()) == list(range(pages))


@pytest.mark.parametrize("rows", [600, 5000])
def test_as_many_new_tokens_as_there_were(dq, rows):
    """Lengths that are the new tokens too, and are written in place."""
    n, batch, page = i32([rows // 4 + 7, 0, rows // 4 - 7, rows // 2]), 4, 16
    most = -(-rows // page) + 1
    before = n.tolist()
    table = torch.arange(batch * most, dtype=torch.int32, device=DEV).view(batch, most)
    free = torch.arange(batch * most, dtype=torch.int32, device=DEV)
    want = [t.clone() for t in dq.int4_cache_extend(table.clone(), n, free, i32([batch * most, 0]), page, n.clone(), rows=rows)]
    starts, slots, count = i32([0] * 5), torch.zeros(rows, dtype=torch.int64, device=DEV), i32([batch * most, 0])
    print("case: doubled", rows, flush=True)
    got = dq.int4_cache_extend(table, n, free, count, page, n, rows=rows, out=(n, starts, slots, count))
    assert got[0].tolist() == [2 * x for x in before]
    for x, y in zip(got, want):
        assert torch.equal(x, y)
