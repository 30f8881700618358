"""A step for which there are too few pages (int4_cache_extend on MI355X), taken back: lengths, count
and free pages of before, pages given back by a sequence that has to wait, and the call once more."""
import numpy as np
import pytest
import torch

from tests.cache_step_model import extend, release
from tests.test_cache_pages_gpu import DEV, dev, dq, state  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,S,spare", [(6, 16, 3), (1100, 32, 500), (5, 64, 0)])
def test_taken_back(dq, batch, S, spare):
    rng = np.random.default_rng(batch)
    lengths = rng.integers(S, 6 * S, size=batch).astype(np.int32)
    added = rng.integers(1, 3 * S, size=batch).astype(np.int32)
    table, free, count = state(rng, lengths, S, 12, spare)
    t, n, f, c, a = dev(table), dev(lengths), dev(free), dev(count), dev(added)
    rows = int(added.sum())
    print("case: taken back", batch, S, spare, flush=True)
    _, _, _, lacking = dq.int4_cache_extend(t, n, f, c, S, a, rows=rows)
    assert lacking[1] > 0
    for x, y in ((n, lengths), (f, free), (c, count)):
        assert np.array_equal(x.cpu().numpy(), y)
    # as many sequences wait as it takes
    waits = np.zeros(batch, bool)
    held = -(-lengths // S)
    need = -(-(lengths + added) // S) - held
    for b in range(batch):
        if spare + held[waits].sum() >= need[~waits].sum():
            break
        waits[b] = True
    n2, c2 = dq.int4_cache_release(t, n, f, c, S, dev(waits))
    a[dev(waits)] = 0
    n3, starts, slots, c3 = dq.int4_cache_extend(t, n2, f, c2, S, a, rows=rows)
    want_n, want_f, want_c = release(table, lengths, free, count, S, waits)
    want = extend(table, want_n, want_f, want_c, S, np.where(waits, 0, added).astype(np.int32), rows)
    assert want[4][1] == 0
    for x, y in zip((n3, starts, slots, c3), want[1:]):
        assert np.array_equal(x.cpu().numpy(), y)
    got = t.cpu().numpy()
    pages = [p for b in range(batch) for p in got[b, :-(-int(n3[b]) // S)]]
    assert pages == [p for b in range(batch) for p in want[0][b, :-(-int(want[1][b]) // S)]]
    rest = f.cpu().numpy()[:int(c3[0])].tolist()
    assert min(pages) >= 0 and sorted(pages + rest) == list(range(len(free)))


def test_not_taken_back(dq):
    """Tokens that lack a page keep lacking it, the others after them have theirs."""
    S = 16
    table, free = torch.full((1, 8), -7, dtype=torch.int32, device=DEV), dev(np.arange(8, dtype=np.int32))
    lengths, count = dev(np.array([0], np.int32)), dev(np.array([1, 0], np.int32))
    lengths, _, slots, count = dq.int4_cache_extend(table, lengths, free, count, S, dev(np.array([40], np.int32)), rows=40)
    assert count.tolist() == [0, 2] and table[0, :3].tolist() == [0, -1, -1] and slots.tolist() == list(range(16)) + [-1] * 24
    count[0] = 8
    lengths, _, slots, count = dq.int4_cache_extend(table, lengths, free, count, S, dev(np.array([10], np.int32)), rows=10)
    assert count.tolist() == [7, 0] and table[0, :4].tolist() == [0, -1, -1, 7]
    assert slots.tolist() == [-1] * 8 + [7 * S, 7 * S + 1]
