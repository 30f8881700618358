"""Plans of the 4-bit cache's attention that no caller means, and calls at once, where
the work takes its longest way: prompts, keys shared out over blocks with the join
after them, and batches planned by a kernel of their own. Model and bounds as in
tests/test_cache_gpu.py."""
import ctypes

import numpy as np
import pytest
import torch

from tests.cache_model import Model, plan
from tests.test_cache_gpu import BF16, DEV, F16, F32, cache_of, check_attention, dev, dq, filled, rounded, say, values  # noqa: F401

pytestmark = pytest.mark.gpu


def workspace_of_call(cache, table, batch, rows, q_heads, starts):
    """Bytes the call itself asks for: above 0 where keys may be shared out."""
    from dequantizing_gemm_amd import cache as binding
    r = binding._RowsStruct(None, table.shape[1], table.shape[1], None, 1 if starts else None, batch, rows)
    return binding.lib.int4_cache_attention_workspace_bytes(cache._ref, ctypes.addressof(r), q_heads)


def with_holes(rng, m_args, lengths, new, page, bad=True):
    """A model filled with sequences whose plan then loses pages in the middle, at the
    start and at the end, claims more tokens than its table covers, and has rows before
    and behind all sequences."""
    heads, D, group, affine = m_args
    lengths = np.array(lengths, np.int32)
    table, pages, starts = plan(rng, np.maximum(lengths, 0), new, page)
    m = Model(pages, page, heads, D, group, affine, fill=0x7E)
    whole = np.concatenate([[0], np.cumsum(np.maximum(lengths, 0))]).astype(np.int32)
    T = int(whole[-1])
    m.write(values(rng, T, heads, D), values(rng, T, heads, D), table, np.maximum(lengths, 0), whole)
    out = [-1, pages, pages + 7, 2 ** 31 - 1, -2 ** 31]
    for b, n in enumerate(lengths):
        used = -(-max(int(n), 0) // page)
        for at in {0, used // 3, used // 3 + 1, used // 2, used - 1}:
            if 0 <= at < used and (b + at) % 3 != 0:
                table[b, at] = out[(b + at) % 5]
    claimed = lengths.copy()
    claimed[-1] = table.shape[1] * page + 77
    return m, table, claimed, (starts + 2).astype(np.int32), int(starts[-1]) + 5


BAD = [  # heads, D, group, affine, ratio, page, dtype, lengths, new rows
    # a few rows on long sequences: shared out, joined
    (1, 64, 64, False, 4, 16, F16, [2600, -5, 1900, 0, 40, 1300], [2, 1, 7, 3, 4, 2]),
    (2, 128, 32, True, 2, 64, BF16, [3000, 700, 1500], [3, 9, 1]),
    # more than 256 query rows a head and sequence: the form for prompts, in one block a tile
    (1, 64, 64, False, 4, 16, F16, [200, 130, -3, 330], [120, 130, 40, 150]),
    (1, 128, 128, True, 3, 32, BF16, [400, 90, 300], [200, 95, 150]),
    # the same, shared out
    (1, 64, 32, False, 4, 64, BF16, [2300, 1500, 100], [90, 70, 110]),
    (1, 192, 64, False, 3, 32, F16, [1900, 300], [130, 100]),
]


@pytest.mark.parametrize("heads,D,group,affine,ratio,page,dtype,lengths,new", BAD)
def test_bad_plans(dq, heads, D, group, affine, ratio, page, dtype, lengths, new):
    rng = np.random.default_rng(200 + D + sum(new))
    m, table, claimed, starts, T = with_holes(rng, (heads, D, group, affine), lengths, new, page)
    cache = cache_of(dq, m)
    n = workspace_of_call(cache, table, len(new), T, heads * ratio, True)
    assert (n > 0) == (table.shape[1] * page > 1024)
    q = rounded(rng.normal(size=(T, heads * ratio, D)).astype(np.float32), dtype)
    say("case: bad plan", heads, D, group, affine, ratio, page, lengths, new)
    check_attention(dq, m, table, claimed, starts, q, dtype, cache=cache)
    check_attention(dq, m, table, claimed, starts, q, dtype, cache=cache, window=150)
    check_attention(dq, m, table, claimed, starts, q, dtype, cache=cache, causal=False)


@pytest.mark.parametrize("one_row", [True, False])
def test_bad_plans_of_many_sequences(dq, one_row):
    """More than 64 sequences, some shared out, with holes, negative lengths and rows
    that no sequence owns."""
    rng = np.random.default_rng(210 + one_row)
    lengths = rng.integers(-3, 40, size=90)
    lengths[[3, 50, 88]] = [1500, 1100, 1700]
    new = np.ones(90, np.int64) if one_row else rng.integers(0, 4, size=90)
    m, table, claimed, starts, T = with_holes(rng, (1, 64, 64, False), lengths, new, 16)
    if one_row:
        starts, T = None, 90
    cache = cache_of(dq, m)
    assert workspace_of_call(cache, table, 90, T, 3, not one_row) > 0
    q = rounded(rng.normal(size=(T, 3, 64)).astype(np.float32), F16)
    say("case: bad plan, many", one_row)
    check_attention(dq, m, table, claimed, starts, q, F16, cache=cache)
    check_attention(dq, m, table, claimed, starts, q, F16, cache=cache, window=100)


@pytest.mark.parametrize("lengths,batch,rows", [([2600, 1900], 1, 1), ([2300, 1500], 1, 90), ([1600, 2000], 70, 1)])
def test_two_streams_that_share_out(dq, lengths, batch, rows):
    """Two calls at once, each with scratch of its own from torch's allocator: keys
    shared out, partial results, the join, and from 65 sequences on the plan."""
    rng = np.random.default_rng(220 + batch + rows)
    cases = []
    for n in lengths:
        lens = [n] + [30] * (batch - 1)
        m, table, starts = filled(rng, 1, 64, 64, False, 16, lens, [rows] * batch)
        q = rounded(rng.normal(size=(rows * batch, 4, 64)).astype(np.float32), F16)
        cache = cache_of(dq, m)
        assert workspace_of_call(cache, table, batch, rows * batch, 4, rows > 1) > 0
        args = (torch.from_numpy(q).to(DEV).half(), cache, dev(table), dev(np.array(lens, np.int32)),
                None if rows == 1 else dev(starts))
        check_attention(dq, m, table, lens, None if rows == 1 else starts, q, F16, cache=cache)
        cases.append((args, dq.int4_cache_attention(*args, return_lse=True)))
    torch.cuda.synchronize()
    say("case: two streams", lengths, batch, rows)
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (args, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(dq.int4_cache_attention(*args, return_lse=True))
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(cases):
        for g in got[i]:
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_write_and_read_of_many_bad_sequences(dq):
    """Writes and reads over more than 64 sequences with holes, negative lengths and
    unowned rows: bytes equal to the model's, unowned rows as they were."""
    rng = np.random.default_rng(230)
    lengths = rng.integers(-3, 90, size=130)
    new = np.minimum(np.maximum(lengths, 0) + 2, rng.integers(0, 70, size=130))
    m, table, claimed, starts, T = with_holes(rng, (2, 64, 32, True), lengths, new, 16)
    cache = cache_of(dq, m)
    k, v = values(rng, T, 2, 64), values(rng, T, 2, 64)
    say("case: bad writes", T)
    dq.int4_cache_write(cache, dev(k), dev(v), dev(table), dev(claimed), dev(starts))
    m.write(k, v, table, claimed, starts)
    torch.cuda.synchronize()
    for s in "kv":
        assert np.array_equal(getattr(cache, s + "_packed").cpu().numpy(), m.packed[s])
        assert np.array_equal(getattr(cache, s + "_scales").cpu().numpy().view(np.uint16), m.scales[s].view(np.uint16))
        assert np.array_equal(getattr(cache, s + "_zeros").cpu().numpy(), m.zeros[s])
    mark = (torch.full((T, 2, 64), 7.0, device=DEV), torch.full((T, 2, 64), 7.0, device=DEV))
    got = dq.int4_cache_read(cache, dev(table), dev(claimed), dev(starts), dtype=F32, out=mark)
    kr, vr, owned = m.read(T, table, claimed, starts)
    assert not owned.all()
    for g, r in zip(got, (kr, vr)):
        r[~owned] = 7.0
        assert np.array_equal(g.cpu().numpy(), r, equal_nan=True)
