"""The forms of the cache's kernels on MI355X: prompts in every width and grouping,
long sequences shared out over several blocks, batches of more sequences than a
wavefront looks through at once, workspaces, graphs, and what the Python calls
refuse. Bounds as in tests/test_cache_gpu.py; joining the parts of a sequence adds
binary32 roundings of 2^-24 each, a few for each part, which the bound's 2^-20
covers."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model, plan
from tests.test_cache_gpu import (BF16, DEV, F16, F32, assert_same_bytes, cache_of, check_attention, dev, dq, filled,
                                  rounded, say, values)

pytestmark = pytest.mark.gpu

PROMPTS = [  # D, group, affine, heads, ratio, dtype, window
    (64, 64, False, 2, 2, F16, 0), (64, 64, True, 1, 2, BF16, 0), (64, 32, False, 1, 3, BF16, 40),
    (64, 32, True, 2, 2, F16, 0), (40, 40, False, 1, 2, F16, 0), (33, 32, True, 1, 2, BF16, 0),
    (96, 96, False, 1, 2, BF16, 0), (96, 32, True, 1, 2, F16, 100), (80, 64, False, 2, 2, F16, 0), (96, 96, True, 1, 3, F16, 0),
    (128, 128, False, 2, 2, BF16, 0), (128, 128, True, 1, 2, F16, 0), (128, 64, False, 1, 2, F16, 70),
    (128, 64, True, 1, 2, BF16, 0), (128, 32, False, 1, 2, BF16, 0), (128, 32, True, 1, 2, F16, 0),
    (100, 64, True, 1, 2, BF16, 0),
    (192, 192, False, 1, 2, BF16, 0), (192, 64, True, 1, 2, F16, 0), (192, 128, False, 1, 2, F16, 0), (160, 32, True, 1, 2, BF16, 0),
    (256, 256, False, 1, 2, F16, 0), (256, 128, True, 1, 2, BF16, 90), (256, 64, False, 1, 2, BF16, 0), (256, 64, True, 1, 2, F16, 0),
    (256, 32, False, 1, 2, F16, 0), (256, 32, True, 1, 2, BF16, 0), (250, 128, False, 1, 2, BF16, 0),
]


@pytest.mark.parametrize("D,group,affine,heads,ratio,dtype,window", PROMPTS)
def test_prompts(dq, D, group, affine, heads, ratio, dtype, window):
    """More than 256 query rows a key/value head and sequence on average, a tile that
    ends inside, one sequence that continues what is cached and one that is new."""
    rng = np.random.default_rng(1000 + D + group + window)
    lengths, new = [230, 290, 3], [140, 290, 3]
    say("case: prompts", D, group, affine, heads, ratio, dtype, window)
    m, table, starts = filled(rng, heads, D, group, affine, 32, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    check_attention(dq, m, table, lengths, starts, q, dtype, window=window)
    if window == 0:
        check_attention(dq, m, table, lengths, starts, q, dtype, causal=False)


LONG = [  # D, group, affine, heads, ratio, page, dtype, lengths, new rows, window
    (128, 128, False, 2, 4, 64, BF16, [2600, 70], [1, 1], 0),
    (128, 32, True, 1, 8, 16, F16, [1700], [3], 0),
    (64, 64, False, 1, 1, 32, F16, [1025, 0, 1600], [1, 1, 1], 0),
    (64, 64, False, 2, 20, 32, BF16, [1500, 1200], [1, 1], 0),
    (128, 64, False, 1, 2, 64, F16, [2300, 1100], [12, 9], 0),
    (96, 96, True, 1, 4, 16, BF16, [2000], [2], 1300),
    (192, 64, False, 1, 3, 16, F16, [1800], [2], 0),
    (256, 128, True, 1, 2, 64, BF16, [1500, 33], [1, 1], 0),
    (72, 32, False, 1, 2, 32, BF16, [1300], [1], 0),
    (128, 128, False, 1, 2, 128, F16, [1900], [90], 0),
    (64, 32, True, 1, 2, 64, BF16, [2100, 1300], [100, 70], 1200),
    (256, 64, False, 1, 1, 64, F16, [1400], [140], 0),
    (128, 128, False, 1, 2, 128, F16, [1900], [150], 0),
    (64, 32, True, 1, 3, 64, BF16, [2100, 1300], [100, 90], 1200),
    (64, 64, False, 1, 2, 64, BF16, [9300], [1], 0),
    (64, 64, False, 1, 2, 64, F16, [9300, 5], [70, 1], 0),
    (64, 64, True, 1, 2, 256, F16, [9300], [130], 0), (64, 64, False, 1, 2, 256, F16, [9300], [140], 0),
]


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,lengths,new,window", LONG)
def test_long_sequences(dq, D, group, affine, heads, ratio, page, dtype, lengths, new, window):
    """Sequences shared out over several blocks (more than 8 from 9300 tokens), with
    a workspace whose contents are not zero, without one, and with one too small."""
    rng = np.random.default_rng(2000 + D + group + sum(lengths))
    say("case: long", D, group, affine, heads, ratio, page, dtype, lengths, new, window)
    m, table, starts = filled(rng, heads, D, group, affine, page, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    st, cache = None if set(new) == {1} else starts, cache_of(dq, m)
    n = dq.cache_attention_workspace_bytes(cache, len(new), len(q), heads * ratio)
    assert n > 0
    memory = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = check_attention(dq, m, table, lengths, st, q, dtype, window=window, cache=cache, workspace=memory[:n])
    assert torch.all(memory[n:] == 0xFF), "written behind the workspace"
    again, lse2 = check_attention(dq, m, table, lengths, st, q, dtype, window=window, cache=cache)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "a second call gives other bits"
    if max(lengths) < 2000:
        for small in (memory[:0], memory[:n - 1]):
            check_attention(dq, m, table, lengths, st, q, dtype, window=window, cache=cache, workspace=small)


@pytest.mark.parametrize("batch,long_at,one_row", [(65, 64, True), (70, 3, False), (200, 130, True), (200, 199, False),
                                                   (1100, 1050, True), (1100, 20, False), (4200, -1, False), (4200, -1, True)])
def test_many_sequences(dq, batch, long_at, one_row):
    """Batches past 64 sequences, most of them short; one of 1500 tokens where long_at
    tells (the table then makes the call share out its keys)."""
    rng = np.random.default_rng(batch + one_row)
    lengths = rng.integers(0, 5, size=batch)
    if long_at >= 0:
        lengths[long_at] = 1500
    new = np.ones(batch, np.int64) if one_row else np.minimum(lengths, rng.integers(0, 4, size=batch))
    say("case: many", batch, long_at, one_row)
    table, pages, starts = plan(rng, lengths, new, 16)
    m = Model(pages, 16, 1, 64, 64, False, fill=0x7E)
    cache = cache_of(dq, m)
    # the whole sequences written by one call, with starts
    whole = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = int(whole[-1])
    k, v = values(rng, T, 1, 64), values(rng, T, 1, 64)
    m.write(k, v, table, lengths, whole)
    dq.int4_cache_write(cache, dev(k), dev(v), dev(table), dev(lengths.astype(np.int32)), dev(whole))
    assert_same_bytes(cache, m)
    kr, vr, _ = m.read(T, table, lengths, whole)
    kg, vg = dq.int4_cache_read(cache, dev(table), dev(lengths.astype(np.int32)), dev(whole), rows=T, dtype=F32)
    assert torch.equal(kg.cpu(), torch.from_numpy(kr)) and torch.equal(vg.cpu(), torch.from_numpy(vr))
    q = rounded(rng.normal(size=(int(starts[-1]), 3, 64)).astype(np.float32), F16)
    check_attention(dq, m, table, lengths, None if one_row else starts, q, F16, cache=cache)


@pytest.mark.parametrize("heads,ratio,batch,rows,longs", [(32, 1, 26, 1, 3), (11, 2, 80, 1, 5), (32, 1, 20, 3, 4), (32, 2, 9, 125, 1), (32, 2, 7, 130, 1)])
def test_a_few_more_tiles_than_fit(dq, heads, ratio, batch, rows, longs):
    """Somewhat more tiles than the GPU holds at once, some of them cut; and the same
    call with a workspace that has no room for as many cuts."""
    rng = np.random.default_rng(50 + batch)
    lengths = rng.integers(rows, rows + 9, size=batch)
    lengths[rng.permutation(batch)[:longs]] = 1100 + rng.integers(0, 200, size=longs)
    D = 128 if rows < 100 else 64
    say("case: crowded", heads, ratio, batch, rows)
    m, table, starts = filled(rng, heads, D, D, False, 16, lengths, [rows] * batch)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), BF16)
    cache, st = cache_of(dq, m), None if rows == 1 else starts
    n = dq.cache_attention_workspace_bytes(cache, batch, len(q), heads * ratio)
    out, lse = check_attention(dq, m, table, lengths, st, q, BF16, cache=cache)
    if rows > 100:
        return
    for room in (n * 2 // 3 + 256 * batch, n // 2):
        ws = torch.full((room,), 0x7F, dtype=torch.uint8, device=DEV)
        check_attention(dq, m, table, lengths, st, q, BF16, cache=cache, workspace=ws)


def test_many_query_heads_of_one(dq):
    """33 query heads to a key/value head and one row a sequence: several tiles a row."""
    rng = np.random.default_rng(31)
    lengths, new = [90, 1, 0, 1100], [1] * 4
    for table_tokens in (16, 64):
        m, table, starts = filled(rng, 1, 64, 64, False, table_tokens, lengths, new)
        q = rounded(rng.normal(size=(4, 33, 64)).astype(np.float32), BF16)
        check_attention(dq, m, table, lengths, None, q, BF16)


def test_sequences_that_share_pages(dq):
    """Two sequences with the first pages in common, as a shared prefix has it."""
    rng = np.random.default_rng(32)
    lengths, new = [100, 81], [4, 1]
    table, pages, starts = plan(rng, lengths, new, 16)
    table[1, :4] = table[0, :4]
    m = Model(pages, 16, 2, 128, 64, True, fill=0x7E)
    for b in (1, 0):                                   # the second write's prefix stands
        whole = np.zeros(3, np.int32)
        whole[b + 1:] = lengths[b]
        m.write(values(rng, lengths[b], 2, 128), values(rng, lengths[b], 2, 128), table, lengths, whole)
    q = rounded(rng.normal(size=(5, 8, 128)).astype(np.float32), F16)
    check_attention(dq, m, table, lengths, starts, q, F16)


def test_broadcast_rows_and_heads(dq):
    """Keys that are one head's for all, queries that are one row's for all."""
    rng = np.random.default_rng(33)
    T, H, D = 37, 3, 64
    table, pages, starts = plan(rng, [T], [T], 16)
    m = Model(pages, 16, H, D, 32, False, fill=0x7E)
    cache = cache_of(dq, m)
    k, v = values(rng, T, 1, D), values(rng, 1, H, D)
    lens = dev(np.array([T], np.int32))
    dq.int4_cache_write(cache, dev(k).expand(T, H, D), dev(v).expand(T, H, D), dev(table), lens, dev(starts))
    m.write(np.repeat(k, H, 1), np.repeat(v, T, 0), table, [T], starts)
    assert_same_bytes(cache, m)
    one = torch.from_numpy(rng.normal(size=(1, 1, D)).astype(np.float32)).to(DEV).half()
    got = dq.int4_cache_attention(one.expand(T, 2 * H, D), cache, dev(table), lens, dev(starts))
    want = dq.int4_cache_attention(one.expand(T, 2 * H, D).contiguous(), cache, dev(table), lens, dev(starts))
    assert torch.equal(got, want)
    check_attention(dq, m, table, [T], starts, one.float().cpu().numpy().repeat(T, 0).repeat(2 * H, 1), F16, cache=cache)


@pytest.mark.parametrize("rows,batch", [(1, 2), (70, 2), (1, 80)])
def test_graphs_that_share_a_workspace(dq, rows, batch):
    """Two graphs captured with one workspace, replayed in turn while the lengths
    change, against the eager call: shared-out keys with few rows, with many, and
    with a large batch."""
    rng = np.random.default_rng(40 + rows)
    top = [2000] * 2 + [20] * (batch - 2)
    m, table, starts = filled(rng, 1, 128, 128, False, 64, top, [rows] * batch)
    cache = cache_of(dq, m)
    st = None if rows == 1 else dev(starts)
    lens, table_d = dev(np.array(top, np.int32)), dev(table)
    ws = dq.cache_attention_workspace(cache, batch, rows * batch, 4)
    qs = [torch.from_numpy(rng.normal(size=(rows * batch, 4, 128)).astype(np.float32)).to(DEV).to(BF16) for _ in range(2)]
    outs, graphs = [torch.zeros_like(q) for q in qs], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for q, out in zip(qs, outs):
            dq.int4_cache_attention(q, cache, table_d, lens, st, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for q, out in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            dq.int4_cache_attention(q, cache, table_d, lens, st, out=out, workspace=ws)
    for n in ([2000, 1400], [1100, 1999], [rows, 1500], [2000, rows]):
        lens.copy_(dev(np.array(n + top[2:], np.int32)))
        for g, q, out in zip(graphs, qs, outs):
            out.zero_()
            g.replay()
        want = [dq.int4_cache_attention(q, cache, table_d, lens, st) for q in qs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), n


def test_the_longest_sequence(dq):
    """2^31 - 1 tokens, all pages the same 16: the softmax is theirs, its sum 2^27
    times as large (2^-27 less for the missing token). A wavefront adds up
    N = 2^25 / 4096 steps (1024 blocks of four), 16 probabilities and 2 products of
    each in binary32: 18 N 2^-24 relative at most, beside the usual bound."""
    rng = np.random.default_rng(60)
    m = Model(1, 16, 1, 64, 64, False, fill=0x7E)
    small = np.zeros((1, 1), np.int32)
    m.write(values(rng, 16, 1, 64), values(rng, 16, 1, 64), small, [16], np.array([0, 16], np.int32))
    q = rounded(rng.normal(size=(1, 2, 64)).astype(np.float32), F16)
    ref, rlse, _, tol, ltol = m.attend(q, small, np.array([16]), None, 0.125)
    table = torch.zeros(1, 1 << 27, dtype=torch.int32, device=DEV)
    lens = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV)
    say("case: the longest")
    out, lse = dq.int4_cache_attention(torch.from_numpy(q).to(DEV).half(), cache_of(dq, m), table, lens, return_lse=True)
    got, many = out.double().cpu().numpy(), 18 * 2.0 ** 25 / 4096 * 2.0 ** -24
    _, v, _ = m.read(16, small, np.array([16]), np.array([0, 16], np.int32))[0:3]
    most = np.abs(v).max()
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -11 * (np.abs(ref) + tol) + 2 * many * most)
    assert np.all(np.abs(lse.cpu().numpy() - (rlse + 27 * np.log(2.0))) <= ltol + 2 * many + 2.0 ** -19)


def test_refusals(dq):
    c = dq.Int4Cache.empty(4, 16, 2, 64, 32)
    table = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    k = torch.zeros(2, 2, 64, device=DEV)
    q = torch.zeros(2, 4, 64, device=DEV, dtype=F16)

    def refused(fn, *a, match, **kw):
        with pytest.raises((ValueError, RuntimeError), match=match):
            fn(*a, **kw)

    w, r, at = dq.int4_cache_write, dq.int4_cache_read, dq.int4_cache_attention
    refused(w, c, k[:, :1], k, table, lens, match="k must be a tensor")
    refused(w, c, k, k[..., :32], table, lens, match="v must be a tensor")
    refused(w, c, k, k.half(), table, lens, match="both the same")
    refused(w, c, k.double(), k.double(), table, lens, match="float32, float16 or bfloat16")
    refused(w, c, k.cpu(), k, table, lens, match="must be on")
    refused(w, c, k, k[:1], table, lens, match="rows")
    refused(w, c, k[:1], k[:1], table, lens, match="one row a sequence")
    refused(w, c, torch.zeros(2, 2, 128, device=DEV)[..., ::2], k, table, lens, match="contiguous in its last")
    refused(w, c, k, k, table.long(), lens, match="page_table must be an int32")
    refused(w, c, k, k, table[0], lens, match="page_table must be an int32")
    refused(w, c, k, k, table.cpu(), lens, match="page_table must be on")
    refused(w, c, k, k, table.t(), lens, match="contiguous in its last")
    refused(w, c, k, k, table[:1].expand(2, 2), lens, match="must not overlap")
    refused(w, c, k, k, table, lens[:1], match="lengths has 1")
    refused(w, c, k, k, table, lens, starts[:2], match="starts has 2")
    refused(w, c, k, k, table, lens, starts.float(), match="starts must be an int32")
    refused(w, "cache", k, k, table, lens, match="Int4Cache")
    refused(r, c, table, lens, starts, match="rows must be given")
    refused(r, c, table, lens, dtype=torch.int8, match="dtype must be")
    refused(r, c, table, lens, rows=3, match="one row a sequence")
    refused(r, c, table, lens, dtype=F32, out=(k, k[:1]), match="must be")
    refused(at, q.float(), c, table, lens, match="float16 or bfloat16")
    refused(at, q[:, :3], c, table, lens, match="no multiple")
    refused(at, q[..., :63], c, table, lens, match="q must be a tensor")
    refused(at, q, c, table, lens, scale=0.0, match="scale")
    refused(at, q, c, table, lens, scale=float("nan"), match="scale")
    refused(at, q, c, table, lens, window=-1, match="window")
    refused(at, q, c, table, lens, window=3, causal=False, match="window")
    refused(at, q, c, table, lens, out=q[:1], match="out must be")
    refused(at, q, c, table, lens, out=q.float(), match="out")
    refused(at, q, c, table, lens, workspace=torch.zeros(256, device=DEV), match="workspace")
    refused(at, q, c, table, lens, workspace=torch.zeros(600, dtype=torch.uint8, device=DEV)[1:], match="aligned")
    refused(dq.cache_attention_workspace, c, 2, 2, 3, match="q_heads")
    refused(dq.Int4Cache.empty, 4, 24, 2, 64, match="page_size")
    refused(dq.Int4Cache.empty, 4, 16, 2, 257, match="head_dim")
    refused(dq.Int4Cache.empty, 4, 16, 2, 128, 48, match="group")
    refused(dq.Int4Cache, c.k_packed, c.k_scales, c.v_packed, c.v_scales, 64, 64, match="shape")
    refused(dq.Int4Cache, c.k_packed, c.k_scales, c.v_packed, c.v_scales, 64, 32, torch.zeros(1, device=DEV), match="both")
    # a table without pages: no keys
    empty = table[:, :0]
    w(c, k, k, empty, lens)
    assert not torch.any(torch.stack(r(c, empty, lens)))
    for causal in (True, False):
        out, lse = at(q + 1, c, empty, lens, causal=causal, return_lse=True)
        assert not torch.any(out) and torch.all(torch.isneginf(lse))
    # nothing to do is no error
    none = torch.zeros(0, 2, 64, device=DEV)
    zeros = torch.zeros(3, dtype=torch.int32, device=DEV)
    w(c, none, none, table, lens, zeros)
    assert at(q[:0], c, table, lens, zeros).shape == (0, 4, 64)
    assert r(c, table, lens, zeros, rows=0)[0].shape == (0, 2, 64)
    assert at(q[:0], c, table[:0], lens[:0]).shape == (0, 4, 64)
