"""Norms, rotation and the cache write in one pass on MI355X (int4_cache_append): the
cache's bytes and the queries must be those of the documented roundings bit for bit,
and both must lie within the bound derived from 64 bits (tests/cache_step_model.py)."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model, plan
from tests.cache_step_model import rope_table, transform, transform64
from tests.test_cache_gpu import BF16, DEV, F16, F32, assert_same_bytes, cache_of, dev, dq, rounded, say, values  # noqa: F401

pytestmark = pytest.mark.gpu


def positions(m, table, lengths, starts, rows):
    got = [m.place(table, lengths, starts, t) for t in range(rows)]
    return got, np.array([-1 if g is None else g[1] for g in got])


def check_append(dq, m, cache, table, lengths, starts, q, k, v, dtype, *, q_norm=None, k_norm=None, eps=1e-6, rope=None,
                 interleaved=False, arrays=None, out=None):
    """One call, its bytes into the model too; q, k, v float32 values of dtype."""
    rows, D = q.shape[0], m.D
    lengths = np.asarray(lengths, np.int32)
    qd, kd, vd = arrays or (torch.from_numpy(x).to(DEV).to(dtype) for x in (q, k, v))
    mark = torch.full(q.shape, 7.0, dtype=dtype, device=DEV) if out is None else out
    got = dq.int4_cache_append(cache, qd, kd, vd, dev(table), dev(lengths), None if starts is None else dev(starts),
                               q_norm=None if q_norm is None else dev(q_norm), k_norm=None if k_norm is None else dev(k_norm),
                               eps=eps, rope=None if rope is None else dev(rope), interleaved=interleaved, out=mark)
    torch.cuda.synchronize()
    assert got is mark
    where, pos = positions(m, table, lengths, starts, rows)
    owned = np.array([g is not None for g in where])
    there = owned & (pos >= 0) & (pos < (len(rope) if rope is not None else 2 ** 40))
    turn = None if rope is None else rope[np.where(there, pos, 0)]
    tq, tk = transform(q, q_norm, eps, turn, interleaved), transform(k, k_norm, eps, turn, interleaved)
    o = got.float().cpu().numpy()
    if out is None:
        assert np.all(o[~owned] == 7.0), "a row that no sequence owns was written"
    assert np.all(o[owned & ~there] == 0.0)
    want = torch.from_numpy(tq).to(dtype).float().numpy()
    assert np.array_equal(o[there], want[there]), "queries"
    exact, tol = transform64(q, q_norm, eps, turn, interleaved)
    tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(exact) + tol) + (2.0 ** -25 if dtype == F16 else 0.0)
    assert np.all(np.abs(o - exact)[there] <= tol[there])
    for t in np.flatnonzero(there):
        if where[t][2] >= 0:
            m.put("k", tk[t], where[t][2], int(pos[t]) % m.S)
            m.put("v", v[t], where[t][2], int(pos[t]) % m.S)
    assert_same_bytes(cache, m)
    # keys: within half a step of the 64-bit values
    exact, tol = transform64(k, k_norm, eps, turn, interleaved)
    for t in np.flatnonzero(there):
        if where[t][2] >= 0:
            y, s = m.values("k", where[t][2], int(pos[t]) % m.S)
            # the scale is rounded to binary16: the largest of a group may lie up to 7.5 * 2^-11 steps past the last code
            top = 15 if m.affine else 7
            bound = s * (0.5 + (0.5 if m.affine else 0.0) + top * 2.0 ** -10) + tol[t] + 2.0 ** -24 * top
            assert np.all(np.abs(y - exact[t]) <= bound)
    return got


APPEND = [  # D, group, affine, heads, q heads, page, dtype, rotary, interleaved, norm, lengths, new rows
    (128, 128, False, 2, 8, 64, BF16, 128, False, True, [1, 17, 40], [1, 1, 1]),
    (128, 64, True, 2, 6, 16, F16, 64, True, True, [200, 64, 33], [150, 30, 1]),
    (128, 32, True, 1, 1, 32, F32, 128, True, True, [90], [90]),
    (64, 64, False, 3, 3, 16, BF16, 64, False, True, [31, 2, 70], [31, 1, 64]),
    (64, 32, True, 2, 4, 128, F16, 16, False, False, [129, 128], [3, 128]),
    (80, 32, True, 2, 5, 16, F32, 80, False, True, [19, 1, 50], [19, 1, 7]),
    (80, 128, False, 2, 2, 16, BF16, 32, False, True, [70], [70]),
    (72, 128, False, 1, 3, 16, BF16, 72, True, False, [33, 40], [33, 2]),
    (96, 64, False, 2, 12, 32, BF16, 96, False, True, [40, 70], [11, 70]),
    (96, 96, True, 1, 2, 32, F16, 48, True, True, [100], [100]),
    (192, 128, True, 2, 2, 16, F16, 128, False, True, [21, 20], [21, 3]),
    (160, 64, False, 1, 4, 16, BF16, 160, False, True, [65], [64]),
    (256, 128, False, 1, 8, 32, BF16, 256, False, True, [65, 9], [64, 9]),
    (256, 32, True, 2, 2, 16, F32, 64, False, False, [18], [18]),
    (250, 64, False, 1, 2, 16, F16, 250, False, True, [40], [16]),
    (33, 32, True, 1, 2, 16, BF16, 32, False, True, [20], [20]),
    (33, 32, False, 1, 1, 16, F32, 6, True, True, [20, 3], [20, 3]),
    (1, 1, False, 2, 2, 16, F32, 0, False, True, [5], [5]),
    (2, 2, True, 1, 3, 16, BF16, 2, False, True, [50], [50]),
    (128, 128, False, 2, 2, 16, BF16, 0, False, True, [20, 4], [20, 4]),
    (128, 128, True, 2, 2, 16, F16, 0, False, False, [20, 4], [20, 4]),
]


def weights(rng, D):
    return (1.0 + 0.4 * rng.normal(size=D)).astype(np.float32)


@pytest.mark.parametrize("D,group,affine,heads,q_heads,page,dtype,rotary,interleaved,norm,lengths,new", APPEND)
def test_append(dq, D, group, affine, heads, q_heads, page, dtype, rotary, interleaved, norm, lengths, new):
    rng = np.random.default_rng(D + group + rotary)
    table, pages, starts = plan(rng, lengths, new, page)
    m = Model(pages, page, heads, D, group, affine, fill=0x5A)
    cache = cache_of(dq, m)
    T = int(starts[-1])
    rope = rope_table(max(lengths) + 5, rotary) if rotary else None
    q, k, v = (rounded(values(rng, T, h, D), dtype) for h in (q_heads, heads, heads))
    say("case: append", D, group, affine, heads, q_heads, page, dtype, rotary, interleaved, norm, lengths, new)
    kw = dict(rope=rope, interleaved=interleaved)
    check_append(dq, m, cache, table, lengths, starts, q, k, v, dtype, q_norm=weights(rng, D) if norm else None,
                 k_norm=weights(rng, D) if norm else None, **kw)
    # only one of the two norms, rows without starts
    B = len(lengths)
    check_append(dq, m, cache, table, lengths, None, q[:B], k[:B], v[:B], dtype, k_norm=weights(rng, D), eps=0.25, **kw)
    check_append(dq, m, cache, table, lengths, None, q[:B], k[:B], v[:B], dtype, q_norm=weights(rng, D), **kw)


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_slices_of_one_projection(dq, dtype, wide):
    """Rows of a fused output, at 16-byte aligned places and at others; queries in place."""
    rng = np.random.default_rng(5)
    H, R, D, T = 2, 3, 64, 40
    table, pages, starts = plan(rng, [T, 30], [T - 10, 10], 16)
    m = Model(pages, 16, H, D, 64, False)
    cache = cache_of(dq, m)
    off = 8 if wide else 3
    x = rounded(values(rng, T, (H * R + 2 * H) * D + off), dtype)
    fused = torch.from_numpy(x).to(DEV).to(dtype)
    rows = fused[:, off:].unflatten(1, (-1, D)) if wide else fused[:, 3:].unflatten(1, (-1, D))
    host = x[:, off:].reshape(T, -1, D)
    arrays = (rows[:, :H * R], rows[:, H * R:H * R + H], rows[:, H * R + H:])
    q, k, v = host[:, :H * R], host[:, H * R:H * R + H], host[:, H * R + H:]
    rope = rope_table(64, 64)
    say("case: slices", dtype, wide)
    kw = dict(q_norm=weights(rng, D), k_norm=weights(rng, D), rope=rope)
    check_append(dq, m, cache, table, [T, 30], starts, q, k, v, dtype, arrays=arrays, **kw)
    own = arrays[0].contiguous()
    check_append(dq, m, cache, table, [T, 30], starts, q, k, v, dtype, arrays=(own, *arrays[1:]), out=own, **kw)
    # weights and angles at addresses that are not 16-byte aligned
    odd = torch.zeros(64 * 65 + 1, device=DEV)[1:].view(64, 65)[:, :64]
    odd.copy_(dev(rope))
    got = dq.int4_cache_append(cache, *arrays, dev(table), dev(np.array([T, 30], np.int32)), dev(starts), rope=odd)
    want = dq.int4_cache_append(cache, *arrays, dev(table), dev(np.array([T, 30], np.int32)), dev(starts), rope=dev(rope))
    assert torch.equal(got, want)


def test_plans_that_no_caller_means(dq):
    """Rows that no sequence owns, positions below 0 and past the rope or the table, pages that are none."""
    rng = np.random.default_rng(6)
    for new in ([3, 2, 4, 1], [70, 20, 40, 30]):   # both forms
        lengths = [60, 2, 200, 90]
        table, pages, starts = plan(rng, lengths, new, 16)
        m = Model(pages, 16, 2, 64, 32, True, fill=0x3C)
        cache = cache_of(dq, m)
        lengths = [60, 2 - new[1], 2000, 90]       # below 0 for the second, past the table for the third
        table[3, 0] = pages + 3
        table[0, 1] = -1
        T = int(starts[-1]) + 6
        q, k, v = (rounded(values(rng, T, h, 64), BF16) for h in (4, 2, 2))
        say("case: plans", new)
        check_append(dq, m, cache, table, lengths, starts + 2, q, k, v, BF16, q_norm=weights(rng, 64), k_norm=weights(rng, 64),
                     rope=rope_table(85, 64))


def test_rows_of_zeros_and_extremes(dq):
    """Zero rows with and without an eps, values near the ends of their type's range."""
    rng = np.random.default_rng(7)
    table, pages, starts = plan(rng, [8], [8], 16)
    for dtype, big in ((F32, 1e18), (BF16, 1e18), (F16, 6e4)):
        m = Model(pages, 16, 1, 64, 64, False)
        cache = cache_of(dq, m)
        q, k, v = (rounded(values(rng, 8, 1, 64), dtype) for _ in range(3))
        q[0] = k[0] = v[0] = 0.0
        q[1] = k[1] = rounded(np.full((1, 64), big, np.float32), dtype)
        q[2] *= 0.0
        q[2, 0, 5] = rounded(np.array([1e-7 if dtype == F16 else 1e-30], np.float32), dtype)[0]
        k[2] = q[2]
        say("case: extremes", dtype)
        check_append(dq, m, cache, table, [8], starts, q, k, v, dtype, q_norm=weights(rng, 64), k_norm=weights(rng, 64),
                     rope=rope_table(9, 64))


def test_no_rows(dq):
    m = Model(2, 16, 1, 64, 64, False, fill=3)
    cache = cache_of(dq, m)
    none = torch.zeros(0, 1, 64, dtype=BF16, device=DEV)
    table, lengths, starts = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    assert dq.int4_cache_append(cache, none, none, none, table, lengths, starts).shape == (0, 1, 64)
    assert_same_bytes(cache, m)


MANY = [  # D, group, affine, heads, query heads, page, dtype, rotary, interleaved, norm, lengths, new rows, elements before the rows
    (128, 64, True, 8, 32, 64, BF16, 128, False, True, [2000, 1800, 150], [2000, 1700, 21], 0),
    (128, 128, False, 4, 60, 16, F16, 64, False, True, [2600, 90], [2581, 70], 0),
    (64, 32, True, 12, 12, 16, F32, 64, False, True, [5000, 5003], [4900, 4801], 0),
    (64, 64, False, 20, 60, 32, BF16, 64, True, False, [4100], [4090], 0),
    (80, 32, True, 10, 30, 16, F16, 80, False, True, [4000, 1800], [4000, 1790], 0),
    (96, 96, False, 10, 40, 16, BF16, 48, False, True, [3000, 900], [2990, 900], 0),
    (96, 64, True, 10, 40, 64, F32, 96, True, True, [3700, 77], [3650, 41], 0),
    (72, 128, False, 10, 40, 16, BF16, 72, False, True, [4000, 900], [3900, 900], 0),
    (192, 64, True, 8, 24, 16, BF16, 192, False, True, [2200, 700], [2190, 700], 0),
    (192, 128, False, 8, 24, 16, F16, 0, False, True, [2200, 700], [2190, 700], 0),
    (256, 128, False, 4, 24, 32, BF16, 256, False, True, [2000, 600], [1999, 599], 0),
    (256, 32, True, 4, 24, 16, F32, 128, True, True, [2000, 600], [1999, 599], 0),
    (250, 64, False, 4, 24, 16, F16, 250, False, True, [2000, 600], [1999, 599], 0),
    (128, 128, True, 8, 32, 64, BF16, 128, False, True, [2000, 1800, 150], [2000, 1700, 21], 3),
    (33, 32, False, 16, 64, 16, F16, 32, False, True, [6600], [6550], 0),
    (2, 2, True, 60, 120, 16, BF16, 2, True, True, [45000], [44900], 0),
]


@pytest.mark.parametrize("D,group,affine,H,HQ,S,dtype,rotary,interleaved,norm,lengths,new,off", MANY)
def test_many_rows(dq, D, group, affine, H, HQ, S, dtype, rotary, interleaved, norm, lengths, new, off):
    """So many rows that they are taken by positions: the same bits as few rows at a time,
    which go row by row; rows that no sequence owns before and behind, pages that are none,
    positions past the rope."""
    rng = np.random.default_rng(D + group)
    table, pages, starts = plan(rng, lengths, new, S)
    starts = starts + 2
    table[0, 1], table[-1, 0] = -1, pages + 5
    T = int(starts[-1]) + 3
    assert T * (HQ + 2 * H) * D > 20000000 and T >= 20 * len(new)
    g = torch.Generator(device=DEV).manual_seed(1)
    fused = torch.randn(T, (HQ + 2 * H) * D + off, generator=g, device=DEV).to(dtype)[:, off:].unflatten(1, (-1, D))
    q, k, v = fused.split([HQ, H, H], 1)
    rope = dev(rope_table(max(lengths) - 37, rotary)) if rotary else None
    q_norm, k_norm = (dev(weights(rng, D)) for _ in range(2)) if norm else (None, None)
    caches = [dq.Int4Cache.empty(pages, S, H, D, group, affine) for _ in range(2)]
    names = [n for n in ("k_packed", "v_packed", "k_scales", "v_scales", "k_zeros", "v_zeros") if getattr(caches[0], n) is not None]
    for c in caches:
        for n in names:
            getattr(c, n).zero_()
    say("case: many rows", D, group, affine, H, HQ, dtype, rotary, interleaved, T)
    kw = dict(q_norm=q_norm, k_norm=k_norm, rope=rope, interleaved=interleaved)
    out = torch.full((T, HQ, D), 7.0, dtype=dtype, device=DEV)
    whole = dq.int4_cache_append(caches[0], q, k, v, dev(table), dev(np.array(lengths, np.int32)), dev(starts), out=out, **kw)
    assert (whole[:2] == 7).all() and (whole[-3:] == 7).all()
    step = max(1, 19000000 // ((HQ + 2 * H) * D))
    for b, n in enumerate(lengths):
        for at in range(0, new[b], step):
            m = min(step, new[b] - at)
            rows = slice(int(starts[b]) + at, int(starts[b]) + at + m)
            part = dq.int4_cache_append(caches[1], q[rows], k[rows], v[rows], dev(table[b:b + 1]),
                                        dev(np.array([n - new[b] + at + m], np.int32)), dev(np.array([0, m], np.int32)), **kw)
            assert torch.equal(whole[rows], part)
    for n in names:
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)), n


def test_append_in_a_graph_and_on_two_streams(dq):
    rng = np.random.default_rng(9)
    lengths = np.array([40, 7, 130], np.int32)
    table, pages, _ = plan(rng, [200, 200, 200], [0, 0, 0], 16)
    m = Model(pages, 16, 2, 64, 32, False)
    cache = cache_of(dq, m)
    rope, w = rope_table(300, 64), weights(rng, 64)
    n, t = dev(lengths), dev(table)
    q, k, v = (torch.zeros(3, h, 64, dtype=BF16, device=DEV) for h in (4, 2, 2))
    args = dict(q_norm=dev(w), k_norm=dev(w), rope=dev(rope))
    dq.int4_cache_append(cache, q, k, v, t, n, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n += 1
        out = dq.int4_cache_append(cache, q, k, v, t, n, **args)
    for s in (m, ):
        zeros = np.zeros((3, 2, 64), np.float32)
        s.write(transform(zeros, w, 1e-6, rope[lengths - 1], False), zeros, table, lengths, None)
    for step in range(4):
        host = [rounded(values(rng, 3, h, 64), BF16) for h in (4, 2, 2)]
        for to, x in zip((q, k, v), host):
            to.copy_(torch.from_numpy(x).to(DEV).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        lengths = lengths + 1
        turn = rope[lengths - 1]
        m.write(transform(host[1], w, 1e-6, turn, False), host[2], table, lengths, None)
        assert_same_bytes(cache, m)
        want = torch.from_numpy(transform(host[0], w, 1e-6, turn, False)).to(BF16).float().numpy()
        assert np.array_equal(out.float().cpu().numpy(), want), step
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(dq.int4_cache_append(cache, q, k, v, t, n, **args))
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    assert_same_bytes(cache, m)
