"""Steps of a serving batch over the 4-bit cache on MI355X, all calls together as a
program makes them: ended sequences give their pages back, the others and new ones get
pages, queries and keys are normalised and rotated, keys and values written, and rows
attend over a prefix that all share. Against the plain models of every call."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model
from tests.cache_step_model import Sinks, extend, release, rope_table, transform
from tests.test_cache_gpu import BF16, DEV, F16, assert_same_bytes, cache_of, check_attention, dev, dq, rounded, say, values  # noqa: F401

pytestmark = pytest.mark.gpu


class Serving:
    """A batch's state on the GPU and in the models."""

    def __init__(self, dq, rng, batch, pages, page, most, heads, ratio, D, group, affine, dtype, prefix):
        self.dq, self.rng, self.page, self.dtype = dq, rng, page, dtype
        self.H, self.R, self.D = heads, ratio, D
        self.m = Model(pages, page, heads, D, group, affine, fill=0x7E)
        common = prefix // page
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((batch, most), -1, np.int32)
        self.table[:, :common] = order[:common]
        for p in order[:common]:
            for slot in range(page):
                self.m.put("k", values(rng, heads, D), int(p), slot)
                self.m.put("v", values(rng, heads, D), int(p), slot)
        self.cache = cache_of(dq, self.m)
        self.prefix = prefix
        self.lengths = np.full(batch, prefix, np.int32)
        self.free = np.full(pages, -1, np.int32)
        self.free[:pages - common] = order[common:]
        self.count = np.array([pages - common, 0], np.int32)
        self.t, self.n, self.f, self.c = dev(self.table), dev(self.lengths), dev(self.free), dev(self.count)
        self.s = torch.tensor([prefix], dtype=torch.int32, device=DEV)
        self.rope = rope_table(most * page, D)
        self.w = [(1 + 0.3 * rng.normal(size=D)).astype(np.float32) for _ in range(2)]
        self.dev = [dev(x) for x in (self.rope, *self.w)]

    def step(self, done, added):
        """The calls of one step, then the same in the models; rows of queries and outputs."""
        dq, rng, S = self.dq, self.rng, self.page
        T = int(added.sum())
        x = [rounded(values(rng, T, h, self.D), self.dtype) for h in (self.H * self.R, self.H, self.H)]
        fused = torch.from_numpy(np.concatenate(x, 1)).to(DEV).to(self.dtype)
        q, k, v = fused.split([self.H * self.R, self.H, self.H], 1)
        d = dev(done)
        # ended sequences' places go to new ones, which begin with the prefix
        self.n, self.c = dq.int4_cache_release(self.t, self.n, self.f, self.c, S, d, shared=self.s)
        self.n = torch.where(d, self.s, self.n)
        self.n, starts, slots, self.c = dq.int4_cache_extend(self.t, self.n, self.f, self.c, S, dev(added), rows=T)
        q = dq.int4_cache_append(self.cache, q, k, v, self.t, self.n, starts, q_norm=self.dev[1], k_norm=self.dev[2],
                                 rope=self.dev[0])
        out, lse = dq.int4_cache_attention(q, self.cache, self.t, self.n, starts, shared=self.s, share_from=1, return_lse=True)
        torch.cuda.synchronize()

        self.lengths, self.free, self.count = release(self.table, self.lengths, self.free, self.count, S, done, self.prefix)
        self.lengths = np.where(done, self.prefix, self.lengths).astype(np.int32)
        self.table, self.lengths, rows, places, self.count = extend(self.table, self.lengths, self.free, self.count, S, added, T)
        for name, a, b in (("table", self.t, self.table), ("lengths", self.n, self.lengths), ("free", self.f, self.free),
                           ("count", self.c, self.count), ("starts", starts, rows), ("slots", slots, places)):
            assert np.array_equal(a.cpu().numpy(), b), name
        pos = np.array([self.m.place(self.table, self.lengths, rows, t)[1] for t in range(T)])
        turn = self.rope[pos]
        self.m.write(transform(x[1], self.w[1], 1e-6, turn, False), x[2], self.table, self.lengths, rows)
        assert_same_bytes(self.cache, self.m)
        host = torch.from_numpy(transform(x[0], self.w[0], 1e-6, turn, False)).to(self.dtype).float().numpy()
        assert np.array_equal(q.float().cpu().numpy(), host), "queries"
        # the outputs against the model, and other forms of attention over the same cache
        again = check_attention(dq, self.m, self.table, self.lengths, rows, host, self.dtype, cache=self.cache, shared=self.s,
                                share_from=1)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        check_attention(dq, Sinks(self.m, 5), self.table, self.lengths, rows, host, self.dtype, cache=self.cache, window=33,
                        sinks=5)
        return T


@pytest.mark.parametrize("batch,heads,ratio,D,group,affine,dtype", [(5, 2, 2, 64, 32, True, BF16), (4, 1, 4, 128, 128, False, F16)])
def test_steps(dq, batch, heads, ratio, D, group, affine, dtype):
    rng = np.random.default_rng(D)
    page, prefix = 16, 48
    run = Serving(dq, rng, batch, 90, page, 45, heads, ratio, D, group, affine, dtype, prefix)
    nobody = np.zeros(batch, bool)
    say("case: prompts")
    run.step(nobody, rng.integers(9, 60, size=batch).astype(np.int32))
    for i in range(3):
        say("case: tokens", i)
        run.step(nobody, np.ones(batch, np.int32))
    done = nobody.copy()
    done[[1, batch - 1]] = True
    say("case: two end, new prompts beside tokens")
    run.step(done, np.where(done, 25, 1).astype(np.int32))
    say("case: drafts, and one that waits")
    run.step(nobody, np.array([4, 0, 3, 4, 2][:batch], np.int32))
    # every page is in one place
    used = [p for b in range(batch) for p in run.table[b, 3:-(-run.lengths[b] // page)]] + list(run.table[0, :3])
    assert sorted(used + list(run.free[:run.count[0]])) == list(range(90))


def test_too_few_pages(dq):
    """Tokens without a page are not written and not seen, and the step after, with pages again, is right."""
    rng = np.random.default_rng(3)
    run = Serving(dq, rng, 3, 9, 16, 20, 1, 2, 64, 64, False, BF16, 32)
    run.step(np.zeros(3, bool), np.array([60, 20, 40], np.int32))
    assert run.count[1] == 2 and run.count[0] == 0
    run.step(np.array([True, False, False]), np.array([10, 1, 1], np.int32))
    assert run.count[1] == 0


def test_steps_in_a_graph(dq):
    """One captured step of token generation, replayed with eager work between, against eager steps."""
    rng = np.random.default_rng(4)
    H, R, D, S, B = 2, 2, 64, 16, 6
    pages, prefix = 600, 1280
    cache, twin = (dq.Int4Cache.empty(pages, S, H, D, 64) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(5)
    order = torch.randperm(pages, device=DEV, generator=g).int()
    rope = dev(rope_table(2000, D))

    def fresh():
        t = torch.full((B, 100), -1, dtype=torch.int32, device=DEV)
        t[:, :80] = order[:80]
        free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        free[:pages - 80] = order[80:]
        return (t, torch.tensor([prefix + 3 * b for b in range(B)], dtype=torch.int32, device=DEV), free,
                torch.tensor([pages - 80, 0], dtype=torch.int32, device=DEV))

    for c in (cache, twin):
        for x in (c.k_packed, c.v_packed):
            x.random_(0, 256, generator=torch.Generator(device=DEV).manual_seed(6))
        for x in (c.k_scales, c.v_scales):
            x.fill_(0.05)
    q, k, v = (torch.zeros(B, h, D, dtype=F16, device=DEV) for h in (H * R, H, H))
    shared = torch.tensor([prefix], dtype=torch.int32, device=DEV)
    starts, slots = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    ws = dq.cache_attention_workspace(cache, B, B, H * R, True, 1)

    def step(c, state):
        t, n, f, count = state
        dq.int4_cache_extend(t, n, f, count, S, out=(n, starts, slots, count))
        turned = dq.int4_cache_append(c, q, k, v, t, n, rope=rope)
        return dq.int4_cache_attention(turned, c, t, n, shared=shared, share_from=1, workspace=ws)

    live, other = fresh(), fresh()
    lengths = live[1].clone()
    first = prefix // S
    # the sequences' pages so far
    for state in (live, other):
        new = state[1] - prefix
        state[1].fill_(prefix)
        dq.int4_cache_extend(state[0], state[1], state[2], state[3], S, new, rows=100, out=(state[1], starts, torch.empty(100, dtype=torch.int64, device=DEV), state[3]))
        assert torch.equal(state[1], lengths) and (state[0][1:, first] >= 0).all()
    step(cache, fresh())
    torch.cuda.synchronize()
    for x, y in ((cache.k_packed, twin.k_packed), (cache.v_packed, twin.v_packed), (cache.k_scales, twin.k_scales), (cache.v_scales, twin.v_scales)):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, live)
    for i in range(5):
        for x in (q, k, v):
            x.normal_(generator=g)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = step(twin, other)
        assert torch.equal(got, want), i
        for a, b in zip(live, other):
            assert torch.equal(a, b), i
        for name in ("k_packed", "v_packed", "k_scales", "v_scales"):
            assert torch.equal(getattr(cache, name), getattr(twin, name)), name


def calls(dq, cache, x, table, lengths, starts, w, rope, shared):
    """Append, read back, attend in each form."""
    q, k, v = x
    q = dq.int4_cache_append(cache, q, k, v, table, lengths, starts, q_norm=w, k_norm=w, rope=rope)
    back = dq.int4_cache_read(cache, table, lengths, starts, rows=q.shape[0], dtype=q.dtype)
    ask = q[-40:].contiguous()
    few = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    return [q, *back, *(dq.int4_cache_attention(a, cache, table, lengths, s, **kw) for a, s in ((q, starts), (ask, few))
                        for kw in (dict(window=300, sinks=70), dict(shared=shared, share_from=1)))]


@pytest.mark.parametrize("rows", [700, 5200])
def test_far_pages(dq, rows):
    """Pages past 2^32 bytes of codes: the same bits as on the first ones, row by row and as prompts."""
    H, HQ, D, S, pages = 8, 32, 128, 64, 140000
    g = torch.Generator(device=DEV).manual_seed(rows)
    cache = dq.Int4Cache.empty(pages, S, H, D, 64, True)
    x = [torch.randn(rows, h, D, device=DEV, generator=g).to(BF16) for h in (HQ, H, H)]
    w, rope = torch.rand(D, device=DEV, generator=g) + 0.5, dev(rope_table(rows, D))
    n = torch.tensor([rows - rows // 3, rows // 3], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, rows - rows // 3, rows], dtype=torch.int32, device=DEV)
    shared = torch.tensor([2 * S], dtype=torch.int32, device=DEV)
    each = -(-rows // S)
    near = torch.arange(2 * each, dtype=torch.int32, device=DEV).view(2, each)
    near[1, :2] = near[0, :2]
    same = torch.cat([t[:2 * S] for t in x[1:]], 1).clone()      # the shared tokens' keys and values
    first = rows - rows // 3
    for i in (1, 2):
        x[i][first:first + 2 * S] = same[:, (i - 1) * H:i * H]
    say("case: far pages", rows)
    want = calls(dq, cache, x, near, n, starts, w, rope, shared)
    got = calls(dq, cache, x, pages - 1 - near, n, starts, w, rope, shared)
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


def test_far_rows(dq):
    """Rows 2^27 elements apart, the last ones past 2^31 elements: the same bits as side by side."""
    H, HQ, D, S, T = 2, 6, 64, 16, 20
    big = torch.empty(T << 27, dtype=F16, device=DEV).view(T, 1 << 27)
    wide = big[:, :(HQ + 2 * H) * D].view(T, HQ + 2 * H, D)
    wide.copy_(torch.randn(T, HQ + 2 * H, D, device=DEV))
    w, rope = torch.ones(D, device=DEV), dev(rope_table(64, D))
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    n = torch.tensor([40, 12], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 8, 20], dtype=torch.int32, device=DEV)
    got = []
    for y in (wide, wide.contiguous()):
        cache = dq.Int4Cache.empty(8, S, H, D, 32, False)
        for t in (cache.k_packed, cache.v_packed, cache.k_scales, cache.v_scales):
            t.zero_()
        x = y.split([HQ, H, H], 1)
        say("case: far rows", y.stride())
        q = dq.int4_cache_append(cache, *x, table, n, starts, q_norm=w, k_norm=w, rope=rope)
        got.append([q, *dq.int4_cache_read(cache, table, n, starts, rows=T, dtype=F16),
                    dq.int4_cache_attention(x[0], cache, table, n, starts, window=5, sinks=3)])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.isfinite(a).all() and torch.equal(a, b), i
